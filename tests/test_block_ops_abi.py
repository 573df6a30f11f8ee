"""CPU checks of the entry points around the feed-forward block: argument refusals (before any launch,
so they run with or without a GPU), workspace and scale sizes, and the plain 64-bit restatements that the
GPU tests compare with."""
import types

import pytest
import torch

import discrete_diffusion_lm_b200 as dg
from discrete_diffusion_lm_b200 import build
from tests import block_ref as ref

FAKE = 1 << 20  # an aligned non-null address that is never dereferenced (calls fail validation first)
A, Bq, Cq, D = FAKE, FAKE + (1 << 16), FAKE + (2 << 16), FAKE + (3 << 16)


@pytest.fixture(scope="module")
def L():
    build.build()
    return dg.lib()


def norm(L, **kw):
    a = dict(x=A, ld_x=64, y=Bq, ld_y=64, act=1, w_post=FAKE, gate=FAKE, w_pre=FAKE, par=1, B=2, C=4, d=64, s=1.0, eps=1e-6,
             x_out=Cq, h=D, ry=FAKE, rx=FAKE, stream=None)
    a.update(kw)
    return L.dg_block_norm(*a.values())


@pytest.mark.parametrize("kw,code,frag", [
    (dict(x=None), 1, "x is required"),
    (dict(act=3), 1, "activation dtype"),
    (dict(par=-1), 1, "parameter dtype"),
    (dict(B=0), 1, "B = 0"),
    (dict(B=257), 1, "B = 257"),
    (dict(C=0), 1, "C = 0"),
    (dict(B=200, C=1 << 30), 1, "overflows"),
    (dict(d=60), 1, "multiple of 8"),
    (dict(d=0), 1, "multiple of 8"),
    (dict(d=16392, ld_x=16392, ld_y=16392), 1, "multiple of 8"),
    (dict(s=float("nan")), 1, "res_scale"),
    (dict(s=float("inf")), 1, "res_scale"),
    (dict(eps=-1e-6), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"),
    (dict(y=None), 1, "y and w_post"),
    (dict(w_post=None), 1, "y and w_post"),
    (dict(y=None, w_post=None, x_out=None), 1, "gate comes only with y"),
    (dict(y=None, w_post=None, gate=None, x_out=None, w_pre=None, h=None), 1, "nothing to compute"),
    (dict(x_out=None), 1, "x_out is required"),
    (dict(y=None, w_post=None, gate=None), 1, "x_out is required"),
    (dict(h=None), 1, "h is required"),
    (dict(w_pre=None), 1, "h is required"),
    (dict(ld_x=56), 1, "row stride"),
    (dict(ld_y=56), 1, "row stride"),
    (dict(ld_x=68), 2, "16 bytes"),
    (dict(x=A + 8), 2, "16 bytes"),
    (dict(y=Bq + 8), 2, "16 bytes"),
    (dict(gate=FAKE + 8), 2, "16-byte"),
    (dict(h=D + 4), 2, "16-byte"),
    (dict(x_out=A, ld_x=72), 1, "ld_x = d"),
    (dict(x_out=Bq), 1, "alias"),
    (dict(h=A), 1, "alias"),
    (dict(h=Cq), 1, "alias"),
])
def test_block_norm_rejects(L, kw, code, frag):
    assert norm(L, **kw) == code, dg.dg_last_error()
    assert frag in dg.dg_last_error()


def back(L, **kw):
    P = FAKE
    a = dict(dxo=A, ld_do=64, dh=Bq, ld_dh=64, x=Cq, ld_x=64, y=D, ld_y=64, act=1, w_post=P, gate=P, w_pre=P, par=1, B=2, C=4, d=64,
             s=1.0, ry=P, rx=P, dx=A + (1 << 20), dy=A + (2 << 20), dw_post=P, dgate=P, dw_pre=P, ws=P, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return L.dg_block_norm_backward(*a.values())


@pytest.mark.parametrize("kw,code,frag", [
    (dict(dx=None), 1, "dx is required"),
    (dict(dh=None), 1, "w_pre needs"),
    (dict(x=None), 1, "w_pre needs"),
    (dict(rx=None), 1, "w_pre needs"),
    (dict(dw_pre=None), 1, "w_pre needs"),
    (dict(w_pre=None), 1, "only with w_pre"),
    (dict(w_pre=None, dh=None, dw_pre=None, dxo=None), 1, "dx_out is required"),
    (dict(ry=None), 1, "y needs"),
    (dict(dy=None), 1, "y needs"),
    (dict(dw_post=None), 1, "y needs"),
    (dict(y=None, w_post=None, gate=None, dgate=None), 1, "only with y"),
    (dict(dgate=None), 1, "dgate"),
    (dict(gate=None), 1, "dgate"),
    (dict(ld_dh=32), 1, "row stride"),
    (dict(ld_do=68), 2, "16 bytes"),
    (dict(dw_pre=FAKE + 4), 2, "16-byte"),
    (dict(dx=A), 1, "alias an input"),
    (dict(dy=D), 1, "alias an input"),
    (dict(dy=A + (1 << 20)), 1, "alias"),
    (dict(ws=None), 3, "workspace"),
    (dict(ws_bytes=16), 3, "workspace"),
    (dict(ws=FAKE + 8), 2, "workspace"),
])
def test_block_norm_backward_rejects(L, kw, code, frag):
    assert back(L, **kw) == code, dg.dg_last_error()
    assert frag in dg.dg_last_error()


def test_mx4_rejects(L):
    q = L.dg_mx4_quantize
    assert q(None, 1, 64, 4, 64, A, Bq, None) == 1
    assert q(FAKE, 1, 64, 4, 64, None, Bq, None) == 1
    assert q(FAKE, 2, 64, 4, 64, A, Bq, None) == 1
    assert q(FAKE, 1, 64, 0, 64, A, Bq, None) == 1
    assert q(FAKE, 1, 64, 4, 48, A, Bq, None) == 1 and "multiple of 32" in dg.dg_last_error()
    assert q(FAKE, 1, 64, 4, 0, A, Bq, None) == 1
    assert q(FAKE, 1, 32, 4, 64, A, Bq, None) == 1 and "ld" in dg.dg_last_error()
    assert q(FAKE, 1, 68, 4, 64, A, Bq, None) == 2
    assert q(FAKE + 8, 1, 64, 4, 64, A, Bq, None) == 2
    assert q(FAKE, 1, 64, 4, 64, A + 8, Bq, None) == 2
    r = L.dg_mx4_dequantize
    assert r(None, FAKE, 4, 64, A, 1, None) == 1
    assert r(FAKE, FAKE, 4, 64, A, 5, None) == 1
    assert r(FAKE, FAKE, 4, 40, A, 1, None) == 1
    assert r(FAKE, FAKE, 4, 64, A + 4, 1, None) == 2
    m = L.dg_mx4_matmul
    assert m(FAKE, FAKE, FAKE, None, 4, 64, 64, A, 1, None) == 1
    assert m(FAKE, FAKE, FAKE, FAKE, 0, 64, 64, A, 1, None) == 1
    assert m(FAKE, FAKE, FAKE, FAKE, 4, 60, 64, A, 1, None) == 1 and "N = 60" in dg.dg_last_error()
    assert m(FAKE, FAKE, FAKE, FAKE, 4, 0, 64, A, 1, None) == 1
    assert m(FAKE, FAKE, FAKE, FAKE, 4, 64, 65, A, 1, None) == 1
    assert m(FAKE, FAKE, FAKE, FAKE, 4, 64, 64, A, 7, None) == 1
    assert m(FAKE, FAKE + 4, FAKE, FAKE, 4, 64, 64, A, 1, None) == 2
    f = L.dg_ffw_mx4
    assert f(FAKE, 0, 64, 64, A, A, A, A, Bq, Cq, 1 << 30, None) == 1
    assert f(FAKE, 4, 96, 64, A, A, A, A, Bq, Cq, 1 << 30, None) == 1
    assert f(FAKE, 4, 64, 16448, A, A, A, A, Bq, Cq, 1 << 30, None) == 1
    assert f(FAKE, 4, 64, 64, A, A, None, A, Bq, Cq, 1 << 30, None) == 1
    assert f(FAKE, 4, 64, 64, A, A, A, A + 8, Bq, Cq, 1 << 30, None) == 2
    assert f(FAKE, 4, 64, 64, A, A, A, A, Bq, Cq, 64, None) == 3
    assert f(FAKE, 4, 64, 64, A, A, A, A, Bq, Cq + 16, 1 << 30, None) == 2


def test_sizes(L):
    assert L.dg_mx4_scale_bytes(1, 32) == 512 and L.dg_mx4_scale_bytes(129, 160) == 4 * 512 and L.dg_mx4_scale_bytes(0, 32) == 0
    for R, K in ((1, 32), (128, 128), (300, 544)):
        n = 1
        for s in dg.dg_mx4_scale_shape(R, K):
            n *= s
        assert n == L.dg_mx4_scale_bytes(R, K)
    assert L.dg_ffw_mx4_workspace_size(0, 64, 64) == 0
    assert L.dg_ffw_mx4_workspace_size(256, 2048, 8192) >= 256 * (2048 + 8192) * 17 // 32
    w = L.dg_block_norm_backward_workspace_size
    assert w(0, 4, 64, 1, 1) == 0 and w(1, 1, 64, 1, 1) == 2 * 64 * 4 and w(1, 1, 64, 5, 1) == 0
    assert w(8, 1536, 2048, 1, 1) >= 2 * 8 * 2048 * 4


def test_backward_workspace_of_the_largest_row_counts(L):
    # the runs of rows are counted without leaving 32 bits up to B*C = 2^31 - 1: as many as fill the device
    w = L.dg_block_norm_backward_workspace_size
    for d, act in ((8, 1), (8, 0), (16384, 0)):
        full = w(1, 1 << 20, d, act, 0)
        assert 0 < full <= 2 * 296 * d * 4
        runs = full // (8 * d)
        for B, C in ((1, 1 << 30), (1, 2**31 - 296), (1, 2**31 - 295), (1, 2**31 - 2), (1, 2**31 - 1), (3, 715827882)):
            assert w(B, C, d, act, 0) == full, (B, C)
            if B == 1:
                assert w(B, C, d, act, 1) == full, (B, C)
        assert w(2, 2**30 - 1, d, act, 1) == 2 * (runs // 2) * 8 * d


def test_binding_rejects_before_any_call(L):
    x, w, f = torch.zeros(8, 64, dtype=torch.bfloat16), torch.ones(64), torch.zeros(8, 64)
    for call in (lambda: dg.dg_block_norm(x, w), lambda: dg.dg_block_norm_backward(x, x, x, w, rstd_x=torch.zeros(8)),
                 lambda: dg.dg_mx4_quantize(f), lambda: dg.dg_mx4_dequantize(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(1, 1, 32, 16, dtype=torch.uint8)),
                 lambda: dg.dg_mx4_matmul((x, x), (x, x)), lambda: dg.dg_ffw_mx4(x, (x, x), (x, x))):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()


def test_binding_rejects_streams_and_tensors_of_another_device():
    with pytest.raises(ValueError, match="the stream is on device 1, the tensors are on device 0"):
        dg._On(0, types.SimpleNamespace(device_index=1))
    other = types.SimpleNamespace(is_cuda=True, device="cuda:1", dtype=torch.float32, shape=torch.Size([4, 8]), get_device=lambda: 1)
    with pytest.raises(ValueError, match="w_pre is on cuda:1, another device"):
        dg._arg(other, "w_pre", 0, other.dtype, other.shape)
    with pytest.raises(ValueError, match="y is on cuda:1, another device"):
        dg._rows_arg(other, "y", 0, other.dtype, other.shape)


# ------------------------------------------------------------------------------------ the restatements themselves
def test_reference_quantisation_by_hand():
    x = torch.zeros(2, 64)
    x[0, :8] = torch.tensor([6.0, 0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5.0])
    x[1, 32:36] = torch.tensor([7.9, -0.4, 3.0, 0.1])
    code, scale = ref.mx4_quantize(x)
    assert scale.tolist() == [[127, 0], [0, 127]]
    assert code[0, :8].tolist() == [7, 0, 2, 2, 8 + 4, 4, 6, 6]
    assert code[1, 32:36].tolist() == [7, 8 + 1, 5, 0]
    v = ref.mx4_values(code, scale)
    assert v[0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, -2.0, 2.0, 4.0, 4.0]
    codes, tiles = ref.mx4_pack(code, scale)
    assert codes[0, :4].tolist() == [0x07, 0x22, 0x4C, 0x66] and tiles.shape == dg.dg_mx4_scale_shape(2, 64)
    back = ref.mx4_unpack(codes, tiles)
    assert torch.equal(back[0], code) and torch.equal(back[1], scale)


@pytest.mark.parametrize("mode,gated", [("both", True), ("both", False), ("pre", False), ("post", True)])
def test_reference_gradients_against_autograd(mode, gated):
    torch.manual_seed(0)
    B, C, d, s, eps = 2, 3, 16, 0.7, 1e-6
    t = lambda *n: torch.randn(*n, dtype=torch.float64, requires_grad=True)  # noqa: E731
    x, y, w_post, gate, w_pre = t(B * C, d), t(B * C, d), t(d), t(B, d), t(d)
    gate_used = gate if gated else None
    dxo, dh = torch.randn(B * C, d, dtype=torch.float64), torch.randn(B * C, d, dtype=torch.float64)
    stream = x if mode == "pre" else ref.block_norm(x, y, w_post, gate_used, C, s, eps)[0]
    loss = (stream * dxo).sum()
    if mode != "post":
        loss = loss + (ref.norm_rows(stream, eps) * w_pre * dh).sum()
    rstd = lambda v: (v.detach().pow(2).mean(1) + eps).rsqrt()  # noqa: E731
    post = mode != "pre"
    got, mag = ref.block_norm_grads(dxo, dh, stream.detach(), w_pre.detach() if mode != "post" else None, rstd(stream),
                                    y.detach() if post else None, w_post.detach(), gate.detach() if gated else None, rstd(y), C, s)
    leaves = {"dx": x, **({"dy": y, "dw_post": w_post} if post else {}), **({"dgate": gate} if post and gated else {}),
              **({"dw_pre": w_pre} if mode != "post" else {})}
    grads = torch.autograd.grad(loss, list(leaves.values()))
    assert set(got) == set(leaves)
    for k, want in zip(leaves, grads):
        assert torch.allclose(got[k], want, rtol=1e-12, atol=1e-12), k
        assert (mag[k] >= got[k].abs() * (1 - 1e-12)).all()
