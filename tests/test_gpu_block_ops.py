"""The operators around the feed-forward block against plain 64-bit restatements (tests/block_ref.py).

Tolerances, from the arithmetic (U = 2^-24 is half a step of fp32, S half a step of the output type):
  * dg_block_norm: a row's sum of squares has at most 32 additions in a thread (16384 columns over
    1024 threads, two rounded operations each) and 10 across threads, so its relative error is below
    74 U and that of rstd below 40 U with the division and root; three more products give every term
    of x_out an error below 48 U of its magnitude, and h below 48 U of its own, plus S for storing.
    h is taken of the unrounded stream: its tolerance also has what the stream's error moves it by.
  * dg_block_norm_backward: the same per-row sums enter each gradient at most twice; 160 U of the sum
    of the terms' magnitudes, plus S for storing.  Column sums add n rows in some order: (n + 160) U
    of the summed magnitudes.
  * dg_mx4_quantize, dg_mx4_dequantize: exact.
  * dg_mx4_matmul: products of E2M1 values are exact and K/64 instruction results are accumulated in
    fp32; each addition may truncate (a whole step, 2 U), so (K/32 + 64) 2 U of sum |a w|, plus S.
  * dg_ffw_mx4: a hidden value is known to (d/32 + 64) 2 U of its summed magnitudes (the derivative of
    gelu is below 1.13) plus 16 U for gelu; where that can cross a midpoint of the 4-bit grid, or move
    its block's largest magnitude across a power of two, the value may be off by the spacing there.
"""
import math
import subprocess
import sys

import pytest
import torch

import discrete_diffusion_lm_b200 as dg
from tests import block_ref as ref
from tests.block_ref import U, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert dg.dg_device_error() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)


def within(got, want, tol, what):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what
    over = ((got - want).abs() - tol).nan_to_num(0.0)
    assert over.max().item() <= 0.0, f"{what}: over by {over.max().item():.3g}, largest error {(got - want).abs().max().item():.3g}"


# ------------------------------------------------------------------------------------ norms, forward
def check_forward(x, y, w_post, gate, w_pre, C, s, eps, out):
    T = x.dtype
    stream, far = x.double(), torch.zeros_like(x, dtype=torch.float64)
    if y is not None:
        want, mag = ref.block_norm(x, y, w_post, gate, C, s, eps)
        within(out["x"], want, 48 * U * mag + half_step(T) * want.abs() + 1e-37, "x")
        r = (y.double().pow(2).mean(1) + eps).rsqrt()
        within(out["rstd_y"], r, 40 * U * r, "rstd_y")
        stream, far = want, 48 * U * mag  # h is taken of the unrounded stream, known to `far`
    if w_pre is not None:
        r = (stream.pow(2).mean(1) + eps).rsqrt()
        r_far = far.pow(2).mean(1).sqrt() * r  # how far the root mean moves with the stream, relative
        want = ref.norm_rows(stream, eps) * w_pre.double()
        tol = (48 * U + half_step(T) + r_far[:, None]) * want.abs() + far * r[:, None] * w_pre.double().abs()
        within(out["h"], want, tol + 1e-37, "h")
        within(out["rstd_x"], r, (40 * U + r_far) * r, "rstd_x")


def norm_inputs(B, C, d, T, P, mode, gated, seed=0):
    g = gen(seed + B * 131 + C * 17 + d)
    R = B * C
    x = randn(g, R, d, dtype=T, std=2.0)
    y = randn(g, R, d, dtype=T, std=0.3) if mode != "pre" else None
    w_post = randn(g, d, dtype=P, std=0.2, mean=1.0) if mode != "pre" else None
    gate = randn(g, B, d, dtype=P, std=0.7) if gated and mode != "pre" else None
    w_pre = randn(g, d, dtype=P, std=0.2, mean=1.0) if mode != "post" else None
    return x, y, w_post, gate, w_pre


# every width class of either type (vectors per row 1 to 4096), one row, odd row counts
SHAPES = [(1, 1, 8), (1, 1, 64), (2, 3, 72), (1, 5, 256), (3, 7, 264), (1, 16, 512), (2, 9, 1000), (1, 2, 1032), (4, 5, 2048),
          (1, 3, 2056), (2, 2, 4096), (1, 3, 5000), (1, 2, 8192), (1, 2, 8200), (1, 3, 16384)]


@pytest.mark.parametrize("T,P", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("B,C,d", SHAPES)
def test_norm_forward(B, C, d, T, P):
    for mode, gated in (("both", True), ("both", False), ("pre", False), ("post", True)):
        x, y, w_post, gate, w_pre = norm_inputs(B, C, d, T, P, mode, gated)
        out = dg.dg_block_norm(x, w_pre, y=y, w_post=w_post, gate=gate, C=C, res_scale=0.7, eps=1e-6)
        assert set(out) == {"both": {"x", "rstd_y", "h", "rstd_x"}, "pre": {"h", "rstd_x"}, "post": {"x", "rstd_y"}}[mode]
        s = torch.tensor(0.7, dtype=F32).item()
        check_forward(x, y, w_post, gate, w_pre, C, s, torch.tensor(1e-6, dtype=F32).item(), out)


# many rows: the form that keeps rows in flight, its widths full and not, canvases that end inside a
# CTA's run of rows, groups of a CTA with no row (3 x 401 of 2048)
MANY = [(3, 500, 64), (256, 5, 72), (5, 300, 256), (4, 400, 512), (3, 401, 1000), (2, 700, 1024), (2, 700, 2048), (3, 401, 2048), (7, 200, 2056),
        (2, 600, 4096), (3, 397, 5000), (1, 1200, 8192), (7, 171, 8200),
        (3, 20001, 64), (200, 300, 72)]


@pytest.mark.parametrize("T,P", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("B,C,d", MANY)
def test_norm_forward_many_rows(B, C, d, T, P):
    s, eps = torch.tensor(0.7, dtype=F32).item(), torch.tensor(1e-6, dtype=F32).item()
    for mode, gated in (("both", True), ("both", False), ("pre", False), ("post", True)):
        x, y, w_post, gate, w_pre = norm_inputs(B, C, d, T, P, mode, gated)
        out = dg.dg_block_norm(x, w_pre, y=y, w_post=w_post, gate=gate, C=C, res_scale=0.7, eps=1e-6)
        check_forward(x, y, w_post, gate, w_pre, C, s, eps, out)
    assert dg.dg_device_error() == 0


@pytest.mark.parametrize("T,d", [(BF16, 72), (BF16, 256), (F32, 128), (BF16, 2048), (F32, 2048)])
def test_norm_row_results_do_not_depend_on_the_number_of_rows(T, d):
    rows = 40000 if d <= 256 else 2000
    x, y, w_post, gate, w_pre = norm_inputs(1, rows, d, T, F32, "both", True)
    many = dg.dg_block_norm(x, w_pre, y=y, w_post=w_post, gate=gate, C=rows, res_scale=0.7)
    for n in (1, 7, 900):
        few = dg.dg_block_norm(x[:n], w_pre, y=y[:n], w_post=w_post, gate=gate, C=n, res_scale=0.7)
        for key, value in few.items():
            assert torch.equal(value, many[key][:n]), key


@pytest.mark.parametrize("rows", [4, 500])
@pytest.mark.parametrize("T", [BF16, F32])
def test_norm_strided_rows_and_in_place_stream(T, rows):
    g = gen(3)
    big, C, d = randn(g, 3 * rows, 3 * 328, dtype=T), 3, 320
    _, _, w_post, gate, w_pre = norm_inputs(4, 3, d, T, F32, "both", True)
    if rows > 4:
        C = 3 * rows // 4
    x, y = big[:, 8:8 + d], big[:, 400:400 + d]
    assert x.stride(0) == 984 and x.data_ptr() % 16 == 0
    kept = big.clone()
    out = dg.dg_block_norm(x, w_pre, y=y, w_post=w_post, gate=gate, C=C, res_scale=-1.5)
    check_forward(x, y, w_post, gate, w_pre, C, -1.5, torch.tensor(1e-6, dtype=F32).item(), out)
    assert torch.equal(big, kept)
    xc = x.contiguous()
    again = dg.dg_block_norm(xc, w_pre, y=y, w_post=w_post, gate=gate, C=C, res_scale=-1.5, out={"x": xc})
    assert again["x"] is xc and torch.equal(xc, out["x"]) and torch.equal(again["h"], out["h"])


def test_norm_zero_rows_nan_rows_and_wide_values():
    d = 512
    x = randn(gen(1), 6, d)
    x[0] = 0
    x[2, 5] = float("nan")
    x[3] = 1e18
    x[4] = 1e-25
    w = torch.ones(d, device=DEV)
    out = dg.dg_block_norm(x, w, eps=0.0)
    # a zero row with eps = 0 has no norm; a NaN stays in its row; other rows are as without them
    assert out["h"][0].isnan().all() and out["h"][2].isnan().all()
    for r in (1, 3, 5):
        within(out["h"][r], ref.norm_rows(x[r:r + 1], 0.0)[0], 48 * U * 4, f"row {r}")
    assert dg.dg_block_norm(x[:1], w, eps=1e-6)["h"].abs().max().item() == 0.0
    within(dg.dg_block_norm(x[4:5], w, eps=1e-6)["h"], x[4:5].double() * 1e3, 1e-6 * 1e-22, "tiny row")


@pytest.mark.parametrize("rows", [12, 1500])
def test_norm_rows_beyond_the_squares_range(rows):
    # rows of 1e-25 and 1e25: their squares leave fp32, and every result but rstd is as at any size
    d, C = 512, rows
    x, y, w_post, _, w_pre = norm_inputs(1, C, d, F32, F32, "both", False)
    size = torch.tensor([1.0, 1e-25, 1e25], device=DEV).repeat(rows // 3)[:, None]
    x, y = x * size, y * size.flip(0)
    out = dg.dg_block_norm(x, w_pre, y=y, w_post=w_post, eps=0.0)
    check_forward(x, y, w_post, None, w_pre, C, 1.0, 0.0, out)
    g = gen(3)
    dxo, dh = randn(g, rows, d), randn(g, rows, d)
    res = dg.dg_block_norm_backward(dxo, dh, out["x"], w_pre, rstd_x=out["rstd_x"], y=y, w_post=w_post, rstd_y=out["rstd_y"])
    check_backward((dxo, dh, out["x"], w_pre, out["rstd_x"], y, w_post, None, out["rstd_y"]), C, 1.0, res, F32)


# ------------------------------------------------------------------------------------ norms, backward
def check_backward(args, C, s, res, T):
    want, mag = ref.block_norm_grads(*args, C, s)
    assert set(res) == set(want)
    n = args[0].shape[0] if args[0] is not None else args[2].shape[0]
    for k, w in want.items():
        tol = (n + 160) * U * mag[k] if k.startswith(("dw", "dg")) else 160 * U * mag[k] + half_step(T) * w.abs()
        within(res[k], w, tol + 1e-37, k)


def backward_case(B, C, d, T, P, mode, gated, seed=0, with_dx=True):
    x, y, w_post, gate, w_pre = norm_inputs(B, C, d, T, P, mode, gated, seed)
    fwd = dg.dg_block_norm(x, w_pre, y=y, w_post=w_post, gate=gate, C=C, res_scale=0.7)
    g = gen(seed + 99)
    dx_out = randn(g, B * C, d, dtype=T, std=0.1) if with_dx or mode == "post" else None
    dh = randn(g, B * C, d, dtype=T, std=0.1) if mode != "post" else None
    return dx_out, dh, fwd.get("x", x), w_pre, fwd.get("rstd_x"), y, w_post, gate, fwd.get("rstd_y")


def run_backward(args, C, **kw):
    dx_out, dh, x, w_pre, rx, y, w_post, gate, ry = args
    return dg.dg_block_norm_backward(dx_out, dh, x, w_pre, rstd_x=rx, y=y, w_post=w_post, gate=gate, rstd_y=ry, C=C, res_scale=0.7, **kw)


@pytest.mark.parametrize("T,P", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("B,C,d", SHAPES + [(3, 37, 1000), (40, 7, 128), (256, 1, 64), (2, 700, 64)])
def test_norm_backward(B, C, d, T, P):
    s = torch.tensor(0.7, dtype=F32).item()
    for mode, gated, with_dx in (("both", True, True), ("both", False, False), ("pre", False, True), ("post", True, True)):
        args = backward_case(B, C, d, T, P, mode, gated, with_dx=with_dx)
        check_backward(args, C, s, run_backward(args, C), T)


# many rows: groups of one, two, four and eight that refill their ring's slots several times over, widths full and
# not; rows of up to 32 vectors, a group several of them; more than 1024 vectors, several rows to a run; runs and
# groups that end short
@pytest.mark.parametrize("T,P", [(BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("B,C,d", [(8, 1536, 2048), (4, 3000, 512), (3, 2500, 1000), (3, 2001, 2056), (5, 3000, 264), (2, 1500, 4096),
                                   (2, 1200, 8192), (2, 300, 16384), (256, 64, 64), (200, 81, 72)])
def test_norm_backward_many_rows(B, C, d, T, P):
    s = torch.tensor(0.7, dtype=F32).item()
    for mode, gated, with_dx in (("both", True, True), ("both", False, False), ("pre", False, True), ("post", True, True)):
        args = backward_case(B, C, d, T, P, mode, gated, with_dx=with_dx)
        check_backward(args, C, s, run_backward(args, C), T)


@pytest.mark.parametrize("which", ["x", "y", "w_post", "gate", "w_pre"])
def test_norm_gradients_against_differences(which):
    # the derivative of a random linear functional of (stream, h) along a random direction, by central
    # differences of the 64-bit forward pass at step 1e-5: their error is of order step^2 (1e-10) of the
    # third derivative, and cancellation leaves 2^-53 / 1e-5 = 1e-11; the gradient's own error is 160 U
    # of its terms' magnitudes.  Both are below 1e-4 of the product's summed magnitudes.
    B, C, d, s, eps = 3, 4, 96, 0.7, 1e-6
    args = backward_case(B, C, d, F32, F32, "both", True)
    dx_out, dh, _, w_pre, _, y, w_post, gate, _ = args
    x, *_ = norm_inputs(B, C, d, F32, F32, "both", True)
    got = run_backward(args, C)
    t = {"x": x.double(), "y": y.double(), "w_post": w_post.double(), "gate": gate.double(), "w_pre": w_pre.double()}
    direction = torch.randn(t[which].shape, generator=gen(5), device=DEV, dtype=torch.float64)

    def loss(step):
        v = dict(t)
        v[which] = t[which] + step * direction
        stream, _ = ref.block_norm(v["x"], v["y"], v["w_post"], v["gate"], C, s, eps)
        return (stream * dx_out.double()).sum() + (ref.norm_rows(stream, eps) * v["w_pre"] * dh.double()).sum()

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    key = {"x": "dx", "y": "dy"}.get(which, "d" + which)
    terms = got[key].double() * direction
    assert (terms.sum() - want).abs().item() <= 1e-4 * terms.abs().sum().item() / terms.numel() ** 0.5 + 1e-9


def test_norm_backward_strided_and_repeatable():
    B, C, d = 4, 50, 640
    args = backward_case(B, C, d, BF16, F32, "both", True)
    res = run_backward(args, C)
    wide = [torch.zeros(B * C, d + 16, dtype=BF16, device=DEV) for _ in range(4)]
    for w, i in zip(wide, (0, 1, 2, 5)):
        w[:, 8:8 + d] = args[i]
    views = [w[:, 8:8 + d] for w in wide]
    strided = list(args)
    for v, i in zip(views, (0, 1, 2, 5)):
        strided[i] = v
    for _ in range(3):
        again = run_backward(strided, C)
        for k in res:
            assert torch.equal(res[k], again[k]), k


# ------------------------------------------------------------------------------------ 4-bit format
def special_values(T):
    g = gen(7)
    x = randn(g, 140, 288, dtype=T, std=3.0)
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0, -0.0, 4.0], device=DEV)
    for r, p in enumerate((0, 5, -30, 100, -120)):  # every midpoint, both signs, at several scales
        blk = torch.cat([grid, -grid, grid[:8]]) * 2.0 ** p
        x[r, :32] = blk.to(T)
        x[r, 31] = 4.0 * 2.0 ** p  # pins the block's scale
    x[5, 32:64] = 0
    x[6, :32] = torch.finfo(T).max
    x[7, :32] = torch.finfo(T).tiny / 4  # subnormal
    x[8, :32] = torch.finfo(T).tiny * 3
    x[9, 3], x[10, 40], x[11, 288 - 1] = float("nan"), float("inf"), float("-inf")
    x[139, 287] = 1e30
    return x


@pytest.mark.parametrize("T", [BF16, F32])
def test_quantize_special_values(T):
    x = special_values(T)
    codes, scales = dg.dg_mx4_quantize(x)
    want = ref.mx4_pack(*ref.mx4_quantize(x))
    assert torch.equal(scales, want[1])
    assert torch.equal(codes, want[0])
    v = dg.dg_mx4_dequantize(codes, scales, dtype=F32)
    assert torch.equal(v.double().nan_to_num(nan=123.0), ref.mx4_values(*ref.mx4_quantize(x)).nan_to_num(nan=123.0))
    assert v[9, :32].isnan().all() and not v[9, 32:].isnan().any()


@pytest.mark.parametrize("T", [BF16, F32])
@pytest.mark.parametrize("R,K", [(1, 32), (1, 2048), (3, 96), (127, 64), (128, 128), (129, 160), (300, 544), (64, 8192), (513, 4128)])
def test_quantize_shapes_and_strides(R, K, T):
    g = gen(R + K)
    wide = randn(g, R, K + 48, dtype=T) * torch.exp(2 * torch.randn(R, 1, generator=g, device=DEV)).to(T)
    want = ref.mx4_pack(*ref.mx4_quantize(wide[:, 16:16 + K]))
    for x in (wide[:, 16:16 + K], wide[:, 16:16 + K].contiguous()):
        out = (torch.full((R, K // 2), 0xAB, dtype=torch.uint8, device=DEV),
               torch.full(dg.dg_mx4_scale_shape(R, K), 0xCD, dtype=torch.uint8, device=DEV))  # every byte is written
        got = dg.dg_mx4_quantize(x, out=out)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for dt in (BF16, F32):
        v = dg.dg_mx4_dequantize(*want, dtype=dt)
        assert torch.equal(v.double(), ref.mx4_values(*ref.mx4_quantize(wide[:, 16:16 + K])))


def test_dequantize_every_code_and_scale():
    code = torch.arange(16, device=DEV).repeat(256, 2)
    scale = torch.arange(256, device=DEV)[:, None]
    codes, tiles = ref.mx4_pack(code, scale)
    v = dg.dg_mx4_dequantize(codes, tiles, dtype=F32)
    want = ref.mx4_values(code, scale).float()  # the largest scales go to infinity in fp32
    assert torch.equal(v.nan_to_num(nan=77.0), want.nan_to_num(nan=77.0))


# ------------------------------------------------------------------------------------ product
def random_mx4(g, R, K, spread=2.0):
    x = torch.randn(R, K, generator=g, device=DEV) * torch.exp(spread * torch.randn(R, K // 32, generator=g, device=DEV)).repeat_interleave(32, 1)
    q = ref.mx4_quantize(x)
    return ref.mx4_pack(*q), ref.mx4_values(*q)


def check_product(a, av, w, wv, dtype, **kw):
    K = av.shape[1]
    out = dg.dg_mx4_matmul(a, w, dtype=dtype, **kw)
    want, mag = av @ wv.T, av.abs() @ wv.abs().T
    within(out, want, (K / 32 + 64) * 2 * U * mag + half_step(dtype) * want.abs(), f"product {list(out.shape)} K={K} {dtype}")
    return out


@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (128, 128, 256), (1, 128, 64), (7, 24, 96), (128, 128, 128), (129, 136, 160),
                                   (16, 256, 2048), (200, 1000, 4096), (300, 520, 544), (1, 2048, 8192), (64, 64, 2080),
                                   (257, 384, 8192), (1000, 2056, 480),
                                   # many tiles: ragged rows and columns, one row in the last pair of row tiles, K ending in
                                   # every part of a stage, more tiles than pairs of CTAs
                                   (2048, 2056, 480), (257, 9608, 96), (4000, 1288, 1184), (2000, 4096, 2048), (2305, 2312, 320),
                                   (5000, 3000, 64), (4096, 2048, 800),
                                   # up to 128 rows: pairs, single CTAs with and without a split, more columns than one wave
                                   (17, 136, 1056), (128, 264, 2112), (100, 4608, 1312), (100, 9736, 2208), (20, 19080, 160)])
def test_product(M, N, K):
    g = gen(M + N + K)
    (a, av), (w, wv) = random_mx4(g, M, K), random_mx4(g, N, K)
    for dtype in (F32, BF16):
        check_product(a, av, w, wv, dtype)
    assert dg.dg_device_error() == 0


def test_product_every_scale_lane():
    # one operand's scales differ in every block, the other's values are ones: a scale read from the wrong
    # row or block shows as a wrong power of two
    M, N, K = 256, 256, 512
    g = gen(4)
    ones = torch.full((N, K), 2, dtype=torch.long, device=DEV)
    sa = torch.randint(120, 135, (M, K // 32), generator=g, device=DEV)
    sb = torch.randint(120, 135, (N, K // 32), generator=g, device=DEV)
    got = dg.dg_mx4_matmul(ref.mx4_pack(ones, sa), ref.mx4_pack(ones, sb), dtype=F32)
    want = ref.mx4_values(ones, sa) @ ref.mx4_values(ones, sb).T
    within(got, want, (K / 32 + 64) * 2 * U * want, "scales")


def test_product_nan_scales_stay_in_their_row_and_column():
    g = gen(6)
    (a, av), (w, wv) = random_mx4(g, 70, 256), random_mx4(g, 72, 256)
    clean = dg.dg_mx4_matmul(a, w, dtype=F32)
    sa, sw = a[1].clone(), w[1].clone()
    sa[0, 1, 5, 4], sw[0, 0, 3, 9] = 255, 255  # row 37, block 4; column 67, block 1
    got = dg.dg_mx4_matmul((a[0], sa), (w[0], sw), dtype=F32)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[37], bad[:, 67] = True, True
    assert torch.equal(got.isnan(), bad)
    assert torch.equal(got[~bad], clean[~bad])


def test_product_writes_nothing_past_its_rows():
    g = gen(8)
    (a, av), (w, wv) = random_mx4(g, 5, 512), random_mx4(g, 40, 512)
    store = torch.full((9, 40), 7.0, device=DEV)
    check_product(a, av, w, wv, F32, out=store[:5])
    assert torch.equal(store[5:], torch.full((4, 40), 7.0, device=DEV))


# ------------------------------------------------------------------------------------ feed-forward block
def spacing(a):
    """Spacing of the E2M1 grid at scaled magnitude a (the larger side)."""
    return torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()


def check_block(z, w1, w1v, w2, w2v, got):
    d, dff = w1v.shape[1], w1v.shape[0]
    zv = ref.mx4_values(*ref.mx4_quantize(z))
    pre, mag1 = zv @ w1v.T, zv.abs() @ w1v.abs().T
    h = ref.gelu(pre)
    off = 1.13 * (d / 32 + 64) * 2 * U * mag1 + 16 * U * h.abs()  # how far the kernel's hidden value may be
    e = ref.mx4_scale_exponents(h)
    hv = ref.mx4_values(*ref.mx4_quantize(h))
    unit = torch.exp2(e).repeat_interleave(32, 1)
    a, da = h.abs() / unit, off / unit
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=z.device)
    near = ((a[..., None] - mids).abs() <= da[..., None]).any(-1)
    slack = torch.where(near, spacing(a) * unit, torch.zeros_like(h))
    # a block whose largest magnitude is near a power of two may take the other scale: every value moves
    # by at most the spacing of the coarser grid
    top, top_off = h.abs().reshape(h.shape[0], -1, 32).max(2)[0], off.reshape(h.shape[0], -1, 32).max(2)[0]
    other = (torch.floor(torch.log2(top + top_off)) != torch.floor(torch.log2((top - top_off).clamp(min=1e-300))))
    slack = torch.where(other.repeat_interleave(32, 1), 2 * spacing(a) * unit + 2 * unit, slack)
    want, mag2 = hv @ w2v.T, hv.abs() @ w2v.abs().T
    tol = (dff / 32 + 64) * 2 * U * mag2 + slack @ w2v.abs().T
    within(got, want, tol * (1 + half_step(BF16)) + half_step(BF16) * want.abs(), "block")
    return (slack > 0).double().mean().item()


@pytest.mark.parametrize("R,d,dff", [(1, 64, 64), (16, 64, 256), (5, 192, 320), (1, 1024, 4096), (130, 512, 2048), (256, 2048, 8192), (300, 128, 576), (2500, 320, 2112), (1100, 1024, 4096),
                                     (16, 2048, 8192), (32, 2048, 8192), (33, 2048, 8192), (31, 192, 64), (17, 4160, 128), (100, 2112, 2048), (128, 64, 128)])
def test_block(R, d, dff):
    g = gen(R + d)
    z = randn(g, R, d, dtype=BF16)
    (w1, w1v), (w2, w2v) = random_mx4(g, dff, d, 0.3), random_mx4(g, d, dff, 0.3)
    # weights of about 1 / sqrt(fan-in): the scale bytes move by a power of two
    k1, k2 = round(math.log2(d) / 2), round(math.log2(dff) / 2)
    (c1, s1), (c2, s2) = ref.mx4_unpack(*w1), ref.mx4_unpack(*w2)
    w1, w1v, w2, w2v = ref.mx4_pack(c1, s1 - k1), w1v * 2.0 ** -k1, ref.mx4_pack(c2, s2 - k2), w2v * 2.0 ** -k2
    got = dg.dg_ffw_mx4(z, w1, w2)
    open_share = check_block(z, w1, w1v, w2, w2v, got)
    assert open_share < 0.05  # the tolerance leaves few hidden values open
    assert dg.dg_device_error() == 0
    zin = z.clone()
    assert torch.equal(dg.dg_ffw_mx4(zin, w1, w2, out=zin), got)


# One to 16 rows, up to 128, pairs of CTAs with 128 and with 256 columns (the kernel's forms of the gelu).
@pytest.mark.parametrize("R", [1, 16, 100, 300, 20000])
def test_block_gelu_far_below_zero(R):
    # With the identity as the second matrix the block returns its quantised hidden layer, exactly; one
    # nonzero input and one weight per column make every pre-activation a known product of powers of two
    # and 1, 1.5 or 2.25.  gelu's factor 1 / (1 + e^(2u)) is known to 3 U of its exponent (at most 126
    # powers of two) plus ex2's 2^-22, 2e-5 together: no value below lies so near a midpoint of the grid.
    # Products are summed in fp32: one past 2^128 (here -2^90 times 2^57 or 2^63) is infinite, its block NaN.
    d = dff = 128
    mixed = [3.0, -6.0, -8.0, -1.0, 0.5, -12.0, -1.5 * 2.0 ** 33, -1.0 * 2.0 ** 60, -1.5 * 2.0 ** 66, 2.0, -4.0, -(2.0 ** 90)]
    far = [-(2.0 ** 60), -1.5 * 2.0 ** 66, -1e10]
    # blocks of far values only, of both kinds, and of huge ones
    v = torch.tensor([-8.0] * 32 + [-6.0] * 32 + (mixed * 3)[:32] + (far * 11)[:32], dtype=torch.float64, device=DEV)
    W1 = torch.zeros(dff, d, dtype=torch.float64, device=DEV)
    W1[:, 0] = v
    w1, w2 = ref.mx4_pack(*ref.mx4_quantize(W1)), ref.mx4_pack(*ref.mx4_quantize(torch.eye(d, device=DEV)))
    v = ref.mx4_values(*ref.mx4_quantize(W1))[:, 0]
    factors = torch.tensor([1.0, 0.75, 1.5, 2.0, 2.0 ** 32, 2.0 ** 57, 2.0 ** 63, 0.0, -1.5 * 2.0 ** 30], dtype=torch.float64, device=DEV)
    factors = factors.repeat(-(-R // 9))[:R]
    z = torch.zeros(R, d, dtype=BF16, device=DEV)
    z[:, 0] = factors.to(BF16)
    x = (factors[:, None] * v).float().double()
    u2 = 2 * (2 / math.pi) ** 0.5 * (x + 0.044715 * x ** 3)
    h = x / (1 + torch.exp(-u2))
    assert torch.equal(h.isnan().any(1), factors.abs() * 2.0 ** 90 >= 2.0 ** 128)
    a = (h.abs().reshape(R, -1, 32) / torch.exp2(ref.mx4_scale_exponents(h))[..., None]).nan_to_num(0.0)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=DEV)
    assert ((a[..., None] / mids - 1).abs() > 2e-5).all()
    top = a.amax(2)
    assert ((top == 0) | ((top > 4.001) & (top < 7.999)) | (top < 3.999)).all()  # (the last: at the smallest scale)
    want = ref.mx4_values(*ref.mx4_quantize(h)).to(BF16)
    want[h.isnan().any(1)] = float("nan")  # a row's sum over its hidden values
    got = dg.dg_ffw_mx4(z, w1, w2)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(), want.nan_to_num()), (got.double() - want.double()).abs().nan_to_num().max()


@pytest.mark.parametrize("R", [8, 200])
def test_block_nan_and_infinite_rows_stay_alone(R):
    g = gen(13)
    z = randn(g, R, 128, dtype=BF16)
    w1, w2 = dg.dg_mx4_quantize(randn(g, 256, 128, std=0.1)), dg.dg_mx4_quantize(randn(g, 128, 256, std=0.1))
    clean = dg.dg_ffw_mx4(z, w1, w2)
    z[3, 5], z[6, 100] = float("nan"), float("-inf")
    got = dg.dg_ffw_mx4(z, w1, w2)
    keep = torch.ones(R, dtype=torch.bool, device=DEV)
    keep[3] = keep[6] = False
    assert got[~keep].isnan().all() and torch.equal(got[keep], clean[keep])


def test_block_is_its_parts_up_to_the_hidden_rounding():
    # against the bf16 block on the same (dequantised) weights: 4-bit rounding of the input and of the
    # hidden layer is the only difference, each about 10 % of a value, so the results are strongly alike
    g = gen(12)
    R, d, dff = 64, 256, 1024
    z = randn(g, R, d, dtype=BF16)
    W1, W2 = randn(g, d, dff, std=d ** -0.5, dtype=BF16), randn(g, dff, d, std=dff ** -0.5, dtype=BF16)
    q1, q2 = dg.dg_mx4_quantize(W1.t().contiguous()), dg.dg_mx4_quantize(W2.t().contiguous())
    four = dg.dg_ffw_mx4(z, q1, q2).double()
    full, _ = dg.dg_ffw(z, dg.dg_mx4_dequantize(*q1).t().contiguous(), dg.dg_mx4_dequantize(*q2).t().contiguous())
    cos = (four * full.double()).sum() / (four.norm() * full.double().norm())
    assert cos.item() > 0.97


# ------------------------------------------------------------------------------------ how they are called
def test_self_conditioning_path_as_used():
    """z = softmax(L) E, norm, 4-bit block, norm with a drop gate into the stream, norm of the next block,
    and the gradients back to the stream, the block's output, the gate and the weights."""
    g = gen(20)
    B, C, V, d, dff = 2, 16, 600, 128, 512
    R = B * C
    L, E = randn(g, R, V, std=2.0), randn(g, V, d, std=0.02)
    x = randn(g, R, d, dtype=BF16)
    w_in, w_post, w_pre = (randn(g, d, dtype=BF16, std=0.1, mean=1.0) for _ in range(3))
    W1, W2 = randn(g, dff, d, std=d ** -0.5), randn(g, d, dff, std=dff ** -0.5)
    w1, w2 = dg.dg_mx4_quantize(W1), dg.dg_mx4_quantize(W2)
    gate = torch.stack([torch.ones(d, device=DEV), torch.zeros(d, device=DEV)]).to(BF16)  # keep, drop
    z = dg.dg_selfcond(L, E, C)
    a = dg.dg_block_norm(z, w_in)
    y = dg.dg_ffw_mx4(a["h"], w1, w2)
    out = dg.dg_block_norm(x, w_pre, y=y, w_post=w_post, gate=gate, C=C, res_scale=0.5)
    check_forward(z, None, None, None, w_in, C, 1.0, torch.tensor(1e-6, dtype=F32).item(), a)
    v = [ref.mx4_values(*ref.mx4_unpack(*w)) for w in (w1, w2)]
    check_block(a["h"], w1, v[0], w2, v[1], y)
    check_forward(x, y, w_post, gate, w_pre, C, 0.5, torch.tensor(1e-6, dtype=F32).item(), out)
    assert torch.equal(out["x"][C:], x[C:])  # the dropped canvas keeps its stream
    dxo, dh = randn(g, R, d, dtype=BF16, std=0.1), randn(g, R, d, dtype=BF16, std=0.1)
    back = dg.dg_block_norm_backward(dxo, dh, out["x"], w_pre, rstd_x=out["rstd_x"], y=y, w_post=w_post, gate=gate,
                                     rstd_y=out["rstd_y"], C=C, res_scale=0.5)
    check_backward((dxo, dh, out["x"], w_pre, out["rstd_x"], y, w_post, gate, out["rstd_y"]), C, 0.5, back, BF16)
    assert back["dy"][C:].abs().max().item() == 0.0
    zg = dg.dg_block_norm_backward(None, back["dy"], z, w_in, rstd_x=a["rstd_x"])
    check_backward((None, back["dy"], z, w_in, a["rstd_x"], None, None, None, None), R, 1.0, zg, BF16)
    assert dg.dg_device_error() == 0


def test_other_stream_two_streams_and_graphs():
    g = gen(21)
    R, d, dff = 200, 512, 1024
    w1, w2 = dg.dg_mx4_quantize(randn(g, dff, d)), dg.dg_mx4_quantize(randn(g, d, dff, std=0.05))
    zs = [randn(g, R, d, dtype=BF16) for _ in range(4)]
    w = randn(g, d, dtype=BF16)
    want = [dg.dg_ffw_mx4(z, w1, w2) for z in zs]
    args = backward_case(4, 50, d, BF16, F32, "both", True)
    grads = run_backward(args, 50)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got, back = [], []
    for k in range(40):  # calls on four streams at once share no scratch
        with torch.cuda.stream(streams[k % 4]):
            got.append(dg.dg_ffw_mx4(zs[k % 4], w1, w2))
        back.append(run_backward(args, 50, stream=streams[(k + 1) % 4]))
    torch.cuda.synchronize()
    for k in range(40):
        assert torch.equal(got[k], want[k % 4])
        assert all(torch.equal(back[k][n], grads[n]) for n in grads)
    graphs, outs = [], []
    static = [z.clone() for z in zs[:2]]
    for k in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            n = dg.dg_block_norm(static[k], w)
            y = dg.dg_ffw_mx4(n["h"], w1, w2)
            o = dg.dg_block_norm(static[k], w, y=y, w_post=w)
            b = dg.dg_block_norm_backward(o["x"], o["h"], o["x"], w, rstd_x=o["rstd_x"], y=y, w_post=w, rstd_y=o["rstd_y"])
        graphs.append(gr)
        outs.append((y, o, b))

    def eager(z):
        n = dg.dg_block_norm(z, w)
        y = dg.dg_ffw_mx4(n["h"], w1, w2)
        o = dg.dg_block_norm(z, w, y=y, w_post=w)
        return y, o, dg.dg_block_norm_backward(o["x"], o["h"], o["x"], w, rstd_x=o["rstd_x"], y=y, w_post=w, rstd_y=o["rstd_y"])

    for rep in range(3):
        for k in range(2):
            static[k].copy_(zs[(rep + k) % 4])
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            ye, oe, be = eager(zs[(rep + k) % 4])
            assert torch.equal(outs[k][0], ye)
            assert all(torch.equal(outs[k][1][n], oe[n]) for n in oe) and all(torch.equal(outs[k][2][n], be[n]) for n in be)
    assert dg.dg_device_error() == 0


def test_first_call_of_a_process_may_be_captured():
    # nothing that a first call sets up needs a call outside of a capture
    code = """
import torch, discrete_diffusion_lm_b200 as dg
z = torch.randn(200, 2048, device='cuda').bfloat16(); big = torch.randn(2000, 2048, device='cuda').bfloat16()
w = torch.ones(2048, device='cuda'); q = torch.zeros(2048, 1024, dtype=torch.uint8, device='cuda'); s = torch.full((16, 16, 32, 16), 127, dtype=torch.uint8, device='cuda')
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = dg.dg_block_norm(big, w); y = dg.dg_ffw_mx4(z, (q, s), (q, s)); o = dg.dg_ffw_mx4(big, (q, s), (q, s))
    b = dg.dg_block_norm_backward(None, big, big, w, rstd_x=a['rstd_x'])
g.replay(); torch.cuda.synchronize()
assert dg.dg_device_error() == 0 and y.abs().max().item() == 0 and torch.equal(a['h'], dg.dg_block_norm(big, w)['h'])
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


def test_offsets_beyond_32_bits():
    # the last rows of arrays of more than 2^31 elements
    rows, d = 300_000, 8192
    x = torch.zeros(rows, d, dtype=BF16, device=DEV)
    x[-3:] = randn(gen(30), 3, d, dtype=BF16)
    w = torch.ones(d, dtype=BF16, device=DEV)
    out = dg.dg_block_norm(x, w)
    assert torch.equal(out["h"][-3:], dg.dg_block_norm(x[-3:].contiguous(), w)["h"]) and out["h"][:-3].abs().max().item() == 0
    res = dg.dg_block_norm_backward(None, x, x, w, rstd_x=out["rstd_x"])
    small = dg.dg_block_norm_backward(None, x[-3:].contiguous(), x[-3:].contiguous(), w, rstd_x=out["rstd_x"][-3:].contiguous())
    assert torch.equal(res["dx"][-3:], small["dx"])
    del out, res
    codes, scales = dg.dg_mx4_quantize(x)
    want = dg.dg_mx4_quantize(x[-3:].contiguous())
    r = torch.arange(rows - 3, rows, device=DEV)
    assert torch.equal(codes[-3:], want[0])
    assert torch.equal(ref.mx4_unpack(codes[-3:], dg.dg_mx4_quantize(x[-3:].contiguous())[1])[1], scales[r // 128, :, r % 32].reshape(3, d // 128, 4, 4)[
        torch.arange(3, device=DEV), :, r // 32 % 4].reshape(3, d // 32).long())
    back = dg.dg_mx4_dequantize(codes, scales)
    assert torch.equal(back[-3:], dg.dg_mx4_dequantize(*want))
    del x, back, codes, scales
    g = gen(31)
    M, N = 70_000, 32_768
    (a, av), (w2, wv) = random_mx4(g, M, 32), random_mx4(g, N, 32)
    out = dg.dg_mx4_matmul(a, w2)
    want = av[-2:] @ wv.T
    within(out[-2:], want, 130 * U * (av[-2:].abs() @ wv.abs().T) + half_step(BF16) * want.abs(), "last rows")


def test_launch_counts():
    g = gen(22)
    x, w = randn(g, 8, 64, dtype=BF16), randn(g, 64, dtype=BF16)
    w1 = dg.dg_mx4_quantize(randn(g, 64, 64))
    torch.cuda.synchronize()

    def count(f):
        n = dg.dg_launch_count()
        f()
        return dg.dg_launch_count() - n

    assert count(lambda: dg.dg_block_norm(x, w)) == 1
    assert count(lambda: dg.dg_mx4_quantize(x)) == 1
    assert count(lambda: dg.dg_mx4_matmul(w1, w1)) == 1
    assert count(lambda: dg.dg_ffw_mx4(x, w1, w1)) == 2
    assert count(lambda: dg.dg_ffw_mx4(x.repeat(5, 1), w1, w1)) == 3
    r = dg.dg_block_norm(x, w)["rstd_x"]
    assert count(lambda: dg.dg_block_norm_backward(None, x, x, w, rstd_x=r)) == 2
