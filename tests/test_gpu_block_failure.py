"""Failure detection of the operators around the feed-forward block, without a GPU fault: copies that are
never issued make the kernels' bounded waits run out (about 10 ms), dg_device_error() reports code 1,
and the next call gives what a call before gave."""
import pytest
import torch

import discrete_diffusion_lm_b200 as dg

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMIT = 20_000_000  # SM cycles, about 10 ms


def stream():
    return torch.cuda.current_stream().cuda_stream


# one CTA per tile; K split over two and four CTAs; pairs of CTAs with 128 and 256 columns
@pytest.mark.parametrize("M,N,K,block", [(16, 128, 256, 0), (128, 8192, 2048, 5), (5, 512, 4096, 9), (200, 4096, 2048, 7), (2048, 4096, 1024, 3)])
def test_product_stall(M, N, K, block):
    g = torch.Generator(device=DEV).manual_seed(1)
    a, w = (dg.dg_mx4_quantize(torch.randn(r, K, generator=g, device=DEV)) for r in (M, N))
    want = dg.dg_mx4_matmul(a, w)
    assert dg.dg_device_error() == 0
    out = torch.empty_like(want)
    args = [t.data_ptr() for t in (*a, *w)] + [M, N, K, out.data_ptr(), dg.DG_BF16, stream()]
    assert dg.lib().dg_test_mx4_stall(*args, block, LIMIT) == 0, dg.dg_last_error()
    assert dg.dg_device_error() == 1
    assert dg.dg_device_error() == 0
    # past the last block nothing is left out, and the limit is long enough
    assert dg.lib().dg_test_mx4_stall(*args, 1 << 20, LIMIT) == 0
    assert dg.dg_device_error() == 0 and torch.equal(out, want)
    assert torch.equal(dg.dg_mx4_matmul(a, w), want)


# the same with the kernel that each size is meant for: (CTAs that share K, or 0 for pairs; columns of a tile)
@pytest.mark.parametrize("M,N,K,block,plan", [
    (16, 128, 256, 0, (1, 128)), (1, 8192, 2048, 2, (2, 128)), (1, 8192, 2048, 5, (2, 128)), (100, 4864, 6624, 15, (2, 128)),
    (200, 2432, 6624, 4, (2, 128)), (5, 512, 4096, 9, (4, 128)), (100, 1024, 6624, 25, (4, 128)),
    (200, 4096, 2048, 7, (0, 128)), (2048, 4096, 1024, 3, (0, 256))])
def test_product_stall_of_every_kernel(M, N, K, block, plan):
    got = torch.zeros(2, dtype=torch.int32)
    assert dg.lib().dg_test_mx4_plan(M, N, K, got[0:].data_ptr(), got[1:].data_ptr()) == 0
    assert tuple(got.tolist()) == plan
    test_product_stall(M, N, K, block)


@pytest.mark.parametrize("rows,d", [(1500, 128), (2000, 512), (1400, 2048), (1300, 4096)])
def test_norm_stall(rows, d):
    g = torch.Generator(device=DEV).manual_seed(2)
    x, w = torch.randn(rows, d, generator=g, device=DEV).bfloat16(), torch.ones(d, device=DEV)
    want = dg.dg_block_norm(x, w)["h"]
    assert dg.dg_device_error() == 0
    h = torch.empty_like(x)
    assert dg.lib().dg_test_block_norm_stall(x.data_ptr(), dg.DG_BF16, w.data_ptr(), dg.DG_F32, rows, d, h.data_ptr(), LIMIT, stream()) == 0
    assert dg.dg_device_error() == 1
    assert torch.equal(h[rows // 2:], want[rows // 2:])  # rows that other CTAs walk are as ever
    assert torch.equal(dg.dg_block_norm(x, w)["h"], want)
    assert dg.dg_device_error() == 0


# the gradients: groups of one, two, four and eight; walks of several times the ring's slots, and one that fits them
@pytest.mark.parametrize("rows,d", [(30000, 512), (20000, 1024), (9000, 2048), (5000, 4096), (2500, 8192), (500, 1000)])
def test_norm_backward_stall(rows, d):
    g = torch.Generator(device=DEV).manual_seed(3)
    x, dh = (torch.randn(rows, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    w = torch.randn(d, generator=g, device=DEV)
    rstd = dg.dg_block_norm(x, w)["rstd_x"]
    want = dg.dg_block_norm_backward(None, dh, x, w, rstd_x=rstd)
    assert dg.dg_device_error() == 0
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(dg.lib().dg_block_norm_backward_workspace_size(1, rows, d, dg.DG_BF16, 0), dtype=torch.uint8, device=DEV)
    rc = dg.lib().dg_test_block_norm_backward_stall(dh.data_ptr(), x.data_ptr(), dg.DG_BF16, w.data_ptr(), dg.DG_F32, rows, d, rstd.data_ptr(),
                                                    dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), ws.numel(), LIMIT, stream())
    assert rc == 0, dg.dg_last_error()
    assert dg.dg_device_error() == 1
    assert torch.equal(dx[rows // 2:], want["dx"][rows // 2:])  # rows that other CTAs walk are as ever
    again = dg.dg_block_norm_backward(None, dh, x, w, rstd_x=rstd, ws=ws)
    assert all(torch.equal(again[k], want[k]) for k in want)
    assert dg.dg_device_error() == 0


def test_hooks_refuse():
    L = dg.lib()
    assert L.dg_test_mx4_stall(*[1 << 20] * 4, 16, 128, 256, 1 << 20, 1, None, -1, 100) == 1
    assert L.dg_test_mx4_stall(*[1 << 20] * 4, 16, 128, 256, 1 << 20, 1, None, 0, 0) == 1
    assert L.dg_test_block_norm_stall(1 << 20, 1, 1 << 20, 1, 8, 64, 1 << 21, 0, None) == 1


def test_backward_hook_refuses():
    a = 1 << 20
    assert dg.lib().dg_test_block_norm_backward_stall(a, a, 1, a, 1, 8, 64, a, 2 * a, a, a, 1 << 20, 0, None) == 1
    assert dg.lib().dg_test_block_norm_backward_stall(a, a, 1, a, 1, 8, 64, a, 2 * a, a, a, 0, 100, None) == 3
