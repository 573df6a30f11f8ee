"""Plain 64-bit restatements of the operators around the feed-forward block: the norms with gate and
residual scale and their gradients, the MXFP4 format, and the products and the block in it.  They run
on the tensors' own device, in torch.float64, and share no code with the library."""
from __future__ import annotations

import torch

U = 2.0 ** -24  # half a step of fp32


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def norm_rows(v, eps):
    v = v.double()
    return v / (v.pow(2).mean(1, keepdim=True) + eps).sqrt()


def per_row(gate, C, R, d, device):
    if gate is None:
        return torch.ones(R, d, dtype=torch.float64, device=device)
    return gate.double().repeat_interleave(C, 0)


def block_norm(x, y, w_post, gate, C, s, eps):
    """The stream after the block and the magnitude of its two terms."""
    R, d = x.shape
    u = s * per_row(gate, C, R, d, x.device) * w_post.double() * norm_rows(y, eps)
    return x.double() + u, x.double().abs() + u.abs()


def block_norm_grads(dx_out, dh, x, w_pre, rstd_x, y, w_post, gate, rstd_y, C, s):
    """Gradients by the formulas, and for each a magnitude that its fp32 rounding errors scale with
    (the same sums over absolute values)."""
    R, d = x.shape if x is not None else dx_out.shape
    dev = (x if x is not None else dx_out).device
    out, mag = {}, {}
    g = torch.zeros(R, d, dtype=torch.float64, device=dev) if dx_out is None else dx_out.double()
    a = g.abs()
    if w_pre is not None:
        rx = rstd_x.double()[:, None]
        m, t = x.double() * rx, dh.double() * w_pre.double()
        g = g + rx * (t - m * (t * m).mean(1, keepdim=True))
        a = a + rx * (t.abs() + m.abs() * (t * m).abs().mean(1, keepdim=True))
        out["dw_pre"], mag["dw_pre"] = (dh.double() * m).sum(0), (dh.double() * m).abs().sum(0)
    out["dx"], mag["dx"] = g, a
    if y is not None:
        ry = rstd_y.double()[:, None]
        v, w, gr = y.double() * ry, w_post.double(), per_row(gate, C, R, d, dev)
        c = s * gr * w
        out["dy"] = ry * (c * g - v * (c * g * v).mean(1, keepdim=True))
        mag["dy"] = ry * (c.abs() * a + v.abs() * (c * v).abs().mul(a).mean(1, keepdim=True))
        out["dw_post"], mag["dw_post"] = (s * gr * g * v).sum(0), (s * gr * v).abs().mul(a).sum(0)
        if gate is not None:
            out["dgate"] = (s * w * g * v).reshape(R // C, C, d).sum(1)
            mag["dgate"] = (s * w * v).abs().mul(a).reshape(R // C, C, d).sum(1)
    return out, mag


# ------------------------------------------------------------------------------------ MXFP4
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def mx4_scale_exponents(x):
    """e of every block of 32 of x [R, K], float64 [R, K/32]; NaN where the block has a NaN or an infinity."""
    top = x.double().reshape(x.shape[0], -1, 32).abs().amax(2)
    m, ex = torch.frexp(top)
    e = torch.where(top == 0, torch.full_like(top, -127.0), (ex - 1 - 2).double().clamp(min=-127.0))
    return torch.where(torch.isfinite(top), e, torch.full_like(top, float("nan")))


def mx4_quantize(x):
    """Codes (int64 [R, K], one value each) and scale bytes (int64 [R, K/32]) by exhaustive search of the
    nearest magnitude; ties go to the even code."""
    R, K = x.shape
    e = mx4_scale_exponents(x)
    bad = torch.isnan(e)
    e = torch.where(bad, torch.zeros_like(e), e)
    b = x.double().reshape(R, -1, 32)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    a = torch.ldexp(b.abs(), -e[..., None].to(torch.int32))
    mags = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    dist = (a[..., None] - mags).abs()
    best = dist.amin(-1, keepdim=True)
    odd = torch.arange(8, device=x.device) % 2
    # among the nearest take an even code: an odd one pays a penalty below any difference of distances
    code = torch.where(dist == best, odd.double(), torch.full_like(dist, 9.0)).argmin(-1)
    code = code + 8 * torch.signbit(b).long()
    code = torch.where(bad[..., None], torch.zeros_like(code), code)
    return code.reshape(R, K), torch.where(bad, torch.full_like(e, 255.0), e + 127).long()


def mx4_values(code, scale):
    """The float64 values of codes [R, K] and scale bytes [R, K/32]."""
    R, K = code.shape
    mags = torch.tensor(MAGNITUDES, dtype=torch.float64, device=code.device)
    v = mags[code & 7] * torch.where(code >= 8, -1.0, 1.0).double()
    s = torch.ldexp(torch.ones_like(scale, dtype=torch.float64), (scale - 127).to(torch.int32))
    s = torch.where(scale == 255, torch.full_like(s, float("nan")), s)
    return (v.reshape(R, -1, 32) * s[..., None]).reshape(R, K)


def mx4_pack(code, scale):
    """Byte tensors in the library's layout, written index by index from its definition."""
    R, K = code.shape
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    tiles = torch.full((-(-R // 128), -(-K // 128), 32, 16), 127, dtype=torch.uint8, device=code.device)
    r = torch.arange(R, device=code.device)[:, None].expand(R, K // 32)
    q = torch.arange(K // 32, device=code.device)[None, :].expand(R, K // 32)
    tiles[r // 128, q // 4, r % 32, (r // 32 % 4) * 4 + q % 4] = scale.to(torch.uint8)
    return codes, tiles


def mx4_unpack(codes, tiles):
    R, half = codes.shape
    K = 2 * half
    code = torch.stack([codes & 15, codes >> 4], 2).reshape(R, K).long()
    r = torch.arange(R, device=codes.device)[:, None].expand(R, K // 32)
    q = torch.arange(K // 32, device=codes.device)[None, :].expand(R, K // 32)
    return code, tiles[r // 128, q // 4, r % 32, (r // 32 % 4) * 4 + q % 4].long()


def gelu(x):
    return 0.5 * x * (1.0 + torch.tanh((2.0 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3)))
