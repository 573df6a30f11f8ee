"""Cases of the operators around the feed-forward block: its norms with gate and residual (forward and
backward), microscaled 4-bit quantisation and products, and the feed-forward block in that format.

`run` computes a case in plain torch operations, or, where `own` is true, through the library's calls.
Microscaled 4-bit values (OCP Microscaling Formats, MXFP4): blocks of 32 values along a row share a power
of two 2^(c - 127) kept as the byte c; a value is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign, two to a
byte, the lower index in the low half.  Scale bytes lie in tiles of 128 rows x 4 blocks: byte
(r % 32) * 16 + (r // 32 % 4) * 4 + block % 4 of tile (r // 128, block // 4), the padding holding 127.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one small canvas of the float workload: a call whose latency is all that counts
        {"name": "norm tiny", "op": "norm", "B": 1, "C": 16, "d": 64, "dtype": "f32", "params": "f32", "mode": "both", "gated": True},
        # the residual streams of 16 canvases between two blocks
        {"name": "norm batched", "op": "norm", "B": 16, "C": 256, "d": 2048, "dtype": "bf16", "params": "bf16", "mode": "both", "gated": True},
        # ragged training rows: odd canvas length, a width off every power of two, no gate
        {"name": "norm back ragged", "op": "norm_back", "B": 3, "C": 37, "d": 1000, "dtype": "f32", "params": "f32", "mode": "both", "gated": False},
        # a training step of 8 sequences of 512 prompt tokens and 4 canvases of 256
        {"name": "norm back train", "op": "norm_back", "B": 8, "C": 1536, "d": 2048, "dtype": "bf16", "params": "f32", "mode": "both", "gated": True},
        # activations of one canvas as they enter the 4-bit block
        {"name": "quantise canvas", "op": "quantise", "R": 256, "K": 2048, "dtype": "bf16"},
        # a weight matrix quantised from its float master copy
        {"name": "quantise weight", "op": "quantise", "R": 8192, "K": 2048, "dtype": "f32"},
        # one token through the widening product
        {"name": "product token", "op": "product", "M": 1, "N": 8192, "K": 2048, "dtype": "bf16"},
        # a ragged row count through the narrowing product, kept in 32 bits
        {"name": "product ragged", "op": "product", "M": 200, "N": 1000, "K": 4096, "dtype": "f32"},
        # 16 canvases through the widening product: the largest
        {"name": "product batched", "op": "product", "M": 4096, "N": 8192, "K": 2048, "dtype": "bf16"},
        # the feed-forward block on a single token, on one canvas, on 16 canvases of the middle width
        {"name": "block token", "op": "block", "R": 1, "d": 1024, "ff": 4096},
        {"name": "block canvas", "op": "block", "R": 256, "d": 2048, "ff": 8192},
        {"name": "block batched", "op": "block", "R": 4096, "d": 1024, "ff": 4096},
    ]


def _log(rng, lo, hi, step=1):
    """A whole multiple of `step`, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + step))) // step * step))) // step * step


def draw(rng):
    op = rng.choice(["norm", "norm_back", "quantise", "product", "block"])
    if op in ("norm", "norm_back"):
        d = _log(rng, 64, 8192, 8)
        rows = _log(rng, 1, min(16384, 12288 * 2048 // d))
        C = _log(rng, 1, rows)
        return {"op": op, "B": max(1, min(256, rows // C)), "C": C, "d": d, "dtype": rng.choice(["bf16", "f32"]) if rows * d <= 1 << 23 else "bf16",
                "params": rng.choice(["bf16", "f32"]), "mode": rng.choice(["both", "both", "both", "pre", "post"]), "gated": rng.random() < 0.6}
    if op == "quantise":
        K = _log(rng, 32, 16384, 32)
        return {"op": op, "R": _log(rng, 1, min(8192, 8192 * 2048 // K)), "K": K, "dtype": rng.choice(["bf16", "f32"])}
    if op == "product":
        K, N = _log(rng, 32, 8192, 32), _log(rng, 8, 8192, 8)
        return {"op": op, "M": _log(rng, 1, max(1, min(8192, 4096 * 8192 * 2048 // (K * N)))), "N": N, "K": K, "dtype": rng.choice(["bf16", "f32"])}
    d = _log(rng, 64, 2048, 64)
    return {"op": op, "R": _log(rng, 1, min(4096, 4096 * 1024 * 2048 // (d * d))), "d": d, "ff": d * rng.choice([2, 3, 4])}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 11)
    return g


def _normal(g, *shape, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=g, device="cuda") * std + mean


def _quantise(x):
    """Codes [R, K/2] and scale bytes [R, K/32] of x [R, K]: the scale is the power of two two below the
    largest magnitude's, values go to the nearest (ties to the even code), beyond 6 to 6; a block
    with a NaN or an infinity has the scale byte 255."""
    R, K = x.shape
    b = x.float().reshape(R, K // 32, 32)
    top = b.abs().amax(dim=2)
    fine = torch.isfinite(top)
    e = (torch.frexp(torch.where(fine, top, torch.ones_like(top)))[1] - 3).clamp(min=-127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    s = torch.where(fine[..., None], b, torch.zeros_like(b)) * torch.ldexp(torch.ones_like(top), -e)[..., None]
    a = s.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    code = (code | (torch.signbit(s).to(torch.uint8) << 3)).reshape(R, K // 2, 2)
    scale = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), scale


def _tiled(scale):
    """Scale bytes [R, K/32] as tiles of 128 rows x 4 blocks."""
    R, n = scale.shape
    rt, kt = -(-R // 128), -(-n // 4)
    p = torch.full((rt * 128, kt * 4), 127, dtype=torch.uint8, device=scale.device)
    p[:R, :n] = scale
    return p.reshape(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(rt, kt, 32, 16).contiguous()


def _untiled(tiles, R, n):
    rt, kt = tiles.shape[:2]
    return tiles.reshape(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:R, :n]


def _values(codes, scale):
    """The values that codes [R, K/2] and scale bytes [R, K/32] stand for, in 32 bits."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    R, half = codes.shape
    v = table[torch.stack([codes & 15, codes >> 4], dim=2).to(torch.int64)].reshape(R, half // 16, 32)
    s = torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.to(torch.int32) - 127)
    s = torch.where(scale == 255, torch.full_like(s, math.nan), s)
    return (v * s[..., None]).reshape(R, 2 * half)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("norm", "norm_back"):
        B, C, d, mode = case["B"], case["C"], case["d"], case["mode"]
        R, T, P = B * C, DTYPES[case["dtype"]], DTYPES[case["params"]]
        both, back = mode == "both", op == "norm_back"
        # a residual stream has a few wide channels; a block's output is smaller and its weights are near 1
        x = (_normal(g, R, d) * (1.0 + 4.0 * (_normal(g, d) > 2.0))).to(T)
        y = (_normal(g, R, d, std=0.5)).to(T) if mode != "pre" else None
        w_post = _normal(g, d, std=0.1, mean=1.0).to(P) if mode != "pre" else None
        w_pre = _normal(g, d, std=0.1, mean=1.0).to(P) if mode != "post" else None
        gate = _normal(g, B, d, std=0.5).to(P) if case["gated"] and mode != "pre" else None
        s = {"case": case, "x": x, "y": y, "w_post": w_post, "w_pre": w_pre, "gate": gate, "C": C, "scale": 0.7}
        if back:  # what the forward pass kept, and gradients of a mean loss
            x64 = x.double()
            if y is not None:
                s["rstd_y"] = ((y.double() ** 2).mean(1) + EPS).rsqrt().float()
                u = y.double() * s["rstd_y"].double()[:, None] * w_post.double() * 0.7
                x64 = x64 + (u if gate is None else u * gate.double().repeat_interleave(C, 0))
                s["x"] = x64.to(T)
            s["rstd_x"] = ((s["x"].double() ** 2).mean(1) + EPS).rsqrt().float() if mode != "post" else None
            s["dx_out"] = _normal(g, R, d, std=1e-2).to(T)
            s["dh"] = _normal(g, R, d, std=1e-2).to(T) if mode != "post" else None
        return s
    if op == "quantise":
        # rows of different size, as activations and weights have
        return {"case": case, "x": (_normal(g, case["R"], case["K"]) * torch.exp(_normal(g, case["R"], 1))).to(DTYPES[case["dtype"]])}
    if op == "product":
        a, w = _quantise(_normal(g, case["M"], case["K"])), _quantise(_normal(g, case["N"], case["K"], std=case["K"] ** -0.5))
        return {"case": case, "a": (a[0], _tiled(a[1])), "w": (w[0], _tiled(w[1]))}
    d, ff = case["d"], case["ff"]
    w1, w2 = _quantise(_normal(g, ff, d, std=d ** -0.5)), _quantise(_normal(g, d, ff, std=ff ** -0.5))
    return {"case": case, "z": _normal(g, case["R"], d).to(torch.bfloat16), "w1": (w1[0], _tiled(w1[1])), "w2": (w2[0], _tiled(w2[1]))}


def _plain_norm(s):
    x, y, gate, T = s["x"].float(), s["y"], s["gate"], s["x"].dtype
    out = {}
    if y is not None:
        r = (y.float().square().mean(1) + EPS).rsqrt()
        u = y.float() * r[:, None] * s["w_post"].float()
        if gate is not None:
            u = u * gate.float().repeat_interleave(s["C"], 0)
        x = x + s["scale"] * u
        out["x"], out["rstd_y"] = x.to(T), r
    if s["w_pre"] is not None:
        r = (x.square().mean(1) + EPS).rsqrt()
        out["h"], out["rstd_x"] = (x * r[:, None] * s["w_pre"].float()).to(T), r
    return out


def _plain_norm_back(s):
    x, y, gate, T, k = s["x"].float(), s["y"], s["gate"], s["x"].dtype, s["scale"]
    R, d = x.shape
    out, g = {}, s["dx_out"].float()
    if s["w_pre"] is not None:
        n, dh = x * s["rstd_x"][:, None], s["dh"].float()
        t = dh * s["w_pre"].float()
        g = g + s["rstd_x"][:, None] * (t - n * (t * n).mean(1, keepdim=True))
        out["dw_pre"] = (dh.double() * n.double()).sum(0).float()
    out["dx"] = g.to(T)
    if y is not None:
        v, w = y.float() * s["rstd_y"][:, None], s["w_post"].float()
        per = (g.double() * v.double()).reshape(R // s["C"], s["C"], d).sum(1)
        t = k * g * w
        if gate is None:
            out["dw_post"] = (k * per.sum(0)).float()
        else:
            t = t * gate.float().repeat_interleave(s["C"], 0)
            out["dw_post"] = (k * per * gate.double()).sum(0).float()
            out["dgate"] = (k * per * w.double()).float()
        out["dy"] = (s["rstd_y"][:, None] * (t - v * (t * v).mean(1, keepdim=True))).to(T)
    return out


def _plain_gelu(x):
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _operand(q, K):
    """A quantised matrix [R, K] with tiled scales, in 32 bits."""
    return _values(q[0], _untiled(q[1], q[0].shape[0], K // 32))


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import discrete_diffusion_lm_b200 as dg

        if op == "norm":
            return dg.dg_block_norm(s["x"], s["w_pre"], y=s["y"], w_post=s["w_post"], gate=s["gate"], C=s["C"], res_scale=s["scale"], eps=EPS)
        if op == "norm_back":
            if s["y"] is None:
                return dg.dg_block_norm_backward(s["dx_out"], s["dh"], s["x"], s["w_pre"], rstd_x=s["rstd_x"])
            return dg.dg_block_norm_backward(s["dx_out"], s["dh"], s["x"], s["w_pre"], rstd_x=s["rstd_x"], y=s["y"], w_post=s["w_post"],
                                             gate=s["gate"], rstd_y=s["rstd_y"], C=s["C"], res_scale=s["scale"])
        if op == "quantise":
            codes, scales = dg.dg_mx4_quantize(s["x"])
            return dg.dg_mx4_dequantize(codes, scales, dtype=s["x"].dtype)
        if op == "product":
            return dg.dg_mx4_matmul(s["a"], s["w"], dtype=DTYPES[c["dtype"]])
        return dg.dg_ffw_mx4(s["z"], s["w1"], s["w2"])
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_back":
        return _plain_norm_back(s)
    if op == "quantise":
        return _values(*_quantise(s["x"])).to(s["x"].dtype)
    if op == "product":
        return (_operand(s["a"], c["K"]) @ _operand(s["w"], c["K"]).t()).to(DTYPES[c["dtype"]])
    z = _values(*_quantise(s["z"]))
    hidden = _values(*_quantise(_plain_gelu(z @ _operand(s["w1"], c["d"]).t())))
    return (hidden @ _operand(s["w2"], c["ff"]).t()).to(torch.bfloat16)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        R, d, e, p = case["B"] * case["C"], case["d"], 4 if case["dtype"] == "f32" else 2, 4 if case["params"] == "f32" else 2
        mode, back = case["mode"], op == "norm_back"
        gate = case["B"] * d if case["gated"] and mode != "pre" else 0
        params = (2 if mode == "both" else 1) * d + gate
        if not back:  # x, y in and the new stream, h out
            return {"bytes": R * d * e * {"both": 4, "post": 3, "pre": 2}[mode] + params * p + R * 4 * (2 if mode == "both" else 1),
                    "flops": R * d * {"both": 9, "post": 5, "pre": 4}[mode]}
        # the two upstream gradients, the stream and y in, dx and dy out, the parameters' gradients out
        return {"bytes": R * d * e * {"both": 6, "post": 4, "pre": 4}[mode] + params * (p + 4) + R * 4 * (2 if mode == "both" else 1),
                "flops": R * d * {"both": 20, "post": 11, "pre": 9}[mode]}
    if op == "quantise":  # the values in and out, the codes and scales that the caller keeps
        n, e = case["R"] * case["K"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": n * (2 * e + 0.5 + 1 / 32), "flops": 4 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * (0.5 + 1 / 32) + M * N * (4 if case["dtype"] == "f32" else 2), "flops": 2 * M * N * K}
    R, d, ff = case["R"], case["d"], case["ff"]
    return {"bytes": 2 * d * ff * (0.5 + 1 / 32) + R * d * 4, "flops": 4 * R * d * ff}


def _power(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)


def _exact_values(x):
    """What x [R, K] becomes in the 4-bit format, in 64 bits: each block's values rounded to a multiple of
    the spacing at their size (half to even), on the grid that the block's largest magnitude sets."""
    R, K = x.shape
    b = x.double().reshape(R, -1, 32)
    top = b.abs().max(dim=2, keepdim=True).values
    unit = _power(torch.frexp(top.clamp(min=2.0 ** -125))[1] - 3)
    a = b / unit
    step = _power(torch.frexp(a.abs().clamp(min=1.0))[1] - 2)
    return ((torch.round(a / step) * step).clamp(-6.0, 6.0) * unit).reshape(R, K)


def _exact_operand(q, K):
    codes, tiles = q
    R = codes.shape[0]
    r, k = torch.arange(R, device="cuda")[:, None], torch.arange(K, device="cuda")[None, :]
    nib = ((codes[:, :, None].int() >> torch.tensor([0, 4], device="cuda")) & 15).reshape(R, K)
    m, e = (nib & 1).double(), (nib >> 1) & 3
    v = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * _power(e - 1)) * (1.0 - 2.0 * (nib >> 3).double())
    blk = k // 32
    byte = ((r // 128 * tiles.shape[1] + blk // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + blk % 4).long()
    return v * _power(tiles.reshape(-1)[byte].int() - 127)


def _exact_normed(v):
    return v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantise":
        return _exact_values(s["x"])
    if op == "product":
        return _exact_operand(s["a"], case["K"]).matmul(_exact_operand(s["w"], case["K"]).T)
    if op == "block":
        t = _exact_values(s["z"]).matmul(_exact_operand(s["w1"], case["d"]).T)
        t = t / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (t + 0.044715 * t.pow(3))))
        return _exact_values(t).matmul(_exact_operand(s["w2"], case["ff"]).T)
    B, C, d = case["B"], case["C"], case["d"]
    f = lambda t: None if t is None else t.double()  # noqa: E731
    x, y, w_post, w_pre = f(s["x"]), f(s["y"]), f(s["w_post"]), f(s["w_pre"])
    gate = torch.ones(B, 1, d, dtype=torch.float64, device="cuda") if s["gate"] is None else f(s["gate"])[:, None, :]
    if op == "norm":
        out = {}
        if y is not None:
            out["rstd_y"] = (y.pow(2).sum(1) / d + EPS).pow(-0.5)
            x = x + (s["scale"] * gate * (_exact_normed(y) * w_post).reshape(B, C, d)).reshape(B * C, d)
            out["x"] = x
        if w_pre is not None:
            out["h"], out["rstd_x"] = _exact_normed(x) * w_pre, (x.pow(2).sum(1) / d + EPS).pow(-0.5)
        return out
    # the gradients by reverse differentiation of the forward formulas at the kept stream
    out = {}
    total = f(s["dx_out"])
    with torch.enable_grad():
        if w_pre is not None:
            x.requires_grad_(True)
            w_pre.requires_grad_(True)
            gx, gw = torch.autograd.grad((_exact_normed(x) * w_pre * f(s["dh"])).sum(), [x, w_pre])
            total, out["dw_pre"] = total + gx, gw
        out["dx"] = total
        if y is not None:
            leaves = [y.requires_grad_(True), w_post.requires_grad_(True), gate.requires_grad_(True)]
            u = (s["scale"] * gate * (_exact_normed(y) * w_post).reshape(B, C, d)).reshape(B * C, d)
            out["dy"], out["dw_post"], gg = torch.autograd.grad((u * total).sum(), leaves)
            if s["gate"] is not None:
                out["dgate"] = gg.reshape(B, d)
    return out
