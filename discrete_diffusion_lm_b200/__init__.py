"""Python binding of libdg, the B200 (sm_100a) sampler library for block-parallel
uniform-noise discrete diffusion (DiffusionGemma Technical Report, sections "Method" and
"Dataset").

The binding only marshals arguments: torch tensors supply device memory and
the current CUDA stream; every step of the computation runs in libdg's CUDA
kernels.  There is no CPU fallback: if libdg.so is missing, a tensor is not on
the GPU, or the device is not sm_100, the calls raise.

Functions carry the C ABI's names (include/dg.h):
    sampler:   dg_sampler_step, dg_sampler_selfcond_step, dg_sampler_step_eb,
               dg_entropy_accept, dg_adaptive_stop, dg_tau_linear, dg_sampler_step_noalloc
    self-conditioning input:   dg_selfcond, dg_ffw, dg_ffw_mx4 (in 4 bits)
    norms around a block:      dg_block_norm, dg_block_norm_backward
    4-bit matrices (MXFP4):    dg_mx4_quantize, dg_mx4_dequantize, dg_mx4_matmul
    training:  dg_forward_noise, dg_canvas_ce, dg_canvas_ce_backward, dg_selfcond_drop
plus the workspace-size queries, dg_last_error, dg_device_error, dg_launch_count, dg_version.

Typical sampler loop over one 256-token canvas (logits from the model each step):

    import discrete_diffusion_lm_b200 as dg
    x = initial_canvas                                   # int32 [256] on the GPU
    for k in range(steps):
        t, dt = 1 - k / steps, 1 / steps
        logits = model(x, z)                             # [256, V] bf16
        out = dg.dg_sampler_selfcond_step(logits, x, E, 256, t, dt, step=k,
                                          inv_tau=dg.dg_tau_linear([t]))
        x, z = out["x_next"], out["z"]                   # next canvas, self-conditioning input

or, with entropy-bounded acceptance and adaptive stopping instead of the Step posterior:

        out = dg.dg_sampler_step_eb(logits, 256, eps=eps, theta=theta, argmax_prev=prev, step=k,
                                    inv_tau=dg.dg_tau_linear([t]))
        if out["stop"].item(): break
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# DG_LIB=checks selects the checks library (device-side index and token-id checks, built with
# `python -m discrete_diffusion_lm_b200.build --checks`); anything else, or unset, the normal one.
LIB_PATH = os.path.join(_PKG, "libdg_checks.so" if os.environ.get("DG_LIB") == "checks" else "libdg.so")

DG_OK = 0
DG_F32, DG_BF16 = 0, 1
DG_SCHED = {"linear": 0, "cosine": 1}
DG_X0 = {"sample": 0, "greedy": 1}
DG_GUMBEL_CHUNK = 512
DG_MAX_CANVASES = 256
DG_MAX_CANVAS_ROWS = 1024
DG_MAX_VOCAB = 1 << 30


class DGError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with status {code}: {msg}")
        self.code = code


_lib = None
_p, _i32, _i64, _u32, _u64, _sz, _int = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                         ctypes.c_uint64, ctypes.c_size_t, ctypes.c_int)
_f32 = ctypes.c_float


def lib() -> ctypes.CDLL:
    """Load libdg.so (built in-tree by discrete_diffusion_lm_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            flag = " --checks" if LIB_PATH.endswith("_checks.so") else ""
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m discrete_diffusion_lm_b200.build{flag}`")
        L = ctypes.CDLL(LIB_PATH)
        L.dg_last_error.restype = ctypes.c_char_p
        L.dg_version.restype = ctypes.c_char_p
        L.dg_launch_count.restype = _u64
        L.dg_device_error.argtypes = [_p]
        L.dg_test_bounded_wait.argtypes = [_u32, _p]
        L.dg_test_merge_stall.argtypes = [_p, _int, _i64, _i32, _i32, _p, _p, _sz, _u32, _p]
        L.dg_test_selfcond_stall.argtypes = [_p, _int, _i64, _i32, _i32, _i32, _p, _p, _p, _int, _i32, _p, _p, _sz,
                                             _p, _i32, _u32]
        L.dg_sampler_step_workspace_size.argtypes = [_i32, _i32]
        L.dg_sampler_step_workspace_size.restype = _sz
        L.dg_sampler_step.argtypes = [_p, _int, _i64, _p, _i32, _i32, _i32, _int, _p, _p, _p, _u64, _u32, _int,
                                      _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]
        L.dg_sampler_step_noalloc.argtypes = [_p, _int, _i64, _p, _i32, _i32, _i32, _int, _p, _p, _p, _u64, _u32,
                                              _int, _p, _p, _p, _p, _p, _p, _p, _p]
        L.dg_selfcond_workspace_size.argtypes = [_i32, _i32, _i32, _int, _int, _int]
        L.dg_selfcond_workspace_size.restype = _sz
        L.dg_selfcond.argtypes = [_p, _int, _i64, _i32, _i32, _i32, _p, _p, _p, _int, _i32, _p, _p, _sz, _p]
        L.dg_forward_noise.argtypes = [_p, _i32, _i32, _i32, _i32, _i32, _int, _p, _u64, _p, _p, _p]
        L.dg_canvas_ce_workspace_size.argtypes = [_i32, _i32, _i32]
        L.dg_canvas_ce_workspace_size.restype = _sz
        L.dg_canvas_ce.argtypes = [_p, _int, _i64, _p, _p, _i32, _i32, _i32, _i32, _i32, _p, _p, _p, _p, _sz, _p]
        L.dg_tau_linear.argtypes = [_p, _i32, ctypes.c_double, ctypes.c_double, _p]
        L.dg_entropy_accept.argtypes = [_p, _p, _i32, _i32, _i32, ctypes.c_double, _u64, _u32, _p, _p, _p, _p]
        L.dg_adaptive_stop.argtypes = [_p, _p, _p, _i32, _i32, ctypes.c_double, _p, _p, _p]
        L.dg_sampler_step_eb.argtypes = [_p, _int, _i64, _i32, _i32, _i32, _p, _u64, _u32, _int, ctypes.c_double,
                                         ctypes.c_double, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]
        L.dg_canvas_ce_backward.argtypes = [_p, _i64, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _p, _p]
        L.dg_selfcond_drop.argtypes = [_p, _i32, _i32, _i32, _u64, _u32, _p, _p]
        L.dg_ffw_workspace_size.argtypes = [_i32, _i32, _i32]
        L.dg_ffw_workspace_size.restype = _sz
        L.dg_ffw.argtypes = [_p, _i32, _i32, _i32, _p, _p, _p, _p, _p, _sz, _p]
        L.dg_sampler_selfcond_step.argtypes = [_p, _int, _i64, _p, _i32, _i32, _i32, _int, _p, _p, _p, _u64, _u32,
                                               _int, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p, _int, _i32, _p, _p,
                                               _sz, _p]
        L.dg_block_norm.argtypes = [_p, _i64, _p, _i64, _int, _p, _p, _p, _int, _i32, _i32, _i32, _f32, _f32, _p, _p,
                                    _p, _p, _p]
        L.dg_block_norm_backward_workspace_size.argtypes = [_i32, _i32, _i32, _int, _int]
        L.dg_block_norm_backward_workspace_size.restype = _sz
        L.dg_block_norm_backward.argtypes = [_p, _i64, _p, _i64, _p, _i64, _p, _i64, _int, _p, _p, _p, _int, _i32,
                                             _i32, _i32, _f32, _p, _p, _p, _p, _p, _p, _p, _p, _sz, _p]
        L.dg_mx4_scale_bytes.argtypes = [_i32, _i32]
        L.dg_mx4_scale_bytes.restype = _sz
        L.dg_mx4_quantize.argtypes = [_p, _int, _i64, _i32, _i32, _p, _p, _p]
        L.dg_mx4_dequantize.argtypes = [_p, _p, _i32, _i32, _p, _int, _p]
        L.dg_mx4_matmul.argtypes = [_p, _p, _p, _p, _i32, _i32, _i32, _p, _int, _p]
        L.dg_test_mx4_stall.argtypes = [_p, _p, _p, _p, _i32, _i32, _i32, _p, _int, _p, _i32, _u32]
        L.dg_test_mx4_plan.argtypes = [_i32, _i32, _i32, _p, _p]
        L.dg_test_block_norm_stall.argtypes = [_p, _int, _p, _int, _i32, _i32, _p, _u32, _p]
        L.dg_test_block_norm_backward_stall.argtypes = [_p, _p, _int, _p, _int, _i32, _i32, _p, _p, _p, _p, _sz, _u32, _p]
        L.dg_ffw_mx4_workspace_size.argtypes = [_i32, _i32, _i32]
        L.dg_ffw_mx4_workspace_size.restype = _sz
        L.dg_ffw_mx4.argtypes = [_p, _i32, _i32, _i32, _p, _p, _p, _p, _p, _p, _sz, _p]
        _lib = L
    return _lib


def dg_last_error() -> str:
    return lib().dg_last_error().decode()


def dg_version() -> str:
    return lib().dg_version().decode()


def dg_launch_count() -> int:
    return int(lib().dg_launch_count())


def dg_device_error() -> int:
    """Synchronize the device and return (and clear) the library's device error word:
    0 = no kernel reported a problem, 1 = a kernel gave up on a bounded wait."""
    code = ctypes.c_int(0)
    _check("dg_device_error", lib().dg_device_error(ctypes.byref(code)))
    return code.value


def _check(fn: str, rc: int):
    if rc != DG_OK:
        raise DGError(fn, rc, dg_last_error())


def _ptr(t: Optional[torch.Tensor]):
    """Device address of a tensor (None stays NULL).  Only CUDA tensors reach the library: a host
    address handed to a kernel would fault the device."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("the library takes CUDA tensors only (got a tensor on %s)" % t.device)
    return ctypes.c_void_p(t.data_ptr())


def _vec(t: Optional[torch.Tensor], name: str, dtype, n: Optional[int] = None):
    """Check a contiguous device vector argument: dtype, and at least n elements when given."""
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if n is not None and t.numel() < n:
        raise ValueError(f"{name} has {t.numel()} elements, {n} are needed")


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DG_BF16
    if t.dtype == torch.float32:
        return DG_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use torch.bfloat16 or torch.float32")


def _row_major_2d(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit stride along the last dim")
    return t.stride(0)


def _host_doubles(vals: Sequence[float], n: int):
    if len(vals) != n:
        raise ValueError(f"expected {n} per-canvas values, got {len(vals)}")
    return (ctypes.c_double * n)(*[float(v) for v in vals])


def _host_floats(vals, n: int):
    if vals is None:
        return None
    if len(vals) != n:
        raise ValueError(f"expected {n} per-canvas values, got {len(vals)}")
    return (ctypes.c_float * n)(*[float(v) for v in vals])


def _expand(v, n):
    if isinstance(v, (int, float)):
        return [float(v)] * n
    return list(v)


# Workspaces are zero-filled once and reused: every successful call leaves their counters at
# zero.  The layout inside a workspace depends on the call's shape, so a cached workspace is
# zero-filled again (on the call's stream) whenever the shape it serves changes.
_WS: dict = {}


def workspace(kind: str, nbytes: int, device, layout=None, stream=None) -> torch.Tensor:
    """A cached zero-filled workspace of at least nbytes for calls of shape `layout`."""
    dev = torch.device(device)
    key = (kind, dev.type, dev.index)
    ws, last = _WS.get(key, (None, None))
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
    elif last != layout:
        with torch.cuda.stream(torch.cuda.current_stream(dev) if stream is None else stream):
            ws.zero_()
    _WS[key] = (ws, layout)
    return ws


def dg_sampler_step_workspace_size(rows: int, V: int) -> int:
    return int(lib().dg_sampler_step_workspace_size(rows, V))


def dg_selfcond_workspace_size(rows: int, V: int, d: int, logits_dtype: int, embed_dtype: int, have_lse: bool) -> int:
    return int(lib().dg_selfcond_workspace_size(rows, V, d, logits_dtype, embed_dtype, int(bool(have_lse))))


def dg_canvas_ce_workspace_size(n_seq: int, C: int, V: int) -> int:
    return int(lib().dg_canvas_ce_workspace_size(n_seq, C, V))


_STEP_OUT_DTYPES = {"x_next": torch.int32, "x0_hat": torch.int32, "argmax": torch.int32, "max_prob": torch.float32,
                    "lse": torch.float32, "entropy": torch.float32, "branch": torch.uint8}


def _check_step_vectors(x_t, out: dict, R: int):
    _vec(x_t, "x_t", torch.int32, R)
    for k, dt_ in _STEP_OUT_DTYPES.items():
        _vec(out.get(k), k, dt_, R)


def dg_sampler_step(logits: torch.Tensor, x_t: torch.Tensor, C: int, t, dt, *, V: Optional[int] = None,
                    schedule: str = "cosine", inv_tau=None, seed: int = 0, step: int = 0, mode: str = "sample",
                    out: Optional[dict] = None, ws: Optional[torch.Tensor] = None, stream=None) -> dict:
    """One sampler step over B = rows / C canvases.  Returns the dict of output tensors
    (x_next, x0_hat, argmax, max_prob, lse, entropy, branch); pass `out` to reuse buffers."""
    ld = _row_major_2d(logits, "logits")
    R = logits.shape[0]
    V = logits.shape[1] if V is None else V
    if R % C:
        raise ValueError("rows must be a multiple of C")
    B = R // C
    dev = logits.device
    if out is None:
        out = {
            "x_next": torch.empty(R, dtype=torch.int32, device=dev),
            "x0_hat": torch.empty(R, dtype=torch.int32, device=dev),
            "argmax": torch.empty(R, dtype=torch.int32, device=dev),
            "max_prob": torch.empty(R, dtype=torch.float32, device=dev),
            "lse": torch.empty(R, dtype=torch.float32, device=dev),
            "entropy": torch.empty(R, dtype=torch.float32, device=dev),
            "branch": torch.empty(R, dtype=torch.uint8, device=dev),
        }
    _check_step_vectors(x_t, out, R)
    nbytes = dg_sampler_step_workspace_size(R, V)
    if ws is None:
        ws = workspace("sampler_step", nbytes, dev, (R, V), stream)
    rc = lib().dg_sampler_step(
        _ptr(logits), _dtype_code(logits), ld, _ptr(x_t), B, C, V, DG_SCHED[schedule],
        _host_doubles(_expand(t, B), B), _host_doubles(_expand(dt, B), B),
        _host_floats(None if inv_tau is None else _expand(inv_tau, B), B),
        ctypes.c_uint64(seed), ctypes.c_uint32(step), DG_X0[mode],
        _ptr(out.get("x_next")), _ptr(out.get("x0_hat")), _ptr(out.get("argmax")), _ptr(out.get("max_prob")),
        _ptr(out.get("lse")), _ptr(out.get("entropy")), _ptr(out.get("branch")),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check("dg_sampler_step", rc)
    return out


def dg_sampler_selfcond_step(logits: torch.Tensor, x_t: torch.Tensor, E: torch.Tensor, C: int, t, dt, *,
                             V: Optional[int] = None, schedule: str = "cosine", inv_tau=None, seed: int = 0,
                             step: int = 0, mode: str = "sample", out: Optional[dict] = None,
                             z: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                             ws_z: Optional[torch.Tensor] = None, stream=None) -> dict:
    """One sampler step and its self-conditioning input z = softmax(L) E in one call (the
    contraction starts while the logits pass finishes).  Returns the dict of dg_sampler_step's
    outputs plus "z"."""
    ld = _row_major_2d(logits, "logits")
    R = logits.shape[0]
    V = logits.shape[1] if V is None else V
    if R % C:
        raise ValueError("rows must be a multiple of C")
    B = R // C
    dev = logits.device
    d = E.shape[1]
    if out is None:
        out = {k: torch.empty(R, dtype=dt_, device=dev) for k, dt_ in
               (("x_next", torch.int32), ("x0_hat", torch.int32), ("argmax", torch.int32),
                ("max_prob", torch.float32), ("lse", torch.float32), ("entropy", torch.float32),
                ("branch", torch.uint8))}
    z = torch.empty((R, d), dtype=torch.bfloat16, device=dev) if z is None else z
    out["z"] = z
    _check_step_vectors(x_t, out, R)
    _vec(z, "z", torch.bfloat16, R * d)
    if ws is None:
        ws = workspace("sampler_step", dg_sampler_step_workspace_size(R, V), dev, (R, V), stream)
    if ws_z is None:
        nz = dg_selfcond_workspace_size(R, V, d, _dtype_code(logits), _dtype_code(E), True)
        ws_z = workspace("selfcond", nz, dev, (R, V, d, False, E.dtype), stream)
    rc = lib().dg_sampler_selfcond_step(
        _ptr(logits), _dtype_code(logits), ld, _ptr(x_t), B, C, V, DG_SCHED[schedule],
        _host_doubles(_expand(t, B), B), _host_doubles(_expand(dt, B), B),
        _host_floats(None if inv_tau is None else _expand(inv_tau, B), B),
        ctypes.c_uint64(seed), ctypes.c_uint32(step), DG_X0[mode],
        _ptr(out.get("x_next")), _ptr(out.get("x0_hat")), _ptr(out.get("argmax")), _ptr(out.get("max_prob")),
        _ptr(out["lse"]), _ptr(out.get("entropy")), _ptr(out.get("branch")),
        _ptr(ws), ws.numel() * ws.element_size(), _ptr(E), _dtype_code(E), d, _ptr(z), _ptr(ws_z),
        ws_z.numel() * ws_z.element_size(), _stream(stream))
    _check("dg_sampler_selfcond_step", rc)
    return out


DG_NOALLOC_SCRATCH_BYTES = 4 * 1024 * 1024


def dg_sampler_step_noalloc(logits: torch.Tensor, x_t: torch.Tensor, C: int, t, dt, *, V: Optional[int] = None,
                            schedule: str = "cosine", inv_tau=None, seed: int = 0, step: int = 0,
                            mode: str = "sample", out: Optional[dict] = None, stream=None) -> dict:
    """The sampler step without a caller workspace: for callers that cannot allocate device
    memory where they sample.  Scratch lives in the library's fixed device array (at most
    DG_NOALLOC_SCRATCH_BYTES); calls share it, so overlapping calls race.  Output tensors are
    the caller's (pass `out` to reuse buffers; otherwise they are created here, as for
    dg_sampler_step)."""
    ld = _row_major_2d(logits, "logits")
    R = logits.shape[0]
    V = logits.shape[1] if V is None else V
    if R % C:
        raise ValueError("rows must be a multiple of C")
    B = R // C
    dev = logits.device
    if out is None:
        out = {k: torch.empty(R, dtype=dt_, device=dev) for k, dt_ in
               (("x_next", torch.int32), ("x0_hat", torch.int32), ("argmax", torch.int32),
                ("max_prob", torch.float32), ("lse", torch.float32), ("entropy", torch.float32),
                ("branch", torch.uint8))}
    _check_step_vectors(x_t, out, R)
    rc = lib().dg_sampler_step_noalloc(
        _ptr(logits), _dtype_code(logits), ld, _ptr(x_t), B, C, V, DG_SCHED[schedule],
        _host_doubles(_expand(t, B), B), _host_doubles(_expand(dt, B), B),
        _host_floats(None if inv_tau is None else _expand(inv_tau, B), B),
        ctypes.c_uint64(seed), ctypes.c_uint32(step), DG_X0[mode],
        _ptr(out.get("x_next")), _ptr(out.get("x0_hat")), _ptr(out.get("argmax")), _ptr(out.get("max_prob")),
        _ptr(out.get("lse")), _ptr(out.get("entropy")), _ptr(out.get("branch")), _stream(stream))
    _check("dg_sampler_step_noalloc", rc)
    return out


def dg_selfcond(logits: torch.Tensor, E: torch.Tensor, C: int, *, V: Optional[int] = None, inv_tau=None,
                lse: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """z = softmax(logits * inv_tau) @ E in bf16 (tcgen05 tensor cores)."""
    ld = _row_major_2d(logits, "logits")
    if E.dim() != 2 or not E.is_contiguous():
        raise ValueError("E must be a contiguous [V, d] tensor")
    R = logits.shape[0]
    V = E.shape[0] if V is None else V
    d = E.shape[1]
    if R % C:
        raise ValueError("rows must be a multiple of C")
    B = R // C
    dev = logits.device
    if z is None:
        z = torch.empty((R, d), dtype=torch.bfloat16, device=dev)
    _vec(z, "z", torch.bfloat16, R * d)
    _vec(lse, "lse", torch.float32, R)
    nbytes = dg_selfcond_workspace_size(R, V, d, _dtype_code(logits), _dtype_code(E), lse is not None)
    if ws is None:
        ws = workspace("selfcond", nbytes, dev, (R, V, d, lse is None, E.dtype), stream)
    rc = lib().dg_selfcond(
        _ptr(logits), _dtype_code(logits), ld, B, C, V,
        _host_floats(None if inv_tau is None else _expand(inv_tau, B), B), _ptr(lse),
        _ptr(E), _dtype_code(E), d, _ptr(z), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check("dg_selfcond", rc)
    return z


def dg_forward_noise(x0: torch.Tensor, P: int, K: int, C: int, V: int, t, *, schedule: str = "cosine",
                     seed: int = 0, x_t: Optional[torch.Tensor] = None, canvas_idx: Optional[torch.Tensor] = None,
                     stream=None):
    """Corrupt the K canvases of each sequence; returns (x_t, canvas_idx)."""
    if x0.dim() != 2 or not x0.is_contiguous() or x0.dtype != torch.int32:
        raise ValueError("x0 must be a contiguous int32 [n_seq, P + K*C] tensor")
    n_seq = x0.shape[0]
    if x_t is None:
        x_t = torch.empty_like(x0)
    if canvas_idx is None:
        canvas_idx = torch.empty(n_seq, dtype=torch.int32, device=x0.device)
    _vec(x_t, "x_t", torch.int32, x0.numel())
    _vec(canvas_idx, "canvas_idx", torch.int32, n_seq)
    rc = lib().dg_forward_noise(_ptr(x0), n_seq, P, K, C, V, DG_SCHED[schedule],
                                _host_doubles(_expand(t, n_seq), n_seq), ctypes.c_uint64(seed), _ptr(x_t),
                                _ptr(canvas_idx), _stream(stream))
    _check("dg_forward_noise", rc)
    return x_t, canvas_idx


def dg_canvas_ce(logits: torch.Tensor, x0: torch.Tensor, canvas_idx: torch.Tensor, P: int, K: int, C: int, *,
                 V: Optional[int] = None, loss_rows=None, loss_seq=None, lse_rows=None,
                 ws: Optional[torch.Tensor] = None, stream=None):
    """Cross-entropy of each sequence's chosen canvas; returns (loss_rows, loss_seq, lse_rows)."""
    ld = _row_major_2d(logits, "logits")
    R = logits.shape[0]
    V = logits.shape[1] if V is None else V
    n_seq = x0.shape[0]
    _vec(x0, "x0", torch.int32)
    _vec(canvas_idx, "canvas_idx", torch.int32, n_seq)
    if R != n_seq * C:
        raise ValueError("logits must have n_seq * C rows")
    dev = logits.device
    loss_rows = torch.empty(R, dtype=torch.float32, device=dev) if loss_rows is None else loss_rows
    loss_seq = torch.empty(n_seq, dtype=torch.float32, device=dev) if loss_seq is None else loss_seq
    lse_rows = torch.empty(R, dtype=torch.float32, device=dev) if lse_rows is None else lse_rows
    nbytes = dg_canvas_ce_workspace_size(n_seq, C, V)
    if ws is None:
        ws = workspace("canvas_ce", nbytes, dev, (n_seq, C, V), stream)
    rc = lib().dg_canvas_ce(_ptr(logits), _dtype_code(logits), ld, _ptr(x0), _ptr(canvas_idx), n_seq, P, K, C, V,
                            _ptr(loss_rows), _ptr(loss_seq), _ptr(lse_rows), _ptr(ws),
                            ws.numel() * ws.element_size(), _stream(stream))
    _check("dg_canvas_ce", rc)
    return loss_rows, loss_seq, lse_rows


# ------------------------------------------------------------------------------ sampler extensions
def dg_tau_linear(t, tau_max: float = 0.8, tau_min: float = 0.4) -> list:
    """Per-canvas inverse temperatures of the linear schedule tau(1) = tau_max, tau(0) = tau_min."""
    tt = _expand(t, 1) if isinstance(t, (int, float)) else list(t)
    n = len(tt)
    out = (ctypes.c_float * n)()
    rc = lib().dg_tau_linear(_host_doubles(tt, n), n, float(tau_max), float(tau_min), out)
    _check("dg_tau_linear", rc)
    return [float(v) for v in out]


def dg_entropy_accept(entropy: torch.Tensor, x0_hat: torch.Tensor, C: int, V: int, eps: float, *, seed: int = 0,
                      step: int = 0, out: Optional[dict] = None, stream=None) -> dict:
    """Entropy-bounded acceptance per canvas; returns {x_next, accepted, n_accepted}."""
    R = entropy.numel()
    if R % C:
        raise ValueError("rows must be a multiple of C")
    B = R // C
    dev = entropy.device
    _vec(entropy, "entropy", torch.float32)
    _vec(x0_hat, "x0_hat", torch.int32, R)
    if out is None:
        out = {"x_next": torch.empty(R, dtype=torch.int32, device=dev),
               "accepted": torch.empty(R, dtype=torch.uint8, device=dev),
               "n_accepted": torch.empty(B, dtype=torch.int32, device=dev)}
    rc = lib().dg_entropy_accept(_ptr(entropy), _ptr(x0_hat), B, C, V, float(eps), ctypes.c_uint64(seed),
                                 ctypes.c_uint32(step), _ptr(out["x_next"]), _ptr(out.get("accepted")),
                                 _ptr(out.get("n_accepted")), _stream(stream))
    _check("dg_entropy_accept", rc)
    return out


def dg_adaptive_stop(entropy: torch.Tensor, argmax: torch.Tensor, argmax_prev: Optional[torch.Tensor], C: int,
                     theta: float, *, stream=None):
    """Adaptive-stopping flags per canvas; returns (stop uint8 [B], mean_entropy float [B])."""
    R = entropy.numel()
    if R % C:
        raise ValueError("rows must be a multiple of C")
    B = R // C
    _vec(entropy, "entropy", torch.float32)
    _vec(argmax, "argmax", torch.int32, R)
    _vec(argmax_prev, "argmax_prev", torch.int32, R)
    stop = torch.empty(B, dtype=torch.uint8, device=entropy.device)
    mean = torch.empty(B, dtype=torch.float32, device=entropy.device)
    rc = lib().dg_adaptive_stop(_ptr(entropy), _ptr(argmax), _ptr(argmax_prev), B, C, float(theta), _ptr(stop),
                                _ptr(mean), _stream(stream))
    _check("dg_adaptive_stop", rc)
    return stop, mean


def dg_sampler_step_eb(logits: torch.Tensor, C: int, *, eps: float, theta: float = 0.0,
                       argmax_prev: Optional[torch.Tensor] = None, V: Optional[int] = None, inv_tau=None,
                       seed: int = 0, step: int = 0, mode: str = "sample", out: Optional[dict] = None,
                       ws: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Entropy-bounded sampler step: statistics and x0_hat draw, then per-canvas acceptance with
    uniform re-noising and the adaptive-stopping flag.  Returns the dict of outputs (x_next,
    x0_hat, argmax, max_prob, lse, entropy, accepted, stop, mean_entropy)."""
    ld = _row_major_2d(logits, "logits")
    R = logits.shape[0]
    V = logits.shape[1] if V is None else V
    if R % C:
        raise ValueError("rows must be a multiple of C")
    B = R // C
    dev = logits.device
    if out is None:
        out = {k: torch.empty(R, dtype=dt, device=dev) for k, dt in
               (("x_next", torch.int32), ("x0_hat", torch.int32), ("argmax", torch.int32),
                ("max_prob", torch.float32), ("lse", torch.float32), ("entropy", torch.float32),
                ("accepted", torch.uint8))}
        out["stop"] = torch.empty(B, dtype=torch.uint8, device=dev)
        out["mean_entropy"] = torch.empty(B, dtype=torch.float32, device=dev)
    _vec(argmax_prev, "argmax_prev", torch.int32, R)
    nbytes = dg_sampler_step_workspace_size(R, V)
    if ws is None:
        ws = workspace("sampler_step", nbytes, dev, (R, V), stream)
    rc = lib().dg_sampler_step_eb(
        _ptr(logits), _dtype_code(logits), ld, B, C, V, _host_floats(None if inv_tau is None else _expand(inv_tau, B), B),
        ctypes.c_uint64(seed), ctypes.c_uint32(step), DG_X0[mode], float(eps), float(theta), _ptr(argmax_prev),
        _ptr(out["x_next"]), _ptr(out["x0_hat"]), _ptr(out.get("argmax")), _ptr(out.get("max_prob")),
        _ptr(out.get("lse")), _ptr(out["entropy"]), _ptr(out.get("accepted")), _ptr(out.get("stop")),
        _ptr(out.get("mean_entropy")), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check("dg_sampler_step_eb", rc)
    return out


def dg_canvas_ce_backward(logits: torch.Tensor, lse_rows: torch.Tensor, x0: torch.Tensor, canvas_idx: torch.Tensor,
                          P: int, K: int, C: int, *, V: Optional[int] = None, g_seq: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Overwrite bf16 logits with d(sum of each sequence's canvas CE) / d logits (times g_seq)."""
    ld = _row_major_2d(logits, "logits")
    if logits.dtype != torch.bfloat16:
        raise TypeError("the in-place CE backward works on bf16 logits")
    V = logits.shape[1] if V is None else V
    n_seq = x0.shape[0]
    _vec(lse_rows, "lse_rows", torch.float32, logits.shape[0])
    _vec(x0, "x0", torch.int32)
    _vec(canvas_idx, "canvas_idx", torch.int32, n_seq)
    _vec(g_seq, "g_seq", torch.float32, n_seq)
    rc = lib().dg_canvas_ce_backward(_ptr(logits), ld, _ptr(lse_rows), _ptr(x0), _ptr(canvas_idx), n_seq, P, K, C, V,
                                     _ptr(g_seq), _stream(stream))
    _check("dg_canvas_ce_backward", rc)
    return logits


def dg_selfcond_drop(z: torch.Tensor, C: int, *, seed: int = 0, step: int = 0,
                     keep: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Zero, in place, the bf16 self-conditioning rows of sequences whose fair coin drops them;
    returns keep (uint8 [n_seq])."""
    if z.dtype != torch.bfloat16 or not z.is_contiguous():
        raise TypeError("z must be a contiguous bf16 tensor [n_seq*C, d]")
    R, d = z.shape
    if R % C:
        raise ValueError("rows must be a multiple of C")
    n_seq = R // C
    keep = torch.empty(n_seq, dtype=torch.uint8, device=z.device) if keep is None else keep
    rc = lib().dg_selfcond_drop(_ptr(z), n_seq, C, d, ctypes.c_uint64(seed), ctypes.c_uint32(step), _ptr(keep),
                                _stream(stream))
    _check("dg_selfcond_drop", rc)
    return keep


def dg_ffw(z: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, *, hidden: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Two-layer feed-forward block gelu(z W1) W2 on the tensor cores (bf16 in and out).
    Returns (out [R, d], hidden [R, d_ff])."""
    for t, n in ((z, "z"), (W1, "W1"), (W2, "W2")):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise TypeError(f"{n} must be a contiguous bf16 tensor")
    R, d = z.shape
    dff = W1.shape[1]
    if W1.shape != (d, dff) or W2.shape != (dff, d):
        raise ValueError("W1 must be [d, d_ff] and W2 [d_ff, d]")
    dev = z.device
    hidden = torch.empty(R, dff, dtype=torch.bfloat16, device=dev) if hidden is None else hidden
    out = torch.empty(R, d, dtype=torch.bfloat16, device=dev) if out is None else out
    nbytes = int(lib().dg_ffw_workspace_size(R, d, dff))
    if ws is None:
        ws = workspace("ffw", nbytes, dev, (R, d, dff), stream)
    rc = lib().dg_ffw(_ptr(z), R, d, dff, _ptr(W1), _ptr(W2), _ptr(hidden), _ptr(out), _ptr(ws),
                      ws.numel() * ws.element_size(), _stream(stream))
    _check("dg_ffw", rc)
    return out, hidden


# ------------------------------------------------------------------------------ the block around the FFW
# These calls run on the device of their tensors, whichever is current, on `stream` or that device's
# current stream; outputs and scratch that they allocate belong to the stream they run on.
_DTYPE = {torch.float32: DG_F32, torch.bfloat16: DG_BF16}


def _dtype_of(t: torch.Tensor, name: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return code


def _arg(t: torch.Tensor, name: str, dev: int, dtype, shape) -> int:
    """Device address of a contiguous tensor argument of the given dtype and shape on device `dev`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dev, dtype, shape)
    raise ValueError(f"{name} must be contiguous")


def _rows_arg(t: torch.Tensor, name: str, dev: int, dtype, shape):
    """Device address and row stride of a 2-D tensor whose last dimension is contiguous."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        _refuse(t, name, dev, dtype, shape)
    s0, s1 = t.stride()
    if s1 != 1:
        raise ValueError(f"{name} must have unit stride along the last dim")
    return t.data_ptr(), (s0 if shape[0] > 1 else shape[1])


def _refuse(t: torch.Tensor, name: str, dev: int, dtype, shape):
    if t.get_device() != dev:
        _wrong_device(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be of shape {list(shape)}, got {list(t.shape)}")


def _wrong_device(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError("the library takes CUDA tensors only (got %s on %s)" % (name, t.device))
    raise ValueError(f"{name} is on {t.device}, another device than the first argument")


# The current stream's handle on a device: without the Stream object that torch.cuda.current_stream builds
# (3 us of a call that costs the GPU as little).
_current_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _device_of(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        _wrong_device(t, name)
    return dev


class _On:
    """The device and stream that a call runs on, where they are not the current ones."""

    def __init__(self, dev: int, stream):
        if stream is not None and stream.device_index != dev:
            raise ValueError(f"the stream is on device {stream.device_index}, the tensors are on device {dev}")
        self.parts = [torch.cuda.device(dev)] + ([torch.cuda.stream(stream)] if stream is not None else [])

    def __enter__(self):
        for p in self.parts:
            p.__enter__()

    def __exit__(self, *exc):
        for p in reversed(self.parts):
            p.__exit__(*exc)


def dg_block_norm(x: torch.Tensor, w_pre: Optional[torch.Tensor] = None, *, y: Optional[torch.Tensor] = None,
                  w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, C: Optional[int] = None,
                  res_scale: float = 1.0, eps: float = 1e-6, out: Optional[dict] = None, stream=None) -> dict:
    """Norms after a block (y given: x + res_scale gate w_post n(y), key "x") and before the next
    (w_pre given: w_pre n(stream), key "h"), with the reciprocal root means "rstd_y" and "rstd_x" that the
    backward pass takes.  x, y: [B*C, d]; gate: [B, d], one row per canvas of C rows.  Pass `out` to
    reuse buffers; out["x"] may be x itself."""
    dev = _device_of(x, "x")
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return dg_block_norm(x, w_pre, y=y, w_post=w_post, gate=gate, C=C, res_scale=res_scale, eps=eps, out=out)
    dtype, shape = x.dtype, x.shape
    act = _dtype_of(x, "x")
    if len(shape) != 2:
        raise ValueError("x must be a 2-D tensor")
    R, d = shape
    px, ld_x = _rows_arg(x, "x", dev, dtype, shape)
    C = R if C is None or gate is None else C  # without a gate rows need no grouping
    if C < 1 or R % C:
        raise ValueError("rows must be a multiple of C")
    given = w_pre if w_pre is not None else w_post
    if given is None:
        raise ValueError("w_pre or w_post (with y) is needed")
    ptype, par = given.dtype, _dtype_of(given, "w_pre" if w_pre is not None else "w_post")
    res, device = {}, x.device

    def new(key, dt, shp):
        t = None if out is None else out.get(key)
        if t is not None:
            p = _arg(t, key, dev, dt, shp)
        else:
            t = torch.empty_like(x, memory_format=torch.contiguous_format) if shp is shape else torch.empty(*shp, dtype=dt, device=device)
            p = t.data_ptr()
        res[key] = t
        return p

    py = pw = pg = pn = po = ph = pry = prx = None
    ld_y = d
    if y is not None:
        if w_post is None:
            raise ValueError("y needs w_post")
        py, ld_y = _rows_arg(y, "y", dev, dtype, shape)
        pw = _arg(w_post, "w_post", dev, ptype, (d,))
        if gate is not None:
            pg = _arg(gate, "gate", dev, ptype, (R // C, d))
        po, pry = new("x", dtype, shape), new("rstd_y", torch.float32, (R,))
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate come only with y")
    if w_pre is not None:
        pn = _arg(w_pre, "w_pre", dev, ptype, (d,))
        ph, prx = new("h", dtype, shape), new("rstd_x", torch.float32, (R,))
    rc = lib().dg_block_norm(px, ld_x, py, ld_y, act, pw, pg, pn, par, R // C, C, d, res_scale, eps, po, ph, pry, prx,
                             _current_stream(dev))
    if rc:
        _check("dg_block_norm", rc)
    return res


def dg_block_norm_backward(dx_out: Optional[torch.Tensor], dh: Optional[torch.Tensor], x: torch.Tensor,
                           w_pre: Optional[torch.Tensor] = None, *, rstd_x: Optional[torch.Tensor] = None,
                           y: Optional[torch.Tensor] = None, w_post: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None, rstd_y: Optional[torch.Tensor] = None,
                           C: Optional[int] = None, res_scale: float = 1.0, out: Optional[dict] = None,
                           ws: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of dg_block_norm: dx_out of its stream (None: zero), dh of its h; x is the stream that h
    was taken of (out["x"] of the forward call, or its x where it had no y).  Returns "dx" and, where
    the call had them, "dw_pre" (w_pre), "dy", "dw_post" (y) and "dgate" (gate); the parameters'
    gradients are float32."""
    dev = _device_of(x, "x")
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return dg_block_norm_backward(dx_out, dh, x, w_pre, rstd_x=rstd_x, y=y, w_post=w_post, gate=gate,
                                          rstd_y=rstd_y, C=C, res_scale=res_scale, out=out, ws=ws)
    dtype, shape = x.dtype, x.shape
    act = _dtype_of(x, "x")
    if len(shape) != 2:
        raise ValueError("x must be a 2-D tensor")
    R, d = shape
    C = R if C is None or gate is None else C  # without a gate rows need no grouping
    if C < 1 or R % C:
        raise ValueError("rows must be a multiple of C")
    given = w_pre if w_pre is not None else w_post
    if given is None:
        raise ValueError("w_pre or w_post (with y) is needed")
    ptype, par = given.dtype, _dtype_of(given, "w_pre" if w_pre is not None else "w_post")
    res, f32, device = {}, torch.float32, x.device

    def new(key, dt, shp):
        t = None if out is None else out.get(key)
        if t is not None:
            p = _arg(t, key, dev, dt, shp)
        else:
            t = torch.empty_like(x, memory_format=torch.contiguous_format) if shp is shape else torch.empty(*shp, dtype=dt, device=device)
            p = t.data_ptr()
        res[key] = t
        return p

    pdo = pdh = px = py = pw = pg = pn = pry = prx = pdy = pdw = pdg = pdn = None
    ld_do = ld_dh = ld_x = ld_y = d
    if dx_out is not None:
        pdo, ld_do = _rows_arg(dx_out, "dx_out", dev, dtype, shape)
    pdx = new("dx", dtype, shape)
    if w_pre is not None:
        if dh is None or rstd_x is None:
            raise ValueError("w_pre needs dh and rstd_x")
        px, ld_x = _rows_arg(x, "x", dev, dtype, shape)
        pdh, ld_dh = _rows_arg(dh, "dh", dev, dtype, shape)
        pn, prx = _arg(w_pre, "w_pre", dev, ptype, (d,)), _arg(rstd_x, "rstd_x", dev, f32, (R,))
        pdn = new("dw_pre", f32, (d,))
    elif dh is not None:
        raise ValueError("dh comes only with w_pre")
    if y is not None:
        if w_post is None or rstd_y is None:
            raise ValueError("y needs w_post and rstd_y")
        py, ld_y = _rows_arg(y, "y", dev, dtype, shape)
        pw, pry = _arg(w_post, "w_post", dev, ptype, (d,)), _arg(rstd_y, "rstd_y", dev, f32, (R,))
        pdy, pdw = new("dy", dtype, shape), new("dw_post", f32, (d,))
        if gate is not None:
            pg = _arg(gate, "gate", dev, ptype, (R // C, d))
            pdg = new("dgate", f32, (R // C, d))
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate come only with y")
    L = lib()
    nbytes = L.dg_block_norm_backward_workspace_size(R // C, C, d, act, pg is not None)
    if ws is None:
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the device of x")
    rc = L.dg_block_norm_backward(pdo, ld_do, pdh, ld_dh, px, ld_x, py, ld_y, act, pw, pg, pn, par, R // C, C, d, res_scale,
                                  pry, prx, pdx, pdy, pdw, pdg, pdn, ws.data_ptr(), ws.numel() * ws.element_size(),
                                  _current_stream(dev))
    if rc:
        _check("dg_block_norm_backward", rc)
    return res


def dg_mx4_scale_shape(rows: int, K: int) -> tuple:
    """Shape of the scale bytes of a [rows, K] MXFP4 matrix: tiles of 128 rows x 4 blocks of 32."""
    return (-(-rows // 128), -(-K // 128), 32, 16)


def dg_mx4_quantize(x: torch.Tensor, *, out=None, stream=None):
    """x [rows, K] (float32 or bfloat16) in MXFP4: (codes uint8 [rows, K/2], scales uint8 in the shape of
    dg_mx4_scale_shape).  Pass out=(codes, scales) to reuse buffers."""
    dev = _device_of(x, "x")
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return dg_mx4_quantize(x, out=out)
    shape = x.shape
    dt = _dtype_of(x, "x")
    if len(shape) != 2:
        raise ValueError("x must be a 2-D tensor")
    R, K = shape
    px, ld = _rows_arg(x, "x", dev, x.dtype, shape)
    u8, scale_shape = torch.uint8, dg_mx4_scale_shape(R, K)
    if out is None:
        codes, scales = torch.empty(R, K // 2, dtype=u8, device=x.device), torch.empty(*scale_shape, dtype=u8, device=x.device)
        pc, ps = codes.data_ptr(), scales.data_ptr()
    else:
        codes, scales = out
        pc, ps = _arg(codes, "codes", dev, u8, (R, K // 2)), _arg(scales, "scales", dev, u8, scale_shape)
    rc = lib().dg_mx4_quantize(px, dt, ld, R, K, pc, ps, _current_stream(dev))
    if rc:
        _check("dg_mx4_quantize", rc)
    return codes, scales


def dg_mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values [rows, K] that MXFP4 codes and scales stand for."""
    dev = _device_of(codes, "codes")
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return dg_mx4_dequantize(codes, scales, dtype=dtype, out=out)
    if len(codes.shape) != 2:
        raise ValueError("codes must be a 2-D tensor")
    R, K = codes.shape[0], 2 * codes.shape[1]
    u8 = torch.uint8
    dt = _DTYPE.get(dtype)
    if dt is None:
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    if out is None:
        out = torch.empty(R, K, dtype=dtype, device=codes.device)
        po = out.data_ptr()
    else:
        po = _arg(out, "out", dev, dtype, (R, K))
    rc = lib().dg_mx4_dequantize(_arg(codes, "codes", dev, u8, codes.shape), _arg(scales, "scales", dev, u8, dg_mx4_scale_shape(R, K)),
                                 R, K, po, dt, _current_stream(dev))
    if rc:
        _check("dg_mx4_dequantize", rc)
    return out


def _mx4_arg(q, name: str, dev: int, rows: int, K: int):
    codes, scales = q
    return (_arg(codes, f"{name} codes", dev, torch.uint8, (rows, K // 2)),
            _arg(scales, f"{name} scales", dev, torch.uint8, dg_mx4_scale_shape(rows, K)))


def dg_mx4_matmul(a, w, *, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """a w^T [M, N] of two MXFP4 matrices a = (codes, scales) [M, K] and w [N, K], fp32 accumulation."""
    (ac, asc), (wc, wsc) = a, w
    dev = _device_of(ac, "a codes")
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return dg_mx4_matmul(a, w, dtype=dtype, out=out)
    if ac.dim() != 2 or wc.dim() != 2:
        raise ValueError("codes must be 2-D tensors")
    (M, half), N, u8, dt = ac.shape, wc.shape[0], torch.uint8, _DTYPE.get(dtype)
    if dt is None:
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    if out is None:
        out = torch.empty(M, N, dtype=dtype, device=ac.device)
        po = out.data_ptr()
    else:
        po = _arg(out, "out", dev, dtype, (M, N))
    K = 2 * half
    rc = lib().dg_mx4_matmul(_arg(ac, "a codes", dev, u8, (M, half)), _arg(asc, "a scales", dev, u8, dg_mx4_scale_shape(M, K)),
                             _arg(wc, "w codes", dev, u8, (N, half)), _arg(wsc, "w scales", dev, u8, dg_mx4_scale_shape(N, K)),
                             M, N, K, po, dt, _current_stream(dev))
    if rc:
        _check("dg_mx4_matmul", rc)
    return out


def dg_ffw_mx4(z: torch.Tensor, w1, w2, *, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """The feed-forward block gelu(z W1) W2 in MXFP4 (z bf16 [R, d], quantised by the call).  w1 = (codes,
    scales) of W1 transposed, [d_ff, d]; w2 of W2 transposed, [d, d_ff]: for weights as dg_ffw takes them,
    dg_mx4_quantize(W.t().contiguous())."""
    dev = _device_of(z, "z")
    if stream is not None or dev != _current_device():
        with _On(dev, stream):
            return dg_ffw_mx4(z, w1, w2, out=out, ws=ws)
    if len(z.shape) != 2:
        raise ValueError("z must be a 2-D tensor")
    R, d = z.shape
    dff = w1[0].shape[0]
    bf16 = torch.bfloat16
    pz = _arg(z, "z", dev, bf16, (R, d))
    p1, ps1 = _mx4_arg(w1, "w1", dev, dff, d)
    p2, ps2 = _mx4_arg(w2, "w2", dev, d, dff)
    if out is None:
        out = torch.empty_like(z)
        po = out.data_ptr()
    else:
        po = _arg(out, "out", dev, bf16, (R, d))
    L = lib()
    if ws is None:
        ws = torch.empty(max(256, L.dg_ffw_mx4_workspace_size(R, d, dff)), dtype=torch.uint8, device=z.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the device of z")
    rc = L.dg_ffw_mx4(pz, R, d, dff, p1, ps1, p2, ps2, po, ws.data_ptr(),
                      ws.numel() * ws.element_size(), _current_stream(dev))
    if rc:
        _check("dg_ffw_mx4", rc)
    return out
