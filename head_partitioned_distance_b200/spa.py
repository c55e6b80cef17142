"""Python binding of libspa.so -- argument marshalling only.

Every function here has the name of the C entry point it calls (see
``include/spa.h``) and does nothing but turn torch tensors into pointers and
sizes and the status code into an exception.  All arithmetic runs in the
library's CUDA kernels; there is no fallback of any kind: importing this
module fails when ``libspa.so`` has not been built, and a call fails when the
library reports an error.
"""
from __future__ import annotations

import array
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m head_partitioned_distance_b200.build` "
        "(nvcc, sm_100a).  There is no non-CUDA fallback.")

_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_i32p = ctypes.POINTER(ctypes.c_int32)
_u8p = ctypes.POINTER(ctypes.c_uint8)
_i64 = ctypes.c_int64
_i64p = ctypes.POINTER(ctypes.c_int64)
_int = ctypes.c_int
_f32 = ctypes.c_float

EXPORTS = {
    "spa_status_string": ([_int], ctypes.c_char_p),
    "spa_version": ([], _int),
    "spa_band_bounds": ([_i64, _int, _i32p, _i32p], _int),
    "spa_attn_fwd": ([_vp, _vp, _vp, _vp, _vp, _int, _int, _i64, _int, _f32, _vp], _int),
    "spa_attn_fwd_ex": ([_vp, _vp, _vp, _vp, _vp, _int, _int, _i64, _int, _f32, _i32p, _i32p, _vp],
                        _int),
    "spa_attn_fwd_merge": ([_vp, _vp, _vp, _vp, _vp, _int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_workspace_bytes": ([_int, _int, _i64], ctypes.c_size_t),
    "spa_attn_bwd": ([_vp] * 10 + [_int, _int, _i64, _int, _f32, _vp], _int),
    "spa_attn_bwd_ex": ([_vp] * 10 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_preprocess": ([_vp, _vp, _vp, _int, _int, _i64, _int, _vp], _int),
    "spa_attn_bwd_dkdv": ([_vp] * 8 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_dq": ([_vp] * 7 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_dq_delta": ([_vp] * 8 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_dkdv_add": ([_vp] * 8 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_dq_add": ([_vp] * 7 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_decode_workspace_bytes": ([_int, _int, _i64, _int, _i32p, _i32p], ctypes.c_size_t),
    "spa_attn_decode": ([_vp] * 7 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_noalloc": ([_vp] * 9 + [_int, _int, _i64, _int, _f32, _vp], _int),
    "spa_attn_bwd_fused_workspace_bytes": ([_int, _int, _i64, _int], ctypes.c_size_t),
    "spa_attn_bwd_stored_workspace_bytes": ([_int, _int, _i64, _int, _i32p, _i32p], ctypes.c_size_t),
    "spa_attn_bwd_stored": ([_vp] * 10 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_stored_steps": ([_vp] * 10 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp, _int], _int),
    "spa_attn_bwd_fused": ([_vp] * 10 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_fused_steps": ([_vp] * 10 + [_int, _int, _i64, _int, _f32, _i32p, _i32p, _vp, _int], _int),
    "spa_attn_union_workspace_bytes": ([_int, _int, _i64, _int], ctypes.c_size_t),
    "spa_union_parts": ([_i64, _int, _i64, _i32p, _i32p, _i32p, _i32p, _i32p, _i32p], _int),
    "spa_attn_union_merge": ([_vp] * 4 + [_int, _int, _i64, _int, _vp], _int),
    "spa_attn_union_add_grads": ([_vp] * 6 + [_int, _int, _i64, _int, _vp], _int),
    "spa_attn_fwd_union": ([_vp] * 5 + [_int, _int, _i64, _int, _f32, _i64, _i32p, _i32p, _vp], _int),
    "spa_attn_bwd_union": ([_vp] * 10 + [_int, _int, _i64, _int, _f32, _i64, _i32p, _i32p, _vp], _int),
    "spa_tile_schedule": ([_i64, _int, _i32p, _i32p, _int, _int, _i32p, _i32p, _u8p, _i32p, _i32p],
                          _int),
    "spa_tile_classes_device": ([_i64, _int, _i32p, _i32p, _int, _int, _vp, _vp], _int),
    "spa_debug_wait_timeout": ([_i64, _vp], _int),
    "spa_device_status": ([_vp], _int),
    "spa_rope_table": ([_vp, _i64, _int, ctypes.c_double, _vp], _int),
    "spa_qk_norm_rope_fwd": ([_vp] * 8 + [_int, _int, _int, _i64, _int, _int, _i64, _i64, _i64p, _i64p, _int, _f32,
                                          _int, _vp], _int),
    "spa_qk_norm_rope_bwd_workspace_bytes": ([_int], ctypes.c_size_t),
    "spa_qk_norm_rope_bwd": ([_vp] * 13 + [_int, _int, _int, _i64, _int, _int, _i64, _i64, _i64p, _i64p, _i64p, _i64p,
                                           _int, _f32, _int, _vp], _int),
    "spa_paged_append": ([_vp] * 12 + [_int, _int, _int, _int, _int, _i64, _int, _int, _int, _i64, _i64p, _i64p, _i64p,
                                       _int, _f32, _int, _vp], _int),
    "spa_paged_attn_workspace_bytes": ([_int, _int], ctypes.c_size_t),
    "spa_paged_attn": ([_vp] * 9 + [_int, _int, _int, _int, _int, _i64, _int, _int, _i64, _int, _f32, _vp, _vp,
                                    _int, _vp], _int),
}
for _name, (_args, _res) in EXPORTS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

SPA_OK, SPA_ERR_INVAL, SPA_ERR_UNSUPPORTED, SPA_ERR_CUDA, SPA_ERR_TIMEOUT = 0, 1, 2, 3, 4


class SpaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {spa_status_string(status)}")


def _check(status: int, where: str):
    if status != SPA_OK:
        raise SpaError(status, where)


def spa_status_string(status: int) -> str:
    return _lib.spa_status_string(status).decode()


def spa_version() -> int:
    return int(_lib.spa_version())


def _i32(arr):
    a = (ctypes.c_int32 * len(arr))(*[int(x) for x in arr])
    return a


def spa_band_bounds(N: int, H: int):
    """Balanced Distance Partitioning bands: (lo, hi) lists of H ints."""
    lo = (ctypes.c_int32 * H)()
    hi = (ctypes.c_int32 * H)()
    _check(_lib.spa_band_bounds(N, H, lo, hi), "spa_band_bounds")
    return list(lo), list(hi)


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return _vp(stream.cuda_stream)


def _dims(q: torch.Tensor):
    if q.dim() != 4:
        raise ValueError("tensors are [B, H, N, d]")
    B, H, N, d = q.shape
    return B, H, N, d


def _need(t: torch.Tensor, shape, dtype, name):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def spa_attn_fwd(q, k, v, o, lse, scale: float, lo=None, hi=None, stream=None):
    """o, lse = band-sparse attention forward (writes into o [B,H,N,d] bf16 and
    lse [B,H,N] fp32).  lo/hi: optional explicit bands (calls spa_attn_fwd_ex)."""
    B, H, N, d = _dims(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    _need(lse, (B, H, N), torch.float32, "lse")
    s = _stream_ptr(stream)
    if lo is None:
        st = _lib.spa_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                               B, H, N, d, scale, s)
        _check(st, "spa_attn_fwd")
    else:
        st = _lib.spa_attn_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                  lse.data_ptr(), B, H, N, d, scale, _i32(lo), _i32(hi), s)
        _check(st, "spa_attn_fwd_ex")
    return o, lse


def spa_attn_fwd_merge(q, k, v, o, lse, scale: float, lo=None, hi=None, stream=None):
    """Forward over bands disjoint from the ones o, lse already hold a
    softmax over; merges into o, lse (the softmax over both sets)."""
    B, H, N, d = _dims(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    _need(lse, (B, H, N), torch.float32, "lse")
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_attn_fwd_merge(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                   B, H, N, d, scale, lo_a, hi_a, _stream_ptr(stream)), "spa_attn_fwd_merge")
    return o, lse


def spa_attn_bwd_workspace_bytes(B: int, H: int, N: int) -> int:
    return int(_lib.spa_attn_bwd_workspace_bytes(B, H, N))


def spa_attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale: float, lo=None, hi=None,
                 stream=None):
    """Gradients of sum(o * dout): writes dq, dk, dv.  workspace: CUDA tensor of
    at least spa_attn_bwd_workspace_bytes(B, H, N) bytes."""
    B, H, N, d = _dims(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"),
                 (dv, "dv")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    _need(lse, (B, H, N), torch.float32, "lse")
    _need_workspace(workspace, B, H, N)
    s = _stream_ptr(stream)
    ptrs = [t.data_ptr() for t in (q, k, v, o, dout, lse, dq, dk, dv, workspace)]
    if lo is None:
        _check(_lib.spa_attn_bwd(*ptrs, B, H, N, d, scale, s), "spa_attn_bwd")
    else:
        _check(_lib.spa_attn_bwd_ex(*ptrs, B, H, N, d, scale, _i32(lo), _i32(hi), s),
               "spa_attn_bwd_ex")
    return dq, dk, dv


def spa_attn_bwd_fused_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(_lib.spa_attn_bwd_fused_workspace_bytes(B, H, N, d))


def spa_attn_bwd_fused(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale: float, lo=None, hi=None,
                       stream=None, steps: int = 7):
    """The backward in one pass over the key tiles (spa_attn_bwd_fused in
    spa.h): same gradients as spa_attn_bwd, dq summed in fp32 by reductions
    (not bit-reproducible from call to call).  workspace: CUDA tensor of at
    least spa_attn_bwd_fused_workspace_bytes(B, H, N, d) bytes."""
    B, H, N, d = _dims(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"),
                 (dv, "dv")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    _need(lse, (B, H, N), torch.float32, "lse")
    if not workspace.is_cuda or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < spa_attn_bwd_fused_workspace_bytes(B, H, N, d):
        raise ValueError("workspace: contiguous CUDA tensor of spa_attn_bwd_fused_workspace_bytes(B, H, N, d) bytes")
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    ptrs = [t.data_ptr() for t in (q, k, v, o, dout, lse, dq, dk, dv, workspace)]
    if steps == 7:
        _check(_lib.spa_attn_bwd_fused(*ptrs, B, H, N, d, scale, lo_a, hi_a, _stream_ptr(stream)),
               "spa_attn_bwd_fused")
    else:  # one or two of its launches (spa_attn_bwd_fused_steps)
        _check(_lib.spa_attn_bwd_fused_steps(*ptrs, B, H, N, d, scale, lo_a, hi_a, _stream_ptr(stream), steps),
               "spa_attn_bwd_fused_steps")
    return dq, dk, dv


def attention_backward_fused(q, k, v, o, dout, lse, scale=None, lo=None, hi=None):
    """Allocate dq / dk / dv / workspace and run spa_attn_bwd_fused."""
    B, H, N, d = _dims(q)
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(spa_attn_bwd_fused_workspace_bytes(B, H, N, d) // 4, dtype=torch.float32, device=q.device)
    return spa_attn_bwd_fused(q, k, v, o, dout, lse, dq, dk, dv, ws, scale, lo, hi)


def spa_attn_bwd_stored_workspace_bytes(B: int, H: int, N: int, d: int, lo=None, hi=None) -> int:
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    return int(_lib.spa_attn_bwd_stored_workspace_bytes(B, H, N, d, lo_a, hi_a))


def spa_attn_bwd_stored(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale: float, lo=None, hi=None,
                        stream=None, steps: int = 7):
    """The backward that stores dS (spa_attn_bwd_stored in spa.h): same
    gradients as spa_attn_bwd, bit-reproducible; the dK/dV pass writes every
    tile pair's dS^T to the workspace and the dQ pass contracts it with k.
    workspace: CUDA tensor of at least
    spa_attn_bwd_stored_workspace_bytes(B, H, N, d, lo, hi) bytes."""
    B, H, N, d = _dims(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"),
                 (dv, "dv")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    _need(lse, (B, H, N), torch.float32, "lse")
    need = spa_attn_bwd_stored_workspace_bytes(B, H, N, d, lo, hi)
    if need == 0 or not workspace.is_cuda or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace: contiguous CUDA tensor of spa_attn_bwd_stored_workspace_bytes(B, H, N, d, "
                         "lo, hi) bytes")
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    ptrs = [t.data_ptr() for t in (q, k, v, o, dout, lse, dq, dk, dv, workspace)]
    if steps == 7:
        _check(_lib.spa_attn_bwd_stored(*ptrs, B, H, N, d, scale, lo_a, hi_a, _stream_ptr(stream)),
               "spa_attn_bwd_stored")
    else:  # one or two of its launches (spa_attn_bwd_stored_steps)
        _check(_lib.spa_attn_bwd_stored_steps(*ptrs, B, H, N, d, scale, lo_a, hi_a, _stream_ptr(stream), steps),
               "spa_attn_bwd_stored_steps")
    return dq, dk, dv


def attention_backward_stored(q, k, v, o, dout, lse, scale=None, lo=None, hi=None):
    """Allocate dq / dk / dv / workspace and run spa_attn_bwd_stored."""
    B, H, N, d = _dims(q)
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(spa_attn_bwd_stored_workspace_bytes(B, H, N, d, lo, hi), dtype=torch.uint8, device=q.device)
    return spa_attn_bwd_stored(q, k, v, o, dout, lse, dq, dk, dv, ws, scale, lo, hi)


SPA_NOALLOC_MAX_ROWS = 1 << 20


def spa_attn_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, scale: float, stream=None):
    """Backward without a workspace argument and without any allocation, for
    callers that cannot call cudaMalloc (see spa_attn_bwd_noalloc in spa.h):
    the row sums D go to a library-owned device array of
    SPA_NOALLOC_MAX_ROWS floats, shared by every call -- calls that overlap on
    the GPU race on it.  B * H * N must not exceed SPA_NOALLOC_MAX_ROWS."""
    B, H, N, d = _dims(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"),
                 (dv, "dv")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    _need(lse, (B, H, N), torch.float32, "lse")
    ptrs = [t.data_ptr() for t in (q, k, v, o, dout, lse, dq, dk, dv)]
    _check(_lib.spa_attn_bwd_noalloc(*ptrs, B, H, N, d, scale, _stream_ptr(stream)),
           "spa_attn_bwd_noalloc")
    return dq, dk, dv


def _need_workspace(workspace, B, H, N):
    if not workspace.is_cuda or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < spa_attn_bwd_workspace_bytes(B, H, N):
        raise ValueError("workspace: contiguous CUDA tensor of spa_attn_bwd_workspace_bytes(B, H, N) bytes")


def _need_step(B, H, N, d, tensors, lse=None, workspace=None):
    """The checks spa_attn_bwd makes, for the step entry points: every tensor
    [B, H, N, d] bf16, contiguous, on the GPU; lse [B, H, N] fp32; the
    workspace large enough for D."""
    for t, n in tensors:
        _need(t, (B, H, N, d), torch.bfloat16, n)
    if lse is not None:
        _need(lse, (B, H, N), torch.float32, "lse")
    if workspace is not None:
        _need_workspace(workspace, B, H, N)


def spa_attn_bwd_preprocess(o, dout, workspace, stream=None):
    B, H, N, d = _dims(o)
    _need_step(B, H, N, d, ((o, "o"), (dout, "dout")), workspace=workspace)
    _check(_lib.spa_attn_bwd_preprocess(o.data_ptr(), dout.data_ptr(), workspace.data_ptr(), B, H, N, d,
                                        _stream_ptr(stream)), "spa_attn_bwd_preprocess")


def spa_attn_bwd_dkdv(q, k, v, dout, lse, workspace, dk, dv, scale: float, lo=None, hi=None,
                      stream=None):
    B, H, N, d = _dims(q)
    _need_step(B, H, N, d, ((q, "q"), (k, "k"), (v, "v"), (dout, "dout"), (dk, "dk"), (dv, "dv")), lse,
               workspace)
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_attn_bwd_dkdv(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                                  lse.data_ptr(), workspace.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                  B, H, N, d, scale, lo_a, hi_a, _stream_ptr(stream)),
           "spa_attn_bwd_dkdv")


def spa_attn_bwd_dq(q, k, v, dout, lse, workspace, dq, scale: float, lo=None, hi=None, stream=None):
    B, H, N, d = _dims(q)
    _need_step(B, H, N, d, ((q, "q"), (k, "k"), (v, "v"), (dout, "dout"), (dq, "dq")), lse, workspace)
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_attn_bwd_dq(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                                lse.data_ptr(), workspace.data_ptr(), dq.data_ptr(), B, H, N, d, scale,
                                lo_a, hi_a, _stream_ptr(stream)), "spa_attn_bwd_dq")


def spa_attn_bwd_dkdv_add(q, k, v, dout, lse, workspace, dk, dv, scale: float, lo=None, hi=None,
                          stream=None):
    """The dk/dv pass adding to dk, dv instead of overwriting them."""
    B, H, N, d = _dims(q)
    _need_step(B, H, N, d, ((q, "q"), (k, "k"), (v, "v"), (dout, "dout"), (dk, "dk"), (dv, "dv")), lse,
               workspace)
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_attn_bwd_dkdv_add(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                                      lse.data_ptr(), workspace.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                      B, H, N, d, scale, lo_a, hi_a, _stream_ptr(stream)),
           "spa_attn_bwd_dkdv_add")


def spa_attn_bwd_dq_add(q, k, v, dout, lse, workspace, dq, scale: float, lo=None, hi=None, stream=None):
    """The dq pass adding to dq instead of overwriting it."""
    B, H, N, d = _dims(q)
    _need_step(B, H, N, d, ((q, "q"), (k, "k"), (v, "v"), (dout, "dout"), (dq, "dq")), lse, workspace)
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_attn_bwd_dq_add(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                                    lse.data_ptr(), workspace.data_ptr(), dq.data_ptr(), B, H, N, d, scale,
                                    lo_a, hi_a, _stream_ptr(stream)), "spa_attn_bwd_dq_add")


def spa_attn_bwd_dq_delta(q, k, v, o, dout, lse, workspace, dq, scale: float, lo=None, hi=None,
                          stream=None):
    B, H, N, d = _dims(q)
    _need_step(B, H, N, d, ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq")), lse,
               workspace)
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_attn_bwd_dq_delta(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                      dout.data_ptr(), lse.data_ptr(), workspace.data_ptr(), dq.data_ptr(),
                                      B, H, N, d, scale, lo_a, hi_a, _stream_ptr(stream)),
           "spa_attn_bwd_dq_delta")


def spa_tile_schedule(N: int, H: int, Bq: int, Bk: int, lo=None, hi=None):
    """Host evaluation of the kernels' tile schedule.  Returns a dict of numpy
    arrays: kt_begin/kt_end [H, nqt], tile_class [H, nqt, nkt], qt_begin/qt_end
    [H, nkt]."""
    import numpy as np
    nqt, nkt = -(-N // Bq), -(-N // Bk)
    kb = np.zeros(H * nqt, np.int32)
    ke = np.zeros(H * nqt, np.int32)
    cls = np.zeros(H * nqt * nkt, np.uint8)
    qb = np.zeros(H * nkt, np.int32)
    qe = np.zeros(H * nkt, np.int32)
    p32 = lambda a: a.ctypes.data_as(_i32p)
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_tile_schedule(N, H, lo_a, hi_a, Bq, Bk, p32(kb), p32(ke), cls.ctypes.data_as(_u8p),
                                  p32(qb), p32(qe)), "spa_tile_schedule")
    return {"kt_begin": kb.reshape(H, nqt), "kt_end": ke.reshape(H, nqt),
            "tile_class": cls.reshape(H, nqt, nkt), "qt_begin": qb.reshape(H, nkt),
            "qt_end": qe.reshape(H, nkt)}


def spa_tile_classes_device(N: int, H: int, Bq: int, Bk: int, out: torch.Tensor, lo=None, hi=None,
                            stream=None):
    nqt, nkt = -(-N // Bq), -(-N // Bk)
    _need(out, (H, nqt, nkt), torch.uint8, "out")
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_tile_classes_device(N, H, lo_a, hi_a, Bq, Bk, out.data_ptr(), _stream_ptr(stream)),
           "spa_tile_classes_device")
    return out


def spa_debug_wait_timeout(limit_ns: int, stream=None):
    """Make one device wait run out of time (see spa.h); check with spa_device_status()."""
    _check(_lib.spa_debug_wait_timeout(limit_ns, _stream_ptr(stream)), "spa_debug_wait_timeout")


def spa_device_status(stream=None) -> int:
    return int(_lib.spa_device_status(_stream_ptr(stream)))


# ------------------------------------------------------------------ conveniences
def attention_forward(q, k, v, scale=None, lo=None, hi=None):
    """Allocate o / lse and run spa_attn_fwd."""
    B, H, N, d = _dims(q)
    scale = d ** -0.5 if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    return spa_attn_fwd(q, k, v, o, lse, scale, lo, hi)


def spa_attn_decode_workspace_bytes(B: int, H: int, N: int, d: int, lo=None, hi=None) -> int:
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    return int(_lib.spa_attn_decode_workspace_bytes(B, H, N, d, lo_a, hi_a))


def spa_attn_decode(q, k, v, pos, o, lse, workspace, scale: float, lo=None, hi=None, stream=None):
    """One new token per sequence: q [B, H, d] at positions pos (int32 [B]) of
    the caches k, v [B, H, N, d]; writes o [B, H, d] and lse [B, H]."""
    B, H, N, d = _dims(k)
    _need(k, (B, H, N, d), torch.bfloat16, "k")
    _need(v, (B, H, N, d), torch.bfloat16, "v")
    _need(q, (B, H, d), torch.bfloat16, "q")
    _need(o, (B, H, d), torch.bfloat16, "o")
    _need(lse, (B, H), torch.float32, "lse")
    _need(pos, (B,), torch.int32, "pos")
    if not workspace.is_cuda or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < spa_attn_decode_workspace_bytes(B, H, N, d, lo, hi):
        raise ValueError("workspace: contiguous CUDA tensor of spa_attn_decode_workspace_bytes(...) bytes")
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_attn_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), pos.data_ptr(), o.data_ptr(),
                                lse.data_ptr(), workspace.data_ptr(), B, H, N, d, scale, lo_a, hi_a,
                                _stream_ptr(stream)), "spa_attn_decode")
    return o, lse


def attention_decode(q, k_cache, v_cache, pos, scale=None, lo=None, hi=None):
    """Allocate o / lse / workspace and run spa_attn_decode."""
    B, H, N, d = _dims(k_cache)
    scale = d ** -0.5 if scale is None else scale
    o = torch.empty((B, H, d), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    nbytes = spa_attn_decode_workspace_bytes(B, H, N, d, lo, hi)
    ws = torch.empty(max(nbytes // 4, 1), dtype=torch.float32, device=q.device)
    return spa_attn_decode(q, k_cache, v_cache, pos, o, lse, ws, scale, lo, hi)


def attention_backward(q, k, v, o, dout, lse, scale=None, lo=None, hi=None):
    """Allocate dq / dk / dv / workspace and run spa_attn_bwd."""
    B, H, N, d = _dims(q)
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(spa_attn_bwd_workspace_bytes(B, H, N) // 4, dtype=torch.float32, device=q.device)
    return spa_attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, ws, scale, lo, hi)


class SPAttentionFunction(torch.autograd.Function):
    """Band-sparse attention as an autograd function (bf16 [B, H, N, d])."""

    @staticmethod
    def forward(ctx, q, k, v, scale, lo, hi, backward="two-pass"):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        o, lse = attention_forward(q, k, v, scale, lo, hi)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.scale, ctx.lo, ctx.hi, ctx.backward = scale, lo, hi, backward
        return o

    @staticmethod
    def backward(ctx, dout):
        q, k, v, o, lse = ctx.saved_tensors
        bwd = BACKWARDS[ctx.backward]
        dq, dk, dv = bwd(q, k, v, o, dout.contiguous(), lse, ctx.scale, ctx.lo, ctx.hi)
        return dq, dk, dv, None, None, None, None


BACKWARDS = {"two-pass": attention_backward, "fused": attention_backward_fused,
             "stored": attention_backward_stored}


def spattention(q, k, v, scale=None, lo=None, hi=None, backward: str = "two-pass"):
    """SPAttention: head h of H attends to causal distances in its Balanced
    Distance Partitioning band (or the explicit bands lo/hi).  backward:
    "two-pass" (spa_attn_bwd, deterministic), "fused" (spa_attn_bwd_fused,
    dq summed by fp32 reductions) or "stored" (spa_attn_bwd_stored,
    deterministic, dS kept in a workspace of about 2 bytes per causal pair)."""
    if backward not in BACKWARDS:
        raise ValueError("backward is 'two-pass', 'fused' or 'stored'")
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    return SPAttentionFunction.apply(q, k, v, scale, lo, hi, backward)


# ------------------------------------------------------------- band + shared window
def spa_attn_union_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(_lib.spa_attn_union_workspace_bytes(B, H, N, d))


def spa_union_parts(N: int, H: int, window: int, lo=None, hi=None):
    """The two disjoint distance intervals per head that the union calls run:
    returns (a1, b1, a2, b2), lists of H ints."""
    out = [(ctypes.c_int32 * H)() for _ in range(4)]
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_union_parts(N, H, int(window), lo_a, hi_a, *out), "spa_union_parts")
    return tuple(list(a) for a in out)


def _union_ws(workspace, B, H, N, d):
    need = spa_attn_union_workspace_bytes(B, H, N, d)
    if not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace: CUDA tensor of spa_attn_union_workspace_bytes(B, H, N, d) bytes")


def spa_attn_fwd_union(q, k, v, o, lse, scale: float, window: int, lo=None, hi=None, stream=None):
    """Each head attends to its band and to the distances [0, window) that every
    head shares; writes o [B,H,N,d] bf16 and lse [B,H,N] fp32."""
    B, H, N, d = _dims(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    _need(lse, (B, H, N), torch.float32, "lse")
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    _check(_lib.spa_attn_fwd_union(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                   B, H, N, d, scale, int(window), lo_a, hi_a, _stream_ptr(stream)),
           "spa_attn_fwd_union")
    return o, lse


def spa_attn_bwd_union(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale: float, window: int, lo=None,
                       hi=None, stream=None):
    """Gradients of sum(o * dout) for spa_attn_fwd_union (o, lse from it)."""
    B, H, N, d = _dims(q)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout"), (dq, "dq"), (dk, "dk"),
                 (dv, "dv")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    _need(lse, (B, H, N), torch.float32, "lse")
    _union_ws(workspace, B, H, N, d)
    lo_a = None if lo is None else _i32(lo)
    hi_a = None if hi is None else _i32(hi)
    ptrs = [t.data_ptr() for t in (q, k, v, o, dout, lse, dq, dk, dv, workspace)]
    _check(_lib.spa_attn_bwd_union(*ptrs, B, H, N, d, scale, int(window), lo_a, hi_a, _stream_ptr(stream)),
           "spa_attn_bwd_union")
    return dq, dk, dv


def _union_workspace(q):
    B, H, N, d = _dims(q)
    nbytes = spa_attn_union_workspace_bytes(B, H, N, d)
    return torch.empty(max(nbytes // 4, 1), dtype=torch.float32, device=q.device)


def attention_forward_union(q, k, v, window: int, scale=None, lo=None, hi=None):
    """Allocate o / lse and run spa_attn_fwd_union."""
    B, H, N, d = _dims(q)
    scale = d ** -0.5 if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    return spa_attn_fwd_union(q, k, v, o, lse, scale, window, lo, hi)


def attention_backward_union(q, k, v, o, dout, lse, window: int, scale=None, lo=None, hi=None):
    """Allocate dq / dk / dv / workspace and run spa_attn_bwd_union."""
    B, H, N, d = _dims(q)
    scale = d ** -0.5 if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    return spa_attn_bwd_union(q, k, v, o, dout, lse, dq, dk, dv, _union_workspace(q), scale, window, lo, hi)


class SPAttentionUnionFunction(torch.autograd.Function):
    """Band plus a local window shared by every head, as an autograd function."""

    @staticmethod
    def forward(ctx, q, k, v, window, scale, lo, hi):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        o, lse = attention_forward_union(q, k, v, window, scale, lo, hi)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.window, ctx.scale, ctx.lo, ctx.hi = window, scale, lo, hi
        return o

    @staticmethod
    def backward(ctx, dout):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = attention_backward_union(q, k, v, o, dout.contiguous(), lse, ctx.window, ctx.scale, ctx.lo,
                                              ctx.hi)
        return dq, dk, dv, None, None, None, None


def spattention_union(q, k, v, window: int, scale=None, lo=None, hi=None):
    """Each head attends to its band and to the distances [0, window) that
    every head shares (spa_attn_fwd_union / spa_attn_bwd_union); differentiable."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    return SPAttentionUnionFunction.apply(q, k, v, int(window), scale, lo, hi)


def spa_attn_union_merge(o, lse, o2, lse2, stream=None):
    """(o, lse) <- softmax over the union of two disjoint parts' (o, lse), (o2, lse2)."""
    B, H, N, d = _dims(o)
    for t, n in ((o, "o"), (o2, "o2")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    for t, n in ((lse, "lse"), (lse2, "lse2")):
        _need(t, (B, H, N), torch.float32, n)
    _check(_lib.spa_attn_union_merge(o.data_ptr(), lse.data_ptr(), o2.data_ptr(), lse2.data_ptr(), B, H, N, d,
                                     _stream_ptr(stream)), "spa_attn_union_merge")
    return o, lse


def spa_attn_union_add_grads(dq, dk, dv, dq2, dk2, dv2, stream=None):
    """dq += dq2, dk += dk2, dv += dv2 (bf16)."""
    B, H, N, d = _dims(dq)
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv"), (dq2, "dq2"), (dk2, "dk2"), (dv2, "dv2")):
        _need(t, (B, H, N, d), torch.bfloat16, n)
    _check(_lib.spa_attn_union_add_grads(dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dq2.data_ptr(),
                                         dk2.data_ptr(), dv2.data_ptr(), B, H, N, d, _stream_ptr(stream)),
           "spa_attn_union_add_grads")
    return dq, dk, dv


# ------------------------------------------------------------- norm and rotation
DTYPES = {torch.bfloat16: 0, torch.float16: 1}  # spa_dtype_t


def _launch(device, where: str, fn, *args):
    """Calls a C entry point with `device` current (the launch goes there)."""
    if torch.cuda.current_device() == device.index:
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status != SPA_OK:
        raise SpaError(status, where)


def _stream_on(device, stream):
    """The stream's handle, or that of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _dtype_code(t: torch.Tensor, name: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None or not t.is_cuda:
        raise ValueError(f"{name}: expected CUDA bfloat16 or float16 tensor, got {t.dtype} on {t.device}")
    return code


def _need_on(t, shape, dtype, device, name):
    """A contiguous tensor of this shape and type on `device`."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _vector_rows(t, strides) -> bool:
    """Rows (the last dimension) contiguous and every row 16-byte aligned."""
    if strides[-1] != 1 or t.data_ptr() % 16:
        return False
    for n, s in zip(t.shape, strides[:-1]):
        if s % 8 and n != 1:
            return False
    return True


_Strides2, _Strides3 = _i64 * 2, _i64 * 3


def _need_rows(t, shape, dtype, device, name):
    """A tensor of this shape and type on `device`, its rows readable in 16-byte
    vectors; returns its address and its strides for a C entry point."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name}: expected {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    strides = t.stride()
    if not _vector_rows(t, strides):
        raise ValueError(f"{name}: the last dimension must be contiguous, rows 16-byte aligned and the other strides "
                         f"multiples of 8, got strides {strides}")
    return t.data_ptr(), _Strides3(*strides[:3]) if len(strides) == 4 else _Strides2(*strides[:2])


def _rope_args(table, positions, B, N, device):
    """(rot, positions pointer, stride between batches) of a checked table and positions."""
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError(f"table: expected [length, rot / 2, 2] (rope_table), got {tuple(table.shape)}")
    _need_on(table, table.shape, torch.float32, device, "table")
    rot = 2 * table.shape[1]
    if positions is None:
        if N > table.shape[0]:
            raise ValueError(f"table: {N} rows need positions up to {N - 1}, the table has {table.shape[0]}")
        return rot, None, 0
    if positions.dtype != torch.int32 or positions.device != device or tuple(positions.shape) not in ((N,), (B, N)) \
            or (N > 1 and positions.stride(-1) != 1):
        raise ValueError(f"positions: expected int32 [{N}] or [{B}, {N}] on {device}, rows contiguous, got "
                         f"{positions.dtype} {tuple(positions.shape)} on {positions.device}")
    return rot, positions.data_ptr(), positions.stride(0) if positions.dim() == 2 else 0


def _qk_dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k are [B, H, N, d]")
    B, Hq, N, d = q.shape
    return B, Hq, k.shape[1], N, d


def spa_rope_table(table, base: float, stream=None):
    """Fill table [length, rot / 2, 2] fp32 with (cos, sin) of pos * base^(-2 i / rot)."""
    if table.dim() != 3 or table.shape[2] != 2 or not table.is_cuda:
        raise ValueError(f"table: expected CUDA tensor [length, rot / 2, 2], got {tuple(table.shape)} on "
                         f"{table.device}")
    _need_on(table, table.shape, torch.float32, table.device, "table")
    _launch(table.device, "spa_rope_table", _lib.spa_rope_table, table.data_ptr(), table.shape[0], 2 * table.shape[1],
            base, _stream_on(table.device, stream))
    return table


def rope_table(length: int, rot: int, base: float = 10000.0, device=None):
    """The rotation's table for positions [0, length) and rot rotated columns."""
    if rot % 2:
        raise ValueError(f"rot: columns are rotated in pairs, got {rot}")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return spa_rope_table(torch.empty((length, rot // 2, 2), dtype=torch.float32, device=device), base)


def spa_qk_norm_rope_fwd(q, k, q_weight, k_weight, table, q_out, k_out, positions=None, eps: float = 1e-6,
                         interleaved: bool = False, stream=None):
    """q_out, k_out = the normed and rotated q [B, Hq, N, d], k [B, Hk, N, d]
    (bf16 or fp16, any strides of whole 16-byte vectors); see spa.h."""
    B, Hq, Hk, N, d = _qk_dims(q, k)
    dt, ty, dev = _dtype_code(q, "q"), q.dtype, q.device
    q_shape, k_shape = (B, Hq, N, d), (B, Hk, N, d)
    pq, sq = _need_rows(q, q_shape, ty, dev, "q")
    pk, sk = _need_rows(k, k_shape, ty, dev, "k")
    pqo, pko = _need_on(q_out, q_shape, ty, dev, "q_out"), _need_on(k_out, k_shape, ty, dev, "k_out")
    pqw = _need_on(q_weight, (d,), torch.float32, dev, "q_weight")
    pkw = _need_on(k_weight, (d,), torch.float32, dev, "k_weight")
    rot, pos, pos_stride = _rope_args(table, positions, B, N, dev)
    _launch(dev, "spa_qk_norm_rope_fwd", _lib.spa_qk_norm_rope_fwd, pq, pk, pqw, pkw, table.data_ptr(), pos, pqo, pko,
            B, Hq, Hk, N, d, rot, table.shape[0], pos_stride, sq, sk, interleaved, eps, dt, _stream_on(dev, stream))
    return q_out, k_out


@functools.lru_cache(maxsize=None)
def spa_qk_norm_rope_bwd_workspace_bytes(d: int) -> int:
    return int(_lib.spa_qk_norm_rope_bwd_workspace_bytes(d))


def spa_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, table, dq, dk, dq_weight, dk_weight, workspace,
                         positions=None, eps: float = 1e-6, interleaved: bool = False, stream=None):
    """Gradients of sum(q_out * dq_out) + sum(k_out * dk_out): writes dq, dk (any
    strides of whole 16-byte vectors) and dq_weight, dk_weight (fp32 [d]).
    workspace: CUDA tensor of spa_qk_norm_rope_bwd_workspace_bytes(d) bytes."""
    B, Hq, Hk, N, d = _qk_dims(q, k)
    _need_rows(dq, (B, Hq, N, d), q.dtype, q.device, "dq")
    _need_rows(dk, (B, Hk, N, d), q.dtype, q.device, "dk")
    _need_on(dq_weight, (d,), torch.float32, q.device, "dq_weight")
    _need_on(dk_weight, (d,), torch.float32, q.device, "dk_weight")
    if workspace.device != q.device or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < spa_qk_norm_rope_bwd_workspace_bytes(d):
        raise ValueError("workspace: contiguous CUDA tensor of spa_qk_norm_rope_bwd_workspace_bytes(d) bytes")
    return _qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, table, dq, dk, dq_weight, dk_weight, workspace,
                             positions, eps, interleaved, stream)


def _qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, table, dq, dk, dq_weight, dk_weight, workspace,
                      positions, eps, interleaved, stream=None):
    """spa_qk_norm_rope_bwd into outputs that are known to fit."""
    B, Hq, Hk, N, d = _qk_dims(q, k)
    dt, ty, dev = _dtype_code(q, "q"), q.dtype, q.device
    q_shape, k_shape = (B, Hq, N, d), (B, Hk, N, d)
    pq, sq = _need_rows(q, q_shape, ty, dev, "q")
    pk, sk = _need_rows(k, k_shape, ty, dev, "k")
    pdqo, pdko = _need_on(dq_out, q_shape, ty, dev, "dq_out"), _need_on(dk_out, k_shape, ty, dev, "dk_out")
    pqw = _need_on(q_weight, (d,), torch.float32, dev, "q_weight")
    pkw = _need_on(k_weight, (d,), torch.float32, dev, "k_weight")
    rot, pos, pos_stride = _rope_args(table, positions, B, N, dev)
    _launch(dev, "spa_qk_norm_rope_bwd", _lib.spa_qk_norm_rope_bwd, pdqo, pdko, pq, pk, pqw, pkw, table.data_ptr(), pos,
            dq.data_ptr(), dk.data_ptr(), dq_weight.data_ptr(), dk_weight.data_ptr(), workspace.data_ptr(), B, Hq, Hk,
            N, d, rot, table.shape[0], pos_stride, sq, sk, _Strides3(*dq.stride()[:3]), _Strides3(*dk.stride()[:3]),
            interleaved, eps, dt, _stream_on(dev, stream))
    return dq, dk, dq_weight, dk_weight


def qk_norm_rope_forward(q, k, q_weight, k_weight, table, positions=None, eps: float = 1e-6,
                         interleaved: bool = False):
    """Allocate q_out / k_out (contiguous) and run spa_qk_norm_rope_fwd."""
    qo = torch.empty_like(q, memory_format=torch.contiguous_format)
    ko = torch.empty_like(k, memory_format=torch.contiguous_format)
    return spa_qk_norm_rope_fwd(q, k, q_weight, k_weight, table, qo, ko, positions, eps, interleaved)


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, table, positions=None, eps: float = 1e-6,
                          interleaved: bool = False):
    """Allocate dq / dk (dense, in the order of q's and k's dimensions) /
    dq_weight / dk_weight / workspace and run spa_qk_norm_rope_bwd."""
    ws = q_weight.new_empty(spa_qk_norm_rope_bwd_workspace_bytes(q.shape[-1]) // 4, dtype=torch.float32)
    return _qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, table, torch.empty_like(q), torch.empty_like(k),
                             torch.empty_like(q_weight), torch.empty_like(k_weight), ws, positions, eps, interleaved)


def _dense(t):
    """t contiguous and on a 16-byte border: itself, or a copy (a part of a longer
    tensor may be contiguous and start anywhere)."""
    if t.is_contiguous() and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


class QKNormRopeFunction(torch.autograd.Function):
    """Norm and rotation of queries and keys as an autograd function."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, table, positions, eps, interleaved):
        q, k = (x if _vector_rows(x, x.stride()) else _dense(x) for x in (q, k))
        q_weight, k_weight, table = _dense(q_weight), _dense(k_weight), _dense(table)
        ctx.save_for_backward(q, k, q_weight, k_weight, table, positions)
        ctx.eps, ctx.interleaved = eps, interleaved
        return qk_norm_rope_forward(q, k, q_weight, k_weight, table, positions, eps, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, table, positions = ctx.saved_tensors
        grads = qk_norm_rope_backward(_dense(dq_out), _dense(dk_out), q, k, q_weight, k_weight, table,
                                      positions, ctx.eps, ctx.interleaved)
        return (*grads, None, None, None, None)


def qk_norm_rope(q, k, q_weight, k_weight, table, positions=None, eps: float = 1e-6, interleaved: bool = False):
    """RMS norm of every query and key head with its weight, then the rotary
    position rotation: what q [B, Hq, N, d] and k [B, Hk, N, d] pass through
    before spattention.  Differentiable in q, k and the weights.  q and k may
    be views of a token-major projection; the outputs are contiguous.  Weights
    of another type are used in fp32.  table: rope_table(...); positions:
    int32 [N] or [B, N], or None for 0 .. N - 1.  As with any autograd function,
    a backward() captured into a CUDA graph needs leaves that no eager graph
    still holds."""
    return QKNormRopeFunction.apply(q, k, q_weight.float(), k_weight.float(), table, positions, eps, interleaved)


# ------------------------------------------------------------- paged cache
def _need_cache(k_pages, v_pages, page_table, cu_q, kv_len, Hk, d, dtype, device):
    """Checks the cache's tensors; returns (B, pages, page, width, their addresses)."""
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_pages and v_pages are [pages, Hk, page, d], page_table is [B, width]")
    pages, page = k_pages.shape[0], k_pages.shape[2]
    B, width = page_table.shape
    shape = (pages, Hk, page, d)
    ptrs = (_need_on(k_pages, shape, dtype, device, "k_pages"), _need_on(v_pages, shape, dtype, device, "v_pages"),
            _need_on(page_table, (B, width), torch.int32, device, "page_table"),
            _need_on(cu_q, (B + 1,), torch.int32, device, "cu_q"),
            _need_on(kv_len, (B,), torch.int32, device, "kv_len"))
    return B, pages, page, width, ptrs


def spa_paged_append(q, k, v, q_weight, k_weight, table, cu_q, kv_len, page_table, q_out, k_pages, v_pages,
                     eps: float = 1e-6, interleaved: bool = False, stream=None):
    """The new tokens' q [T, Hq, d] and k [T, Hk, d] normed and rotated at their
    positions; q to q_out, k and v to their places in the pages (spa.h)."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v are [T, H, d]")
    T, Hq, d = q.shape
    Hk = k.shape[1]
    dt, ty, dev = _dtype_code(q, "q"), q.dtype, q.device
    pq, sq = _need_rows(q, (T, Hq, d), ty, dev, "q")
    pk, sk = _need_rows(k, (T, Hk, d), ty, dev, "k")
    pv, sv = _need_rows(v, (T, Hk, d), ty, dev, "v")
    po = _need_on(q_out, (T, Hq, d), ty, dev, "q_out")
    pqw = _need_on(q_weight, (d,), torch.float32, dev, "q_weight")
    pkw = _need_on(k_weight, (d,), torch.float32, dev, "k_weight")
    B, pages, page, width, (pkp, pvp, ppt, pcu, pkv) = _need_cache(k_pages, v_pages, page_table, cu_q, kv_len, Hk, d,
                                                                  ty, dev)
    rot, _, _ = _rope_args(table, None, 1, 0, dev)
    _launch(dev, "spa_paged_append", _lib.spa_paged_append, pq, pk, pv, pqw, pkw, table.data_ptr(), pcu, pkv, ppt, po,
            pkp, pvp, B, T, Hq, Hk, d, pages, page, width, rot, table.shape[0], sq, sk, sv, interleaved, eps, dt,
            _stream_on(dev, stream))
    return q_out


def paged_append(q, k, v, k_pages, v_pages, page_table, cu_q, kv_len, q_weight, k_weight, table, eps: float = 1e-6,
                 interleaved: bool = False, out=None):
    """Norm and rotate the new tokens' queries and keys, store keys and values in
    the paged cache, return the queries (allocated unless given as out; rows
    behind the last sequence are not written).  The weights are fp32."""
    out = torch.empty_like(q, memory_format=torch.contiguous_format) if out is None else out
    return spa_paged_append(q, k, v, q_weight, k_weight, table, cu_q, kv_len, page_table, out, k_pages, v_pages, eps,
                            interleaved)


@functools.lru_cache(maxsize=64)
def spa_paged_attn_workspace_bytes(max_q: int, d: int) -> int:
    return int(_lib.spa_paged_attn_workspace_bytes(max_q, d))


def spa_paged_attn(q, k_pages, v_pages, page_table, cu_q, kv_len, max_q: int, o, lse, workspace, N: int, scale: float,
                   lo=None, hi=None, stream=None):
    """Attention of the new tokens' q [T, Hq, d] over the paged cache: writes
    o [T, Hq, d] and lse [T, Hq] fp32 (spa.h).  Bands: lo / hi per query head,
    or the Balanced Distance Partitioning ones of length N."""
    if q.dim() != 3 or k_pages.dim() != 4:
        raise ValueError("q is [T, Hq, d], k_pages and v_pages are [pages, Hk, page, d]")
    T, Hq, d = q.shape
    Hk = k_pages.shape[1]
    dt, ty, dev = _dtype_code(q, "q"), q.dtype, q.device
    pq, po = _need_on(q, (T, Hq, d), ty, dev, "q"), _need_on(o, (T, Hq, d), ty, dev, "o")
    pl = _need_on(lse, (T, Hq), torch.float32, dev, "lse")
    B, pages, page, width, (pkp, pvp, ppt, pcu, pkv) = _need_cache(k_pages, v_pages, page_table, cu_q, kv_len, Hk, d,
                                                                  ty, dev)
    if workspace.device != dev or not workspace.is_contiguous() or \
            workspace.numel() * workspace.element_size() < spa_paged_attn_workspace_bytes(max_q, d):
        raise ValueError("workspace: contiguous CUDA tensor of spa_paged_attn_workspace_bytes(max_q, d) bytes")
    if (lo is not None and len(lo) != Hq) or (hi is not None and len(hi) != Hq):
        raise ValueError(f"lo and hi: {Hq} entries, one for each query head")
    lo_a, hi_a = (None if x is None else array.array("i", x) for x in (lo, hi))
    _launch(dev, "spa_paged_attn", _lib.spa_paged_attn, pq, pkp, pvp, ppt, pcu, pkv, po, pl, workspace.data_ptr(), B, T,
            max_q, Hq, Hk, pages, page, width, N, d, scale, lo_a and lo_a.buffer_info()[0],
            hi_a and hi_a.buffer_info()[0], dt, _stream_on(dev, stream))
    return o, lse


def paged_attention(q, k_pages, v_pages, page_table, cu_q, kv_len, max_q: int, scale=None, lo=None, hi=None, N=None,
                    out=None, lse=None):
    """Attention of the new tokens (one or many per sequence) over the paged
    cache; allocates o / lse (unless given as out, lse) and the workspace and
    runs spa_paged_attn.  max_q: no sequence may have more new tokens; rows past
    that many of a sequence, and rows behind the last sequence, are not written.
    N: the length that the model's bands belong to; it may be left out where lo
    and hi give the bands (it then only bounds them: what the page table can
    hold)."""
    if N is None and (lo is None or hi is None):
        raise ValueError("N: without both lo and hi the bands follow from the length that the model was trained with")
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    N = page_table.shape[-1] * k_pages.shape[2] if N is None else N
    out = torch.empty_like(q, memory_format=torch.contiguous_format) if out is None else out
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if lse is None else lse
    ws = lse.new_empty(spa_paged_attn_workspace_bytes(max_q, d) // 4)
    return spa_paged_attn(q, k_pages, v_pages, page_table, cu_q, kv_len, max_q, out, lse, ws, N, scale, lo, hi)
