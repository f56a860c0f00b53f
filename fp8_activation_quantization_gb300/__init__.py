"""GB300-native per-token-group FP8 activation quantization.

A thin ctypes binding over ``libtkq.so`` (C ABI in ``include/tkq.h``).  Every
step of the computation runs in the library's CUDA kernels; this module only
marshals pointers, sizes and the current CUDA stream, and allocates output
tensors with PyTorch.  There is no CPU fallback: if the library is missing or a
call fails, an exception is raised.

Low-level names mirror the C ABI (``tkq_per_token_cast``, ``tkq_swiglu_cast``,
``tkq_swiglu_cast_t``: raw device pointers, return the status code).  The
tensor-level helpers follow the call shape of the TileKernels quant API
(``per_token_cast(x, fmt='e4m3', num_per_channels=128) -> (out, out_sf)``,
"DeepSeek开源TileKernels：用Python写的GPU算子逼近硬件性能上限", quick start).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

__all__ = [
    "TkqError", "library_path", "load_library", "tkq_per_token_cast", "tkq_swiglu_cast",
    "tkq_swiglu_cast_t", "tkq_swiglu_backward_cast", "tkq_status_string", "per_token_cast",
    "swiglu_forward_and_per_token_cast", "swiglu_backward_and_per_token_cast",
    "tkq_read_device_status", "tkq_selftest_wait_timeout", "FMT_E4M3", "FMT_E5M2", "GROUP",
    "tkq_per_channel_cast", "tkq_per_block_cast", "tkq_cast_back", "per_channel_cast",
    "per_block_cast", "cast_back", "OUT_F32", "OUT_BF16", "tkq_swiglu_cast_clamp",
    "tkq_swiglu_cast_t_clamp", "tkq_swiglu_cast_t_ex", "tkq_per_token_cast_f32", "tkq_swiglu_values", "swiglu_values",
    "use_checked_library", "tkq_checked_build", "tkq_read_check_address",
    "tkq_swiglu_backward_values", "swiglu_backward_values", "tkq_fp8_encode", "fp8_encode",
    "tkq_route_topk", "tkq_route_topk_backward", "route_topk", "route_topk_backward",
    "tkq_swiglu_cast_checkpoint", "tkq_swiglu_checkpoint_backward",
    "tkq_swiglu_checkpoint_backward_cast", "swiglu_forward_cast_and_checkpoint",
    "swiglu_backward_from_checkpoint", "tkq_residual_norm_cast", "tkq_residual_norm_workspace",
    "tkq_residual_norm_backward", "residual_norm_and_cast", "residual_norm_backward",
]

FMT_E4M3 = 0
FMT_E5M2 = 1
GROUP = 128
_FMTS = {"e4m3": FMT_E4M3, "e5m2": FMT_E5M2}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libtkq.so")
# the access-checked test build of the same sources (see include/tkq.h)
_LIB_CHECKED_PATH = os.path.join(_HERE, "_lib", "libtkq_checked.so")
_lock = threading.RLock()
_lib = None          # the library every call of this module goes to
_opened = {}         # path -> loaded library


class TkqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {tkq_status_string(status)} (status {status})")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libtkq.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = _open(_LIB_PATH)
        return _lib


@contextlib.contextmanager
def use_checked_library():
    """Route this module's calls to the access-checked build libtkq_checked.so
    (built by ``_build.build(checked=True)``) inside the ``with`` block."""
    global _lib
    with _lock:
        prev = _lib
        _lib = _open(_LIB_CHECKED_PATH)
    try:
        yield _lib
    finally:
        with _lock:
            _lib = prev


def _open(path):
    with _lock:
        if path in _opened:
            return _opened[path]
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        p, i64, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.tkq_per_token_cast.argtypes = [p, p, p, i64, i64, i, i, p]
        lib.tkq_per_token_cast.restype = i
        lib.tkq_swiglu_cast.argtypes = [p, p, p, p, i64, i64, i, i, p]
        lib.tkq_swiglu_cast.restype = i
        lib.tkq_swiglu_cast_t.argtypes = [p, p, p, p, p, p, i64, i64, i, i, p]
        lib.tkq_swiglu_cast_t.restype = i
        lib.tkq_status_string.argtypes = [i]
        lib.tkq_status_string.restype = ctypes.c_char_p
        lib.tkq_version.argtypes = []
        lib.tkq_version.restype = i
        lib.tkq_swiglu_backward_cast.argtypes = [p, p, p, p, p, i64, i64, i, i, p]
        lib.tkq_swiglu_backward_cast.restype = i
        u = ctypes.c_uint
        lib.tkq_per_token_cast_ex.argtypes = [p, p, p, i64, i64, i, i, u, p]
        lib.tkq_per_token_cast_ex.restype = i
        lib.tkq_swiglu_cast_ex.argtypes = [p, p, p, p, i64, i64, i, i, u, p]
        lib.tkq_swiglu_cast_ex.restype = i
        lib.tkq_swiglu_backward_cast_ex.argtypes = [p, p, p, p, p, i64, i64, i, i, u, p]
        lib.tkq_swiglu_backward_cast_ex.restype = i
        lib.tkq_sf_bytes.argtypes = [i64, i64, u]
        lib.tkq_sf_bytes.restype = i64
        lib.tkq_read_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), i]
        lib.tkq_read_device_status.restype = i
        lib.tkq_selftest_wait_timeout.argtypes = [i64, p]
        lib.tkq_selftest_wait_timeout.restype = i
        lib.tkq_per_channel_cast.argtypes = [p, p, p, i64, i64, i, i, i, p]
        lib.tkq_per_channel_cast.restype = i
        lib.tkq_per_block_cast.argtypes = [p, p, p, i64, i64, i, i, p]
        lib.tkq_per_block_cast.restype = i
        lib.tkq_cast_back.argtypes = [p, p, p, i64, i64, i, i, i, i, p]
        lib.tkq_cast_back.restype = i
        f32 = ctypes.c_float
        lib.tkq_swiglu_cast_clamp.argtypes = [p, p, p, p, i64, i64, i, i, u, f32, p, p]
        lib.tkq_swiglu_cast_clamp.restype = i
        lib.tkq_swiglu_cast_t_clamp.argtypes = [p, p, p, p, p, p, i64, i64, i, i, u, f32, p, p]
        lib.tkq_swiglu_cast_t_clamp.restype = i
        lib.tkq_swiglu_cast_t_ex.argtypes = [p, p, p, p, p, p, i64, i64, i, i, u, p]
        lib.tkq_swiglu_cast_t_ex.restype = i
        lib.tkq_per_token_cast_f32.argtypes = [p, p, p, i64, i64, i, i, u, p]
        lib.tkq_per_token_cast_f32.restype = i
        lib.tkq_swiglu_values.argtypes = [p, p, p, i64, i64, p]
        lib.tkq_swiglu_values.restype = i
        lib.tkq_swiglu_backward_values.argtypes = [p, p, p, p, i64, i64, p]
        lib.tkq_swiglu_backward_values.restype = i
        lib.tkq_fp8_encode.argtypes = [p, p, i64, i, p]
        lib.tkq_fp8_encode.restype = i
        lib.tkq_route_topk.argtypes = [p, p, p, p, p, i64, i64, i64, i, i, i, i, i, u, f32, p]
        lib.tkq_route_topk.restype = i
        lib.tkq_route_topk_backward.argtypes = [p, p, p, p, i64, i64, i64, i, i, u, f32, p]
        lib.tkq_route_topk_backward.restype = i
        lib.tkq_swiglu_cast_checkpoint.argtypes = [p, p, p, p, p, p, i64, i64, i, i, i, u, p]
        lib.tkq_swiglu_cast_checkpoint.restype = i
        lib.tkq_swiglu_checkpoint_backward.argtypes = [p] * 7 + [i64, i64, i, i, p]
        lib.tkq_swiglu_checkpoint_backward.restype = i
        lib.tkq_swiglu_checkpoint_backward_cast.argtypes = [p] * 8 + [i64, i64, i, i, i, u, p]
        lib.tkq_swiglu_checkpoint_backward_cast.restype = i
        lib.tkq_residual_norm_cast.argtypes = [p] * 11 + [i64, i64, i, i, u, u, f32, f32, p]
        lib.tkq_residual_norm_cast.restype = i
        lib.tkq_residual_norm_workspace.argtypes = [i64, i64]
        lib.tkq_residual_norm_workspace.restype = i64
        lib.tkq_residual_norm_backward.argtypes = [p] * 15 + [i64, i64, u, f32, p]
        lib.tkq_residual_norm_backward.restype = i
        lib.tkq_checked_build.argtypes = []
        lib.tkq_checked_build.restype = i
        lib.tkq_read_check_address.argtypes = [ctypes.POINTER(ctypes.c_uint64), i]
        lib.tkq_read_check_address.restype = i
        _opened[path] = lib
        return lib


DEVICE_TIMEOUT = 1
ERR_TIMEOUT = 7    # tkq_read_device_status: the status word holds DEVICE_TIMEOUT
DEVICE_OUT_OF_BOUNDS = 2


def tkq_checked_build() -> bool:
    return bool((_lib or load_library()).tkq_checked_build())


def tkq_read_check_address(clear: bool = False) -> int:
    """Synchronize the current device and return the first address an access
    check refused (bit 63 set for a store; 0 if none, and always 0 in the
    release build)."""
    v = ctypes.c_uint64(0)
    st = (_lib or load_library()).tkq_read_check_address(ctypes.byref(v), 1 if clear else 0)
    if st:
        raise TkqError(st, "tkq_read_check_address")
    return int(v.value)


def tkq_read_device_status(clear: bool = False) -> int:
    """Synchronize the current device and return its status word (bit
    DEVICE_TIMEOUT: a bounded wait inside a kernel gave up; the C call then
    returns ERR_TIMEOUT, which here is the word's bit, not an exception)."""
    v = ctypes.c_uint32(0)
    st = (_lib or load_library()).tkq_read_device_status(ctypes.byref(v), 1 if clear else 0)
    if st and st != ERR_TIMEOUT:
        raise TkqError(st, "tkq_read_device_status")
    return int(v.value)


def tkq_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return (_lib or load_library()).tkq_selftest_wait_timeout(int(limit_ns), stream)


def tkq_status_string(status: int) -> str:
    return (_lib or load_library()).tkq_status_string(int(status)).decode()


# ---------------------------------------------------------------------------
# C-ABI mirrors: raw device pointers (ints or None), sizes, stream handle.
# ---------------------------------------------------------------------------

def tkq_per_token_cast(x, out, sf, T, C, group=GROUP, fmt=FMT_E4M3, stream=None) -> int:
    return (_lib or load_library()).tkq_per_token_cast(x, out, sf, T, C, group, fmt, stream)


def tkq_swiglu_cast(x, w, out, sf, T, H, group=GROUP, fmt=FMT_E4M3, stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_cast(x, w, out, sf, T, H, group, fmt, stream)


def tkq_swiglu_cast_t(x, w, out, sf, out_t, sf_t, T, H, group=GROUP, fmt=FMT_E4M3,
                      stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_cast_t(x, w, out, sf, out_t, sf_t, T, H, group, fmt, stream)


def tkq_swiglu_backward_cast(x, dy, w, out, sf, T, H, group=GROUP, fmt=FMT_E4M3,
                             stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_backward_cast(x, dy, w, out, sf, T, H, group, fmt, stream)


def tkq_per_token_cast_f32(x, out, sf, T, C, group=GROUP, fmt=FMT_E4M3, sf_flags=0,
                           stream=None) -> int:
    return (_lib or load_library()).tkq_per_token_cast_f32(x, out, sf, T, C, group, fmt, sf_flags, stream)


def tkq_swiglu_values(x, w, y, T, H, stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_values(x, w, y, T, H, stream)


def tkq_fp8_encode(x, out, n, fmt=FMT_E4M3, stream=None) -> int:
    return (_lib or load_library()).tkq_fp8_encode(x, out, n, fmt, stream)


def tkq_swiglu_backward_values(x, dy, w, y, T, H, stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_backward_values(x, dy, w, y, T, H, stream)


def tkq_swiglu_cast_clamp(x, w, out, sf, T, H, group=GROUP, fmt=FMT_E4M3, sf_flags=0,
                          clamp_value=0.0, clamp_count=None, stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_cast_clamp(x, w, out, sf, T, H, group, fmt, sf_flags,
                                                clamp_value, clamp_count, stream)


def tkq_swiglu_cast_t_clamp(x, w, out, sf, out_t, sf_t, T, H, group=GROUP, fmt=FMT_E4M3,
                            sf_flags=0, clamp_value=0.0, clamp_count=None, stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_cast_t_clamp(x, w, out, sf, out_t, sf_t, T, H, group,
                                                            fmt, sf_flags, clamp_value, clamp_count,
                                                            stream)


def tkq_swiglu_cast_t_ex(x, w, out, sf, out_t, sf_t, T, H, group=GROUP, fmt=FMT_E4M3, sf_flags=0,
                         stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_cast_t_ex(x, w, out, sf, out_t, sf_t, T, H, group,
                                                         fmt, sf_flags, stream)


def tkq_per_channel_cast(x, out, sf, T, C, group=GROUP, fmt=FMT_E4M3, transpose=0,
                         stream=None) -> int:
    return (_lib or load_library()).tkq_per_channel_cast(x, out, sf, T, C, group, fmt, int(transpose),
                                               stream)


def tkq_per_block_cast(x, out, sf, T, C, block=GROUP, fmt=FMT_E4M3, stream=None) -> int:
    return (_lib or load_library()).tkq_per_block_cast(x, out, sf, T, C, block, fmt, stream)


OUT_F32 = 0
OUT_BF16 = 1


def tkq_cast_back(codes, sf, out, T, C, group_rows=1, group_cols=GROUP, fmt=FMT_E4M3,
                  out_dtype=OUT_F32, stream=None) -> int:
    return (_lib or load_library()).tkq_cast_back(codes, sf, out, T, C, group_rows, group_cols, fmt,
                                        out_dtype, stream)


SF_ROUND_POW2 = 1
SF_UE8M0_PACKED = 2
SF_COL_MAJOR = 4
Q_RECIPROCAL = 8   # plain casts: codes of x * fl32(1/s) instead of fl32(x/s)


def tkq_sf_bytes(T, groups_per_row, sf_flags=0) -> int:
    return (_lib or load_library()).tkq_sf_bytes(T, groups_per_row, sf_flags)


def tkq_per_token_cast_ex(x, out, sf, T, C, group=GROUP, fmt=FMT_E4M3, sf_flags=0,
                          stream=None) -> int:
    return (_lib or load_library()).tkq_per_token_cast_ex(x, out, sf, T, C, group, fmt, sf_flags, stream)


def tkq_swiglu_cast_ex(x, w, out, sf, T, H, group=GROUP, fmt=FMT_E4M3, sf_flags=0,
                       stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_cast_ex(x, w, out, sf, T, H, group, fmt, sf_flags, stream)


def tkq_swiglu_backward_cast_ex(x, dy, w, out, sf, T, H, group=GROUP, fmt=FMT_E4M3, sf_flags=0,
                                stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_backward_cast_ex(x, dy, w, out, sf, T, H, group, fmt,
                                                      sf_flags, stream)


ROUTE_SIGMOID = 1
ROUTE_RENORM = 2
NORM_POST = 1
NORM_PRE = 2
NORM_RES_F32 = 4


def tkq_route_topk(logits, bias, ids, weights, counts, T, E, ld, dtype, k, n_groups=1,
                   topk_groups=1, group_top=2, route_flags=0, scale=1.0, stream=None) -> int:
    return (_lib or load_library()).tkq_route_topk(logits, bias, ids, weights, counts, T, E, ld,
                                                   dtype, k, n_groups, topk_groups, group_top,
                                                   route_flags, scale, stream)


def tkq_route_topk_backward(logits, ids, dweights, dlogits, T, E, ld, dtype, k, route_flags=0,
                            scale=1.0, stream=None) -> int:
    return (_lib or load_library()).tkq_route_topk_backward(logits, ids, dweights, dlogits, T, E,
                                                            ld, dtype, k, route_flags, scale,
                                                            stream)


def tkq_swiglu_cast_checkpoint(x, w, out, sf, ckpt, ckpt_sf, T, H, group=GROUP, fmt=FMT_E4M3,
                               ckpt_fmt=FMT_E4M3, sf_flags=0, stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_cast_checkpoint(x, w, out, sf, ckpt, ckpt_sf, T, H,
                                                               group, fmt, ckpt_fmt, sf_flags,
                                                               stream)


def tkq_swiglu_checkpoint_backward(ckpt, ckpt_sf, dy, w, dx, y, dw, T, H, group=GROUP,
                                   ckpt_fmt=FMT_E4M3, stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_checkpoint_backward(ckpt, ckpt_sf, dy, w, dx, y, dw,
                                                                   T, H, group, ckpt_fmt, stream)


def tkq_swiglu_checkpoint_backward_cast(ckpt, ckpt_sf, dy, w, dx, dx_sf, y, dw, T, H, group=GROUP,
                                        ckpt_fmt=FMT_E4M3, fmt=FMT_E4M3, sf_flags=0,
                                        stream=None) -> int:
    return (_lib or load_library()).tkq_swiglu_checkpoint_backward_cast(
        ckpt, ckpt_sf, dy, w, dx, dx_sf, y, dw, T, H, group, ckpt_fmt, fmt, sf_flags, stream)


def tkq_residual_norm_cast(r, h, w_post, gate, w_pre, r_out, out, sf, x_out, rstd_post, rstd_pre,
                           T, C, group=GROUP, fmt=FMT_E4M3, sf_flags=0, norm_flags=0,
                           res_scale=1.0, eps=1e-6, stream=None) -> int:
    return (_lib or load_library()).tkq_residual_norm_cast(
        r, h, w_post, gate, w_pre, r_out, out, sf, x_out, rstd_post, rstd_pre, T, C, group, fmt,
        sf_flags, norm_flags, res_scale, eps, stream)


def tkq_residual_norm_workspace(T, C) -> int:
    return (_lib or load_library()).tkq_residual_norm_workspace(T, C)


def tkq_residual_norm_backward(dr, dx, r, h, w_post, gate, w_pre, rstd_post, rstd_pre, dr_out, dh,
                               dgate, dw_post, dw_pre, workspace, T, C, norm_flags=0,
                               res_scale=1.0, stream=None) -> int:
    return (_lib or load_library()).tkq_residual_norm_backward(
        dr, dx, r, h, w_post, gate, w_pre, rstd_post, rstd_pre, dr_out, dh, dgate, dw_post, dw_pre,
        workspace, T, C, norm_flags, res_scale, stream)


def _sf_shape(T: int, groups_per_row: int, sf_flags: int):
    """Shape and element type of the scales in the layout `sf_flags` selects:
    fp32 [T, G], fp32 [G, T4], int32 [T, W] or int32 [W, T4] (T4 = T rounded
    up to 4, W = G / 4 rounded up)."""
    T4 = (T + 3) // 4 * 4
    W = (groups_per_row + 3) // 4
    if sf_flags & SF_UE8M0_PACKED:
        return ((W, T4) if sf_flags & SF_COL_MAJOR else (T, W)), "int32"
    return ((groups_per_row, T4) if sf_flags & SF_COL_MAJOR else (T, groups_per_row)), "float32"


def sf_tensor(T: int, groups_per_row: int, sf_flags: int, device):
    """An empty scale tensor shaped for the layout `sf_flags` selects:
    fp32 [T, G], fp32 [G, T4], int32 [T, W] or int32 [W, T4]."""
    import torch
    shape, dt = _sf_shape(T, groups_per_row, sf_flags)
    return torch.empty(shape, dtype=getattr(torch, dt), device=device)


# ---------------------------------------------------------------------------
# Tensor-level helpers (PyTorch supplies device memory and the stream).
# ---------------------------------------------------------------------------

def _fmt_code(fmt) -> int:
    if isinstance(fmt, str):
        if fmt not in _FMTS:
            raise ValueError(f"unknown fmt {fmt!r}: expected 'e4m3' or 'e5m2'")
        return _FMTS[fmt]
    return int(fmt)


def _fp8_dtype(fmt_code: int):
    import torch
    return torch.float8_e4m3fn if fmt_code == FMT_E4M3 else torch.float8_e5m2


def _check_input(x, name="x", allow_f32=False):
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    ok = (torch.bfloat16, torch.float32) if allow_f32 else (torch.bfloat16,)
    if x.dtype not in ok or x.dim() != 2 or not x.is_contiguous():
        raise TypeError(f"{name} must be a contiguous 2-D "
                        + ("bfloat16 or float32" if allow_f32 else "bfloat16") + " tensor")


def _check_out(t, name, x, nbytes, itemsize=None, dtype=None):
    """A caller-supplied output buffer: a contiguous CUDA tensor on x's device
    of at least `nbytes` bytes (the kernels write exactly the bytes the call's
    shape and layout give, so a smaller buffer would be written past its end).
    `itemsize` / `dtype` pin the element size or type where the layout fixes
    them; scale buffers of any element type are accepted by size."""
    import torch
    if not isinstance(t, torch.Tensor) or t.device != x.device or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA tensor on x's device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if itemsize is not None and t.element_size() != itemsize:
        raise TypeError(f"{name} must have {itemsize}-byte elements")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes; "
                         f"the call writes {nbytes}")


def _check_sf_out(t, name, x, rows, groups_per_row, sf_flags):
    shape, _ = _sf_shape(rows, groups_per_row, sf_flags)
    _check_out(t, name, x, 4 * shape[0] * shape[1])


def _stream_handle(dev):
    """The current stream of `dev` as an int (ctypes passes it as void*).
    torch's raw-stream query avoids building a Stream object per call; the
    public call is used where that query does not exist."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(dev.index if dev.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(dev).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


_NO_CONTEXT = contextlib.nullcontext()


def _device_ctx(dev):
    """The launch must happen on the tensors' device: switch only if it is not
    the current one (entering torch.cuda.device costs more than the launch)."""
    import torch
    if dev.index is None or dev.index == torch.cuda.current_device():
        return _NO_CONTEXT
    return torch.cuda.device(dev)


def _sf_flags(round_sf: bool, use_packed_ue8m0: bool, use_tma_aligned_col_major_sf: bool) -> int:
    """The TileKernels cast-config options ("DeepSeek开源TileKernels..." §3.1) as
    the C ABI's TKQ_SF_* flags."""
    return ((SF_ROUND_POW2 if round_sf else 0) | (SF_UE8M0_PACKED if use_packed_ue8m0 else 0)
            | (SF_COL_MAJOR if use_tma_aligned_col_major_sf else 0))


def _check_weights(topk_weights, T, x):
    import torch
    if topk_weights is not None:
        if (topk_weights.dtype != torch.float32 or topk_weights.numel() != T
                or not topk_weights.is_contiguous() or topk_weights.device != x.device):
            raise TypeError("topk_weights must be a contiguous fp32 tensor of T elements on x's device")


def per_token_cast(x, fmt="e4m3", num_per_channels: int = GROUP, out=None, out_sf=None,
                   round_sf: bool = False, use_packed_ue8m0: bool = False,
                   use_tma_aligned_col_major_sf: bool = False, use_sf_inv: bool = False):
    """bf16 or fp32 [T, C] -> (FP8 codes [T, C], scales).  Scales are fp32
    [T, C/128] unless a scale-layout option is set (see ``sf_tensor`` for the
    shapes).  Codes are those of the exact quotient x / s, or with
    ``use_sf_inv`` those of the product x * fl32(1 / s) (TKQ_Q_RECIPROCAL)."""
    import torch
    _check_input(x, allow_f32=True)
    f = _fmt_code(fmt)
    T, C = x.shape
    flags = _sf_flags(round_sf, use_packed_ue8m0, use_tma_aligned_col_major_sf)
    if use_sf_inv:
        flags |= Q_RECIPROCAL
    G = C // max(num_per_channels, 1)
    if out is None:
        out = torch.empty((T, C), dtype=_fp8_dtype(f), device=x.device)
    else:
        _check_out(out, "out", x, T * C, itemsize=1)
    if out_sf is None:
        out_sf = sf_tensor(T, G, flags, x.device)
    else:
        _check_sf_out(out_sf, "out_sf", x, T, G, flags)
    with _device_ctx(x.device):
        call = tkq_per_token_cast_f32 if x.dtype == torch.float32 else tkq_per_token_cast_ex
        st = call(_ptr(x), _ptr(out), _ptr(out_sf), T, C, num_per_channels, f, flags,
                  _stream_handle(x.device))
    if st:
        raise TkqError(st, "tkq_per_token_cast")
    return out, out_sf


def swiglu_forward_and_per_token_cast(x, fmt="e4m3", num_per_channels: int = GROUP,
                                      topk_weights=None, with_transpose: bool = False,
                                      out=None, out_sf=None, out_t=None, out_sf_t=None,
                                      round_sf: bool = False, use_packed_ue8m0: bool = False,
                                      use_tma_aligned_col_major_sf: bool = False,
                                      use_clamp: bool = False, swiglu_clamp_value=None,
                                      clamp_count=None):
    """bf16 [T, 2H] (gate | up) -> (codes [T, H], scales [T, H/128]) and, with
    ``with_transpose``, also (codes_t [H, T], scales_t [H, T/128]).
    ``topk_weights``: optional fp32 [T] routing weight per row.  The scale-layout
    options apply to the row scales and, with ``with_transpose``, to the column
    scales as an [H, T/128] matrix (see ``sf_tensor`` for the shapes).  Codes
    are those of the product y * fl32(1 / s) (the TileKernels sf_inv reading).
    ``use_clamp``: clamp the gate to <= swiglu_clamp_value and the up projection
    to [-swiglu_clamp_value, swiglu_clamp_value] before the SwiGLU; the number of
    changed values is added to ``clamp_count`` (a zeroed int64 CUDA tensor of one
    element) when given."""
    import torch
    _check_input(x)
    clamp = None
    if use_clamp:
        if swiglu_clamp_value is None:
            raise ValueError("use_clamp needs swiglu_clamp_value")
        clamp = float(swiglu_clamp_value)
        if clamp_count is not None and (clamp_count.dtype != torch.int64 or clamp_count.numel() != 1
                                        or clamp_count.device != x.device):
            raise TypeError("clamp_count must be a one-element int64 tensor on x's device")
    elif clamp_count is not None:
        raise ValueError("clamp_count needs use_clamp")
    f = _fmt_code(fmt)
    T, H2 = x.shape
    if H2 % 2:
        raise ValueError("x must have an even number of columns (gate | up)")
    H = H2 // 2
    g = max(num_per_channels, 1)
    _check_weights(topk_weights, T, x)
    flags = _sf_flags(round_sf, use_packed_ue8m0, use_tma_aligned_col_major_sf)
    if out is None:
        out = torch.empty((T, H), dtype=_fp8_dtype(f), device=x.device)
    else:
        _check_out(out, "out", x, T * H, itemsize=1)
    if out_sf is None:
        out_sf = sf_tensor(T, H // g, flags, x.device)
    else:
        _check_sf_out(out_sf, "out_sf", x, T, H // g, flags)
    with _device_ctx(x.device):
        stream = _stream_handle(x.device)
        if not with_transpose:
            if clamp is None:
                st = tkq_swiglu_cast_ex(_ptr(x), _ptr(topk_weights), _ptr(out), _ptr(out_sf), T,
                                        H, num_per_channels, f, flags, stream)
            else:
                st = tkq_swiglu_cast_clamp(_ptr(x), _ptr(topk_weights), _ptr(out), _ptr(out_sf),
                                           T, H, num_per_channels, f, flags, clamp,
                                           _ptr(clamp_count), stream)
            if st:
                raise TkqError(st, "tkq_swiglu_cast")
            return out, out_sf
        if out_t is None:
            out_t = torch.empty((H, T), dtype=_fp8_dtype(f), device=x.device)
        else:
            _check_out(out_t, "out_t", x, H * T, itemsize=1)
        if out_sf_t is None:
            out_sf_t = sf_tensor(H, T // g, flags, x.device)
        else:
            _check_sf_out(out_sf_t, "out_sf_t", x, H, T // g, flags)
        if clamp is None:
            st = tkq_swiglu_cast_t_ex(_ptr(x), _ptr(topk_weights), _ptr(out), _ptr(out_sf),
                                      _ptr(out_t), _ptr(out_sf_t), T, H, num_per_channels, f,
                                      flags, stream)
        else:
            st = tkq_swiglu_cast_t_clamp(_ptr(x), _ptr(topk_weights), _ptr(out), _ptr(out_sf),
                                         _ptr(out_t), _ptr(out_sf_t), T, H, num_per_channels, f,
                                         flags, clamp, _ptr(clamp_count), stream)
        if st:
            raise TkqError(st, "tkq_swiglu_cast_t")
        return out, out_sf, out_t, out_sf_t


def swiglu_backward_and_per_token_cast(x, dy, fmt="e4m3", num_per_channels: int = GROUP,
                                       topk_weights=None, out=None, out_sf=None,
                                       round_sf: bool = False, use_packed_ue8m0: bool = False,
                                       use_tma_aligned_col_major_sf: bool = False):
    """Gradients of y = silu(gate) * up [* w] from dy, cast per token.
    x: bf16 [T, 2H] (gate | up); dy: bf16 [T, H] -> (codes [T, 2H] of [dg | du],
    scales [T, 2H/128] or the chosen scale layout); codes of the products by
    fl32(1 / s), like the forward cast."""
    import torch
    _check_input(x)
    _check_input(dy, "dy")
    f = _fmt_code(fmt)
    T, H2 = x.shape
    H = H2 // 2
    if H2 % 2 or tuple(dy.shape) != (T, H) or dy.device != x.device:
        raise ValueError("dy must be [T, H] for x [T, 2H], on the same device")
    _check_weights(topk_weights, T, x)
    g = max(num_per_channels, 1)
    flags = _sf_flags(round_sf, use_packed_ue8m0, use_tma_aligned_col_major_sf)
    if out is None:
        out = torch.empty((T, 2 * H), dtype=_fp8_dtype(f), device=x.device)
    else:
        _check_out(out, "out", x, T * 2 * H, itemsize=1)
    if out_sf is None:
        out_sf = sf_tensor(T, 2 * H // g, flags, x.device)
    else:
        _check_sf_out(out_sf, "out_sf", x, T, 2 * H // g, flags)
    with _device_ctx(x.device):
        st = tkq_swiglu_backward_cast_ex(_ptr(x), _ptr(dy), _ptr(topk_weights), _ptr(out),
                                         _ptr(out_sf), T, H, num_per_channels, f, flags,
                                         _stream_handle(x.device))
    if st:
        raise TkqError(st, "tkq_swiglu_backward_cast")
    return out, out_sf


def per_channel_cast(x, fmt="e4m3", num_per_channels: int = GROUP, transpose: bool = False,
                     out=None, out_sf=None):
    """bf16 [T, C] -> codes and scales of groups of 128 tokens per channel:
    (codes [T, C], scales [T/128, C]), or with ``transpose`` the column-major
    copy (codes [C, T], scales [C, T/128]).  T must be a multiple of 128."""
    import torch
    _check_input(x)
    f = _fmt_code(fmt)
    T, C = x.shape
    g = max(num_per_channels, 1)
    if out is None:
        out = torch.empty((C, T) if transpose else (T, C), dtype=_fp8_dtype(f), device=x.device)
    else:
        _check_out(out, "out", x, T * C, itemsize=1)
    if out_sf is None:
        out_sf = torch.empty((C, T // g) if transpose else (T // g, C), dtype=torch.float32,
                             device=x.device)
    else:
        _check_out(out_sf, "out_sf", x, 4 * C * (T // g))
    with _device_ctx(x.device):
        st = tkq_per_channel_cast(_ptr(x), _ptr(out), _ptr(out_sf), T, C, num_per_channels, f,
                                  int(transpose), _stream_handle(x.device))
    if st:
        raise TkqError(st, "tkq_per_channel_cast")
    return out, out_sf


def per_block_cast(x, fmt="e4m3", block_size: int = GROUP, out=None, out_sf=None):
    """bf16 [T, C] -> (codes [T, C], scales [ceil(T/128), C/128]), one scale per
    128 x 128 block."""
    import torch
    _check_input(x)
    f = _fmt_code(fmt)
    T, C = x.shape
    b = max(block_size, 1)
    if out is None:
        out = torch.empty((T, C), dtype=_fp8_dtype(f), device=x.device)
    else:
        _check_out(out, "out", x, T * C, itemsize=1)
    if out_sf is None:
        out_sf = torch.empty(((T + b - 1) // b, C // b), dtype=torch.float32, device=x.device)
    else:
        _check_out(out_sf, "out_sf", x, 4 * ((T + b - 1) // b) * (C // b))
    with _device_ctx(x.device):
        st = tkq_per_block_cast(_ptr(x), _ptr(out), _ptr(out_sf), T, C, block_size, f,
                                _stream_handle(x.device))
    if st:
        raise TkqError(st, "tkq_per_block_cast")
    return out, out_sf


def cast_back(x, sf, fmt=None, group_size=(1, GROUP), out_dtype=None, out=None):
    """FP8 codes [T, C] and fp32 scales -> decode(code) * scale as fp32 (default)
    or bf16.  ``group_size`` = (rows, cols) of one scale group: (1, 128)
    per-token, (128, 1) per-channel, (128, 128) per-block.  ``fmt`` defaults to
    the codes' dtype (float8_e4m3fn or float8_e5m2; uint8 codes need fmt)."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise TypeError("x must be a contiguous 2-D CUDA tensor of FP8 codes")
    if x.element_size() != 1:
        raise TypeError("x must hold one-byte FP8 codes")
    if fmt is None:
        if x.dtype == torch.float8_e4m3fn:
            fmt = "e4m3"
        elif x.dtype == torch.float8_e5m2:
            fmt = "e5m2"
        else:
            raise ValueError("fmt is required for codes that are not an FP8 dtype")
    f = _fmt_code(fmt)
    if (not isinstance(sf, torch.Tensor) or sf.dtype != torch.float32 or not sf.is_contiguous()
            or sf.device != x.device):
        raise TypeError("sf must be a contiguous fp32 tensor on the codes' device")
    gr, gc = group_size
    T, C = x.shape
    if (-(-T // max(gr, 1)), C // max(gc, 1)) != tuple(sf.shape[-2:]) or sf.dim() != 2:
        raise ValueError(f"sf must have shape [ceil(T/{gr}), C/{gc}]")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    if out is None:
        out = torch.empty((T, C), dtype=out_dtype, device=x.device)
    else:
        _check_out(out, "out", x, T * C * (4 if out_dtype == torch.float32 else 2),
                   dtype=out_dtype)
    code = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    with _device_ctx(x.device):
        st = tkq_cast_back(_ptr(x), _ptr(sf), _ptr(out), T, C, gr, gc, f, code,
                           _stream_handle(x.device))
    if st:
        raise TkqError(st, "tkq_cast_back")
    return out


def _check_like(t, name, shape, dtypes, device):
    """A tensor operand: contiguous, of one of `dtypes` and of `shape`, on `device`."""
    import torch
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape
            and t.device == device and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA tensor on the inputs' device")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(map(str, dtypes))}")
    raise ValueError(f"{name} must have shape {list(shape)}")


def _check_logits(logits, scores):
    """T, E, row stride, dtype code and score flag of the logits of a routing call."""
    import torch
    if (not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dim() != 2
            or logits.dtype not in (torch.bfloat16, torch.float32)):
        raise TypeError("logits must be a 2-D bfloat16 or float32 CUDA tensor")
    T, E = logits.shape
    ld = logits.stride(0) if T > 1 else E
    if E > 1 and logits.stride(1) != 1:
        raise TypeError("logits must be contiguous along the experts")
    if scores not in ("softmax", "sigmoid"):
        raise ValueError(f"unknown scores {scores!r}: expected 'softmax' or 'sigmoid'")
    return (T, E, ld, OUT_BF16 if logits.dtype == torch.bfloat16 else OUT_F32,
            ROUTE_SIGMOID if scores == "sigmoid" else 0)


def route_topk(logits, k: int, scores: str = "softmax", bias=None, num_groups: int = 1,
               topk_groups: int = 1, num_topk_sum: int = 2, renormalize: bool = True,
               scale: float = 1.0, counts=None, ids=None, weights=None):
    """Route each of T tokens to k of E experts: logits bf16 or fp32 [T, E] (rows
    may be strided) -> (ids int32 [T, k], weights fp32 [T, k]).

    ``scores``: 'softmax' over the experts or the 'sigmoid' of each logit.
    ``bias`` (fp32 [E]) is added for the choice only.  With ``num_groups`` > 1 the
    ``topk_groups`` best groups of consecutive experts are searched, a group's
    score being the sum of its ``num_topk_sum`` (1 or 2) largest keys.  Experts
    come in falling order, ties to the lowest index; the weights are
    ``scale`` times the scores, divided by their sum with ``renormalize``.
    ``counts`` (int32 [E], zeroed by the caller) receives the tokens of each
    expert by addition.  A logit of -inf or NaN takes its expert out of the
    row; ids left over are -1 with weight 0."""
    import torch
    T, E, ld, dtype, flags = _check_logits(logits, scores)
    dev = logits.device
    if bias is not None:
        _check_like(bias, "bias", (E,), (torch.float32,), dev)
    if counts is not None:
        _check_like(counts, "counts", (E,), (torch.int32,), dev)
    if renormalize:
        flags |= ROUTE_RENORM
    k = int(k)
    if ids is None:
        ids = torch.empty((T, max(k, 0)), dtype=torch.int32, device=dev)
    else:
        _check_out(ids, "ids", logits, 4 * T * k, dtype=torch.int32)
    if weights is None:
        weights = torch.empty((T, max(k, 0)), dtype=torch.float32, device=dev)
    else:
        _check_out(weights, "weights", logits, 4 * T * k, dtype=torch.float32)
    lib = _lib or load_library()
    with _device_ctx(dev):
        st = lib.tkq_route_topk(_ptr(logits), _ptr(bias), _ptr(ids), _ptr(weights), _ptr(counts), T, E,
                                ld, dtype, k, num_groups, topk_groups, num_topk_sum, flags, scale,
                                _stream_handle(dev))
    if st:
        raise TkqError(st, "tkq_route_topk")
    return ids, weights


def route_topk_backward(logits, ids, dweights, scores: str = "softmax", renormalize: bool = True,
                        scale: float = 1.0, out=None):
    """Gradient of ``route_topk``'s weights: (logits, its ids, dweights fp32
    [T, k]) -> dlogits [T, E] in the logits' type.  ``scores``, ``renormalize``
    and ``scale`` as given to the forward."""
    import torch
    T, E, ld, dtype, flags = _check_logits(logits, scores)
    dev = logits.device
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise TypeError("ids must be an int32 [T, k] tensor")
    k = ids.shape[1]
    _check_like(ids, "ids", (T, k), (torch.int32,), dev)
    _check_like(dweights, "dweights", (T, k), (torch.float32,), dev)
    if renormalize:
        flags |= ROUTE_RENORM
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=dev)
    else:
        _check_out(out, "out", logits, T * E * logits.element_size(), dtype=logits.dtype)
    lib = _lib or load_library()
    with _device_ctx(dev):
        st = lib.tkq_route_topk_backward(_ptr(logits), _ptr(ids), _ptr(dweights), _ptr(out), T, E, ld,
                                         dtype, k, flags, scale, _stream_handle(dev))
    if st:
        raise TkqError(st, "tkq_route_topk_backward")
    return out


def swiglu_forward_cast_and_checkpoint(x, fmt="e4m3", num_per_channels: int = GROUP,
                                       topk_weights=None, ckpt_fmt="e4m3", round_sf: bool = False,
                                       use_packed_ue8m0: bool = False,
                                       use_tma_aligned_col_major_sf: bool = False):
    """``swiglu_forward_and_per_token_cast`` that also keeps its input in 8 bits
    for the backward: bf16 [T, 2H] (gate | up) -> (codes [T, H], scales,
    checkpoint codes [T, 2H], checkpoint scales fp32 [T, 2H/128]).  The
    checkpoint is ``per_token_cast(x, ckpt_fmt)``, bit for bit; the scale-layout
    options apply to the cast's scales."""
    import torch
    _check_input(x)
    f, cf = _fmt_code(fmt), _fmt_code(ckpt_fmt)
    T, H2 = x.shape
    if H2 % 2:
        raise ValueError("x must have an even number of columns (gate | up)")
    H, dev = H2 // 2, x.device
    g = max(num_per_channels, 1)
    _check_weights(topk_weights, T, x)
    flags = _sf_flags(round_sf, use_packed_ue8m0, use_tma_aligned_col_major_sf)
    out = torch.empty((T, H), dtype=_fp8_dtype(f), device=dev)
    out_sf = sf_tensor(T, H // g, flags, dev)
    ckpt = torch.empty((T, H2), dtype=_fp8_dtype(cf), device=dev)
    ckpt_sf = torch.empty((T, 2 * (H // g)), dtype=torch.float32, device=dev)
    lib = _lib or load_library()
    with _device_ctx(dev):
        st = lib.tkq_swiglu_cast_checkpoint(_ptr(x), _ptr(topk_weights), _ptr(out), _ptr(out_sf),
                                            _ptr(ckpt), _ptr(ckpt_sf), T, H, num_per_channels, f, cf,
                                            flags, _stream_handle(dev))
    if st:
        raise TkqError(st, "tkq_swiglu_cast_checkpoint")
    return out, out_sf, ckpt, ckpt_sf


def swiglu_backward_from_checkpoint(ckpt, ckpt_sf, dy, fmt=None, num_per_channels: int = GROUP,
                                    topk_weights=None, ckpt_fmt=None,
                                    with_weight_grad: bool = False, with_y: bool = False,
                                    round_sf: bool = False, use_packed_ue8m0: bool = False,
                                    use_tma_aligned_col_major_sf: bool = False):
    """Backward of y = silu(gate) * up [* w] from its 8-bit checkpoint (codes
    [T, 2H], scales fp32 [T, 2H/128]) and dy bf16 [T, H]
    -> (dx, dx_sf, dw, y).

    dx is [dg | du]: bf16 [T, 2H] with dx_sf None (``fmt`` None), or its
    per-token cast in ``fmt`` with the scales dx_sf.  dw: with
    ``with_weight_grad`` the gradient of the routing weights (fp32 [T]), else
    None.  y: with ``with_y`` the forward's output again in bf16 [T, H], for the
    weight gradient of the product that follows, else None."""
    import torch
    _check_input(dy, "dy")
    T, H = dy.shape
    dev = dy.device
    if ckpt_fmt is None and isinstance(ckpt, torch.Tensor):
        ckpt_fmt = {torch.float8_e4m3fn: "e4m3", torch.float8_e5m2: "e5m2"}.get(ckpt.dtype)
        if ckpt_fmt is None:
            raise ValueError("ckpt_fmt is required for codes that are not an FP8 dtype")
    cf = _fmt_code(ckpt_fmt)
    g = max(num_per_channels, 1)
    _check_like(ckpt, "ckpt", (T, 2 * H), (_fp8_dtype(cf), torch.uint8), dev)
    _check_like(ckpt_sf, "ckpt_sf", (T, 2 * (H // g)), (torch.float32,), dev)
    _check_weights(topk_weights, T, dy)
    flags = _sf_flags(round_sf, use_packed_ue8m0, use_tma_aligned_col_major_sf)
    dw = torch.empty((T,), dtype=torch.float32, device=dev) if with_weight_grad else None
    y = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if with_y else None
    if fmt is None:
        if flags:
            raise ValueError("the scale-layout options need fmt")
        dx, dx_sf = torch.empty((T, 2 * H), dtype=torch.bfloat16, device=dev), None
    else:
        f = _fmt_code(fmt)
        dx = torch.empty((T, 2 * H), dtype=_fp8_dtype(f), device=dev)
        dx_sf = sf_tensor(T, 2 * (H // g), flags, dev)
    lib = _lib or load_library()
    with _device_ctx(dev):
        stream = _stream_handle(dev)
        if fmt is None:
            st = lib.tkq_swiglu_checkpoint_backward(_ptr(ckpt), _ptr(ckpt_sf), _ptr(dy),
                                                    _ptr(topk_weights), _ptr(dx), _ptr(y), _ptr(dw), T,
                                                    H, num_per_channels, cf, stream)
        else:
            st = lib.tkq_swiglu_checkpoint_backward_cast(_ptr(ckpt), _ptr(ckpt_sf), _ptr(dy),
                                                         _ptr(topk_weights), _ptr(dx), _ptr(dx_sf),
                                                         _ptr(y), _ptr(dw), T, H, num_per_channels, cf,
                                                         f, flags, stream)
    if st:
        raise TkqError(st, "tkq_swiglu_checkpoint_backward")
    return dx, dx_sf, dw, y


def _check_stream(r, name):
    """The residual stream: a contiguous bf16 or fp32 [T, C] tensor."""
    _check_input(r, name, allow_f32=True)
    return r.shape


def residual_norm_and_cast(r, h=None, w_post=None, gate=None, w_pre=None, post_norm: bool = True,
                           res_scale: float = 1.0, eps: float = 1e-6, fmt="e4m3",
                           with_bf16: bool = False, num_per_channels: int = GROUP,
                           round_sf: bool = False, use_packed_ue8m0: bool = False,
                           use_tma_aligned_col_major_sf: bool = False):
    """The norms around a block, its gate and its residual scale, ending in the
    cast of the next product's input:

        r' = r + res_scale * norm(h) * w_post * sigmoid(gate)
        x  = norm(r') * w_pre

    with norm(v) = v / sqrt(mean(v^2) + eps) over the channels.  r: the residual
    stream, bf16 or fp32 [T, C]; h: the block's output, bf16 [T, C] (None before
    the first block: r' is r); gate: bf16 [T, C] or None; w_post, w_pre: fp32
    [C] or None; ``post_norm`` False leaves h as it is.
    -> (r', codes, scales, x, rstd_post, rstd_pre): the FP8 cast of x unless
    ``fmt`` is None, x in bf16 with ``with_bf16``, and the two norms' factors
    (fp32 [T]) that the backward takes; what is not asked for is None, and
    without ``fmt`` and ``with_bf16`` there is no second norm."""
    import torch
    T, C = _check_stream(r, "r")
    dev = r.device
    bf16, f32 = (torch.bfloat16,), (torch.float32,)
    flags = NORM_RES_F32 if r.dtype == torch.float32 else 0
    r_out = r
    rstd_post = rstd_pre = out = sf = x = None
    if h is not None:
        _check_like(h, "h", (T, C), bf16, dev)
        r_out = torch.empty_like(r)
        if post_norm:
            flags |= NORM_POST
            rstd_post = torch.empty((T,), dtype=torch.float32, device=dev)
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate need h")
    if gate is not None:
        _check_like(gate, "gate", (T, C), bf16, dev)
    if w_post is not None:
        _check_like(w_post, "w_post", (C,), f32, dev)
    if w_pre is not None:
        _check_like(w_pre, "w_pre", (C,), f32, dev)
    f, sf_flags = FMT_E4M3, 0
    if fmt is not None or with_bf16:
        flags |= NORM_PRE
        rstd_pre = torch.empty((T,), dtype=torch.float32, device=dev)
        if fmt is not None:
            f = _fmt_code(fmt)
            sf_flags = _sf_flags(round_sf, use_packed_ue8m0, use_tma_aligned_col_major_sf)
            out = torch.empty((T, C), dtype=_fp8_dtype(f), device=dev)
            sf = sf_tensor(T, C // max(num_per_channels, 1), sf_flags, dev)
        if with_bf16:
            x = torch.empty((T, C), dtype=torch.bfloat16, device=dev)
    elif w_pre is not None:
        raise ValueError("w_pre needs fmt or with_bf16")
    lib = _lib or load_library()
    with _device_ctx(dev):
        st = lib.tkq_residual_norm_cast(_ptr(r), _ptr(h), _ptr(w_post), _ptr(gate), _ptr(w_pre),
                                        None if h is None else _ptr(r_out), _ptr(out), _ptr(sf),
                                        _ptr(x), _ptr(rstd_post), _ptr(rstd_pre), T, C,
                                        num_per_channels, f, sf_flags, flags, res_scale, eps,
                                        _stream_handle(dev))
    if st:
        raise TkqError(st, "tkq_residual_norm_cast")
    return r_out, out, sf, x, rstd_post, rstd_pre


def residual_norm_backward(dr, r, h=None, dx=None, w_post=None, gate=None, w_pre=None,
                           rstd_post=None, rstd_pre=None, res_scale: float = 1.0):
    """Gradients of ``residual_norm_and_cast``: dr (the stream's type, or None) and
    dx (bf16, or None where the forward had no second norm) are the gradients of
    its r' and x, r is its r', and h, gate, the weights, the factors and
    ``res_scale`` are the forward's (rstd_post None: there was no post-norm).
    -> (dr of the forward's r, dh, dgate, dw_post, dw_pre); None for what has no
    counterpart.  The cast is passed through."""
    import torch
    lead = dr if dr is not None else r
    T, C = _check_stream(lead, "dr" if dr is not None else "r")
    dev = lead.device
    bf16, f32 = (torch.bfloat16,), (torch.float32,)
    flags = NORM_RES_F32 if lead.dtype == torch.float32 else 0
    dh = dgate = dw_post = dw_pre = work = None
    if dx is not None:
        flags |= NORM_PRE
        _check_like(dx, "dx", (T, C), bf16, dev)
        _check_like(r, "r", (T, C), (lead.dtype,), dev)
        _check_like(rstd_pre, "rstd_pre", (T,), f32, dev)
        if w_pre is not None:
            _check_like(w_pre, "w_pre", (C,), f32, dev)
            dw_pre = torch.empty((C,), dtype=torch.float32, device=dev)
    elif dr is None:
        raise ValueError("dr or dx is needed")
    elif w_pre is not None:
        raise ValueError("w_pre needs dx")
    if h is not None:
        _check_like(h, "h", (T, C), bf16, dev)
        dh = torch.empty_like(h)
        if rstd_post is not None:
            flags |= NORM_POST
            _check_like(rstd_post, "rstd_post", (T,), f32, dev)
        if gate is not None:
            _check_like(gate, "gate", (T, C), bf16, dev)
            dgate = torch.empty_like(gate)
        if w_post is not None:
            _check_like(w_post, "w_post", (C,), f32, dev)
            dw_post = torch.empty((C,), dtype=torch.float32, device=dev)
    elif w_post is not None or gate is not None or rstd_post is not None:
        raise ValueError("w_post, gate and rstd_post need h")
    dr_out = torch.empty_like(lead)
    lib = _lib or load_library()
    with _device_ctx(dev):
        if T == 0:  # sums over no rows
            for dw in (dw_post, dw_pre):
                if dw is not None:
                    dw.zero_()
        elif dw_post is not None or dw_pre is not None:
            work = torch.empty((max(tkq_residual_norm_workspace(T, C), 0),), dtype=torch.uint8,
                               device=dev)
        st = lib.tkq_residual_norm_backward(_ptr(dr), _ptr(dx), _ptr(r) if dx is not None else None,
                                            _ptr(h), _ptr(w_post), _ptr(gate), _ptr(w_pre),
                                            _ptr(rstd_post), _ptr(rstd_pre), _ptr(dr_out), _ptr(dh),
                                            _ptr(dgate), _ptr(dw_post), _ptr(dw_pre), _ptr(work), T, C,
                                            flags, res_scale, _stream_handle(dev))
    if st:
        raise TkqError(st, "tkq_residual_norm_backward")
    return dr_out, dh, dgate, dw_post, dw_pre


def swiglu_values(x, topk_weights=None):
    """Diagnostic: the fp32 SwiGLU values [T, H] exactly as the SwiGLU casts
    compute them before quantizing (x: bf16 [T, 2H] gate | up)."""
    import torch
    _check_input(x)
    T, H2 = x.shape
    if H2 % 2:
        raise ValueError("x must have an even number of columns (gate | up)")
    _check_weights(topk_weights, T, x)
    y = torch.empty((T, H2 // 2), dtype=torch.float32, device=x.device)
    with _device_ctx(x.device):
        st = tkq_swiglu_values(_ptr(x), _ptr(topk_weights), _ptr(y), T, H2 // 2,
                               _stream_handle(x.device))
    if st:
        raise TkqError(st, "tkq_swiglu_values")
    return y


def swiglu_backward_values(x, dy, topk_weights=None):
    """Diagnostic: the fp32 gradients [dg | du] ([T, 2H]) exactly as the SwiGLU
    backward cast computes them before quantizing (x: bf16 [T, 2H] gate | up,
    dy: bf16 [T, H])."""
    import torch
    _check_input(x)
    _check_input(dy, "dy")
    T, H2 = x.shape
    H = H2 // 2
    if H2 % 2 or tuple(dy.shape) != (T, H) or dy.device != x.device:
        raise ValueError("dy must be [T, H] for x [T, 2H], on the same device")
    _check_weights(topk_weights, T, x)
    y = torch.empty((T, H2), dtype=torch.float32, device=x.device)
    with _device_ctx(x.device):
        st = tkq_swiglu_backward_values(_ptr(x), _ptr(dy), _ptr(topk_weights), _ptr(y), T, H,
                                        _stream_handle(x.device))
    if st:
        raise TkqError(st, "tkq_swiglu_backward_values")
    return y


def fp8_encode(x, fmt="e4m3"):
    """Diagnostic: the FP8 codes (uint8, same shape) of an fp32 CUDA tensor,
    unscaled, by the conversion every cast ends with."""
    import torch
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous fp32 CUDA tensor")
    f = _fmt_code(fmt)
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    with _device_ctx(x.device):
        st = tkq_fp8_encode(_ptr(x), _ptr(out), x.numel(), f, _stream_handle(x.device))
    if st:
        raise TkqError(st, "tkq_fp8_encode")
    return out
