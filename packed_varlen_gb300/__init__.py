"""Python binding of libpackedattn (packed variable-length attention, sm_103a).

Argument marshalling only: every function checks tensor dtypes, shapes and
devices, passes raw device pointers and the current CUDA stream to the C ABI
declared in ``include/packedattn.h`` and raises ``PackedAttnError`` on a
non-OK status.  Every step runs in the library's CUDA kernels; there is no
other implementation behind these names.  Names are the C entry points
without their ``pa_`` prefix.
"""
from __future__ import annotations

import ctypes
import functools
import math
import operator
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libpackedattn.so")

PA_OK = 0
STATUS_NAMES = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED",
                3: "PA_ERR_MISALIGNED", 4: "PA_ERR_CUDA", 5: "PA_ERR_DEVICE"}
DEVICE_ERRORS = {0: "PA_DEVICE_OK", 1: "PA_DEVICE_ERR_CU_SEQLENS", 2: "PA_DEVICE_ERR_MAX_LEN",
                 3: "PA_DEVICE_ERR_TIMEOUT", 4: "PA_DEVICE_ERR_LENGTH",
                 5: "PA_DEVICE_ERR_CAPACITY", 6: "PA_DEVICE_ERR_SMEM_ALIGN",
                 7: "PA_DEVICE_ERR_SEGMENT", 8: "PA_DEVICE_ERR_PAGE"}
MAX_BATCH = 1024
VARLEN_TILE_M = 256


class PackedAttnError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        msg = f"{fn} returned {STATUS_NAMES.get(status, status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))
        self.status = status


_lib = None

_c_i32 = ctypes.c_int32
_c_i64 = ctypes.c_int64
_c_ptr = ctypes.c_void_p
_c_f32 = ctypes.c_float
# An integer argument of 32 or 64 bits has a place of 8 bytes on both machines that
# the library is built for (x86-64 and AArch64 Linux), in a register or on the stack.
_c_word = ctypes.c_void_p

_SIGNATURES = {
    "pa_varlen_attn_fwd": ([_c_ptr] * 6 + [_c_i32] * 7 + [_c_f32, _c_ptr], _c_i32),
    "pa_block_window_attn_fwd": ([_c_ptr] * 4 + [_c_i32] * 7 + [_c_f32, _c_ptr], _c_i32),
    "pa_block_window_attn_fwd_f32": ([_c_ptr] * 4 + [_c_i32] * 7 + [_c_f32, _c_ptr], _c_i32),
    "pa_cu_seqlens_from_lengths": ([_c_ptr, _c_ptr, _c_i32, _c_ptr], _c_i32),
    "pa_pack": ([_c_ptr, _c_ptr, _c_ptr, _c_i32, _c_i32, _c_i32, _c_i64, _c_ptr], _c_i32),
    "pa_unpack": ([_c_ptr, _c_ptr, _c_ptr, _c_i32, _c_i32, _c_i32, _c_i64, _c_ptr], _c_i32),
    "pa_varlen_num_work_items": ([_c_ptr, _c_i32, _c_i32, _c_i32], _c_i64),
    "pa_varlen_work_order": ([_c_ptr, _c_ptr, _c_i32, _c_i32, _c_i32, _c_ptr, _c_i64, _c_ptr],
                             _c_i32),
    "pa_get_device_status": ([ctypes.POINTER(_c_i32)], _c_i32),
    "pa_status_string": ([_c_i32], ctypes.c_char_p),
    "pa_selftest_wait_timeout": ([_c_i32, _c_ptr], _c_i32),
    "pa_last_cuda_error": ([], ctypes.c_char_p),
    "pa_cfg_combine": ([_c_ptr] * 8 + [_c_i32] * 5 + [_c_ptr], _c_i32),
    "pa_rope_packed": ([_c_ptr] * 5 + [_c_i32] * 5 + [_c_f32, _c_ptr], _c_i32),
    "pa_linear_bf16": ([_c_ptr] * 4 + [_c_i32] * 3 + [_c_ptr], _c_i32),
    # Integers of these three go as _c_word: ctypes converts it in 50 ns and c_int32 in
    # 110, which in a call of 21 to 29 arguments is a tenth of its host time.
    "pa_kv_cache_write": ([_c_ptr] * 9 + [_c_word] * 11 + [_c_ptr], _c_i32),
    "pa_kv_cache_read": ([_c_ptr] * 9 + [_c_word] * 9 + [_c_ptr], _c_i32),
    "pa_paged_attn_fwd": ([_c_ptr] * 9 + [_c_word] * 14 + [_c_f32, _c_ptr, _c_word, _c_ptr],
                          _c_i32),
    "pa_paged_attn_workspace_bytes": ([_c_i32] * 8, _c_i64),
    # (as the three above)
    "pa_prompt_attn_fwd": ([_c_ptr] * 6 + [_c_word] * 12 + [_c_f32, _c_ptr], _c_i32),
    "pa_rope_axes": ([_c_ptr] * 7 + [_c_word] * 11 + [_c_f32, _c_ptr], _c_i32),
    "pa_linear_act_bf16": ([_c_ptr] * 5 + [_c_word] * 7 + [_c_ptr], _c_i32),
    "pa_linear_gated_bf16": ([_c_ptr] * 4 + [_c_word] * 6 + [_c_ptr], _c_i32),
}


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libpackedattn.so (built in-tree by ``packed_varlen_gb300.build``).

    Raises if the library is missing: there is no fallback implementation."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing; build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != PA_OK:
        detail = ""
        if status == 4 and _lib is not None:
            detail = _lib.pa_last_cuda_error().decode()
        raise PackedAttnError(fn, status, detail)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, name: str, dtype, dims=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got {t.dim()}")


def varlen_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor,
                    max_q: int, max_k: int, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Packed varlen attention (pa_varlen_attn_fwd).  q [Tq, H, D], k/v
    [Tk, H, D] bf16; cu_seqlens int32 [B + 1] on the device.  Rows of ``out``
    beyond cu_seqlens_q[B] are not written (a fresh ``out`` is zero-filled)."""
    lib = load_library()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 3)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    Tq, H, D = q.shape
    if k.shape[1:] != (H, D) or v.shape != k.shape:
        raise ValueError("k and v must be [Tk, H, D] with q's H and D")
    if cu_seqlens_k.numel() != cu_seqlens_q.numel():
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    if out is None:
        out = torch.zeros_like(q)
    _need(out, "out", torch.bfloat16, 3)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    st = lib.pa_varlen_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                                cu_seqlens_q.numel() - 1, Tq, k.shape[0], int(max_q),
                                int(max_k), H, D, float(scale), _stream(stream))
    _check("pa_varlen_attn_fwd", st)
    return out


def block_window_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block: int,
                          look_back: int, look_ahead: int, scale: Optional[float] = None,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Block-window attention (pa_block_window_attn_fwd); q/k/v [batch, n, H, D] bf16."""
    lib = load_library()
    for t, nme in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, nme, torch.bfloat16, 4)
    if k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must have the same [batch, n, H, D] shape")
    batch, n, H, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, 4)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    st = lib.pa_block_window_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                      batch, n, int(block), int(look_back), int(look_ahead),
                                      H, D, float(scale), _stream(stream))
    _check("pa_block_window_attn_fwd", st)
    return out


def block_window_attn_fwd_f32(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block: int,
                              look_back: int, look_ahead: int, scale: Optional[float] = None,
                              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fp32 block-window attention (pa_block_window_attn_fwd_f32); q/k/v
    [batch, n, H, D] float32."""
    lib = load_library()
    for t, nme in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, nme, torch.float32, 4)
    if k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must have the same [batch, n, H, D] shape")
    batch, n, H, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.float32, 4)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    st = lib.pa_block_window_attn_fwd_f32(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                          out.data_ptr(), batch, n, int(block), int(look_back),
                                          int(look_ahead), H, D, float(scale), _stream(stream))
    _check("pa_block_window_attn_fwd_f32", st)
    return out


def cu_seqlens_from_lengths(lengths: torch.Tensor, out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """cu[0] = 0, cu[b+1] = cu[b] + lengths[b] (pa_cu_seqlens_from_lengths)."""
    lib = load_library()
    _need(lengths, "lengths", torch.int32, 1)
    if out is None:
        out = torch.empty(lengths.numel() + 1, dtype=torch.int32, device=lengths.device)
    _need(out, "out", torch.int32, 1)
    if out.numel() != lengths.numel() + 1:
        raise ValueError("out must have batch + 1 entries")
    st = lib.pa_cu_seqlens_from_lengths(lengths.data_ptr(), out.data_ptr(), lengths.numel(),
                                        _stream(stream))
    _check("pa_cu_seqlens_from_lengths", st)
    return out


def _row_bytes(t: torch.Tensor, lead: int) -> int:
    n = 1
    for s in t.shape[lead:]:
        n *= s
    return n * t.element_size()


def pack(padded: torch.Tensor, cu_seqlens: torch.Tensor, total: int,
         out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """padded [B, S_max, ...] -> flat [total, ...] (pa_pack).  ``total`` must be
    at least cu_seqlens[B] (the caller knows it from the host-side lengths)."""
    lib = load_library()
    _need(padded, "padded", padded.dtype)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    B, s_max = padded.shape[0], padded.shape[1]
    if cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    if out is None:
        out = torch.empty((int(total),) + tuple(padded.shape[2:]), dtype=padded.dtype,
                          device=padded.device)
    _need(out, "out", padded.dtype)
    if out.shape[0] != total or out.shape[1:] != padded.shape[2:]:
        raise ValueError("out must be [total, *padded.shape[2:]]")
    st = lib.pa_pack(padded.data_ptr(), out.data_ptr(), cu_seqlens.data_ptr(), B, s_max,
                     int(total), _row_bytes(padded, 2), _stream(stream))
    _check("pa_pack", st)
    return out


def unpack(flat: torch.Tensor, cu_seqlens: torch.Tensor, padded_out: torch.Tensor,
           stream=None) -> torch.Tensor:
    """flat [total, ...] -> rows [0, L_b) of each slot of padded_out [B, S_max, ...]
    (pa_unpack); padding rows of padded_out are left as they are."""
    lib = load_library()
    _need(flat, "flat", flat.dtype)
    _need(padded_out, "padded_out", flat.dtype)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    B, s_max = padded_out.shape[0], padded_out.shape[1]
    if cu_seqlens.numel() != B + 1 or padded_out.shape[2:] != flat.shape[1:]:
        raise ValueError("shape mismatch between flat, padded_out and cu_seqlens")
    st = lib.pa_unpack(flat.data_ptr(), padded_out.data_ptr(), cu_seqlens.data_ptr(), B, s_max,
                       flat.shape[0], _row_bytes(flat, 1), _stream(stream))
    _check("pa_unpack", st)
    return padded_out


def rope_packed(q: torch.Tensor, k: torch.Tensor, cu_seqlens_q: torch.Tensor,
                cu_seqlens_k: torch.Tensor, pos_offset: Optional[torch.Tensor] = None,
                base: float = 10000.0, stream=None):
    """Rotary embedding with request-local positions, in place on packed q
    [Tq, H, D] and k [Tk, H, D] bf16 (pa_rope_packed).  Returns (q, k)."""
    lib = load_library()
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 3)
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    if k.shape[1:] != q.shape[1:] or cu_seqlens_k.numel() != cu_seqlens_q.numel():
        raise ValueError("q/k heads, dims or batch differ")
    B = cu_seqlens_q.numel() - 1
    ptr = None
    if pos_offset is not None:
        _need(pos_offset, "pos_offset", torch.int32, 1)
        if pos_offset.numel() != B:
            raise ValueError("pos_offset must have one entry per sequence")
        ptr = pos_offset.data_ptr()
    st = lib.pa_rope_packed(q.data_ptr(), k.data_ptr(), cu_seqlens_q.data_ptr(),
                            cu_seqlens_k.data_ptr(), ptr, B, q.shape[0], k.shape[0], q.shape[1],
                            q.shape[2], float(base), _stream(stream))
    _check("pa_rope_packed", st)
    return q, k


def cfg_combine(flat: torch.Tensor, cu_seqlens: torch.Tensor, img_off: torch.Tensor,
                pos_seq: torch.Tensor, neg_seq: torch.Tensor, cfg_scale: torch.Tensor,
                cfg_normalize: torch.Tensor, img_max: int, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Per-request image-span unpack with the CFG combine (pa_cfg_combine).
    flat [T, ...] bf16 -> out [R, img_max, ...] bf16; index tensors int32 and
    cfg_scale float32 on the device.  Rows of ``out`` past each request's
    image span are left as they are (a fresh ``out`` is zero-filled)."""
    lib = load_library()
    _need(flat, "flat", torch.bfloat16)
    _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
    for t, n in ((img_off, "img_off"), (pos_seq, "pos_seq"), (neg_seq, "neg_seq"),
                 (cfg_normalize, "cfg_normalize")):
        _need(t, n, torch.int32, 1)
    _need(cfg_scale, "cfg_scale", torch.float32, 1)
    B, R = cu_seqlens.numel() - 1, pos_seq.numel()
    if img_off.numel() != B or neg_seq.numel() != R or cfg_scale.numel() != R or \
            cfg_normalize.numel() != R:
        raise ValueError("segment metadata sizes do not match")
    row = _row_bytes(flat, 1) // 2
    if out is None:
        out = torch.zeros((R, int(img_max)) + tuple(flat.shape[1:]), dtype=torch.bfloat16,
                          device=flat.device)
    _need(out, "out", torch.bfloat16)
    if out.shape[0] != R or out.shape[1] != img_max or out.shape[2:] != flat.shape[1:]:
        raise ValueError("out must be [R, img_max, *flat.shape[1:]]")
    st = lib.pa_cfg_combine(flat.data_ptr(), out.data_ptr(), cu_seqlens.data_ptr(),
                            img_off.data_ptr(), pos_seq.data_ptr(), neg_seq.data_ptr(),
                            cfg_scale.data_ptr(), cfg_normalize.data_ptr(), B, R, flat.shape[0],
                            int(img_max), row, _stream(stream))
    _check("pa_cfg_combine", st)
    return out


def varlen_num_work_items(cu_seqlens_q_host, H: int, tile_m: int = VARLEN_TILE_M) -> int:
    """Host-side work item count (pa_varlen_num_work_items); cu on the host."""
    lib = load_library()
    arr = (ctypes.c_int32 * len(cu_seqlens_q_host))(*[int(x) for x in cu_seqlens_q_host])
    n = lib.pa_varlen_num_work_items(ctypes.cast(arr, ctypes.c_void_p),
                                     len(cu_seqlens_q_host) - 1, H, tile_m)
    if n < 0:
        raise PackedAttnError("pa_varlen_num_work_items", 1)
    return int(n)


def varlen_work_order(cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, H: int,
                      capacity: int, tile_m: int = VARLEN_TILE_M, stream=None) -> torch.Tensor:
    """The attention kernel's work list as an int32 [capacity, 3] tensor of
    (sequence, head, q_tile) rows (pa_varlen_work_order)."""
    lib = load_library()
    _need(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _need(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    items = torch.full((max(1, capacity), 3), -1, dtype=torch.int32, device=cu_seqlens_q.device)
    st = lib.pa_varlen_work_order(cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(),
                                  cu_seqlens_q.numel() - 1, H, tile_m, items.data_ptr(),
                                  capacity, _stream(stream))
    _check("pa_varlen_work_order", st)
    return items[:capacity]


def get_device_status() -> int:
    """Synchronize, read and clear the device status word (pa_get_device_status).
    Returns the device error code (0 = none)."""
    lib = load_library()
    code = ctypes.c_int32(0)
    st = lib.pa_get_device_status(ctypes.byref(code))
    if st not in (PA_OK, 5):
        raise PackedAttnError("pa_get_device_status", st)
    return int(code.value)


def selftest_wait_timeout(timeout_us: int = 1000, stream=None) -> None:
    """Launch the bounded-wait self-test (pa_selftest_wait_timeout)."""
    lib = load_library()
    _check("pa_selftest_wait_timeout",
           lib.pa_selftest_wait_timeout(int(timeout_us), _stream(stream)))


def status_string(status: int) -> str:
    return load_library().pa_status_string(int(status)).decode()


def linear_bf16(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = x w^T + bias (pa_linear_bf16); x [M, K], w [N, K], bias [N], bf16."""
    lib = load_library()
    _need(x, "x", torch.bfloat16, 2)
    _need(w, "w", torch.bfloat16, 2)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w must be [N, {K}], got {tuple(w.shape)}")
    _fits_32_bits("pa_linear_bf16", M, N, K)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, 1)
        if bias.shape[0] != N:
            raise ValueError("bias must be [N]")
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    st = lib.pa_linear_bf16(x.data_ptr(), w.data_ptr(),
                            bias.data_ptr() if bias is not None else None, out.data_ptr(),
                            M, N, K, _stream(stream))
    _check("pa_linear_bf16", st)
    return out


# ---------------------------------------------------------------- paged K/V cache
# A step of single tokens takes some ten microseconds on the GPU, so these calls
# keep their checks short: what is usual passes one test, and the functions that
# allow for the rest, and name what is wrong, run only where it fails.
_CACHE_FORMATS = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}
_BF16, _I32, _U8 = torch.bfloat16, torch.int32, torch.uint8
_current_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
_NOT_USUAL = (AttributeError, KeyError, TypeError, ValueError)


def _rows_stride(t: torch.Tensor, name: str, dev: int) -> int:
    """Elements from one token to the next of a packed [T, H, D] bf16 tensor
    whose rows (one token) are contiguous."""
    try:
        T, H, D = t.shape
        sT, sH, sD = t.stride()
        if sD == 1 and sH == D and t.dtype is _BF16 and t.get_device() == dev:
            return sT if T > 1 else H * D
    except _NOT_USUAL:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dims, got {t.dim()}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors, not {t.device}")
    T, H, D = t.shape
    if not t.is_contiguous():
        sT, sH, sD = t.stride()
        if (D > 1 and sD != 1) or (H > 1 and sH != D):
            raise ValueError(f"the rows of {name} must be contiguous")
        return sT if T > 1 else H * D
    return H * D


def _need_index(t: torch.Tensor, name: str, n: int, dev: int):
    try:
        if t.dtype is _I32 and t.shape == (n,) and t.get_device() == dev and t.is_contiguous():
            return
    except _NOT_USUAL:
        pass
    _need(t, name, _I32, 1)
    raise ValueError(f"{name} must be [{n}] on the device of the other tensors, got {list(t.shape)} on {t.device}")


def _need_out(t: torch.Tensor, name: str, shape, dev: int):
    try:
        if t.dtype is _BF16 and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return
    except _NOT_USUAL:
        pass
    _need(t, name, _BF16, len(shape))
    raise ValueError(f"{name} must be {list(shape)} on the device of the other tensors")


def _batch_of(cu: torch.Tensor, name: str) -> int:
    try:
        return cu.shape[0] - 1
    except (AttributeError, IndexError, TypeError):
        _need(cu, name, _I32, 1)
        raise


def _page_stride(t: torch.Tensor, name: str) -> int:
    P, page, H, D = t.shape
    s = t.stride()
    if (D > 1 and s[3] != 1) or (H > 1 and s[2] != D) or (page > 1 and s[1] != H * D):
        raise ValueError(f"each page of {name} must be contiguous")
    return s[0] if P > 1 else page * H * D


def _need_cache(k_cache, v_cache, k_exp, v_exp, page_table, batch):
    """Checks the cache's tensors against each other; returns (device index,
    format, num_pages, page_size, Hkv, D, page_stride, table_pages, k_exp
    address, v_exp address)."""
    try:
        shape, dtype, dev = k_cache.shape, k_cache.dtype, k_cache.get_device()
        P, page, H, D = shape
        B, width = page_table.shape
        if dev >= 0 and v_cache.shape == shape and v_cache.dtype is dtype and \
                v_cache.get_device() == dev and k_cache.is_contiguous() and \
                v_cache.is_contiguous() and B == batch and page_table.dtype is _I32 and \
                page_table.get_device() == dev and page_table.is_contiguous():
            if dtype is _BF16:
                if k_exp is None and v_exp is None:
                    return dev, 0, P, page, H, D, page * H * D, width, None, None
            elif dtype is torch.float8_e4m3fn:
                of_rows = (P, H, page)
                if k_exp.dtype is _U8 and v_exp.dtype is _U8 and k_exp.shape == of_rows and \
                        v_exp.shape == of_rows and k_exp.get_device() == dev and \
                        v_exp.get_device() == dev and k_exp.is_contiguous() and \
                        v_exp.is_contiguous():
                    return (dev, 1, P, page, H, D, page * H * D, width, k_exp.data_ptr(),
                            v_exp.data_ptr())
    except _NOT_USUAL:
        pass
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{n} must be a CUDA tensor")
    dev = k_cache.get_device()
    dtype, shape = k_cache.dtype, k_cache.shape
    fmt = _CACHE_FORMATS.get(dtype)
    if fmt is None or v_cache.dtype not in _CACHE_FORMATS:
        raise TypeError("k_cache and v_cache must be torch.bfloat16 or torch.float8_e4m3fn, "
                        f"got {dtype} and {v_cache.dtype}")
    if len(shape) != 4:
        raise ValueError("k_cache must be [num_pages, page_size, Hkv, D]")
    if v_cache.shape != shape or v_cache.dtype is not dtype or v_cache.get_device() != dev:
        raise ValueError("k_cache and v_cache must have the same shape, type and device")
    P, page, H, D = shape
    if k_cache.is_contiguous() and v_cache.is_contiguous():
        stride = page * H * D
    else:
        stride = _page_stride(k_cache, "k_cache")
        if _page_stride(v_cache, "v_cache") != stride:
            raise ValueError("k_cache and v_cache must have the same page stride")
    ke = ve = None
    if fmt == 1:
        if k_exp is None or v_exp is None:
            raise ValueError("an 8-bit cache needs k_exp and v_exp")
        for t, n in ((k_exp, "k_exp"), (v_exp, "v_exp")):
            _need(t, n, _U8, 3)
            if t.get_device() != dev or t.shape != (P, H, page):
                raise ValueError(f"{n} must be [num_pages, Hkv, page_size] on the cache's device")
        ke, ve = k_exp.data_ptr(), v_exp.data_ptr()
    elif k_exp is not None or v_exp is not None:
        raise ValueError("a bf16 cache has no k_exp and v_exp")
    _need(page_table, "page_table", _I32, 2)
    if page_table.get_device() != dev or page_table.shape[0] != batch:
        raise ValueError("page_table must be [batch, table_pages] on the cache's device")
    return dev, fmt, P, page, H, D, stride, page_table.shape[1], ke, ve


def _raw_stream(dev: int, stream) -> int:
    if stream is None:
        return _current_stream(dev)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _call_on(dev: int, fn, args) -> int:
    """The C call with another device current than the caller's."""
    with torch.cuda.device(dev):
        return fn(*args)


def _new(make, shape, dtype, dev: int, stream, raw: int) -> torch.Tensor:
    """A tensor that belongs to the stream that uses it, so that its memory is
    not handed on while it is in use."""
    device = torch.device("cuda", dev)
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(raw, device=device)):
        return make(shape, dtype=dtype, device=device)


def _fits_32_bits(name: str, *counts: int):
    # ctypes cuts integers to the parameter's width without a word
    for n in counts:
        if n >> 31:
            raise PackedAttnError(name, 1 if n < 0 else 2)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(*sizes: int) -> int:
    # arithmetic on the sizes alone; the call through ctypes costs a microsecond
    return load_library().pa_paged_attn_workspace_bytes(*sizes)


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, cu_seqlens: torch.Tensor, page_table: torch.Tensor,
                   pos_offset: Optional[torch.Tensor] = None,
                   k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None,
                   stream=None):
    """Packed new rows k, v [T, Hkv, D] bf16 into a paged cache (pa_kv_cache_write):
    row j of sequence b goes to position pos_offset[b] + j.  k_cache, v_cache
    [num_pages, page_size, Hkv, D] bf16, or float8_e4m3fn with exponent bytes
    k_exp, v_exp [num_pages, Hkv, page_size] uint8; k and v may be slices of a
    wider tensor along its last dimensions.  Returns (k_cache, v_cache)."""
    lib = _lib or load_library()
    B = _batch_of(cu_seqlens, "cu_seqlens")
    dev, fmt, P, page, H, D, ps, width, ke, ve = _need_cache(k_cache, v_cache, k_exp, v_exp,
                                                             page_table, B)
    ks, vs = _rows_stride(k, "k", dev), _rows_stride(v, "v", dev)
    T = k.shape[0]
    if k.shape != (T, H, D) or v.shape != (T, H, D):
        raise ValueError("k and v must be [T, Hkv, D] with the cache's Hkv and D")
    _need_index(cu_seqlens, "cu_seqlens", B + 1, dev)
    off = None
    if pos_offset is not None:
        _need_index(pos_offset, "pos_offset", B, dev)
        off = pos_offset.data_ptr()
    args = (k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ke, ve,
            cu_seqlens.data_ptr(), off, page_table.data_ptr(), B, T, ks, vs, P, page, width, ps, H,
            D, fmt, _raw_stream(dev, stream))
    fn = lib.pa_kv_cache_write
    st = fn(*args) if _current_device() == dev else _call_on(dev, fn, args)
    if st != PA_OK:
        _check("pa_kv_cache_write", st)
    return k_cache, v_cache


def kv_cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, cu_seqlens: torch.Tensor,
                  page_table: torch.Tensor, total: int,
                  pos_offset: Optional[torch.Tensor] = None,
                  k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None,
                  k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                  stream=None):
    """Cached rows as packed bf16 rows (pa_kv_cache_read): positions
    [pos_offset[b], pos_offset[b] + L_b) of each sequence, L_b from cu_seqlens, as
    rows cu_seqlens[b].. of k_out and v_out [total, Hkv, D].  Rows past
    cu_seqlens[B] are left as they are (fresh outputs are zero-filled).
    Returns (k_out, v_out)."""
    lib = _lib or load_library()
    total = int(total)
    if total >> 31:
        _fits_32_bits("pa_kv_cache_read", total)
    B = _batch_of(cu_seqlens, "cu_seqlens")
    dev, fmt, P, page, H, D, ps, width, ke, ve = _need_cache(k_cache, v_cache, k_exp, v_exp,
                                                             page_table, B)
    _need_index(cu_seqlens, "cu_seqlens", B + 1, dev)
    off = None
    if pos_offset is not None:
        _need_index(pos_offset, "pos_offset", B, dev)
        off = pos_offset.data_ptr()
    raw = _raw_stream(dev, stream)
    shape = (total, H, D)
    if k_out is None:
        k_out = _new(torch.zeros, shape, _BF16, dev, stream, raw)
    else:
        _need_out(k_out, "k_out", shape, dev)
    if v_out is None:
        v_out = _new(torch.zeros, shape, _BF16, dev, stream, raw)
    else:
        _need_out(v_out, "v_out", shape, dev)
    args = (k_cache.data_ptr(), v_cache.data_ptr(), ke, ve, k_out.data_ptr(), v_out.data_ptr(),
            cu_seqlens.data_ptr(), off, page_table.data_ptr(), B, shape[0], P, page, width, ps, H, D,
            fmt, raw)
    fn = lib.pa_kv_cache_read
    st = fn(*args) if _current_device() == dev else _call_on(dev, fn, args)
    if st != PA_OK:
        _check("pa_kv_cache_read", st)
    return k_out, v_out


def paged_attn_workspace_bytes(batch: int, total_q: int, max_q: int, max_k: int, Hq: int,
                               Hkv: int, D: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace of paged_attn_fwd over a cache of `dtype`, in bytes
    (pa_paged_attn_workspace_bytes)."""
    sizes = [int(x) for x in (batch, total_q, max_q, max_k, Hq, Hkv, D)]
    _fits_32_bits("pa_paged_attn_workspace_bytes", *sizes)
    n = load_library().pa_paged_attn_workspace_bytes(*sizes, _CACHE_FORMATS.get(dtype, -1))
    if n < 0:
        raise PackedAttnError("pa_paged_attn_workspace_bytes", 1)
    return int(n)


def paged_attn_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   cu_seqlens_q: torch.Tensor, seq_lens: torch.Tensor,
                   page_table: torch.Tensor, max_q: int, max_k: int,
                   k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None,
                   causal: bool = True, scale: Optional[float] = None,
                   out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of packed new tokens q [Tq, Hq, D] bf16 over a paged cache
    (pa_paged_attn_fwd).  seq_lens int32 [B]: keys of each sequence, its new
    tokens' own among them (causal) or not (causal=False).  q may be a slice of
    a wider tensor along its last dimensions.  Rows of ``out`` beyond
    cu_seqlens_q[B] are not written (a fresh ``out`` is zero-filled).
    ``workspace`` (uint8, paged_attn_workspace_bytes) is allocated per call
    unless given; calls that may overlap need one each."""
    lib = _lib or load_library()
    max_q, max_k = int(max_q), int(max_k)
    if (max_q | max_k) >> 31:
        _fits_32_bits("pa_paged_attn_fwd", max_q, max_k)
    B = _batch_of(cu_seqlens_q, "cu_seqlens_q")
    dev, fmt, P, page, H, D, ps, width, ke, ve = _need_cache(k_cache, v_cache, k_exp, v_exp,
                                                             page_table, B)
    qs = _rows_stride(q, "q", dev)
    Tq, Hq, Dq = shape = q.shape
    if Dq != D or Hq < 1 or Hq % H:
        raise ValueError("q must be [Tq, Hq, D] with the cache's D and Hq a multiple of its Hkv")
    _need_index(cu_seqlens_q, "cu_seqlens_q", B + 1, dev)
    _need_index(seq_lens, "seq_lens", B, dev)
    if scale is None:
        scale = D ** -0.5
    raw = _raw_stream(dev, stream)
    if out is None:
        out = _new(torch.zeros, shape, _BF16, dev, stream, raw)
    else:
        _need_out(out, "out", shape, dev)
    wp, wn = None, 0
    if workspace is None:
        wn = _workspace_bytes(B, Tq, max_q, max_k, Hq, H, D, fmt)
        if wn > 0:
            workspace = _new(torch.empty, (wn,), _U8, dev, stream, raw)
            wp = workspace.data_ptr()
    else:
        if workspace.dtype is not _U8 or workspace.get_device() != dev or \
                not workspace.is_contiguous():
            _need(workspace, "workspace", _U8)
            raise ValueError("workspace must be on the cache's device")
        wp, wn = workspace.data_ptr(), workspace.numel()
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ke, ve, out.data_ptr(),
            cu_seqlens_q.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(), B, Tq, max_q, max_k,
            qs, P, page, width, ps, Hq, H, D, fmt, 1 if causal else 0, float(scale), wp, wn, raw)
    fn = lib.pa_paged_attn_fwd
    st = fn(*args) if _current_device() == dev else _call_on(dev, fn, args)
    if st != PA_OK:
        _check("pa_paged_attn_fwd", st)
    return out


# ---------------------------------------------------------------- a layer over packed prompts
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _device_of(t: torch.Tensor, name: str) -> int:
    try:
        dev = t.get_device()
        if dev >= 0:
            return dev
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _rows(t: torch.Tensor, name: str, dev: int):
    """T, H, D of a packed bf16 tensor, and elements from one token to the next."""
    try:
        T, H, D = t.shape
        sT, sH, sD = t.stride()
        if sD == 1 and sH == D and t.dtype is _BF16 and t.get_device() == dev:
            return T, H, D, sT if T > 1 else H * D
    except _NOT_USUAL:
        pass
    stride = _rows_stride(t, name, dev)
    return (*t.shape, stride)


def prompt_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    cu_seqlens_q: torch.Tensor, cu_seqlens_k: torch.Tensor, max_q: int,
                    max_k: int, causal: bool = True, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of packed prompts, causal and with grouped heads (pa_prompt_attn_fwd).
    q [Tq, Hq, D], k, v [Tk, Hkv, D] bf16, each possibly a slice of a wider tensor
    along its last dimensions; cu_seqlens int32 [B + 1].  Causal order lines up
    the ends: query i of a sequence sees key j iff j <= Lk - Lq + i.  Rows of
    ``out`` beyond cu_seqlens_q[B] are not written (a fresh ``out`` is zero-filled)."""
    lib = _lib or load_library()
    max_q, max_k = int(max_q), int(max_k)
    dev = _device_of(q, "q")
    Tq, Hq, D, qs = _rows(q, "q", dev)
    Tk, Hkv, Dk, ks = _rows(k, "k", dev)
    Tv, Hv, Dv, vs = _rows(v, "v", dev)
    if Dk != D or Dv != D or Tv != Tk or Hv != Hkv or Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError("k and v must be [Tk, Hkv, D] with q's D and Hq a multiple of Hkv")
    B = _batch_of(cu_seqlens_q, "cu_seqlens_q")
    if (max_q | max_k | B | Tq | Tk | Hq | D) >> 31:
        _fits_32_bits("pa_prompt_attn_fwd", max_q, max_k, B, Tq, Tk, Hq, D)
    _need_index(cu_seqlens_q, "cu_seqlens_q", B + 1, dev)
    if cu_seqlens_k is not cu_seqlens_q:
        _need_index(cu_seqlens_k, "cu_seqlens_k", B + 1, dev)
    if scale is None:
        scale = D ** -0.5
    raw = _raw_stream(dev, stream)
    if out is None:
        out = _new(torch.zeros, (Tq, Hq, D), _BF16, dev, stream, raw)
    else:
        _need_out(out, "out", (Tq, Hq, D), dev)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), cu_seqlens_q.data_ptr(),
            cu_seqlens_k.data_ptr(), B, Tq, Tk, max_q, max_k, qs, ks, vs, Hq, Hkv, D,
            1 if causal else 0, float(scale), raw)
    fn = lib.pa_prompt_attn_fwd
    st = fn(*args) if _current_device() == dev else _call_on(dev, fn, args)
    if st != PA_OK:
        _check("pa_prompt_attn_fwd", st)
    return out


_int_arrays = {}    # host int32 arrays by their values: a program has a few


def _host_ints(values):
    """The values as a host int32 array, how many they are, and its address."""
    # (whole numbers before they are looked up: 16.0 and 16 are one key of a dict, and a
    # tensor that stands for a number may have another value by the next call)
    ints = tuple(map(operator.index, values))
    known = _int_arrays.get(ints)
    if known is None:
        _fits_32_bits("pa_rope_axes", *[abs(v) for v in ints])
        arr = (ctypes.c_int32 * len(ints))(*ints)
        if len(_int_arrays) >= 256:
            _int_arrays.clear()
        known = _int_arrays[ints] = (arr, len(ints), ctypes.addressof(arr))
    return known


def rope_axes(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, axis_dims,
              base: float = 10000.0, halves: bool = False, shared: bool = False,
              num_tokens: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
              k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions with several axes on packed q [T, Hq, D] and k [T, Hkv, D]
    bf16 (pa_rope_axes), each possibly a slice of a wider tensor along its last
    dimensions, and k possibly None.  positions int32 [axes, T]; axis_dims: the
    elements of a head that each axis turns.  ``halves``: pairs are (i, i + R/2)
    instead of (2i, 2i + 1); ``shared``: one spectrum over all axes.  In place
    unless q_out / k_out are given.  ``num_tokens`` (int32, one element, for
    instance cu_seqlens[-1:]): rows from there on are left as they are.
    Returns (q_out, k_out)."""
    lib = _lib or load_library()
    dev = _device_of(q, "q")
    T, Hq, D, qs = _rows(q, "q", dev)
    qp = qo_p = q.data_ptr()
    qo = qs
    if q_out is None:
        q_out = q
    elif q_out is not q:
        To, Ho, Do, qo = _rows(q_out, "q_out", dev)
        if To != T or Ho != Hq or Do != D:
            raise ValueError("q_out must have q's shape")
        qo_p = q_out.data_ptr()
    kp = ko_p = None
    ks = ko = Hkv = 0
    if k is not None:
        Tk, Hkv, Dk, ks = _rows(k, "k", dev)
        kp = ko_p = k.data_ptr()
        ko = ks
        To, Ho, Do = Tk, Hkv, Dk
        if k_out is None:
            k_out = k
        elif k_out is not k:
            To, Ho, Do, ko = _rows(k_out, "k_out", dev)
            ko_p = k_out.data_ptr()
        if Tk != T or Dk != D or To != T or Ho != Hkv or Do != D:
            raise ValueError("k and k_out must be [T, Hkv, D] with q's T and D")
    elif k_out is not None:
        raise ValueError("k_out without k")
    if (T | Hq | Hkv | D) >> 31:
        _fits_32_bits("pa_rope_axes", T, Hq, Hkv, D)
    dims, axes, dims_at = _host_ints(axis_dims)    # (dims: kept until the call is made)
    try:
        usual = positions.dtype is _I32 and positions.shape == (axes, T) and \
            positions.get_device() == dev and positions.is_contiguous()
    except _NOT_USUAL:
        usual = False
    if not usual:
        _need(positions, "positions", _I32, 2)
        raise ValueError("positions must be [axes, T] on q's device")
    n_at = None
    if num_tokens is not None:
        _need(num_tokens, "num_tokens", _I32)
        if num_tokens.numel() != 1 or num_tokens.get_device() != dev:
            raise ValueError("num_tokens must be one element on q's device")
        n_at = num_tokens.data_ptr()
    args = (qp, kp, qo_p, ko_p, positions.data_ptr(), n_at, dims_at, axes, T,
            qs, ks, qo, ko, Hq, Hkv, D, 1 if halves else 0, 1 if shared else 0, float(base),
            _raw_stream(dev, stream))
    fn = lib.pa_rope_axes
    st = fn(*args) if _current_device() == dev else _call_on(dev, fn, args)
    if st != PA_OK:
        _check("pa_rope_axes", st)
    return q_out, k_out


def _matrix(t: torch.Tensor, name: str, dev: int):
    """M, N of a bf16 matrix whose rows are contiguous, and elements from one row to the
    next."""
    try:
        M, N = t.shape
        s0, s1 = t.stride()
        if s1 == 1 and t.dtype is _BF16 and t.get_device() == dev:
            return M, N, s0 if M > 1 else N
    except _NOT_USUAL:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {t.dim()}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on x's device, not {t.device}")
    M, N = t.shape
    if N > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return M, N, t.stride(0) if M > 1 else N


def _weight(w: torch.Tensor, name: str, K: int, dev: int) -> int:
    try:
        N, k = w.shape
        if k == K and w.dtype is _BF16 and w.get_device() == dev and w.is_contiguous():
            return N
    except _NOT_USUAL:
        pass
    _need(w, name, _BF16, 2)
    if w.shape[1] != K or w.get_device() != dev:
        raise ValueError(f"{name} must be [N, {K}] on x's device, got {list(w.shape)}")
    return w.shape[0]


def _need_vector(t: torch.Tensor, name: str, dtype, n: int, dev: int):
    try:
        if t.dtype is dtype and t.shape == (n,) and t.get_device() == dev and t.is_contiguous():
            return
    except _NOT_USUAL:
        pass
    _need(t, name, dtype, 1)
    raise ValueError(f"{name} must be [{n}] on x's device")


def _activation(act: str) -> int:
    try:
        return ACTIVATIONS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}") from None


def linear_act_bf16(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    act: str = "none", residual: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = residual + act(x w^T + bias) (pa_linear_act_bf16); x [M, K], w [N, K], bias
    [N], residual [M, N] bf16; act: a name in ACTIVATIONS.  x, residual and out
    may be slices of wider matrices; out may be residual itself."""
    lib = _lib or load_library()
    dev = _device_of(x, "x")
    M, K, xs = _matrix(x, "x", dev)
    N = _weight(w, "w", K, dev)
    if (M | N | K) >> 31:
        _fits_32_bits("pa_linear_act_bf16", M, N, K)
    code = _activation(act)
    b = r = None
    rs = 0
    if bias is not None:
        _need_vector(bias, "bias", _BF16, N, dev)
        b = bias.data_ptr()
    if residual is not None:
        Mr, Nr, rs = _matrix(residual, "residual", dev)
        if Mr != M or Nr != N:
            raise ValueError("residual must be [M, N]")
        r = residual.data_ptr()
    raw = _raw_stream(dev, stream)
    if out is None:
        out = _new(torch.empty, (M, N), _BF16, dev, stream, raw)
    Mo, No, ys = _matrix(out, "out", dev)
    if Mo != M or No != N:
        raise ValueError("out must be [M, N]")
    args = (x.data_ptr(), w.data_ptr(), b, r, out.data_ptr(), M, N, K, xs, rs, ys, code, raw)
    fn = lib.pa_linear_act_bf16
    st = fn(*args) if _current_device() == dev else _call_on(dev, fn, args)
    if st != PA_OK:
        _check("pa_linear_act_bf16", st)
    return out


def linear_gated_bf16(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                      act: str = "silu", out: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """y = act(x w_gate^T) * (x w_up^T) (pa_linear_gated_bf16); x [M, K], w_gate, w_up
    [N, K] bf16 (two tensors, or the halves of one); act: a name in ACTIVATIONS.
    x and out may be slices of wider matrices."""
    lib = _lib or load_library()
    dev = _device_of(x, "x")
    M, K, xs = _matrix(x, "x", dev)
    N = _weight(w_gate, "w_gate", K, dev)
    if _weight(w_up, "w_up", K, dev) != N:
        raise ValueError("w_gate and w_up must have the same shape")
    if (M | N | K) >> 31:
        _fits_32_bits("pa_linear_gated_bf16", M, N, K)
    code = _activation(act)
    raw = _raw_stream(dev, stream)
    if out is None:
        out = _new(torch.empty, (M, N), _BF16, dev, stream, raw)
    Mo, No, ys = _matrix(out, "out", dev)
    if Mo != M or No != N:
        raise ValueError("out must be [M, N]")
    args = (x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), out.data_ptr(), M, N, K, xs, ys,
            code, raw)
    fn = lib.pa_linear_gated_bf16
    st = fn(*args) if _current_device() == dev else _call_on(dev, fn, args)
    if st != PA_OK:
        _check("pa_linear_gated_bf16", st)
    return out
