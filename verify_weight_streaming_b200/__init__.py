"""Python binding of libmrgemm.so (ctypes; argument marshalling only).

Every function has the name of the C entry point it calls (see
``include/mrgemm.h``).  Tensors are torch CUDA tensors: torch supplies device
memory and the current stream, the library does all of the arithmetic.  16-bit
inputs may be ``torch.bfloat16`` / ``torch.float16`` or raw ``torch.int16``
patterns.  A status other than MR_OK raises ``MrError``.  If the compiled
library is missing the import fails: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

from ._build import LIB, build  # noqa: F401

MR_OK, MR_ERR_INVALID_ARG, MR_ERR_MISALIGNED, MR_ERR_UNSUPPORTED, MR_ERR_CUDA, MR_ERR_TIMEOUT = range(6)
MR_F16, MR_BF16, MR_F32 = 0, 1, 2
MR_GEMV_PDL = 0x1
MR_GEMV_SIGMOID = 0x2
MR_ROUTER_TWO_LAUNCH = 0x4
MR_W4_GROUP_MASK, MR_W4_ZEROS, MR_W4_SCALE_F16 = 0xFF, 0x100, 0x200
MR_MOE_SOFTMAX = 0x1
MR_DEVERR_GEMV_TIMEOUT, MR_DEVERR_GEMM_TIMEOUT, MR_DEVERR_TOPK_TIMEOUT, MR_DEVERR_SELFTEST = 1, 2, 4, 8

EXPORTS = (
    "mrgemv_bf16", "mrgemv_bf16_ex", "mrgemv_bf16_plan", "router_topk", "router_topk_ex",
    "router_topk_merge", "router_gemv_topk",
    "router_gemv_topk_workspace_bytes", "router_gemv_topk_noalloc", "router_gemv_topk_noalloc_max_logits", "gemm_f16_grouped",
    "gemm_f16_grouped_select_tile", "cast_f32_bf16", "gemm_f16_ex", "gemm_f16", "gemm_f16_num_tiles",
    "gemm_f16_tile_name", "gemm_f16_select_tile", "mr_poll_errors", "mr_selftest_wait_timeout",
    "mr_status_str", "mr_version", "w4_packed_bytes", "w4_pack", "mrgemv_w4",
    "moe_window_workspace_bytes", "moe_window_bf16", "moe_window_w4",
    "token_logprobs",
)


class MrError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {status_str(status)}")


def _load() -> ctypes.CDLL:
    from . import _build
    if _build.stale():
        # Sources newer than the library (or no library): compile it now with
        # nvcc.  Without a toolkit this raises; there is no fallback path.
        try:
            _build.build()
        except Exception as exc:
            raise ImportError(f"{LIB} is missing or stale and could not be built: {exc}") from exc
    L = ctypes.CDLL(LIB)
    P, I64, I32, U32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
    L.mrgemv_bf16.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, P]
    L.mrgemv_bf16_ex.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, U32, P]
    L.mrgemv_bf16_plan.argtypes = [I32, I32, I32, U32, I32, I32, P]
    L.router_topk.argtypes = [P, I64, I32, I32, I32, P, P, I64, P]
    L.router_topk_ex.argtypes = [P, I64, I32, I32, I32, P, P, I64, I32, P]
    L.router_topk_merge.argtypes = [P, P, I32, I32, I32, I64, I64, I32, P, P, I64, P]
    L.router_gemv_topk.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, I32, P, P, I64, P,
                                   ctypes.c_size_t, U32, P]
    L.router_gemv_topk_workspace_bytes.argtypes = [I32, I32, I32]
    L.router_gemv_topk_workspace_bytes.restype = ctypes.c_size_t
    L.router_gemv_topk_noalloc.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, I32, P, P, I64, U32, P]
    L.router_gemv_topk_noalloc_max_logits.argtypes = []
    L.router_gemv_topk_noalloc_max_logits.restype = ctypes.c_size_t
    L.gemm_f16.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, I32, I32, I32, P]
    L.gemm_f16_grouped.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, I32, I32, I32, I32, P]
    L.gemm_f16_grouped_select_tile.argtypes = [I32, I32, I32, I32]
    L.cast_f32_bf16.argtypes = [P, I64, P, I64, I32, I32, P]
    L.gemm_f16_ex.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, I32, I32, I32, I32, P]
    L.gemm_f16_num_tiles.argtypes = []
    L.gemm_f16_tile_name.argtypes = [I32]
    L.gemm_f16_tile_name.restype = ctypes.c_char_p
    L.gemm_f16_select_tile.argtypes = [I32, I32, I32]
    L.mr_poll_errors.argtypes = [P, ctypes.POINTER(U32)]
    L.mr_selftest_wait_timeout.argtypes = [I32, P]
    L.mr_status_str.argtypes = [ctypes.c_int]
    L.mr_status_str.restype = ctypes.c_char_p
    L.mr_version.argtypes = []
    L.mr_version.restype = ctypes.c_char_p
    L.w4_packed_bytes.argtypes = [I32, I32, U32, I32]
    L.w4_packed_bytes.restype = ctypes.c_size_t
    L.w4_pack.argtypes = [P, P, P, P, ctypes.c_size_t, I32, I32, I32, U32, I32, P]
    L.mrgemv_w4.argtypes = [P, I64, P, ctypes.c_size_t, P, I64, I32, I32, I32, I32, U32, U32, P]
    SZ = ctypes.c_size_t
    L.moe_window_workspace_bytes.argtypes = [I32, I32, I32, I32]
    L.moe_window_workspace_bytes.restype = SZ
    L.moe_window_bf16.argtypes = [P, I64, P, P, I64, P, I64, I64, P, I64, I64, P, I64, I32, I32, I32, I32, I32, I32,
                                  I32, U32, P, SZ, P]
    L.moe_window_w4.argtypes = [P, I64, P, P, I64, P, SZ, P, SZ, P, I64, I32, I32, I32, I32, I32, I32, U32, I32, U32,
                                P, SZ, P]
    L.token_logprobs.argtypes = [P, I64, I32, I32, I32, ctypes.c_float, P, I64, I32, P, I64, P, P, I32, P, P, I64, P]
    for name in ("w4_pack", "mrgemv_w4", "moe_window_bf16", "moe_window_w4", "token_logprobs"):
        getattr(L, name).restype = ctypes.c_int
    for name in ("mrgemv_bf16", "mrgemv_bf16_ex", "mrgemv_bf16_plan", "router_topk", "router_topk_ex",
                 "router_topk_merge", "router_gemv_topk",
                 "router_gemv_topk_noalloc", "gemm_f16_grouped", "gemm_f16_grouped_select_tile",
                 "cast_f32_bf16", "gemm_f16_ex", "gemm_f16", "gemm_f16_num_tiles",
                 "gemm_f16_select_tile", "mr_poll_errors", "mr_selftest_wait_timeout"):
        getattr(L, name).restype = ctypes.c_int
    return L


lib = _load()


def status_str(status: int) -> str:
    return lib.mr_status_str(int(status)).decode()


def version() -> str:
    return lib.mr_version().decode()


def _check(status: int, call: str) -> None:
    if status != MR_OK:
        raise MrError(status, call)


_current_raw_stream = None


def _current_stream_handle() -> int:
    """The current CUDA stream of the current device, as torch sees it."""
    global _current_raw_stream
    if _current_raw_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        dev = getattr(torch._C, "_cuda_getDevice", None)
        if raw is not None and dev is not None:
            _current_raw_stream = lambda: raw(dev())  # noqa: E731  (one C++ call each, per launch)
        else:
            _current_raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _current_raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream_handle()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _rows(t, name):
    st = t.stride()
    if len(st) != 2 or st[1] != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    sh = t.shape
    return sh[0], sh[1], st[0]


_dtype_codes: dict = {}


def _dtype_code(t) -> int:
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.float16: MR_F16, torch.bfloat16: MR_BF16, torch.float32: MR_F32,
                             torch.int16: MR_BF16})
    return _dtype_codes.get(t.dtype, -1)


def mrgemv_bf16(A, Wt, C, stream=None, flags: int = 0) -> None:
    """C[m,n] (fp32) = A[m,k] (bf16) . Wt[n,k]^T (bf16); m <= 16."""
    m, k, lda = _rows(A, "A")
    n, kw, ldw = _rows(Wt, "Wt")
    mc, nc, ldc = _rows(C, "C")
    if kw != k or mc != m or nc != n:
        raise ValueError(f"shape mismatch A{tuple(A.shape)} Wt{tuple(Wt.shape)} C{tuple(C.shape)}")
    st = lib.mrgemv_bf16_ex(A.data_ptr(), lda, Wt.data_ptr(), ldw, C.data_ptr(), ldc,
                            m, n, k, flags, _stream(stream))
    _check(st, "mrgemv_bf16")


PLAN_FIELDS = ("grid", "threads", "smem_bytes", "ring_slots", "k_warps", "column_warps",
               "row_bucket", "columns_per_group")


def mrgemv_bf16_plan(m: int, n: int, k: int, flags: int, sm_count: int, smem_optin: int) -> dict:
    """The launch plan of mrgemv_bf16_ex for these sizes on a described device."""
    out = (ctypes.c_int32 * 8)()
    _check(lib.mrgemv_bf16_plan(m, n, k, flags, sm_count, smem_optin, out), "mrgemv_bf16_plan")
    return dict(zip(PLAN_FIELDS, list(out)))


def router_topk(logits, topk: int, idx, val=None, stream=None) -> None:
    """idx[m,topk] (int32), val[m,topk] (fp32, optional) = per-row top-k of logits[m,n]."""
    m, n, ldl = _rows(logits, "logits")
    mi, ki, ldo = _rows(idx, "idx")
    if mi != m or ki < topk:
        raise ValueError("idx shape mismatch")
    vptr = None
    if val is not None:
        mv, kv, ldv = _rows(val, "val")
        if mv != m or kv < topk or ldv != ldo:
            raise ValueError("val must match idx's shape and stride")
        vptr = val.data_ptr()
    st = lib.router_topk(logits.data_ptr(), ldl, m, n, topk, idx.data_ptr(), vptr, ldo, _stream(stream))
    _check(st, "router_topk")


def router_topk_ex(logits, topk: int, idx, val=None, index_base: int = 0, stream=None) -> None:
    """router_topk of a shard of columns: indices are written as index_base + column."""
    m, n, ldl = _rows(logits, "logits")
    mi, ki, ldo = _rows(idx, "idx")
    if mi != m or ki < topk:
        raise ValueError("idx shape mismatch")
    vptr = None
    if val is not None:
        mv, kv, ldv = _rows(val, "val")
        if mv != m or kv < topk or ldv != ldo:
            raise ValueError("val must match idx's shape and stride")
        vptr = val.data_ptr()
    st = lib.router_topk_ex(logits.data_ptr(), ldl, m, n, topk, idx.data_ptr(), vptr, ldo, index_base,
                            _stream(stream))
    _check(st, "router_topk_ex")


def router_topk_merge(cand_val, cand_idx, topk: int, idx, val=None, stream=None) -> None:
    """Per-row top-k of candidate lists laid out [groups, m, per_group] (fp32
    values, int32 global indices, -1 = empty), e.g. an all-gather of every
    shard's router_topk_ex output."""
    if cand_val.dim() != 3 or tuple(cand_idx.shape) != tuple(cand_val.shape):
        raise ValueError("cand_val and cand_idx must be [groups, m, per_group] of the same shape")
    if cand_val.stride() != cand_idx.stride() or cand_val.stride(2) != 1:
        raise ValueError("candidates need a common layout with unit stride in the last dimension")
    groups, m, per = cand_val.shape
    mi, ki, ldo = _rows(idx, "idx")
    if mi != m or ki < topk:
        raise ValueError("idx shape mismatch")
    vptr = None
    if val is not None:
        mv, kv, ldv = _rows(val, "val")
        if mv != m or kv < topk or ldv != ldo:
            raise ValueError("val must match idx's shape and stride")
        vptr = val.data_ptr()
    st = lib.router_topk_merge(cand_val.data_ptr(), cand_idx.data_ptr(), m, groups, per, cand_val.stride(1),
                               cand_val.stride(0), topk, idx.data_ptr(), vptr, ldo, _stream(stream))
    _check(st, "router_topk_merge")


MR_ROUTER_TICKET_BYTES = 256


def router_gemv_topk_workspace_bytes(m: int, n: int, logits_provided: bool) -> int:
    return int(lib.router_gemv_topk_workspace_bytes(m, n, 1 if logits_provided else 0))


def router_gemv_topk(A, Wt, topk: int, idx, val=None, logits=None, workspace=None, stream=None,
                     flags: int = 0) -> None:
    """GEMV + per-row top-k in one launch (or, with MR_ROUTER_TWO_LAUNCH, the
    GEMV kernel then the top-k kernel).  ``workspace``: a zeroed contiguous CUDA tensor
    of at least router_gemv_topk_workspace_bytes(...) bytes (each fused call
    leaves its tag array zero again)."""
    m, k, lda = _rows(A, "A")
    n, kw, ldw = _rows(Wt, "Wt")
    if kw != k:
        raise ValueError("A and Wt disagree on k")
    mi, ki, ldo = _rows(idx, "idx")
    if mi != m or ki < topk:
        raise ValueError("idx shape mismatch")
    lptr, ldl = None, n
    if logits is not None:
        ml, nl, ldl = _rows(logits, "logits")
        if ml != m or nl != n:
            raise ValueError("logits shape mismatch")
        lptr = logits.data_ptr()
    vptr = None
    if val is not None:
        mv, kv, ldv = _rows(val, "val")
        if mv != m or kv < topk or ldv != ldo:
            raise ValueError("val must match idx's shape and stride")
        vptr = val.data_ptr()
    if workspace is None:
        raise ValueError("router_gemv_topk needs a zero-initialised workspace tensor")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    wbytes = workspace.numel() * workspace.element_size()
    st = lib.router_gemv_topk(A.data_ptr(), lda, Wt.data_ptr(), ldw, lptr, ldl, m, n, k, topk,
                              idx.data_ptr(), vptr, ldo, workspace.data_ptr(), wbytes, flags,
                              _stream(stream))
    _check(st, "router_gemv_topk")


def gemm_f16(A, Wt, C, tile_id: int = -1, in_dtype: int | None = None, stream=None, raster: int = 0) -> None:
    """C[M,N] = A[M,K] . Wt[N,K]^T on tcgen05; dtypes from the tensors (int16 = bf16 bits)."""
    M, K, lda = _rows(A, "A")
    N, kw, ldw = _rows(Wt, "Wt")
    mc, nc, ldc = _rows(C, "C")
    if kw != K or mc != M or nc != N:
        raise ValueError("shape mismatch")
    idt = _dtype_code(A) if in_dtype is None else in_dtype
    st = lib.gemm_f16_ex(A.data_ptr(), lda, Wt.data_ptr(), ldw, C.data_ptr(), ldc, M, N, K,
                         idt, _dtype_code(C), tile_id, raster, _stream(stream))
    _check(st, "gemm_f16")


def gemm_f16_grouped(A, Wts, Cs, tile_id: int = -1, in_dtype: int | None = None, stream=None) -> None:
    """Cs[g] = A . Wts[g]^T for every g in one launch (lists of equal-shape tensors)."""
    M, K, lda = _rows(A, "A")
    if len(Wts) != len(Cs) or not Wts:
        raise ValueError("Wts and Cs must be non-empty lists of the same length")
    N, kw, ldw = _rows(Wts[0], "Wts[0]")
    _, _, ldc = _rows(Cs[0], "Cs[0]")
    for w, c in zip(Wts, Cs):
        if tuple(w.shape) != (N, K) or w.stride(0) != ldw or tuple(c.shape) != (M, N) or c.stride(0) != ldc:
            raise ValueError("every Wts[g] must be [N,K] and every Cs[g] [M,N] with common strides")
    G = len(Wts)
    wp = (ctypes.c_void_p * G)(*[w.data_ptr() for w in Wts])
    cp = (ctypes.c_void_p * G)(*[c.data_ptr() for c in Cs])
    idt = _dtype_code(A) if in_dtype is None else in_dtype
    st = lib.gemm_f16_grouped(A.data_ptr(), lda, wp, ldw, cp, ldc, M, N, K, G, idt, _dtype_code(Cs[0]),
                              tile_id, _stream(stream))
    _check(st, "gemm_f16_grouped")


def gemm_f16_grouped_select_tile(M: int, N: int, K: int, G: int) -> int:
    return int(lib.gemm_f16_grouped_select_tile(M, N, K, G))


def cast_f32_bf16(X, Y, stream=None) -> None:
    """Y (bf16 or int16 bits) = X (fp32) rounded to nearest even."""
    rows, cols, ldx = _rows(X, "X")
    ry, cy, ldy = _rows(Y, "Y")
    if (ry, cy) != (rows, cols):
        raise ValueError("X and Y shapes differ")
    _check(lib.cast_f32_bf16(X.data_ptr(), ldx, Y.data_ptr(), ldy, rows, cols, _stream(stream)), "cast_f32_bf16")


def gemm_f16_num_tiles() -> int:
    return int(lib.gemm_f16_num_tiles())


def gemm_f16_tile_name(tile_id: int):
    r = lib.gemm_f16_tile_name(tile_id)
    return None if r is None else r.decode()


def gemm_f16_select_tile(M: int, N: int, K: int) -> int:
    return int(lib.gemm_f16_select_tile(M, N, K))


def mr_poll_errors(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error bits."""
    flags = ctypes.c_uint32(0)
    st = lib.mr_poll_errors(_stream(stream), ctypes.byref(flags))
    if st not in (MR_OK, MR_ERR_TIMEOUT):
        raise MrError(st, "mr_poll_errors")
    return int(flags.value)


def mr_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    _check(lib.mr_selftest_wait_timeout(limit_us, _stream(stream)), "mr_selftest_wait_timeout")


class _T:
    """What the calls below need of torch, filled on the first of them."""
    bf16 = f16 = f32 = i32 = u8 = device = stream = None


def _types():
    if _T.device is None:
        import torch
        _T.bf16, _T.f16, _T.f32, _T.i32, _T.u8 = (torch.bfloat16, torch.float16, torch.float32, torch.int32,
                                                  torch.uint8)
        _T.stream, _T.device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    return _T


def _on(stream, first, *others):
    """The stream handle for a call on these tensors (None is skipped), which must be on the current CUDA device:
    the kernels run there."""
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            raise ValueError(f"tensors on {first.device} and {t.device}")
    if d < 0 or d != _T.device():
        raise ValueError(f"the tensors are on {first.device}, not on the current CUDA device")
    return _T.stream(d) if stream is None else _stream(stream)


def _matrix(t, name):
    """_rows, where the stride of a dimension of size one may be anything."""
    st, sh = t.stride(), t.shape
    if len(sh) != 2 or (st[1] != 1 and sh[1] != 1):
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    return sh[0], sh[1], st[0] if sh[0] > 1 else sh[1]


def _int32(*sizes):
    """The C entry points take int32, and ctypes would cut a larger size to its low bits."""
    if max(sizes) > 0x7FFFFFFF or min(sizes) < -0x80000000:
        raise ValueError(f"a size of {sizes} is beyond 32 bits")


def w4_format(group: int, zeros: bool, scale_dtype) -> int:
    """The format word of a 4-bit weight: group size, zero points or not, torch.bfloat16 or torch.float16 scales."""
    T = _types()
    if scale_dtype not in (T.bf16, T.f16):
        raise ValueError("scales must be bfloat16 or float16")
    if not 0 <= group <= MR_W4_GROUP_MASK:  # beyond it the group would run into the flags
        raise ValueError(f"a group of {group} values does not fit a format word")
    return group | (MR_W4_ZEROS if zeros else 0) | (MR_W4_SCALE_F16 if scale_dtype is T.f16 else 0)


def w4_packed_bytes(n: int, k: int, fmt: int, paired: bool = False) -> int:
    _int32(n, k)
    return int(lib.w4_packed_bytes(n, k, fmt, 1 if paired else 0))


def w4_pack(q, scales, zeros, packed, paired: bool = False, stream=None) -> None:
    """packed (uint8) = the weights q[..., n, k/2] (uint8, low half first), scales[..., n, k/G] (bf16 or f16) and
    zeros[..., n, k/G] (uint8, or None) in the order mrgemv_w4 and moe_window_w4 read."""
    T = _types()
    if q.dim() not in (2, 3) or q.dtype is not T.u8 or packed.dtype is not T.u8:
        raise ValueError("q must be uint8 [n, k/2] or [count, n, k/2], packed uint8")
    n, k = q.shape[-2], 2 * q.shape[-1]
    count = q.shape[0] if q.dim() == 3 else 1
    groups = scales.shape[-1]
    _int32(count, n, k)
    if tuple(scales.shape[:-1]) != tuple(q.shape[:-1]) or groups < 1 or k % groups:
        raise ValueError("scales must be [..., n, k/G]")
    if zeros is not None and (zeros.shape != scales.shape or zeros.dtype is not T.u8):
        raise ValueError("zeros must be uint8 of the scales' shape")
    for t in (q, scales, packed) if zeros is None else (q, scales, packed, zeros):
        if not t.is_contiguous():
            raise ValueError("q, scales, zeros and packed must be contiguous")
    fmt = w4_format(k // groups, zeros is not None, scales.dtype)
    stream = _on(stream, q, scales, zeros, packed)
    st = lib.w4_pack(q.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(), packed.data_ptr(),
                     packed.numel(), count, n, k, fmt, 1 if paired else 0, stream)
    _check(st, "w4_pack")


def mrgemv_w4(A, packed, C, fmt: int, stream=None, flags: int = 0) -> None:
    """C[m,n] (fp32) = A[m,k] (bf16 or f16) . (the packed 4-bit n x k weight)^T; m <= 16."""
    m, k, lda = _matrix(A, "A")
    mc, n, ldc = _matrix(C, "C")
    if mc != m:
        raise ValueError(f"shape mismatch A{tuple(A.shape)} C{tuple(C.shape)}")
    if (m | n | k) >> 31:
        _int32(m, n, k)
    T = _types()
    if C.dtype is not T.f32 or packed.dtype is not T.u8 or not packed.is_contiguous():
        raise ValueError("C must be float32, packed a contiguous uint8 tensor")
    stream = _on(stream, A, packed, C)
    st = lib.mrgemv_w4(A.data_ptr(), lda, packed.data_ptr(), packed.numel(), C.data_ptr(), ldc, m, n, k, _dtype_code(A),
                       fmt, flags, stream)
    _check(st, "mrgemv_w4")


def moe_window_workspace_bytes(m: int, topk: int, hidden: int, inter: int) -> int:
    _int32(m, topk, hidden, inter)
    return int(lib.moe_window_workspace_bytes(m, topk, hidden, inter))


def _window(X, ids, weights, Y, workspace):
    m, hidden, ldx = _matrix(X, "X")
    mi, topk, ldr = _matrix(ids, "ids")
    my, hy, ldy = _matrix(Y, "Y")
    if mi != m or my != m or hy != hidden:
        raise ValueError(f"shape mismatch X{tuple(X.shape)} ids{tuple(ids.shape)} Y{tuple(Y.shape)}")
    if _matrix(weights, "weights") != (m, topk, ldr):
        raise ValueError("weights must match ids' shape and stride")
    T = _types()
    if X.dtype is not T.bf16 or ids.dtype is not T.i32 or weights.dtype is not T.f32:
        raise ValueError("X must be bfloat16, ids int32 and weights float32")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _int32(m, topk, hidden)
    return m, topk, hidden, ldx, ldr, ldy


def moe_window_bf16(X, ids, weights, Wup, Wdown, Y, workspace, expert_base: int = 0, flags: int = 0,
                    stream=None) -> None:
    """Y[m,hidden] (fp32 or bf16) = the experts ids[m,topk] (int32) of X[m,hidden] (bf16), weighted by
    weights[m,topk] (fp32; their softmax with MR_MOE_SOFTMAX).  Wup[experts,2*inter,hidden] holds the gate rows
    before the up rows, Wdown is [experts,hidden,inter].  ``workspace``: a contiguous CUDA tensor of at least
    moe_window_workspace_bytes(...) bytes."""
    m, topk, hidden, ldx, ldr, ldy = _window(X, ids, weights, Y, workspace)
    su, sd = Wup.stride(), Wdown.stride()
    if len(su) != 3 or len(sd) != 3 or su[2] != 1 or sd[2] != 1:
        raise ValueError("Wup and Wdown must be 3-D tensors with unit column stride")
    experts, rows, inter = Wdown.shape
    if Wup.shape != (experts, 2 * inter, hidden) or rows != hidden:
        raise ValueError(f"shape mismatch Wup{tuple(Wup.shape)} Wdown{tuple(Wdown.shape)}")
    if Wup.dtype is not _T.bf16 or Wdown.dtype is not _T.bf16:
        raise ValueError("Wup and Wdown must be bfloat16")
    _int32(experts, inter, expert_base)
    stream = _on(stream, X, ids, weights, Wup, Wdown, Y, workspace)
    eu, ed = (su[0], sd[0]) if experts > 1 else (0, 0)
    st = lib.moe_window_bf16(X.data_ptr(), ldx, ids.data_ptr(), weights.data_ptr(), ldr, Wup.data_ptr(), su[1], eu,
                             Wdown.data_ptr(), sd[1], ed, Y.data_ptr(), ldy, m, topk, experts, hidden, inter,
                             expert_base, _dtype_code(Y), flags, workspace.data_ptr(), workspace.nbytes, stream)
    _check(st, "moe_window_bf16")


def moe_window_w4(X, ids, weights, up, down, Y, workspace, experts: int, inter: int, fmt: int, expert_base: int = 0,
                  flags: int = 0, stream=None) -> None:
    """moe_window_bf16 with the experts' weights packed by w4_pack (``up`` paired, ``down`` not)."""
    m, topk, hidden, ldx, ldr, ldy = _window(X, ids, weights, Y, workspace)
    if up.dtype is not _T.u8 or down.dtype is not _T.u8 or not (up.is_contiguous() and down.is_contiguous()):
        raise ValueError("up and down must be contiguous uint8 tensors")
    _int32(experts, inter, expert_base)
    stream = _on(stream, X, ids, weights, up, down, Y, workspace)
    st = lib.moe_window_w4(X.data_ptr(), ldx, ids.data_ptr(), weights.data_ptr(), ldr, up.data_ptr(), up.numel(),
                           down.data_ptr(), down.numel(), Y.data_ptr(), ldy, m, topk, experts, hidden, inter,
                           expert_base, fmt, _dtype_code(Y), flags, workspace.data_ptr(), workspace.nbytes, stream)
    _check(st, "moe_window_w4")


def token_logprobs(logits, tokens=None, logprob=None, scale: float = 1.0, lse=None, entropy=None, top_idx=None,
                   top_logprob=None, stream=None) -> None:
    """Log probabilities (fp32) of logits[m,n] (fp32, bf16 or f16) times ``scale``, into whichever outputs are given:
    logprob[m,t] of tokens[m,t] (int32), lse[m], entropy[m], and the top_idx.shape[1] best alternatives
    top_idx[m,k] (int32), top_logprob[m,k]."""
    m, n, ldl = _matrix(logits, "logits")
    dtype = _dtype_code(logits)
    if dtype == MR_BF16 and not logits.is_floating_point():  # no raw bit patterns here
        dtype = -1
    T = _types()
    tptr = lptr = iptr = vptr = sptr = eptr = None
    ntok = ldt = ldp = topk = ldo = 0
    if (tokens is None) != (logprob is None):
        raise ValueError("tokens and logprob go together")
    if tokens is not None:
        shape = tokens.shape
        if len(shape) != 2 or shape[0] != m or logprob.shape != shape:
            raise ValueError("tokens and logprob must be [m, t]")
        if tokens.dtype is not T.i32 or logprob.dtype is not T.f32:
            raise ValueError("tokens must be int32, logprob float32")
        ntok = shape[1]
        if ntok:
            ldt, cols = tokens.stride()
            ldp, cols1 = logprob.stride()
            if (cols != 1 or cols1 != 1) and ntok != 1:
                raise ValueError("tokens and logprob must have unit column stride")
            if m == 1:  # strides of dimensions of size one may be anything
                ldt = ldp = ntok
            tptr, lptr = tokens.data_ptr(), logprob.data_ptr()
    if lse is not None:
        if lse.shape != (m,) or (lse.stride(0) != 1 and m != 1) or lse.dtype is not T.f32:
            raise ValueError("lse must be a contiguous [m] float32 tensor")
        sptr = lse.data_ptr()
    if entropy is not None:
        if entropy.shape != (m,) or (entropy.stride(0) != 1 and m != 1) or entropy.dtype is not T.f32:
            raise ValueError("entropy must be a contiguous [m] float32 tensor")
        eptr = entropy.data_ptr()
    if top_idx is None:
        if top_logprob is not None:
            raise ValueError("top_logprob needs top_idx")
    else:
        shape = top_idx.shape
        if len(shape) != 2 or shape[0] != m or top_idx.dtype is not T.i32:
            raise ValueError("top_idx must be [m, k] int32")
        if top_logprob is not None and (top_logprob.shape != shape or top_logprob.dtype is not T.f32):
            raise ValueError("top_logprob must be float32 of top_idx's shape")
        topk = shape[1]
        if topk:
            ldo, cols = top_idx.stride()
            iptr = top_idx.data_ptr()
            if top_logprob is not None:
                ldv, cols1 = top_logprob.stride()
                if (cols1 != 1 and topk != 1) or (ldv != ldo and m != 1):
                    raise ValueError("top_logprob must have top_idx's stride")
                vptr = top_logprob.data_ptr()
            if cols != 1 and topk != 1:
                raise ValueError("top_idx must have unit column stride")
            if m == 1:
                ldo = topk
    if (m | n | ntok | topk) >> 31:
        _int32(m, n, ntok, topk)
    stream = _on(stream, logits, tokens, logprob, lse, entropy, top_idx, top_logprob)
    st = lib.token_logprobs(logits.data_ptr(), ldl, dtype, m, n, scale, tptr, ldt, ntok, lptr, ldp, sptr, eptr, topk,
                            iptr, vptr, ldo, stream)
    _check(st, "token_logprobs")
