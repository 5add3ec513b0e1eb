"""Python binding of libpagedattn.so (ctypes).

Argument marshalling only: torch tensors supply device pointers, strides and
the current CUDA stream; every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the library is missing or a call
fails, an exception is raised.

    reshape_and_cache(key, value, k_cache, v_cache, slot_mapping)
    paged_attention(q, k_cache, v_cache, block_tables, seq_lens,
                    query_start_loc, scale, max_query_len, max_seq_len)
    prepare_reshape_and_cache(...) / prepare_paged_attention(...)
        the same calls validated once, re-issued by calling the result
    build_step_metadata(...), qk_norm_rope(...), qk_norm_rope_and_cache(...)
        what a step needs before them: tables, slots and positions from the
        request lengths; the norm and rotation of queries and keys
    QuantCache, reshape_and_cache_quant(...), dequantize_kv(...),
    paged_attention_quant(...)
        the cache in 4 bits: its write, read-back and attention

k_cache / v_cache are [num_blocks, 16, Hkv, Dh] BF16 views (they may be
slices of one interleaved [num_blocks, 2, 16, Hkv, Dh] pool) with identical
strides and a contiguous head dimension.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedattn.so")

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_WORKSPACE = 3
PA_ERR_BAD_METADATA = 4
PA_ERR_TIMEOUT = 5
PA_ERR_CUDA = 6

EXPORTED = ("pa_init", "pa_reshape_and_cache", "pa_paged_attention_workspace_size",
            "pa_paged_attention", "pa_paged_attention_noalloc", "pa_reshape_and_paged_attention",
            "pa_gather_kv_head", "pa_check_errors", "pa_set_fold_wait_limit_ns",
            "pa_copy_to_device", "pa_status_string", "pa_last_launch_info", "pa_build_step_metadata",
            "pa_qk_norm_rope", "pa_qk_norm_rope_and_cache", "pa_reshape_and_cache_quant", "pa_dequantize_kv",
            "pa_paged_attention_quant_workspace_size", "pa_paged_attention_quant")
NOALLOC_SCRATCH_BYTES = 8 << 20


class PaKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kv_tile", ctypes.c_int32),
                ("block_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class PaQuantCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("block_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


_lib = None
_lock = threading.Lock()


def load(path: str = LIB_PATH):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m paged_kv_cache_178_gb300.build` (needs nvcc)")
        lib = ctypes.CDLL(path)
        i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        lib.pa_init.restype = i32
        lib.pa_init.argtypes = []
        lib.pa_reshape_and_cache.restype = i32
        lib.pa_reshape_and_cache.argtypes = [vp, i64, vp, i64, i64, ctypes.POINTER(PaKvCache), vp, vp]
        lib.pa_paged_attention_workspace_size.restype = sz
        lib.pa_paged_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.pa_paged_attention.restype = i32
        lib.pa_paged_attention.argtypes = [vp, i64, i64, i32, ctypes.POINTER(PaKvCache), vp, i32, vp,
                                           vp, i32, i32, i32, ctypes.c_float, vp, vp, vp, sz, vp]
        lib.pa_paged_attention_noalloc.restype = i32
        lib.pa_paged_attention_noalloc.argtypes = [vp, i64, i64, i32, ctypes.POINTER(PaKvCache), vp, i32,
                                                   vp, vp, i32, i32, i32, ctypes.c_float, vp, vp, vp]
        lib.pa_reshape_and_paged_attention.restype = i32
        lib.pa_reshape_and_paged_attention.argtypes = [
            vp, i64, vp, i64, i64, vp, vp, i64, i64, i32, ctypes.POINTER(PaKvCache), vp, i32, vp, vp, i32,
            i32, i32, ctypes.c_float, vp, vp, vp, sz, vp]
        lib.pa_gather_kv_head.restype = i32
        lib.pa_gather_kv_head.argtypes = [ctypes.POINTER(PaKvCache), i32, vp, i32, vp, i32, vp, vp, i64, vp,
                                          vp, vp]
        lib.pa_check_errors.restype = i32
        lib.pa_check_errors.argtypes = [vp, ctypes.POINTER(i64)]
        lib.pa_set_fold_wait_limit_ns.restype = ctypes.c_uint64
        lib.pa_set_fold_wait_limit_ns.argtypes = [ctypes.c_uint64]
        lib.pa_copy_to_device.restype = i32
        lib.pa_copy_to_device.argtypes = [vp, vp, sz, i32, vp]
        f32, qc = ctypes.c_float, ctypes.POINTER(PaQuantCache)
        lib.pa_build_step_metadata.restype = i32
        lib.pa_build_step_metadata.argtypes = [vp, vp, i32, vp, i32, vp, i32, vp, vp, i64, vp, vp, i64, vp, vp, vp]
        lib.pa_qk_norm_rope.restype = i32
        lib.pa_qk_norm_rope.argtypes = [vp, i64, i32, vp, i64, i32, i32, i64, vp, vp, i64, i32, i32, vp, vp, f32, f32,
                                        vp, i64, vp, i64, vp]
        lib.pa_qk_norm_rope_and_cache.restype = i32
        lib.pa_qk_norm_rope_and_cache.argtypes = [vp, i64, i32, vp, i64, vp, i64, i64, vp, vp, i64, i32, i32, vp, vp,
                                                  f32, f32, vp, i64, ctypes.POINTER(PaKvCache), vp, vp]
        lib.pa_reshape_and_cache_quant.restype = i32
        lib.pa_reshape_and_cache_quant.argtypes = [vp, i64, vp, i64, i64, qc, vp, vp]
        lib.pa_dequantize_kv.restype = i32
        lib.pa_dequantize_kv.argtypes = [qc, vp, i32, vp, i32, vp, vp, i64, vp, vp, vp]
        lib.pa_paged_attention_quant_workspace_size.restype = sz
        lib.pa_paged_attention_quant_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i64]
        lib.pa_paged_attention_quant.restype = i32
        lib.pa_paged_attention_quant.argtypes = [vp, i64, i64, i32, qc, vp, i32, vp, vp, i32, i32, i32, i64, f32, vp,
                                                 vp, vp, sz, vp]
        lib.pa_status_string.restype = ctypes.c_char_p
        lib.pa_status_string.argtypes = [i32]
        lib.pa_last_launch_info.restype = None
        lib.pa_last_launch_info.argtypes = [ctypes.c_char_p, sz]
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != PA_OK:
        raise PagedAttnError(status, what)


def _stream_handle(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def init() -> None:
    _check(load().pa_init(), "pa_init")


def set_fold_wait_limit_ns(limit_ns: int) -> int:
    """Time limit of the split-KV fold's cross-CTA wait and of the direct 4-bit
    attention's waits for pages (default 2 s); returns the previous limit.  0
    makes the waiting CTAs give up at once (a test of the timeout path)."""
    return int(load().pa_set_fold_wait_limit_ns(int(limit_ns)))


def last_launch_info() -> str:
    buf = ctypes.create_string_buffer(256)
    load().pa_last_launch_info(buf, 256)
    return buf.value.decode()


def cache_struct(k_cache: torch.Tensor, v_cache: torch.Tensor, kv_tile: int = 0) -> PaKvCache:
    """Describe a [num_blocks, 16, Hkv, Dh] K/V pair for the C ABI.  kv_tile:
    the attention's KV tile (0: the head dim's default; 64 or 128 at Dh=128)."""
    for t in (k_cache, v_cache):
        if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 4:
            raise ValueError("caches must be 4-D BF16 CUDA tensors [num_blocks, 16, Hkv, Dh]")
        if t.stride(3) != 1:
            raise ValueError("the head dimension of the caches must be contiguous")
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("K and V caches must have the same shape and strides")
    nb, bs, hkv, dh = k_cache.shape
    return PaKvCache(k_cache.data_ptr(), v_cache.data_ptr(), nb, bs, hkv, dh, int(kv_tile), k_cache.stride(0),
                     k_cache.stride(1), k_cache.stride(2))


def _validate_write(key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor) -> int:
    """Checks the cache-write inputs; returns the token count."""
    for t in (key, value):
        if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 3 or t.stride(2) != 1 \
                or t.stride(1) != t.shape[2]:
            raise ValueError("key/value must be [N, Hkv, Dh] BF16 CUDA tensors with contiguous heads")
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_cuda or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 CUDA tensor")
    n = key.shape[0]
    if value.shape[0] != n or slot_mapping.numel() != n:
        raise ValueError("key, value and slot_mapping disagree on the token count")
    return n


def _validate_attention(q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                        query_start_loc: torch.Tensor) -> Tuple[int, int, int, int]:
    """Checks the attention inputs; returns (Tq, Hq, Dh, num_seqs)."""
    if q.dtype != torch.bfloat16 or not q.is_cuda or q.dim() != 3 or q.stride(2) != 1 \
            or q.stride(1) != q.shape[2]:
        raise ValueError("q must be a [Tq, Hq, Dh] BF16 CUDA tensor with contiguous heads")
    tq, hq, dh = q.shape
    for name, t in (("block_tables", block_tables), ("seq_lens", seq_lens),
                    ("query_start_loc", query_start_loc)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    num_seqs = seq_lens.numel()
    if query_start_loc.numel() != num_seqs + 1 or block_tables.dim() != 2 \
            or block_tables.shape[0] != num_seqs:
        raise ValueError("metadata shapes disagree")
    return tq, hq, dh, num_seqs


def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Write key/value [N, Hkv, Dh] into the caches at slot_mapping [N] (int64);
    negative slots are skipped."""
    c = cache_struct(k_cache, v_cache)
    n = _validate_write(key, value, slot_mapping)
    _check(load().pa_reshape_and_cache(key.data_ptr(), key.stride(0), value.data_ptr(), value.stride(0),
                                       n, ctypes.byref(c), slot_mapping.data_ptr(),
                                       _stream_handle(stream)), "pa_reshape_and_cache")


def workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                   max_query_len: int, max_seq_len: int) -> int:
    return int(load().pa_paged_attention_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                        max_query_len, max_seq_len))


def new_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                  max_query_len: int, max_seq_len: int, device=None) -> torch.Tensor:
    """Zero-filled scratch for pa_paged_attention (reusable across calls)."""
    n = workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len, max_seq_len)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_tables: torch.Tensor, seq_lens: torch.Tensor,
                    query_start_loc: torch.Tensor, scale: float, max_query_len: int,
                    max_seq_len: int, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                    workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None, kv_tile: int = 0
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal GQA attention of q [Tq, Hq, Dh] over the paged caches.
    Returns (out [Tq, Hq, Dh] BF16, lse [Tq, Hq] fp32 or None).  kv_tile
    selects the fixed arithmetic's KV tile (see cache_struct)."""
    c = cache_struct(k_cache, v_cache, kv_tile)
    tq, hq, dh, num_seqs = _validate_attention(q, block_tables, seq_lens, query_start_loc)
    if out is None:
        out = torch.empty((tq, hq, dh), dtype=torch.bfloat16, device=q.device)
    elif out.shape != (tq, hq, dh) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [Tq, Hq, Dh] BF16 tensor")
    if lse is None and want_lse:
        lse = torch.empty((tq, hq), dtype=torch.float32, device=q.device)
    if lse is not None and (lse.shape != (tq, hq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous [Tq, Hq] fp32 tensor")
    _check_result_tensor("out", out)
    if lse is not None:
        _check_result_tensor("lse", lse)
    need = workspace_size(num_seqs, hq, c.num_kv_heads, dh, max_query_len, max_seq_len)
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(load().pa_paged_attention(
        q.data_ptr(), tq, q.stride(0), hq, ctypes.byref(c), block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), query_start_loc.data_ptr(), num_seqs,
        int(max_query_len), int(max_seq_len), float(scale), out.data_ptr(),
        lse.data_ptr() if lse is not None else 0, ws_ptr, ws_len, _stream_handle(stream)),
        "pa_paged_attention")
    return out, lse


def paged_attention_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor,
                            query_start_loc: torch.Tensor, scale: float, max_query_len: int,
                            max_seq_len: int, out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None, kv_tile: int = 0) -> int:
    """paged_attention for callers that cannot allocate: no workspace and no
    output allocation here (out, and lse if wanted, are passed in); the
    library's built-in scratch array is used instead.  Returns the status
    code (PA_ERR_WORKSPACE when the bounds need more than
    NOALLOC_SCRATCH_BYTES) rather than raising."""
    c = cache_struct(k_cache, v_cache, kv_tile)
    tq, hq, dh = q.shape
    return int(load().pa_paged_attention_noalloc(
        q.data_ptr(), tq, q.stride(0), hq, ctypes.byref(c), block_tables.data_ptr(),
        block_tables.shape[1], seq_lens.data_ptr(), query_start_loc.data_ptr(), seq_lens.numel(),
        int(max_query_len), int(max_seq_len), float(scale), out.data_ptr(),
        lse.data_ptr() if lse is not None else 0, _stream_handle(stream)))


class PreparedCall:
    """A library call validated and marshalled once.  Calling it re-issues the
    same C-ABI call with the same pointers: the tensors' contents may change
    between calls, their storage must stay alive and in place (the object
    keeps references to them)."""

    def __init__(self, fn, args, what: str, keep):
        # The arguments are converted here, and the call goes through a function
        # object without argument types, which would convert them each time
        # (22 arguments: 2.1 us a call, 1.1 so).  from_param is the prototypes'
        # own conversion: what they take (numpy and torch integers too) or refuse.
        self._args = tuple(t.from_param(a) for t, a in zip(fn.argtypes, args))
        self._fn = load()[fn.__name__]
        self._fn.restype = fn.restype
        self._what, self._keep = what, keep

    def __call__(self) -> None:
        st = self._fn(*self._args)
        if st != PA_OK:
            raise PagedAttnError(st, self._what)


def _check_result_tensor(name: str, t: torch.Tensor) -> None:
    """out / lse: device memory, or page-locked host memory the kernels write
    directly (mapped into the device's address space)."""
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or a pinned host tensor")


def prepare_copy_to_device(dst: torch.Tensor, src: torch.Tensor,
                           stream: Optional[torch.cuda.Stream] = None, src_ready: bool = False) -> PreparedCall:
    """pa_copy_to_device of all of src's bytes into dst (a CUDA tensor of the
    same byte size; src a pinned host tensor or a CUDA tensor), validated now
    and issued by each call of the result.  src_ready: no kernel in flight
    writes src (e.g. host memory the host fills), so it is read at once."""
    nbytes = src.numel() * src.element_size()
    if not dst.is_cuda or not dst.is_contiguous() or not src.is_contiguous() \
            or dst.numel() * dst.element_size() != nbytes:
        raise ValueError("dst must be a contiguous CUDA tensor of src's byte size")
    if not (src.is_cuda or src.is_pinned()):
        raise ValueError("src must be a pinned host tensor or a CUDA tensor")
    lib = load()
    return PreparedCall(lib.pa_copy_to_device,
                        (dst.data_ptr(), src.data_ptr(), nbytes, 1 if src_ready else 0, _stream_handle(stream)),
                        "pa_copy_to_device", (dst, src))


def copy_to_device(dst: torch.Tensor, src: torch.Tensor, stream: Optional[torch.cuda.Stream] = None,
                   src_ready: bool = False) -> None:
    """Copy src (pinned host or CUDA) into the CUDA tensor dst with the
    library's staging kernel."""
    prepare_copy_to_device(dst, src, stream, src_ready)()


def prepare_reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                              v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                              stream: Optional[torch.cuda.Stream] = None) -> PreparedCall:
    """reshape_and_cache, validated now and issued by each call of the result."""
    c = cache_struct(k_cache, v_cache)
    n = _validate_write(key, value, slot_mapping)
    lib = load()
    args = (key.data_ptr(), key.stride(0), value.data_ptr(), value.stride(0), n, ctypes.byref(c),
            slot_mapping.data_ptr(), _stream_handle(stream))
    return PreparedCall(lib.pa_reshape_and_cache, args, "pa_reshape_and_cache",
                        (key, value, k_cache, v_cache, slot_mapping, c))


def prepare_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor,
                            query_start_loc: torch.Tensor, scale: float, max_query_len: int,
                            max_seq_len: int, out: torch.Tensor, lse: Optional[torch.Tensor],
                            workspace: Optional[torch.Tensor],
                            stream: Optional[torch.cuda.Stream] = None, kv_tile: int = 0) -> PreparedCall:
    """paged_attention into given out / lse / workspace, validated now and
    issued by each call of the result."""
    c = cache_struct(k_cache, v_cache, kv_tile)
    tq, hq, dh, num_seqs = _validate_attention(q, block_tables, seq_lens, query_start_loc)
    if out.shape != (tq, hq, dh) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [Tq, Hq, Dh] BF16 tensor")
    if lse is not None and (lse.shape != (tq, hq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous [Tq, Hq] fp32 tensor")
    _check_result_tensor("out", out)
    if lse is not None:
        _check_result_tensor("lse", lse)
    need = workspace_size(num_seqs, hq, c.num_kv_heads, dh, max_query_len, max_seq_len)
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if ws_len < need:
        raise ValueError(f"workspace needs {need} bytes")
    lib = load()
    args = (q.data_ptr(), tq, q.stride(0), hq, ctypes.byref(c), block_tables.data_ptr(),
            block_tables.shape[1], seq_lens.data_ptr(), query_start_loc.data_ptr(), num_seqs,
            int(max_query_len), int(max_seq_len), ctypes.c_float(float(scale)), out.data_ptr(),
            lse.data_ptr() if lse is not None else 0, workspace.data_ptr() if workspace is not None else 0,
            ws_len, _stream_handle(stream))
    return PreparedCall(lib.pa_paged_attention, args, "pa_paged_attention",
                        (q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, out, lse, workspace, c))


def _composition_args(key, value, slot_mapping, q, k_cache, v_cache, block_tables, seq_lens,
                      query_start_loc, scale, max_query_len, max_seq_len, out, lse, workspace, stream, kv_tile):
    c = cache_struct(k_cache, v_cache, kv_tile)
    n = _validate_write(key, value, slot_mapping)
    tq, hq, dh, num_seqs = _validate_attention(q, block_tables, seq_lens, query_start_loc)
    if out.shape != (tq, hq, dh) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [Tq, Hq, Dh] BF16 tensor")
    if lse is not None and (lse.shape != (tq, hq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous [Tq, Hq] fp32 tensor")
    _check_result_tensor("out", out)
    if lse is not None:
        _check_result_tensor("lse", lse)
    need = workspace_size(num_seqs, hq, c.num_kv_heads, dh, max_query_len, max_seq_len)
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if ws_len < need:
        raise ValueError(f"workspace needs {need} bytes")
    args = (key.data_ptr(), key.stride(0), value.data_ptr(), value.stride(0), n, slot_mapping.data_ptr(),
            q.data_ptr(), tq, q.stride(0), hq, ctypes.byref(c), block_tables.data_ptr(),
            block_tables.shape[1], seq_lens.data_ptr(), query_start_loc.data_ptr(), num_seqs,
            int(max_query_len), int(max_seq_len), ctypes.c_float(float(scale)), out.data_ptr(),
            lse.data_ptr() if lse is not None else 0, workspace.data_ptr() if workspace is not None else 0,
            ws_len, _stream_handle(stream))
    keep = (key, value, slot_mapping, q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, out, lse,
            workspace, c)
    return args, keep


def reshape_and_paged_attention(key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor,
                                q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                query_start_loc: torch.Tensor, scale: float, max_query_len: int,
                                max_seq_len: int, out: Optional[torch.Tensor] = None,
                                lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                                workspace: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None, kv_tile: int = 0
                                ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """reshape_and_cache of key/value at slot_mapping, then paged_attention of q
    over the updated caches, in one library call whose attention grid starts
    its set-up while the cache write runs.  Returns (out, lse or None)."""
    tq, hq, dh = q.shape
    if out is None:
        out = torch.empty((tq, hq, dh), dtype=torch.bfloat16, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((tq, hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        need = workspace_size(seq_lens.numel(), hq, k_cache.shape[2], dh, max_query_len, max_seq_len)
        if need > 0:
            workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    args, _keep = _composition_args(key, value, slot_mapping, q, k_cache, v_cache, block_tables, seq_lens,
                                    query_start_loc, scale, max_query_len, max_seq_len, out, lse, workspace,
                                    stream, kv_tile)
    _check(load().pa_reshape_and_paged_attention(*args), "pa_reshape_and_paged_attention")
    return out, lse


def prepare_reshape_and_paged_attention(key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor,
                                        q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                        block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                        query_start_loc: torch.Tensor, scale: float, max_query_len: int,
                                        max_seq_len: int, out: torch.Tensor, lse: Optional[torch.Tensor],
                                        workspace: Optional[torch.Tensor],
                                        stream: Optional[torch.cuda.Stream] = None,
                                        kv_tile: int = 0) -> PreparedCall:
    """reshape_and_paged_attention into given out / lse / workspace, validated
    now and issued by each call of the result."""
    args, keep = _composition_args(key, value, slot_mapping, q, k_cache, v_cache, block_tables, seq_lens,
                                   query_start_loc, scale, max_query_len, max_seq_len, out, lse, workspace,
                                   stream, kv_tile)
    return PreparedCall(load().pa_reshape_and_paged_attention, args, "pa_reshape_and_paged_attention", keep)


def _validate_gather(k_cache: torch.Tensor, kv_head: int, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                     packed_k: torch.Tensor, packed_v: torch.Tensor, compact_tables: torch.Tensor,
                     compact_offsets: torch.Tensor) -> int:
    """Checks the gather inputs; returns the packed capacity in pages."""
    num_seqs = seq_lens.numel()
    for name, t in (("block_tables", block_tables), ("seq_lens", seq_lens), ("compact_tables", compact_tables),
                    ("compact_offsets", compact_offsets)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if block_tables.dim() != 2 or block_tables.shape[0] != num_seqs or compact_tables.shape != block_tables.shape \
            or compact_offsets.numel() != num_seqs + 1:
        raise ValueError("metadata shapes disagree")
    dh = k_cache.shape[3]
    for t in (packed_k, packed_v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4 \
                or tuple(t.shape[1:]) != (16, 1, dh):
            raise ValueError("packed buffers must be contiguous BF16 CUDA tensors [capacity_pages, 16, 1, Dh]")
    if packed_k.shape != packed_v.shape:
        raise ValueError("packed K and V must have the same capacity")
    if not 0 <= kv_head < k_cache.shape[2]:
        raise ValueError("kv_head out of range")
    return packed_k.shape[0]


def gather_kv_head(k_cache: torch.Tensor, v_cache: torch.Tensor, kv_head: int, block_tables: torch.Tensor,
                   seq_lens: torch.Tensor, packed_k: torch.Tensor, packed_v: torch.Tensor,
                   compact_tables: torch.Tensor, compact_offsets: torch.Tensor,
                   stream: Optional[torch.cuda.Stream] = None) -> None:
    """Pack the pages that block_tables/seq_lens select for one KV head into
    packed_k/packed_v [capacity_pages, 16, 1, Dh] (a one-head pool of their
    own), writing the compact table [B, max_blocks] and page offsets [B + 1]."""
    c = cache_struct(k_cache, v_cache)
    cap = _validate_gather(k_cache, kv_head, block_tables, seq_lens, packed_k, packed_v, compact_tables,
                           compact_offsets)
    _check(load().pa_gather_kv_head(ctypes.byref(c), kv_head, block_tables.data_ptr(), block_tables.shape[1],
                                    seq_lens.data_ptr(), seq_lens.numel(), packed_k.data_ptr(),
                                    packed_v.data_ptr(), cap, compact_tables.data_ptr(),
                                    compact_offsets.data_ptr(), _stream_handle(stream)), "pa_gather_kv_head")


def prepare_gather_kv_head(k_cache: torch.Tensor, v_cache: torch.Tensor, kv_head: int, block_tables: torch.Tensor,
                           seq_lens: torch.Tensor, packed_k: torch.Tensor, packed_v: torch.Tensor,
                           compact_tables: torch.Tensor, compact_offsets: torch.Tensor,
                           stream: Optional[torch.cuda.Stream] = None) -> "PreparedCall":
    """gather_kv_head validated and marshalled once; calling the result
    re-issues the same C-ABI call (tensor contents may change, not storage)."""
    c = cache_struct(k_cache, v_cache)
    cap = _validate_gather(k_cache, kv_head, block_tables, seq_lens, packed_k, packed_v, compact_tables,
                           compact_offsets)
    keep = (c, k_cache, v_cache, block_tables, seq_lens, packed_k, packed_v, compact_tables, compact_offsets)
    args = (ctypes.byref(c), kv_head, block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(),
            seq_lens.numel(), packed_k.data_ptr(), packed_v.data_ptr(), cap, compact_tables.data_ptr(),
            compact_offsets.data_ptr(), _stream_handle(stream))
    return PreparedCall(load().pa_gather_kv_head, args, "pa_gather_kv_head", keep)


def _require_i32(**tensors: torch.Tensor) -> None:
    for name, t in tensors.items():
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")


def _require_same_device(*tensors: Optional[torch.Tensor]) -> None:
    """The library launches on the current device: every tensor must be there."""
    here = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.is_cuda and t.device.index != here:
            raise ValueError(f"tensors must be on the current CUDA device (cuda:{here}), got {t.device}")


def _empty(shape, dtype: torch.dtype, device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """Memory for a call on `stream`, taken from that stream's share of the
    allocator: no earlier or later user of it on another stream can meet the call."""
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def prepare_build_step_metadata(context_lens: torch.Tensor, query_lens: torch.Tensor, block_tables: torch.Tensor,
                                free_pages: torch.Tensor, num_blocks: int, slot_mapping: torch.Tensor,
                                positions: torch.Tensor, seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                                cursor_out: torch.Tensor, cursor_in: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None) -> PreparedCall:
    """build_step_metadata, validated now and issued by each call of the result."""
    _require_i32(context_lens=context_lens, query_lens=query_lens, block_tables=block_tables, free_pages=free_pages,
                 positions=positions, seq_lens=seq_lens, query_start_loc=query_start_loc, cursor_out=cursor_out)
    if cursor_in is not None:
        _require_i32(cursor_in=cursor_in)
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_cuda or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int64 CUDA tensor")
    _require_same_device(context_lens, query_lens, block_tables, free_pages, slot_mapping, positions, seq_lens,
                         query_start_loc, cursor_out, cursor_in)
    n = context_lens.numel()
    if query_lens.numel() != n or seq_lens.numel() != n or query_start_loc.numel() != n + 1 \
            or block_tables.dim() != 2 or block_tables.shape[0] != n or positions.numel() != slot_mapping.numel() \
            or cursor_out.numel() != 1 or (cursor_in is not None and cursor_in.numel() != 1):
        raise ValueError("metadata shapes disagree")
    args = (context_lens.data_ptr(), query_lens.data_ptr(), n, block_tables.data_ptr(), block_tables.shape[1],
            free_pages.data_ptr(), free_pages.numel(), cursor_in.data_ptr() if cursor_in is not None else 0,
            cursor_out.data_ptr(), int(num_blocks), slot_mapping.data_ptr(), positions.data_ptr(),
            slot_mapping.numel(), seq_lens.data_ptr(), query_start_loc.data_ptr(), _stream_handle(stream))
    return PreparedCall(load().pa_build_step_metadata, args, "pa_build_step_metadata",
                        (context_lens, query_lens, block_tables, free_pages, slot_mapping, positions, seq_lens,
                         query_start_loc, cursor_out, cursor_in))


def build_step_metadata(context_lens: torch.Tensor, query_lens: torch.Tensor, block_tables: torch.Tensor,
                        free_pages: torch.Tensor, num_blocks: int, slot_mapping: torch.Tensor,
                        positions: torch.Tensor, seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                        cursor_out: torch.Tensor, cursor_in: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> None:
    """One step's metadata from context_lens and query_lens [B] (int32): pages
    from free_pages (from index cursor_in on) enter block_tables [B, max_blocks];
    slot_mapping (int64) and positions [N] of the new tokens (-1 past them),
    seq_lens [B], query_start_loc [B + 1] and cursor_out [1] are written.
    seq_lens may be context_lens, cursor_out may be cursor_in."""
    prepare_build_step_metadata(context_lens, query_lens, block_tables, free_pages, num_blocks, slot_mapping,
                                positions, seq_lens, query_start_loc, cursor_out, cursor_in, stream)()


def rope_table(max_positions: int, rot_dim: int, theta: float = 10000.0, device=None) -> torch.Tensor:
    """The [max_positions, rot_dim] fp32 cos/sin table of qk_norm_rope for the
    angles p * theta**(-2i/rot_dim), computed in 64 bits and rounded once."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * float(theta) ** (-i / rot_dim)
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _head_rows(name: str, t: torch.Tensor) -> None:
    if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 3 or t.stride(2) != 1 \
            or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name} must be a [T, heads, Dh] BF16 CUDA tensor with contiguous heads")


def _tok_stride(t: torch.Tensor) -> int:
    """Token stride; that of one token does not matter (torch may report any)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1] * t.shape[2])


def _rope_args(q, k, positions, cos_sin, q_out, q_weight, k_weight):
    for name, t in (("q", q), ("k", k), ("q_out", q_out)):
        _head_rows(name, t)
    _require_i32(positions=positions)
    n, dh = q.shape[0], q.shape[2]
    if k.shape[0] != n or k.shape[2] != dh or q_out.shape != q.shape or positions.numel() != n:
        raise ValueError("q, k, q_out and positions disagree")
    if cos_sin.dtype != torch.float32 or not cos_sin.is_cuda or not cos_sin.is_contiguous() or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be a contiguous [max_positions, rot_dim] fp32 CUDA tensor")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype != torch.bfloat16 or not w.is_cuda or not w.is_contiguous() or w.numel() != dh):
            raise ValueError(f"{name} must be a contiguous [Dh] BF16 CUDA tensor")
    return n, dh


def _ptr(t: Optional[torch.Tensor]) -> int:
    return t.data_ptr() if t is not None else 0


def prepare_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                         q_out: torch.Tensor, k_out: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                         k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                         weight_offset: float = 0.0, stream: Optional[torch.cuda.Stream] = None) -> PreparedCall:
    """qk_norm_rope, validated now and issued by each call of the result."""
    n, dh = _rope_args(q, k, positions, cos_sin, q_out, q_weight, k_weight)
    _head_rows("k_out", k_out)
    if k_out.shape != k.shape:
        raise ValueError("k_out must have k's shape")
    _require_same_device(q, k, positions, cos_sin, q_out, k_out, q_weight, k_weight)
    args = (q.data_ptr(), _tok_stride(q), q.shape[1], k.data_ptr(), _tok_stride(k), k.shape[1], dh, n,
            positions.data_ptr(), cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], 1 if interleaved else 0,
            _ptr(q_weight), _ptr(k_weight), ctypes.c_float(weight_offset), ctypes.c_float(eps), q_out.data_ptr(),
            _tok_stride(q_out), k_out.data_ptr(), _tok_stride(k_out), _stream_handle(stream))
    return PreparedCall(load().pa_qk_norm_rope, args, "pa_qk_norm_rope",
                        (q, k, positions, cos_sin, q_out, k_out, q_weight, k_weight))


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False, weight_offset: float = 0.0,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMS norm of every head row of q [T, Hq, Dh] and k [T, Hkv, Dh] (where a
    weight is given), then the rotation by positions [T] (int32, -1: padding, the
    row is left untouched) with cos_sin (see rope_table).  q_out / k_out may be
    q / k.  Returns (q_out, k_out)."""
    q_out = _empty(q.shape, q.dtype, q.device, stream) if q_out is None else q_out
    k_out = _empty(k.shape, k.dtype, k.device, stream) if k_out is None else k_out
    prepare_qk_norm_rope(q, k, positions, cos_sin, q_out, k_out, q_weight, k_weight, eps, interleaved, weight_offset,
                         stream)()
    return q_out, k_out


def prepare_qk_norm_rope_and_cache(q: torch.Tensor, k: torch.Tensor, value: torch.Tensor, positions: torch.Tensor,
                                   cos_sin: torch.Tensor, q_out: torch.Tensor, k_cache: torch.Tensor,
                                   v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                                   q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                                   eps: float = 1e-6, interleaved: bool = False, weight_offset: float = 0.0,
                                   stream: Optional[torch.cuda.Stream] = None) -> PreparedCall:
    """qk_norm_rope_and_cache, validated now and issued by each call of the result."""
    c = cache_struct(k_cache, v_cache)
    n, dh = _rope_args(q, k, positions, cos_sin, q_out, q_weight, k_weight)
    _head_rows("value", value)
    if value.shape != k.shape or k.shape[1] != c.num_kv_heads or dh != c.head_dim:
        raise ValueError("k and value must be [T, Hkv, Dh] of the cache")
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_cuda or not slot_mapping.is_contiguous() \
            or slot_mapping.numel() != n:
        raise ValueError("slot_mapping must be a contiguous int64 CUDA tensor of one slot per token")
    _require_same_device(q, k, value, positions, cos_sin, q_out, k_cache, v_cache, slot_mapping, q_weight, k_weight)
    args = (q.data_ptr(), _tok_stride(q), q.shape[1], k.data_ptr(), _tok_stride(k), value.data_ptr(),
            _tok_stride(value), n, positions.data_ptr(), cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1],
            1 if interleaved else 0, _ptr(q_weight), _ptr(k_weight), ctypes.c_float(weight_offset),
            ctypes.c_float(eps), q_out.data_ptr(), _tok_stride(q_out), ctypes.byref(c), slot_mapping.data_ptr(),
            _stream_handle(stream))
    return PreparedCall(load().pa_qk_norm_rope_and_cache, args, "pa_qk_norm_rope_and_cache",
                        (q, k, value, positions, cos_sin, q_out, k_cache, v_cache, slot_mapping, q_weight, k_weight, c))


def qk_norm_rope_and_cache(q: torch.Tensor, k: torch.Tensor, value: torch.Tensor, positions: torch.Tensor,
                           cos_sin: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           slot_mapping: torch.Tensor, q_out: Optional[torch.Tensor] = None,
                           q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, interleaved: bool = False, weight_offset: float = 0.0,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """qk_norm_rope and the cache write in one pass: the rotated keys and the
    values go to slot_mapping of the BF16 pool.  Returns q_out."""
    q_out = _empty(q.shape, q.dtype, q.device, stream) if q_out is None else q_out
    prepare_qk_norm_rope_and_cache(q, k, value, positions, cos_sin, q_out, k_cache, v_cache, slot_mapping, q_weight,
                                   k_weight, eps, interleaved, weight_offset, stream)()
    return q_out


def quant_record_bytes(head_dim: int) -> int:
    """Bytes of one page's K (or V) of one head in a 4-bit pool."""
    return 9 * int(head_dim)


class QuantCache:
    """A paged KV cache in 4 bits: byte pools k_pool, v_pool [num_blocks, Hkv,
    9*Dh] (two tensors, or the slices [:, 0] and [:, 1] of one [num_blocks, 2,
    Hkv, 9*Dh] tensor) with identical strides, and the power-of-two factors
    k_scale, v_scale of all their values."""

    def __init__(self, k_pool: torch.Tensor, v_pool: torch.Tensor, head_dim: int, k_scale: float = 1.0,
                 v_scale: float = 1.0):
        for t in (k_pool, v_pool):
            if t.dtype != torch.uint8 or not t.is_cuda or t.dim() != 3 or t.stride(2) != 1 \
                    or t.shape[2] != quant_record_bytes(head_dim):
                raise ValueError("4-bit pools must be [num_blocks, Hkv, 9*Dh] uint8 CUDA tensors with contiguous records")
        if k_pool.shape != v_pool.shape or k_pool.stride() != v_pool.stride() or k_pool.device != v_pool.device:
            raise ValueError("K and V pools must have the same shape, strides and device")
        self.k_pool, self.v_pool = k_pool, v_pool
        self.head_dim, self.num_kv_heads, self.num_blocks = int(head_dim), k_pool.shape[1], k_pool.shape[0]
        self.struct = PaQuantCache(k_pool.data_ptr(), v_pool.data_ptr(), k_pool.shape[0], 16, k_pool.shape[1],
                                   int(head_dim), 0, k_pool.stride(0), k_pool.stride(1), float(k_scale),
                                   float(v_scale))


def new_quant_cache(num_blocks: int, num_kv_heads: int, head_dim: int, k_scale: float = 1.0, v_scale: float = 1.0,
                    device=None) -> QuantCache:
    """A zero-filled interleaved 4-bit cache (every value reads as 0)."""
    pool = torch.zeros((num_blocks, 2, num_kv_heads, quant_record_bytes(head_dim)), dtype=torch.uint8,
                       device=device if device is not None else "cuda")
    return QuantCache(pool[:, 0], pool[:, 1], head_dim, k_scale, v_scale)


def prepare_reshape_and_cache_quant(key: torch.Tensor, value: torch.Tensor, cache: QuantCache,
                                    slot_mapping: torch.Tensor,
                                    stream: Optional[torch.cuda.Stream] = None) -> PreparedCall:
    """reshape_and_cache_quant, validated now and issued by each call of the result."""
    n = key.shape[0]
    for name, t in (("key", key), ("value", value)):
        _head_rows(name, t)
        if tuple(t.shape) != (n, cache.num_kv_heads, cache.head_dim):
            raise ValueError(f"{name} must be [N, Hkv, Dh] of the cache")
    if slot_mapping.dtype != torch.int64 or not slot_mapping.is_cuda or not slot_mapping.is_contiguous() \
            or slot_mapping.numel() != n:
        raise ValueError("slot_mapping must be a contiguous int64 CUDA tensor of one slot per token")
    _require_same_device(key, value, cache.k_pool, slot_mapping)
    args = (key.data_ptr(), _tok_stride(key), value.data_ptr(), _tok_stride(value), n, ctypes.byref(cache.struct),
            slot_mapping.data_ptr(), _stream_handle(stream))
    return PreparedCall(load().pa_reshape_and_cache_quant, args, "pa_reshape_and_cache_quant",
                        (key, value, cache, slot_mapping))


def reshape_and_cache_quant(key: torch.Tensor, value: torch.Tensor, cache: QuantCache, slot_mapping: torch.Tensor,
                            stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantise key/value [N, Hkv, Dh] into the 4-bit cache at slot_mapping [N]
    (int64); negative slots are skipped."""
    prepare_reshape_and_cache_quant(key, value, cache, slot_mapping, stream)()


def prepare_dequantize_kv(cache: QuantCache, block_tables: torch.Tensor, seq_lens: torch.Tensor, k_out: torch.Tensor,
                          v_out: torch.Tensor, compact_tables: torch.Tensor, compact_offsets: torch.Tensor,
                          stream: Optional[torch.cuda.Stream] = None) -> PreparedCall:
    """dequantize_kv, validated now and issued by each call of the result."""
    _require_i32(block_tables=block_tables, seq_lens=seq_lens, compact_tables=compact_tables,
                 compact_offsets=compact_offsets)
    num_seqs = seq_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != num_seqs or compact_tables.shape != block_tables.shape \
            or compact_offsets.numel() != num_seqs + 1:
        raise ValueError("metadata shapes disagree")
    for t in (k_out, v_out):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4 \
                or tuple(t.shape[1:]) != (16, cache.num_kv_heads, cache.head_dim):
            raise ValueError("k_out/v_out must be contiguous BF16 CUDA tensors [capacity_pages, 16, Hkv, Dh]")
    if k_out.shape != v_out.shape:
        raise ValueError("k_out and v_out must have the same capacity")
    _require_same_device(cache.k_pool, block_tables, seq_lens, k_out, v_out, compact_tables, compact_offsets)
    args = (ctypes.byref(cache.struct), block_tables.data_ptr(), block_tables.shape[1], seq_lens.data_ptr(), num_seqs,
            k_out.data_ptr(), v_out.data_ptr(), k_out.shape[0], compact_tables.data_ptr(), compact_offsets.data_ptr(),
            _stream_handle(stream))
    return PreparedCall(load().pa_dequantize_kv, args, "pa_dequantize_kv",
                        (cache, block_tables, seq_lens, k_out, v_out, compact_tables, compact_offsets))


def dequantize_kv(cache: QuantCache, block_tables: torch.Tensor, seq_lens: torch.Tensor, k_out: torch.Tensor,
                  v_out: torch.Tensor, compact_tables: torch.Tensor, compact_offsets: torch.Tensor,
                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Read the pages that block_tables/seq_lens select back into k_out/v_out
    [capacity_pages, 16, Hkv, Dh] (a BF16 pool of their own), writing the compact
    table [B, max_blocks] and page offsets [B + 1]."""
    prepare_dequantize_kv(cache, block_tables, seq_lens, k_out, v_out, compact_tables, compact_offsets, stream)()


def quant_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_query_len: int,
                         max_seq_len: int, max_pages: int = 0) -> int:
    return int(load().pa_paged_attention_quant_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                              max_query_len, max_seq_len, max_pages))


def new_quant_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_query_len: int,
                        max_seq_len: int, max_pages: int = 0, device=None) -> torch.Tensor:
    """Scratch for paged_attention_quant (reusable across calls, one after another)."""
    n = quant_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len, max_seq_len, max_pages)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device if device is not None else "cuda")


def prepare_paged_attention_quant(q: torch.Tensor, cache: QuantCache, block_tables: torch.Tensor,
                                  seq_lens: torch.Tensor, query_start_loc: torch.Tensor, scale: float,
                                  max_query_len: int, max_seq_len: int, out: torch.Tensor,
                                  lse: Optional[torch.Tensor], workspace: torch.Tensor, max_pages: int = 0,
                                  stream: Optional[torch.cuda.Stream] = None) -> PreparedCall:
    """paged_attention_quant into given out / lse / workspace, validated now
    and issued by each call of the result."""
    tq, hq, dh, num_seqs = _validate_attention(q, block_tables, seq_lens, query_start_loc)
    if dh != cache.head_dim:
        raise ValueError("q and the cache disagree on the head dim")
    if out.shape != (tq, hq, dh) or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous [Tq, Hq, Dh] BF16 tensor")
    if lse is not None and (lse.shape != (tq, hq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous [Tq, Hq] fp32 tensor")
    _check_result_tensor("out", out)
    if lse is not None:
        _check_result_tensor("lse", lse)
    _require_same_device(q, cache.k_pool, block_tables, seq_lens, query_start_loc, out, lse, workspace)
    if workspace is not None and (not workspace.is_cuda or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    need = quant_workspace_size(num_seqs, hq, cache.num_kv_heads, dh, max_query_len, max_seq_len, max_pages)
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if ws_len < need:
        raise ValueError(f"workspace needs {need} bytes")
    args = (q.data_ptr(), tq, _tok_stride(q), hq, ctypes.byref(cache.struct), block_tables.data_ptr(),
            block_tables.shape[1], seq_lens.data_ptr(), query_start_loc.data_ptr(), num_seqs, int(max_query_len),
            int(max_seq_len), int(max_pages), ctypes.c_float(float(scale)), out.data_ptr(), _ptr(lse),
            _ptr(workspace), ws_len, _stream_handle(stream))
    return PreparedCall(load().pa_paged_attention_quant, args, "pa_paged_attention_quant",
                        (q, cache, block_tables, seq_lens, query_start_loc, out, lse, workspace))


def paged_attention_quant(q: torch.Tensor, cache: QuantCache, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                          query_start_loc: torch.Tensor, scale: float, max_query_len: int, max_seq_len: int,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          want_lse: bool = True, workspace: Optional[torch.Tensor] = None, max_pages: int = 0,
                          stream: Optional[torch.cuda.Stream] = None
                          ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal GQA attention of q [Tq, Hq, Dh] over the 4-bit cache.  Returns
    (out [Tq, Hq, Dh] BF16, lse [Tq, Hq] fp32 or None)."""
    tq, hq, dh = q.shape
    if out is None:
        out = _empty((tq, hq, dh), torch.bfloat16, q.device, stream)
    if lse is None and want_lse:
        lse = _empty((tq, hq), torch.float32, q.device, stream)
    if workspace is None:
        n = quant_workspace_size(seq_lens.numel(), hq, cache.num_kv_heads, dh, max_query_len, max_seq_len, max_pages)
        workspace = _empty((max(n, 256),), torch.uint8, q.device, stream)
    prepare_paged_attention_quant(q, cache, block_tables, seq_lens, query_start_loc, scale, max_query_len,
                                  max_seq_len, out, lse, workspace, max_pages, stream)()
    return out, lse


def check_errors(stream: Optional[torch.cuda.Stream] = None) -> Tuple[int, int]:
    """Synchronise the stream, read and clear the device error latch.
    Returns (status, first_bad_index)."""
    idx = ctypes.c_int64(-1)
    st = load().pa_check_errors(_stream_handle(stream), ctypes.byref(idx))
    return int(st), int(idx.value)
