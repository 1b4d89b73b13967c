"""Python binding of the io_aware_online_b200 C-ABI attention library.

Argument marshalling only: every step of the computation runs in the CUDA kernels
of ``libfa_b200.so`` (built by ``io_aware_online_b200.build``).  PyTorch supplies
device memory and the current stream; outputs the caller does not pass are
allocated with ``torch.empty`` before the call.  There is no fallback: if the
library is missing or a call fails, an exception is raised.

Functions mirror include/fa.h:
    fa_fwd(q, k, v, ...)                  dense [B,S,H,d] or varlen [total,H,d]
    fa_fwd_host(q, k, v, ...)             dense, q/k/v/out in host memory (transfers
                                          overlapped with the kernels)
    fa_fwd_kvcache(q, k_cache, v_cache, ...)
    fa_fwd_kvcache_static(q, k_cache, v_cache, ...)   (no workspace; fixed device scratch)
    fa_combine(out_partial, lse_partial, ...)
    fa_kvcache_num_splits(...), fa_kvcache_workspace_size(...)
    fa_qk_norm_rope(q, k, ...), fa_qk_norm_rope_bwd(dq_out, dk_out, q, k, ...)
    fa_kvcache_append_quant(...), fa_kvcache_read_quant(...), fa_fwd_kvcache_quant(...),
    fa_qk_norm_rope_append_quant(...)     the 8-bit KV cache
    fa_device_status(clear=True), fa_set_wait_timeout_ms(ms), fa_version()
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

__all__ = ["FAError", "fa_fwd", "fa_fwd_host", "fa_fwd_host_workspace_size", "fa_fwd_kvcache", "fa_fwd_kvcache_static", "fa_combine",
           "fa_kvcache_num_splits",
           "fa_kvcache_workspace_size", "fa_qk_norm_rope", "fa_qk_norm_rope_bwd",
           "fa_qk_norm_rope_append_quant", "fa_kvcache_append_quant", "fa_kvcache_read_quant",
           "fa_fwd_kvcache_quant", "fa_kvcache_quant_workspace_size",
           "fa_device_status", "fa_set_wait_timeout_ms",
           "fa_version", "library_path", "load"]

FA_FP16, FA_BF16, FA_FP32 = 0, 1, 2
FA_DEV_WAIT_TIMEOUT, FA_DEV_BAD_BLOCK = 1, 2
FA_DEV_BAD_POSITION = 16
_KV_FORMAT = {torch.float8_e4m3fn: 0, torch.int8: 1}
_DT = {torch.float16: FA_FP16, torch.bfloat16: FA_BF16, torch.float32: FA_FP32}
_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libfa_b200.so")
_lib = None


class FAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[fa error {code}] {msg}")
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libfa_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: run `python -m io_aware_online_b200.build` "
                          "(there is no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64p, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_int64), ctypes.c_float
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i64p, i64p,
                           i64p, i64p, vp, vp, i32, i32, f32, i32, i32, i32, f32, vp, vp]
    lib.fa_fwd.restype = i32
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, f32, f32, f32, i32, i32, i32, i32, i32, i32,
                               i64p, i64p, i64p, i64p, vp, vp, i32, i32, f32, i32, i32, i32, f32,
                               vp, vp]
    lib.fa_fwd_fp8.restype = i32
    lib.fa_fwd_host_workspace_size.argtypes = [i32] * 7
    lib.fa_fwd_host_workspace_size.restype = ctypes.c_size_t
    lib.fa_fwd_host.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, i32,
                                i32, i32, f32, vp, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_host.restype = i32
    lib.fa_kvcache_num_splits.argtypes = [i32] * 8
    lib.fa_kvcache_num_splits.restype = i32
    lib.fa_kvcache_workspace_size.argtypes = [i32] * 8
    lib.fa_kvcache_workspace_size.restype = ctypes.c_size_t
    lib.fa_fwd_kvcache.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, i32, i32,
                                   i32, i32, vp, f32, i32, i32, i32, f32, vp, i32, vp,
                                   ctypes.c_size_t, vp]
    lib.fa_fwd_kvcache.restype = i32
    lib.fa_fwd_kvcache_static.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp,
                                          i32, i32, i32, i32, vp, f32, i32, i32, i32, f32, vp,
                                          i32, vp]
    lib.fa_fwd_kvcache_static.restype = i32
    lib.fa_kvcache_append.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, i32, i32, i32,
                                      i32, vp, vp]
    lib.fa_kvcache_append.restype = i32
    lib.fa_fwd_kvcache_append.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, i32,
                                          i32, i32, vp, i32, i32, i32, i32, vp, f32, i32, i32,
                                          i32, f32, vp, i32, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_kvcache_append.restype = i32
    lib.fa_kvcache_static_scratch_bytes.argtypes = []
    lib.fa_kvcache_static_scratch_bytes.restype = ctypes.c_size_t
    lib.fa_combine.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i64p, i64p, vp]
    lib.fa_combine.restype = i32
    lib.fa_last_error.argtypes = []
    lib.fa_last_error.restype = ctypes.c_char_p
    lib.fa_device_status.argtypes = [i32, ctypes.POINTER(ctypes.c_uint)]
    lib.fa_device_status.restype = i32
    lib.fa_set_wait_timeout_ms.argtypes = [i32]
    lib.fa_set_wait_timeout_ms.restype = i32
    lib.fa_bwd_workspace_size.argtypes = [i32, i32, i32]
    lib.fa_bwd_workspace_size.restype = ctypes.c_size_t
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                           vp, vp, i32, i32, f32, i32, i32, i32, f32, vp, vp, ctypes.c_size_t, vp]
    lib.fa_bwd.restype = i32
    szt = ctypes.c_size_t
    rope = [vp, vp, i32, i32, f32, vp, vp, i32, i32, i32, vp]
    paging = [vp, i32, i32, i32, i32]
    lib.fa_qk_norm_rope.argtypes = [vp] * 4 + [i32] * 6 + [vp] * 4 + rope + [vp]
    lib.fa_qk_norm_rope.restype = i32
    lib.fa_qk_norm_rope_bwd_workspace_size.argtypes = [i32] * 3
    lib.fa_qk_norm_rope_bwd_workspace_size.restype = szt
    lib.fa_qk_norm_rope_bwd.argtypes = [vp] * 8 + [i32] * 6 + [vp] * 6 + rope + [vp, szt, vp]
    lib.fa_qk_norm_rope_bwd.restype = i32
    lib.fa_kvcache_append_quant.argtypes = [vp] * 6 + [i32] * 6 + [vp] * 3 + [vp] + paging + [vp, vp]
    lib.fa_kvcache_append_quant.restype = i32
    lib.fa_qk_norm_rope_append_quant.argtypes = ([vp] * 8 + [i32] * 7 + [vp] * 5 + rope + [vp] +
                                                 paging + [vp, vp])
    lib.fa_qk_norm_rope_append_quant.restype = i32
    lib.fa_kvcache_read_quant.argtypes = [vp] * 6 + [i32] * 6 + [vp, vp, vp] + paging + [vp]
    lib.fa_kvcache_read_quant.restype = i32
    lib.fa_kvcache_quant_workspace_size.argtypes = [i32] * 5
    lib.fa_kvcache_quant_workspace_size.restype = szt
    lib.fa_fwd_kvcache_quant.argtypes = ([vp] * 7 + [i32] * 7 + [vp] + paging +
                                         [vp, f32, i32, i32, i32, f32, vp, vp, szt, vp])
    lib.fa_fwd_kvcache_quant.restype = i32
    lib.fa_selftest_wait_timeout.argtypes = [i32, vp]
    lib.fa_selftest_wait_timeout.restype = i32
    lib.fa_version.argtypes = []
    lib.fa_version.restype = i32
    _lib = lib
    return lib


def _check(rc: int):
    if rc != 0:
        raise FAError(rc, load().fa_last_error().decode(errors="replace"))


def _ptr(t) -> ctypes.c_void_p | None:
    """Device address of a CUDA tensor (None stays NULL).  Host tensors, pinned ones
    included, are refused: every pointer of the C ABI is read by the kernels."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"tensor arguments must be CUDA tensors, got one on {t.device}")
    return ctypes.c_void_p(t.data_ptr())


def _i64(vals) -> ctypes.Array:
    return (ctypes.c_int64 * len(vals))(*[int(x) for x in vals])


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return ctypes.c_void_p(handle)


def _scale(softmax_scale) -> float:
    return float("nan") if softmax_scale is None else float(softmax_scale)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"inputs must be float16 or bfloat16, got {t.dtype}")
    return _DT[t.dtype]


def fa_version() -> int:
    return load().fa_version()


def fa_set_wait_timeout_ms(ms: int) -> None:
    _check(load().fa_set_wait_timeout_ms(int(ms)))


def fa_device_status(clear: bool = True) -> int:
    """Synchronise and return the device status bits (FA_DEV_*), clearing them."""
    flags = ctypes.c_uint(0)
    rc = load().fa_device_status(int(bool(clear)), ctypes.byref(flags))
    if rc not in (0, 5):
        _check(rc)
    return int(flags.value)


def fa_fwd(q, k, v, *, out=None, lse=None, cu_seqlens_q=None, cu_seqlens_k=None,
           max_seqlen_q=None, max_seqlen_k=None, softmax_scale=None, causal=False,
           window_size=(-1, -1), softcap=0.0, alibi_slopes=None, return_lse=True, stream=None,
           _fp8=None):
    """Exact attention forward (sections 3.1 / 3.2 of the interface page).

    Dense: q [B, Sq, H, d], k/v [B, Sk, Hkv, d] -> out like q, lse [B, H, Sq].
    Varlen: q [total_q, H, d], k/v [total_k, Hkv, d], int32 cu_seqlens [B+1],
    max_seqlen_q/k -> out like q, lse [H, total_q].
    """
    lib = load()
    fp8 = _fp8
    dt = _DT[torch.bfloat16] if fp8 is not None else _dtype(q)
    varlen = cu_seqlens_q is not None or cu_seqlens_k is not None
    if varlen:
        total_q, H, d = q.shape
        total_k, Hkv = k.shape[0], k.shape[1]
        B = cu_seqlens_q.numel() - 1
        sq, sk = total_q, total_k
        qs = (0, q.stride(0), q.stride(1))
        ks = (0, k.stride(0), k.stride(1))
        vs = (0, v.stride(0), v.stride(1))
        if max_seqlen_q is None or max_seqlen_k is None:
            raise ValueError("varlen needs max_seqlen_q and max_seqlen_k")
    else:
        B, sq, H, d = q.shape
        sk, Hkv = k.shape[1], k.shape[2]
        qs = (q.stride(0), q.stride(1), q.stride(2))
        ks = (k.stride(0), k.stride(1), k.stride(2))
        vs = (v.stride(0), v.stride(1), v.stride(2))
        max_seqlen_q = max_seqlen_k = 0
    for t in (q, k, v):
        if t.stride(-1) != 1:
            raise ValueError("the head_dim axis must be contiguous")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    os_ = (0, out.stride(0), out.stride(1)) if varlen else (out.stride(0), out.stride(1),
                                                            out.stride(2))
    if lse is None and return_lse:
        shape = (H, sq) if varlen else (B, H, sq)
        lse = torch.empty(shape, dtype=torch.float32, device=q.device)
    args = (_i64(qs), _i64(ks), _i64(vs), _i64(os_), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
            int(max_seqlen_q), int(max_seqlen_k), _scale(softmax_scale), int(bool(causal)),
            int(window_size[0]), int(window_size[1]), float(softcap), _ptr(alibi_slopes),
            _stream(stream))
    if fp8 is None:
        _check(lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), dt, B, sq, sk, H, Hkv,
                          d, *args))
    else:
        _check(lib.fa_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), *fp8, B, sq, sk,
                              H, Hkv, d, *args))
    return out, lse


def _host_ptr(t) -> ctypes.c_void_p | None:
    """Address of a contiguous CPU tensor (page-locked ones let the copies overlap)."""
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("fa_fwd_host takes contiguous CPU tensors")
    return ctypes.c_void_p(t.data_ptr())


def fa_fwd_host_workspace_size(batch, seqlen_q, seqlen_k, num_heads, num_heads_k, head_dim,
                               with_lse=True) -> int:
    return int(load().fa_fwd_host_workspace_size(batch, seqlen_q, seqlen_k, num_heads,
                                                 num_heads_k, head_dim, int(bool(with_lse))))


def fa_fwd_host(q, k, v, *, out=None, lse=None, softmax_scale=None, causal=False,
                window_size=(-1, -1), softcap=0.0, alibi_slopes=None, return_lse=True,
                workspace=None, stream=None):
    """fa_fwd on dense q [B, Sq, H, d], k/v [B, Sk, Hkv, d] in host memory; out (and lse
    [B, H, Sq], and alibi_slopes [H]) in host memory too.  The library copies the batch
    through a device workspace (on the current CUDA device) chunk by chunk, overlapping
    the copies with the kernels.  When `stream` (default: the current stream) has passed
    the call, out and lse hold the results."""
    lib = load()
    dt = _dtype(q)
    B, sq, H, d = q.shape
    sk, Hkv = k.shape[1], k.shape[2]
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if lse is None and return_lse:
        lse = torch.empty((B, H, sq), dtype=torch.float32, pin_memory=True)
    if workspace is None:
        n = fa_fwd_host_workspace_size(B, sq, sk, H, Hkv, d, lse is not None)
        workspace = torch.empty(max(n, 1), dtype=torch.uint8,
                                device=torch.device("cuda", torch.cuda.current_device()))
    if alibi_slopes is not None and (alibi_slopes.is_cuda or alibi_slopes.dtype != torch.float32):
        raise ValueError("fa_fwd_host takes fp32 CPU alibi_slopes")
    _check(lib.fa_fwd_host(_host_ptr(q), _host_ptr(k), _host_ptr(v), _host_ptr(out),
                           _host_ptr(lse), dt, B, sq, sk, H, Hkv, d, _scale(softmax_scale),
                           int(bool(causal)), int(window_size[0]), int(window_size[1]),
                           float(softcap), _host_ptr(alibi_slopes), _ptr(workspace),
                           workspace.numel(), _stream(stream)))
    return out, lse


def fa_fwd_fp8(q, k, v, *, q_descale=1.0, k_descale=1.0, v_descale=1.0, **kw):
    """fa_fwd on float8_e4m3fn q, k, v (head_dim 128) with per-tensor descale
    factors (the real inputs are q * q_descale etc.); out is bf16.  Other keywords
    as for fa_fwd."""
    for t in (q, k, v):
        if t.dtype != torch.float8_e4m3fn:
            raise TypeError("fa_fwd_fp8 takes float8_e4m3fn q, k, v")
    if kw.get("out") is None:
        kw["out"] = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    return fa_fwd(q, k, v, _fp8=(float(q_descale), float(k_descale), float(v_descale)), **kw)


def fa_kvcache_num_splits(batch, seqlen_q, num_heads, num_heads_k, head_dim, max_seqlen_k,
                          page_size=0, num_splits=0) -> int:
    return load().fa_kvcache_num_splits(batch, seqlen_q, num_heads, num_heads_k, head_dim,
                                        max_seqlen_k, page_size, num_splits)


def fa_kvcache_workspace_size(batch, seqlen_q, num_heads, num_heads_k, head_dim, max_seqlen_k,
                              page_size=0, num_splits=0) -> int:
    return int(load().fa_kvcache_workspace_size(batch, seqlen_q, num_heads, num_heads_k,
                                                head_dim, max_seqlen_k, page_size, num_splits))


def _cache_geometry(k_cache, block_table):
    if block_table is not None:
        return k_cache.shape[2], k_cache.shape[0], k_cache.shape[1], block_table.shape[1], 0
    return k_cache.shape[2], 0, 0, 0, k_cache.shape[1]   # Hkv, num_blocks, page, max_blocks, sk_max


def fa_kvcache_append(k_cache, v_cache, k, v, cache_seqlens, *, block_table=None, stream=None):
    """Write k, v [B, S_new, Hkv, d] into the cache at positions cache_seqlens[b] + t
    (cache_seqlens = keys already cached; it is not advanced here)."""
    lib = load()
    dt = _dtype(k)
    B, s_new, Hkv, d = k.shape
    for t in (k_cache, v_cache, k, v):
        if not t.is_contiguous():
            raise ValueError("the caches and the new keys/values must be contiguous")
    _, num_blocks, page, max_blocks, sk_max = _cache_geometry(k_cache, block_table)
    _check(lib.fa_kvcache_append(_ptr(k_cache), _ptr(v_cache), _ptr(k), _ptr(v), dt, B, s_new,
                                 Hkv, d, _ptr(block_table), max_blocks, page, num_blocks, sk_max,
                                 _ptr(cache_seqlens), _stream(stream)))


def fa_fwd_kvcache(q, k_cache, v_cache, k=None, v=None, *, cache_seqlens=None, block_table=None,
                   softmax_scale=None, causal=False, window_size=(-1, -1), softcap=0.0,
                   alibi_slopes=None, num_splits=0, out=None, lse=None, return_lse=True,
                   workspace=None, stream=None):
    """Split-KV attention against a paged or contiguous KV cache (section 3.3).
    q [B, Sq, H, d]; paged pools [num_blocks, page, Hkv, d] with int32 block_table
    [B, max_blocks]; or contiguous caches [B, Sk_max, Hkv, d].  With k and v
    [B, S_new, Hkv, d] given, they are first written into the cache after the
    cache_seqlens[b] keys already there, and the attention covers
    cache_seqlens[b] + S_new keys (cache_seqlens itself is not advanced)."""
    lib = load()
    dt = _dtype(q)
    B, sq, H, d = q.shape
    for t in (q, k_cache, v_cache):
        if not t.is_contiguous():
            raise ValueError("q and the caches must be contiguous")
    if (k is None) != (v is None):
        raise ValueError("give both k and v, or neither")
    if k is not None and not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k and v must be contiguous")
    if block_table is not None:
        num_blocks, page, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
        max_blocks = block_table.shape[1]
        sk_max = 0
        max_k = max_blocks * page
    else:
        num_blocks, page, max_blocks = 0, 0, 0
        sk_max, Hkv = k_cache.shape[1], k_cache.shape[2]
        max_k = sk_max
    need = fa_kvcache_workspace_size(B, sq, H, Hkv, d, max_k, page, num_splits)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, sq), dtype=torch.float32, device=q.device)
    if k is None:
        _check(lib.fa_fwd_kvcache(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse),
                                  dt, B, sq, H, Hkv, d, _ptr(block_table), max_blocks, page,
                                  num_blocks, sk_max, _ptr(cache_seqlens), _scale(softmax_scale),
                                  int(bool(causal)), int(window_size[0]), int(window_size[1]),
                                  float(softcap), _ptr(alibi_slopes), int(num_splits),
                                  _ptr(workspace), ws_bytes, _stream(stream)))
    else:
        _check(lib.fa_fwd_kvcache_append(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k), _ptr(v),
                                         k.shape[1], _ptr(out), _ptr(lse), dt, B, sq, H, Hkv, d,
                                         _ptr(block_table), max_blocks, page, num_blocks, sk_max,
                                         _ptr(cache_seqlens), _scale(softmax_scale),
                                         int(bool(causal)), int(window_size[0]),
                                         int(window_size[1]), float(softcap),
                                         _ptr(alibi_slopes), int(num_splits), _ptr(workspace),
                                         ws_bytes, _stream(stream)))
    return out, lse


def fa_fwd_kvcache_static(q, k_cache, v_cache, *, cache_seqlens=None, block_table=None,
                          softmax_scale=None, causal=False, window_size=(-1, -1), softcap=0.0,
                          alibi_slopes=None, num_splits=0, out=None, lse=None,
                          return_lse=True, stream=None):
    """fa_fwd_kvcache for callers that cannot allocate device memory at the call:
    the scratch comes from the library's fixed device array (see include/fa.h).
    Outputs not passed in are allocated here by torch, before the call."""
    lib = load()
    dt = _dtype(q)
    B, sq, H, d = q.shape
    for t in (q, k_cache, v_cache):
        if not t.is_contiguous():
            raise ValueError("q and the caches must be contiguous")
    if block_table is not None:
        num_blocks, page, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
        max_blocks, sk_max = block_table.shape[1], 0
    else:
        num_blocks, page, max_blocks = 0, 0, 0
        sk_max, Hkv = k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, sq), dtype=torch.float32, device=q.device)
    _check(lib.fa_fwd_kvcache_static(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(lse),
                                     dt, B, sq, H, Hkv, d, _ptr(block_table), max_blocks, page,
                                     num_blocks, sk_max, _ptr(cache_seqlens),
                                     _scale(softmax_scale), int(bool(causal)),
                                     int(window_size[0]), int(window_size[1]), float(softcap),
                                     _ptr(alibi_slopes), int(num_splits), _stream(stream)))
    return out, lse


def fa_combine(out_partial, lse_partial, *, out_dtype=torch.float32, out=None, lse=None,
               return_lse=True, stream=None):
    """LSE-weighted combine (section 3.4): out_partial [B, S, H, d, splits] and
    lse_partial [B, S, H, splits] (any strides) -> out [B, S, H, d], lse [B, H, S]."""
    lib = load()
    B, S, H, d, splits = out_partial.shape
    if out is None:
        out = torch.empty((B, S, H, d), dtype=out_dtype, device=out_partial.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=out_partial.device)
    if out_partial.dtype != torch.float32 or lse_partial.dtype != torch.float32:
        raise TypeError("partials must be float32")
    _check(lib.fa_combine(_ptr(out_partial), _ptr(lse_partial), _ptr(out), _ptr(lse),
                          _DT[out.dtype], B, S, H, d, splits, _i64(out_partial.stride()),
                          _i64(lse_partial.stride()), _stream(stream)))
    return out, lse


def fa_selftest_wait_timeout(timeout_ms=20, stream=None):
    """Launch the bounded-wait self-test (include/fa.h): after timeout_ms the waiting
    CTA raises FA_DEV_WAIT_TIMEOUT in the device status word and exits."""
    _check(load().fa_selftest_wait_timeout(int(timeout_ms), _stream(stream)))


def fa_bwd(dout, q, k, v, out, lse, *, cu_seqlens_q=None, cu_seqlens_k=None,
           max_seqlen_q=None, max_seqlen_k=None, softmax_scale=None, causal=False,
           window_size=(-1, -1), softcap=0.0, alibi_slopes=None, dq=None, dk=None, dv=None,
           workspace=None, stream=None):
    """Gradients (dq, dk, dv) of the forward for output gradient dout (same mask,
    scale, softcap and ALiBi arguments as the forward call).
    Dense: q, out, dout [B, Sq, H, d], k, v [B, Sk, Hkv, d] contiguous, lse [B, H, Sq].
    Varlen: q, out, dout [total_q, H, d], k, v [total_k, Hkv, d], int32 cu_seqlens
    [B+1], max_seqlen_q/k, lse [H, total_q] (fa_fwd's varlen outputs)."""
    lib = load()
    dt = _dtype(q)
    varlen = cu_seqlens_q is not None or cu_seqlens_k is not None
    if varlen:
        if cu_seqlens_q is None or cu_seqlens_k is None:
            raise ValueError("varlen needs cu_seqlens_q and cu_seqlens_k")
        if max_seqlen_q is None or max_seqlen_k is None:
            raise ValueError("varlen needs max_seqlen_q and max_seqlen_k")
        B = cu_seqlens_q.numel() - 1
        sq, H, d = q.shape
        sk, Hkv = k.shape[0], k.shape[1]
        ws_b = 1
    else:
        B, sq, H, d = q.shape
        sk, Hkv = k.shape[1], k.shape[2]
        max_seqlen_q = max_seqlen_k = 0
        ws_b = B
    for t in (dout, q, k, v, out, lse):
        if not t.is_contiguous():
            raise ValueError("fa_bwd takes contiguous tensors")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = lib.fa_bwd_workspace_size(ws_b, sq, H)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.fa_bwd(_ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dq),
                      _ptr(dk), _ptr(dv), dt, B, sq, sk, H, Hkv, d, _ptr(cu_seqlens_q),
                      _ptr(cu_seqlens_k), int(max_seqlen_q), int(max_seqlen_k),
                      _scale(softmax_scale), int(bool(causal)), int(window_size[0]),
                      int(window_size[1]), float(softcap), _ptr(alibi_slopes), _ptr(workspace),
                      ws_bytes, _stream(stream)))
    return dq, dk, dv


# ------------------------------------------------------------------ arguments of the calls below
# A decoding step calls these many times for a few microseconds of GPU work each, so the checks
# read each property once and hand plain integers to ctypes.
_STRIDES = {}  # (a, b, c) -> the address of an int64[3] holding them


class _Address(int):
    """The address of an array, which lives as long as this number."""


def _s3(a, b, c) -> int:
    """Address of an int64[3] holding (a, b, c), for as long as the caller keeps it; equal triples
    share one."""
    at = _STRIDES.get((a, b, c))
    if at is None:
        if len(_STRIDES) >= 16384:
            _STRIDES.clear()
        array = (ctypes.c_int64 * 3)(a, b, c)
        at = _STRIDES[(a, b, c)] = _Address(ctypes.addressof(array))
        at.array = array
    return at


def _like(t):
    """A new contiguous tensor of t's shape, dtype and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _device_of(t) -> int:
    i = t.get_device()
    if i < 0:
        raise ValueError(f"tensor arguments must be CUDA tensors, got one on {t.device}")
    return i


def _want(name, t, shape, dtype, dev):
    """Checks a contiguous tensor; returns its address (0, NULL, for None)."""
    if t is None:
        return 0
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call's first tensor on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(name, t, dtype, dev):
    """A [B, S, heads, d] or [T, heads, d] (one packed batch) tensor of any row strides, checked:
    its four sizes and the address of its (batch, seq, head) strides.  The strides of axes of
    one entry, which are never stepped along, are given as the contiguous ones."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call's first tensor on cuda:{dev}")
    shape, st = t.shape, t.stride()
    if len(shape) == 3:
        S, H, d = shape
        B, sb = 1, 0
        ss, sh, se = st
    elif len(shape) == 4:
        B, S, H, d = shape
        sb, ss, sh, se = st
    else:
        raise ValueError(f"{name} must be [B, S, heads, d] or [T, heads, d], got {tuple(shape)}")
    if se != 1:
        raise ValueError(f"{name}: the head_dim axis must be contiguous")
    return (B, S, H, d), _s3(sb if B > 1 else S * H * d, ss if S > 1 else H * d, sh if H > 1 else d)


def _positions(t, q, B, S, dev):
    return 0 if t is None else _want("positions", t, (S,) if q.dim() == 3 else (B, S), torch.int32, dev)


def _is_packed(name, t, cu_seqlens_new):
    if t.dim() != (4 if cu_seqlens_new is None else 3):
        raise ValueError(f"{name}: new rows are [B, S_new, heads, d], or packed [total, heads, d] "
                         "with cu_seqlens_new")


def _size(fn, dev, *args) -> int:
    """The bytes fn(*args) that a call on the tensors' device needs (they go by its SMs)."""
    if torch.cuda.current_device() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _launch(fn, dev, *args):
    """Calls fn(*args, stream) for the current stream of the tensors' device, with that device
    current (the C ABI launches there)."""
    if torch.cuda.current_device() == dev:
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(dev)))
        return
    with torch.cuda.device(dev):
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(dev)))


def _handle(stream) -> int:
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _int32(n) -> int:
    """n within 32 bits (ctypes would cut a larger one down to its low bits)."""
    return min(max(n, -0x80000000), 0x7fffffff)


def _on(fn, args):
    """fn(**args) on args["stream"], another stream than the current one perhaps.  What the call
    allocates has to be that stream's (memory freed on the current stream may still be in use
    there); its arguments and what it returns are freed for work of both."""
    stream = args.pop("stream")
    first = next((t for t in args.values() if torch.is_tensor(t)), None)
    if first is None or not first.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors")
    dev, handle = first.device, _handle(stream)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the call's first tensor on {dev}")
    current = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        result = fn(**args)
    if handle != current.cuda_stream:
        for t in args.values():
            if torch.is_tensor(t):
                t.record_stream(stream)
        for t in result if isinstance(result, tuple) else (result,):
            if t is not None:
                t.record_stream(current)
    return result


def _workspace(w, nbytes, device, dev):
    """The caller's workspace, checked, or one of this call alone (it goes back to the allocator
    when the call returns, for work behind the call's own)."""
    if w is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if w.get_device() != dev or not w.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}, got one on {w.device}")
    return w


# ------------------------------------------------------------------ q/k norm and rotation
def _rope_args(d, dtype, dev, q_weight, k_weight, eps, norm, cos, sin, interleaved):
    """The C arguments from q_weight to interleaved."""
    wdt = torch.float32
    pq = pk = 0
    if q_weight is not None:
        wdt = q_weight.dtype
        pq = _want("q_weight", q_weight, (d,), wdt, dev)
    if k_weight is not None:
        if q_weight is None:
            wdt = k_weight.dtype
        pk = _want("k_weight", k_weight, (d,), wdt, dev)
    if wdt is not torch.float32 and wdt is not dtype:
        raise TypeError(f"the norm weights must be float32 or {dtype}, got {wdt}")
    rot = rows = pc = ps = 0
    if cos is not None and sin is not None:
        shape = cos.shape
        if len(shape) != 2:
            raise ValueError("cos and sin must be [max_positions, rotary_dim / 2]")
        pc = _want("cos", cos, shape, torch.float32, dev)
        ps = _want("sin", sin, shape, torch.float32, dev)
        rows, rot = shape[0], 2 * shape[1]
    elif cos is not None or sin is not None:
        raise ValueError("give both cos and sin, or neither")
    return pq, pk, _DT[wdt], 1 if norm else 0, eps, pc, ps, rot, rows, 1 if interleaved else 0


def fa_qk_norm_rope(q, k, *, q_weight=None, k_weight=None, eps=1e-6, norm=True, cos=None, sin=None,
                    positions=None, interleaved=False, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [B, S, H, d] and k [B, S, Hkv, d] (or packed [T, heads, d])
    and the rotation of their first 2 * cos.shape[1] elements, in one pass (include/fa.h).
    cos, sin: fp32 [max_positions, rotary_dim / 2]; positions int32 [B, S] (or [T]; None:
    the index along S).  q and k may be strided views; the outputs are allocated contiguous
    unless given, and may be q and k themselves.  Returns (q_out, k_out)."""
    if stream is not None:
        return _on(fa_qk_norm_rope, locals())
    lib = load()
    dt, dtype, dev = _dtype(q), q.dtype, _device_of(q)
    qs, sq = _rows("q", q, dtype, dev)
    ks, sk = _rows("k", k, dtype, dev)
    qos, sqo, kos, sko = qs, 0, ks, 0  # strides 0 (NULL): contiguous
    if q_out is None:
        q_out = _like(q)
    else:
        qos, sqo = _rows("q_out", q_out, dtype, dev)
    if k_out is None:
        k_out = _like(k)
    else:
        kos, sko = _rows("k_out", k_out, dtype, dev)
    B, S, H, d = qs
    if ks[0] != B or ks[1] != S or ks[3] != d or qos != qs or kos != ks:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and their outputs {tuple(q_out.shape)}, "
                         f"{tuple(k_out.shape)} do not fit together")
    _launch(lib.fa_qk_norm_rope, dev, q.data_ptr(), k.data_ptr(), q_out.data_ptr(),
            k_out.data_ptr(), dt, B, S, H, ks[2], d, sq, sk, sqo, sko,
            *_rope_args(d, dtype, dev, q_weight, k_weight, eps, norm, cos, sin, interleaved),
            _positions(positions, q, B, S, dev))
    return q_out, k_out


def fa_qk_norm_rope_bwd(dq_out, dk_out, q, k, *, q_weight=None, k_weight=None, eps=1e-6, norm=True,
                        cos=None, sin=None, positions=None, interleaved=False, dq=None, dk=None,
                        workspace=None, stream=None):
    """Gradients of fa_qk_norm_rope for output gradients dq_out, dk_out; q and k are its
    inputs and the keywords those of the forward call.  Returns (dq, dk, dq_weight,
    dk_weight), the weight gradients fp32 [d] (None for a weight that was None)."""
    if stream is not None:
        return _on(fa_qk_norm_rope_bwd, locals())
    lib = load()
    dt, dtype, dev = _dtype(q), q.dtype, _device_of(q)
    qs, sq = _rows("q", q, dtype, dev)
    ks, sk = _rows("k", k, dtype, dev)
    dqs, sdq, dks, sdk = qs, 0, ks, 0  # strides 0 (NULL): contiguous
    if dq is None:
        dq = _like(q)
    else:
        dqs, sdq = _rows("dq", dq, dtype, dev)
    if dk is None:
        dk = _like(k)
    else:
        dks, sdk = _rows("dk", dk, dtype, dev)
    B, S, H, d = qs
    strides = []
    for name, t, like in (("dq_out", dq_out, qs), ("dk_out", dk_out, ks)):
        shape, st = _rows(name, t, dtype, dev)
        if shape != like:
            raise ValueError(f"{name} must have its input's shape, got {tuple(t.shape)}")
        strides.append(st)
    if ks[0] != B or ks[1] != S or ks[3] != d or dqs != qs or dks != ks:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and their gradients {tuple(dq.shape)}, "
                         f"{tuple(dk.shape)} do not fit together")
    dwq = None if q_weight is None else torch.empty(d, dtype=torch.float32, device=q.device)
    dwk = None if k_weight is None else torch.empty(d, dtype=torch.float32, device=q.device)
    args = _rope_args(d, dtype, dev, q_weight, k_weight, eps, norm, cos, sin, interleaved)
    workspace = _workspace(workspace, _size(lib.fa_qk_norm_rope_bwd_workspace_size, dev, B, S, d), q.device, dev)
    _launch(lib.fa_qk_norm_rope_bwd, dev, dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(),
            k.data_ptr(), dq.data_ptr(), dk.data_ptr(), 0 if dwq is None else dwq.data_ptr(),
            0 if dwk is None else dwk.data_ptr(), dt, B, S, H, ks[2], d, *strides, sq, sk, sdq, sdk,
            *args, _positions(positions, q, B, S, dev),
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dq, dk, dwq, dwk


# ------------------------------------------------------------------ the 8-bit KV cache
def _quant_cache(k_cache, v_cache, k_scale, v_scale, block_table, batch, dev):
    """Checks the cache tensors; returns (pointers, format, Hkv, d, strides, paging)."""
    dtype, shape = k_cache.dtype, k_cache.shape
    fmt = _KV_FORMAT.get(dtype)
    if fmt is None:
        raise TypeError(f"an 8-bit cache is float8_e4m3fn or int8, got {dtype}")
    if len(shape) != 4:
        raise ValueError("a cache is [num_blocks, page, Hkv, d] or [B, Sk_max, Hkv, d]")
    n, rows, Hkv, d = shape
    sb, sr, sh, se = st = k_cache.stride()
    if v_cache.shape != shape or v_cache.dtype is not dtype:
        raise ValueError(f"v_cache must be like k_cache, {tuple(shape)} {dtype}, got "
                         f"{tuple(v_cache.shape)} {v_cache.dtype}")
    if se != 1 or v_cache.stride() != st:
        raise ValueError("the caches need a contiguous head_dim axis and the same strides")
    if k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise ValueError(f"the caches are on {k_cache.device} and {v_cache.device}, the call's first "
                         f"tensor on cuda:{dev}")
    scales = (n, Hkv, rows)
    ptrs = (k_cache.data_ptr(), v_cache.data_ptr(), _want("k_scale", k_scale, scales, torch.float32, dev),
            _want("v_scale", v_scale, scales, torch.float32, dev))
    if 0 in ptrs and k_cache.numel() > 0:
        raise ValueError("k_scale and v_scale are needed")
    strides = _s3(sb if n > 1 else max(1, rows) * Hkv * d, sr if rows > 1 else Hkv * d,
                  sh if Hkv > 1 else d)
    if block_table is not None:
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_blocks]")
        width = block_table.shape[1]
        paging = (_want("block_table", block_table, (batch, width), torch.int32, dev), width, rows, n, 0)
    else:
        if n != batch:
            raise ValueError(f"a contiguous cache of {n} sequences for a batch of {batch}")
        paging = (0, 0, 0, 0, rows)
    return ptrs, fmt, Hkv, d, strides, paging


def fa_kvcache_append_quant(k_cache, v_cache, k_scale, v_scale, k, v, cache_seqlens, *, block_table=None,
                            cu_seqlens_new=None, stream=None):
    """Quantise k, v [B, S_new, Hkv, d] (packed [total, Hkv, d] with int32 cu_seqlens_new [B + 1])
    and write them into the 8-bit cache after each sequence's cache_seqlens[b] rows (not advanced
    here).  Caches: float8_e4m3fn or int8 [num_blocks, page, Hkv, d] with block_table, or
    [B, Sk_max, Hkv, d], any strides of whole 16 bytes; scales fp32 [num_blocks, Hkv, page] or
    [B, Hkv, Sk_max].  See include/fa.h."""
    if stream is not None:
        return _on(fa_kvcache_append_quant, locals())
    lib = load()
    dt, dtype, dev = _dtype(k), k.dtype, _device_of(k)
    B = cache_seqlens.numel()
    ptrs, fmt, Hkv, d, cst, paging = _quant_cache(k_cache, v_cache, k_scale, v_scale, block_table, B, dev)
    _is_packed("k", k, cu_seqlens_new)
    ks, sk = _rows("k", k, dtype, dev)
    vs, sv = _rows("v", v, dtype, dev)
    if ks != (1 if cu_seqlens_new is not None else B, ks[1], Hkv, d) or vs != ks or v.shape != k.shape:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} do not fit the cache {tuple(k_cache.shape)} "
                         f"and a batch of {B}")
    _launch(lib.fa_kvcache_append_quant, dev, *ptrs, k.data_ptr(), v.data_ptr(), dt, fmt, B, ks[1],
            Hkv, d, sk, sv, cst, _want("cu_seqlens_new", cu_seqlens_new, (B + 1,), torch.int32, dev),
            *paging, _want("cache_seqlens", cache_seqlens, (B,), torch.int32, dev))


def fa_qk_norm_rope_append_quant(q, k, v, k_cache, v_cache, k_scale, v_scale, cache_seqlens, *,
                                 q_weight=None, k_weight=None, eps=1e-6, norm=True, cos=None, sin=None,
                                 positions=None, interleaved=False, block_table=None,
                                 cu_seqlens_new=None, q_out=None, stream=None):
    """fa_qk_norm_rope on q and k, then fa_kvcache_append_quant of that k and of v, in one launch
    and with the same results.  positions None: the rows' places in the cache.  Returns q_out."""
    if stream is not None:
        return _on(fa_qk_norm_rope_append_quant, locals())
    lib = load()
    dt, dtype, dev = _dtype(q), q.dtype, _device_of(q)
    B = cache_seqlens.numel()
    ptrs, fmt, Hkv, d, cst, paging = _quant_cache(k_cache, v_cache, k_scale, v_scale, block_table, B, dev)
    _is_packed("q", q, cu_seqlens_new)
    qs, sq = _rows("q", q, dtype, dev)
    ks, sk = _rows("k", k, dtype, dev)
    vs, sv = _rows("v", v, dtype, dev)
    qos, sqo = qs, 0  # strides 0 (NULL): contiguous
    if q_out is None:
        q_out = _like(q)
    else:
        qos, sqo = _rows("q_out", q_out, dtype, dev)
    S, H = qs[1], qs[2]
    nb = 1 if cu_seqlens_new is not None else B
    if (qs != (nb, S, H, d) or ks != (nb, S, Hkv, d) or vs != ks or qos != qs or k.dim() != q.dim()
            or v.dim() != q.dim()):
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)} and q_out "
                         f"{tuple(q_out.shape)} do not fit the cache {tuple(k_cache.shape)} and a batch of {B}")
    _launch(lib.fa_qk_norm_rope_append_quant, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            q_out.data_ptr(), *ptrs, dt, fmt, B, S, H, Hkv, d, sq, sk, sv, sqo, cst,
            *_rope_args(d, dtype, dev, q_weight, k_weight, eps, norm, cos, sin, interleaved),
            _positions(positions, q, B, S, dev),
            _want("cu_seqlens_new", cu_seqlens_new, (B + 1,), torch.int32, dev), *paging,
            _want("cache_seqlens", cache_seqlens, (B,), torch.int32, dev))
    return q_out


def fa_kvcache_read_quant(k_cache, v_cache, k_scale, v_scale, cu_seqlens, *, dtype=torch.bfloat16, total=None,
                          seq_start=None, block_table=None, k_out=None, v_out=None, stream=None):
    """Rows seq_start[b] .. of every sequence (None: from its first) as packed 16-bit k, v
    [total, Hkv, d], sequence b's at cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32).  total:
    the packed row count, needed when k_out and v_out are not given."""
    if stream is not None:
        return _on(fa_kvcache_read_quant, locals())
    lib = load()
    dev = _device_of(k_cache)
    B = cu_seqlens.numel() - 1
    ptrs, fmt, Hkv, d, cst, paging = _quant_cache(k_cache, v_cache, k_scale, v_scale, block_table, B, dev)
    if k_out is None and v_out is None:
        if total is None:
            raise ValueError("fa_kvcache_read_quant needs total, or k_out and v_out")
        k_out = torch.empty((total, Hkv, d), dtype=dtype, device=k_cache.device)
        v_out = torch.empty((total, Hkv, d), dtype=dtype, device=k_cache.device)
    elif k_out is None or v_out is None:
        raise ValueError("give both k_out and v_out, or neither")
    n = k_out.shape[0]
    if total is not None and total != n:
        raise ValueError(f"total is {total}, k_out has {n} rows")
    dt = _dtype(k_out)
    shape = (n, Hkv, d)
    _launch(lib.fa_kvcache_read_quant, dev, *ptrs, _want("k_out", k_out, shape, k_out.dtype, dev),
            _want("v_out", v_out, shape, k_out.dtype, dev), dt, fmt, B, n, Hkv, d, cst,
            _want("cu_seqlens", cu_seqlens, (B + 1,), torch.int32, dev),
            _want("seq_start", seq_start, (B,), torch.int32, dev), *paging)
    return k_out, v_out


def fa_kvcache_quant_workspace_size(batch, seqlen_q, num_heads, num_heads_k, head_dim) -> int:
    return int(load().fa_kvcache_quant_workspace_size(batch, seqlen_q, num_heads, num_heads_k, head_dim))


def fa_fwd_kvcache_quant(q, k_cache, v_cache, k_scale, v_scale, *, cache_seqlens=None, block_table=None,
                         softmax_scale=None, causal=False, window_size=(-1, -1), softcap=0.0,
                         alibi_slopes=None, out=None, lse=None, return_lse=True, workspace=None,
                         stream=None):
    """fa_fwd_kvcache over an 8-bit cache (fa_kvcache_append_quant): q [B, Sq, H, d] attends the
    values that the first cache_seqlens[b] rows stand for.  Returns (out, lse [B, H, Sq])."""
    if stream is not None:
        return _on(fa_fwd_kvcache_quant, locals())
    lib = load()
    dt, dtype, dev = _dtype(q), q.dtype, _device_of(q)
    shape = q.shape
    B, sq, H, d = shape
    ptrs, fmt, Hkv, cd, cst, paging = _quant_cache(k_cache, v_cache, k_scale, v_scale, block_table, B, dev)
    if cd != d:
        raise ValueError(f"q has head_dim {d}, the cache {cd}")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if out is None:
        out = _like(q)
    if lse is None and return_lse:
        lse = q.new_empty((B, H, sq), dtype=torch.float32)
    workspace = _workspace(workspace, _size(lib.fa_kvcache_quant_workspace_size, dev, B, sq, H, Hkv, d), q.device, dev)
    _launch(lib.fa_fwd_kvcache_quant, dev, q.data_ptr(), *ptrs, _want("out", out, shape, dtype, dev),
            _want("lse", lse, (B, H, sq), torch.float32, dev), dt, fmt, B, sq, H, Hkv, d, cst, *paging,
            _want("cache_seqlens", cache_seqlens, (B,), torch.int32, dev),
            math.nan if softmax_scale is None else softmax_scale, 1 if causal else 0, _int32(window_size[0]),
            _int32(window_size[1]), softcap, _want("alibi_slopes", alibi_slopes, (H,), torch.float32, dev),
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out, lse
