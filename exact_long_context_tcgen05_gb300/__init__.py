"""Exact long-context attention forward on one GB300 (sm_103a): thin Python binding of libcqsa_gb300.

The functions below carry the C ABI's names (``include/cqsa.h``) and only marshal arguments:
torch tensors or integer addresses become pointers, the current torch CUDA stream becomes the
``cudaStream_t``, and a non-OK status raises :class:`CqsaError` with the library's message. Every
step of the computation runs in the library's CUDA kernels. If the compiled library is missing the
import of the binding fails loudly (there is no fallback of any kind).
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libcqsa_gb300.so")

CQSA_OK, CQSA_ERR_INVALID, CQSA_ERR_UNSUPPORTED, CQSA_ERR_CUDA, CQSA_ERR_OOM, CQSA_ERR_TIMEOUT, CQSA_ERR_DEVICE = (
    0, -1, -2, -3, -4, -5, -6)
CQSA_F16, CQSA_BF16, CQSA_F32, CQSA_E4M3 = 0, 1, 2, 3
CQSA_LAYOUT_BHND, CQSA_LAYOUT_BNHD = 0, 1
CQSA_ENGINE_CLASSIC, CQSA_ENGINE_WAVE = 0, 1

EXPORTED = ("cqsa_attn_fwd", "cqsa_attn_fwd_chunk", "cqsa_merge_partials", "cqsa_stream_attn_fwd",
            "cqsa_attn_fwd_chunked_static", "cqsa_quorum_check", "cqsa_quorum_schedule", "cqsa_quorum_attn_fwd",
            "cqsa_quorum_attn_fwd_ex", "cqsa_release_cache", "cqsa_attn_bwd_workspace_size", "cqsa_attn_bwd", "cqsa_attn_bwd_dvec",
            "cqsa_attn_bwd_chunk", "cqsa_attn_bwd_cast", "cqsa_stream_attn_bwd", "cqsa_stream_attn_bwd_ex",
            "cqsa_status_string", "cqsa_last_error", "cqsa_device_error", "cqsa_set_timeout_ms",
            "cqsa_debug_set_fault", "cqsa_version", "cqsa_set_stream_kv_resident_bytes", "cqsa_attn_packed_fwd",
            "cqsa_attn_packed_bwd_workspace_size", "cqsa_attn_packed_bwd", "cqsa_kv_cache_write",
            "cqsa_kv_cache_read", "cqsa_attn_paged_workspace_size", "cqsa_attn_paged_fwd")
CQSA_STATIC_SCRATCH_BYTES = 32 << 20


class CqsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_name(status)}: {message}")
        self.status = status


class cqsa_stream_stats(ctypes.Structure):
    _fields_ = [("wall_ms", ctypes.c_double), ("compute_ms", ctypes.c_double), ("h2d_ms", ctypes.c_double),
                ("stall_ms", ctypes.c_double), ("h2d_bytes", ctypes.c_longlong), ("d2h_bytes", ctypes.c_longlong),
                ("peak_device_bytes", ctypes.c_longlong), ("n_chunks", ctypes.c_int), ("n_launches", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class cqsa_quorum_stats(ctypes.Structure):
    _fields_ = [("wall_ms", ctypes.c_double), ("compute_ms", ctypes.c_double), ("copy_ms", ctypes.c_double),
                ("copy_bytes", ctypes.c_longlong), ("peak_device_bytes", ctypes.c_longlong),
                ("chunk_tokens", ctypes.c_longlong), ("acc_host_bytes", ctypes.c_longlong),
                ("n_subproblems", ctypes.c_int), ("n_pairs", ctypes.c_int),
                ("n_chunk_loads", ctypes.c_int), ("n_launches", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


_vp, _i, _ll, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libcqsa_gb300.so is not built ({LIB_PATH}); run "
                          "`python -m exact_long_context_tcgen05_gb300.build` (needs nvcc)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.cqsa_attn_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp]
    lib.cqsa_attn_fwd_chunk.argtypes = [_vp, _vp, _vp, _ll, _ll, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _i, _vp]
    lib.cqsa_merge_partials.argtypes = [_vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _vp]
    lib.cqsa_stream_attn_fwd.argtypes = [_vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _ll, _i, _i, _f, _i, _ll,
                                         ctypes.POINTER(cqsa_stream_stats), _vp]
    lib.cqsa_attn_fwd_chunked_static.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _vp]
    lib.cqsa_quorum_check.argtypes = [_i, _vp, _i]
    lib.cqsa_quorum_schedule.argtypes = [_i, _vp, _i, _i, _i, _i, _vp, _ll]
    lib.cqsa_quorum_schedule.restype = _ll
    lib.cqsa_quorum_attn_fwd.argtypes = [_vp, _vp, _vp, _i, _i, _vp, _vp, _i, _i, _i, _ll, _i, _i, _f, _i, _i, _vp,
                                         _i, _i, _i, _i, ctypes.POINTER(cqsa_quorum_stats), _vp]
    lib.cqsa_quorum_attn_fwd_ex.argtypes = [_vp, _vp, _vp, _i, _i, _vp, _vp, _i, _i, _i, _ll, _i, _i, _f, _i, _i,
                                            _vp, _i, _i, _i, _i, _i, _ll, ctypes.POINTER(cqsa_quorum_stats), _vp]
    lib.cqsa_attn_bwd_workspace_size.argtypes = [_i, _i, _i, _i]
    lib.cqsa_attn_bwd_workspace_size.restype = ctypes.c_size_t
    lib.cqsa_attn_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _i, _i, _i, _i,
                                  _i, _f, _i, _vp]
    lib.cqsa_attn_bwd_dvec.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]
    lib.cqsa_attn_bwd_chunk.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _ll, _ll, _i, _i, _i, _i, _i, _i, _f, _i, _vp,
                                        _vp, _vp, _vp]
    lib.cqsa_attn_bwd_cast.argtypes = [_vp, _vp, _ll, _i, _vp]
    lib.cqsa_stream_attn_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _ll, _i, _i, _f, _i,
                                         _ll, _vp]
    lib.cqsa_stream_attn_bwd_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _ll, _i, _i, _f, _i,
                                            _ll, ctypes.POINTER(cqsa_stream_stats), _vp]
    lib.cqsa_set_stream_kv_resident_bytes.argtypes = [_ll]
    lib.cqsa_set_stream_kv_resident_bytes.restype = None
    lib.cqsa_attn_packed_fwd.argtypes = [_vp, _vp, _vp, _ll, _ll, _ll, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp]
    lib.cqsa_attn_packed_bwd_workspace_size.argtypes = [_i] * 5
    lib.cqsa_attn_packed_bwd_workspace_size.restype = ctypes.c_size_t
    lib.cqsa_attn_packed_bwd.argtypes = [_vp, _vp, _vp, _ll, _ll, _ll, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                         _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp]
    lib.cqsa_kv_cache_write.argtypes = [_vp, _vp, _ll, _ll, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i,
                                        _i, _i, _i, _vp]
    lib.cqsa_kv_cache_read.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                                       _vp]
    lib.cqsa_attn_paged_workspace_size.argtypes = [_i] * 10
    lib.cqsa_attn_paged_workspace_size.restype = ctypes.c_size_t
    lib.cqsa_attn_paged_fwd.argtypes = [_vp, _ll, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i,
                                        _i, _i, _i, _i, _i, _f, _i, _i, _vp, ctypes.c_size_t, _vp]
    lib.cqsa_release_cache.argtypes = []
    lib.cqsa_release_cache.restype = _i
    lib.cqsa_status_string.argtypes = [_i]
    lib.cqsa_status_string.restype = ctypes.c_char_p
    lib.cqsa_last_error.argtypes = []
    lib.cqsa_last_error.restype = ctypes.c_char_p
    lib.cqsa_device_error.argtypes = [ctypes.POINTER(_i), ctypes.POINTER(_i), _i]
    lib.cqsa_set_timeout_ms.argtypes = [ctypes.c_uint]
    lib.cqsa_set_timeout_ms.restype = None
    lib.cqsa_debug_set_fault.argtypes = [_i]
    lib.cqsa_debug_set_fault.restype = _i
    lib.cqsa_version.argtypes = []
    lib.cqsa_version.restype = ctypes.c_char_p
    for name in ("cqsa_attn_fwd", "cqsa_attn_fwd_chunk", "cqsa_merge_partials", "cqsa_stream_attn_fwd",
                 "cqsa_attn_fwd_chunked_static", "cqsa_device_error", "cqsa_quorum_check", "cqsa_quorum_attn_fwd",
                 "cqsa_quorum_attn_fwd_ex"):
        getattr(lib, name).restype = _i
    return lib


lib = _load()


def status_name(status: int) -> str:
    return lib.cqsa_status_string(status).decode()


def last_error() -> str:
    return lib.cqsa_last_error().decode()


def _check(rc: int) -> int:
    if rc != CQSA_OK:
        raise CqsaError(rc, last_error())
    return rc


def _ptr(x) -> int | None:
    """Address of a torch tensor / numpy array / int (None and 0 stay NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x or None
    if hasattr(x, "data_ptr"):
        return x.data_ptr() or None
    if hasattr(x, "ctypes"):
        return x.ctypes.data or None
    raise TypeError(f"cannot take the address of {type(x).__name__}")


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def dtype_code(torch_dtype) -> int:
    import torch
    if torch_dtype == torch.float16:
        return CQSA_F16
    if torch_dtype == torch.bfloat16:
        return CQSA_BF16
    if torch_dtype == torch.float32:
        return CQSA_F32
    raise ValueError(f"unsupported dtype {torch_dtype}")


def cqsa_attn_fwd(q, k, v, out, lse, B, H, N, d, causal, scale, dtype, stream=None) -> int:
    return _check(lib.cqsa_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d, int(bool(causal)),
                                    float(scale), dtype, _stream(stream)))


def cqsa_attn_fwd_chunk(q_blk, k_blk, v_blk, q_off, kv_off, B, H, Nq, Nkv, d, causal, scale, dtype, O_part, LSE_part,
                        accumulate, stream=None) -> int:
    return _check(lib.cqsa_attn_fwd_chunk(_ptr(q_blk), _ptr(k_blk), _ptr(v_blk), q_off, kv_off, B, H, Nq, Nkv, d,
                                          int(bool(causal)), float(scale), dtype, _ptr(O_part), _ptr(LSE_part),
                                          int(bool(accumulate)), _stream(stream)))


def cqsa_merge_partials(O_parts, LSE_parts, n, out, lse, B, H, Nq, d, out_dtype, stream=None) -> int:
    po = (ctypes.c_void_p * max(n, 1))(*[_ptr(o) for o in O_parts][:n])
    pl = (ctypes.c_void_p * max(n, 1))(*[_ptr(x) for x in LSE_parts][:n])
    return _check(lib.cqsa_merge_partials(ctypes.cast(po, _vp), ctypes.cast(pl, _vp), n, _ptr(out), _ptr(lse), B, H,
                                          Nq, d, out_dtype, _stream(stream)))


def cqsa_stream_attn_fwd(q_host, k_host, v_host, layout, out, lse, out_on_host, B, H, N, d, causal, scale, dtype,
                         chunk_tokens, stats=None, stream=None) -> int:
    st = stats if stats is not None else cqsa_stream_stats()
    return _check(lib.cqsa_stream_attn_fwd(_ptr(q_host), _ptr(k_host), _ptr(v_host), layout, _ptr(out), _ptr(lse),
                                           int(bool(out_on_host)), B, H, N, d, int(bool(causal)), float(scale), dtype,
                                           chunk_tokens, ctypes.byref(st), _stream(stream)))


def cqsa_attn_fwd_chunked_static(q, k, v, out, lse, B, H, N, d, causal, scale, dtype, chunk_tokens,
                                 stream=None) -> int:
    """No-allocation chunked forward (scratch in the library's static device array)."""
    return _check(lib.cqsa_attn_fwd_chunked_static(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d,
                                                   int(bool(causal)), float(scale), dtype, chunk_tokens,
                                                   _stream(stream)))


def _int_array(values):
    vals = [int(x) for x in values]
    return (ctypes.c_int * max(len(vals), 1))(*vals), len(vals)


def cqsa_quorum_check(c, interest_set) -> int:
    """CQSA_OK if interest_set is a perfect difference set modulo c (raises CqsaError otherwise)."""
    arr, l = _int_array(interest_set)
    return _check(lib.cqsa_quorum_check(c, ctypes.cast(arr, _vp), l))


def cqsa_quorum_schedule(c, interest_set, itr, n_chunks, causal):
    """The quorum schedule as a list of (subproblem, query chunk, key chunk) triples (host only)."""
    arr, l = _int_array(interest_set)
    n = lib.cqsa_quorum_schedule(c, ctypes.cast(arr, _vp), l, itr, n_chunks, int(bool(causal)), None, 0)
    if n < 0:
        raise CqsaError(int(n), last_error())
    buf = (ctypes.c_int * max(3 * n, 1))()
    m = lib.cqsa_quorum_schedule(c, ctypes.cast(arr, _vp), l, itr, n_chunks, int(bool(causal)),
                                 ctypes.cast(buf, _vp), n)
    if m != n:
        raise CqsaError(int(m) if m < 0 else CQSA_ERR_INVALID, last_error())
    return [(buf[3 * i], buf[3 * i + 1], buf[3 * i + 2]) for i in range(n)]


def cqsa_quorum_attn_fwd(q, k, v, layout, inputs_on_host, out, lse, out_on_host, B, H, N, d, causal, scale, dtype,
                         c, interest_set, itr, acc_on_host=False, max_parallel=1, stats=None, stream=None) -> int:
    st = stats if stats is not None else cqsa_quorum_stats()
    arr, l = _int_array(interest_set)
    return _check(lib.cqsa_quorum_attn_fwd(_ptr(q), _ptr(k), _ptr(v), layout, int(bool(inputs_on_host)), _ptr(out),
                                           _ptr(lse), int(bool(out_on_host)), B, H, N, d, int(bool(causal)),
                                           float(scale), dtype, c, ctypes.cast(arr, _vp), l, itr,
                                           int(bool(acc_on_host)), int(max_parallel), ctypes.byref(st),
                                           _stream(stream)))


def cqsa_quorum_attn_fwd_ex(q, k, v, layout, inputs_on_host, out, lse, out_on_host, B, H, N, d, causal, scale,
                            dtype, c, interest_set, itr, acc_on_host=False, max_parallel=1, engine=CQSA_ENGINE_WAVE,
                            wave_tokens=0, stats=None, stream=None) -> int:
    st = stats if stats is not None else cqsa_quorum_stats()
    arr, l = _int_array(interest_set)
    return _check(lib.cqsa_quorum_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), layout, int(bool(inputs_on_host)),
                                              _ptr(out), _ptr(lse), int(bool(out_on_host)), B, H, N, d,
                                              int(bool(causal)), float(scale), dtype, c, ctypes.cast(arr, _vp), l,
                                              itr, int(bool(acc_on_host)), int(max_parallel), int(engine),
                                              int(wave_tokens), ctypes.byref(st), _stream(stream)))


def cqsa_attn_bwd_workspace_size(B, H, N, d) -> int:
    return int(lib.cqsa_attn_bwd_workspace_size(B, H, N, d))


def cqsa_attn_bwd(q, k, v, out, dout, lse, dq, dk, dv, workspace, workspace_bytes, B, H, N, d, causal, scale, dtype,
                  stream=None) -> int:
    return _check(lib.cqsa_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                                    _ptr(dv), _ptr(workspace), int(workspace_bytes), B, H, N, d, int(bool(causal)),
                                    float(scale), dtype, _stream(stream)))


def cqsa_attn_bwd_dvec(out_blk, dout_blk, dvec_blk, B, H, Nq, d, dtype, stream=None) -> int:
    return _check(lib.cqsa_attn_bwd_dvec(_ptr(out_blk), _ptr(dout_blk), _ptr(dvec_blk), B, H, Nq, d, dtype,
                                         _stream(stream)))


def cqsa_attn_bwd_chunk(q_blk, k_blk, v_blk, dout_blk, lse_blk, dvec_blk, q_off, kv_off, B, H, Nq, Nkv, d, causal,
                        scale, dtype, dq_acc, dk_acc, dv_acc, stream=None) -> int:
    return _check(lib.cqsa_attn_bwd_chunk(_ptr(q_blk), _ptr(k_blk), _ptr(v_blk), _ptr(dout_blk), _ptr(lse_blk),
                                          _ptr(dvec_blk), q_off, kv_off, B, H, Nq, Nkv, d, int(bool(causal)),
                                          float(scale), dtype, _ptr(dq_acc), _ptr(dk_acc), _ptr(dv_acc),
                                          _stream(stream)))


def cqsa_attn_bwd_cast(acc, out, n, dtype, stream=None) -> int:
    return _check(lib.cqsa_attn_bwd_cast(_ptr(acc), _ptr(out), n, dtype, _stream(stream)))


def cqsa_stream_attn_bwd(q, k, v, out, dout, lse, dq, dk, dv, B, H, N, d, causal, scale, dtype, chunk_tokens,
                         stream=None) -> int:
    """Host-resident backward (all tensors in host memory, pinned for speed)."""
    return _check(lib.cqsa_stream_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq),
                                           _ptr(dk), _ptr(dv), B, H, N, d, int(bool(causal)), float(scale), dtype,
                                           chunk_tokens, _stream(stream)))


def cqsa_stream_attn_bwd_ex(q, k, v, out, dout, lse, dq, dk, dv, B, H, N, d, causal, scale, dtype, chunk_tokens,
                            stats=None, stream=None):
    """cqsa_stream_attn_bwd that also fills a cqsa_stream_stats (kernel, copy and stall times); returns it."""
    st = stats if stats is not None else cqsa_stream_stats()
    _check(lib.cqsa_stream_attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq),
                                       _ptr(dk), _ptr(dv), B, H, N, d, int(bool(causal)), float(scale), dtype,
                                       chunk_tokens, ctypes.byref(st), _stream(stream)))
    return st


def cqsa_attn_packed_fwd(q, k, v, q_stride, k_stride, v_stride, out, lse, cu_seqlens, n_seqs, T, Hq, Hkv, d, causal, scale,
                         dtype, stream=None) -> int:
    return _check(lib.cqsa_attn_packed_fwd(_ptr(q), _ptr(k), _ptr(v), q_stride, k_stride, v_stride, _ptr(out), _ptr(lse),
                                           _ptr(cu_seqlens), n_seqs, T, Hq, Hkv, d, int(bool(causal)), float(scale), dtype,
                                           _stream(stream)))


def cqsa_attn_packed_bwd_workspace_size(n_seqs, T, Hq, Hkv, d) -> int:
    return int(lib.cqsa_attn_packed_bwd_workspace_size(n_seqs, T, Hq, Hkv, d))


def cqsa_attn_packed_bwd(q, k, v, q_stride, k_stride, v_stride, out, dout, lse, dq, dk, dv, workspace, workspace_bytes,
                         cu_seqlens, n_seqs, T, Hq, Hkv, d, causal, scale, dtype, stream=None) -> int:
    return _check(lib.cqsa_attn_packed_bwd(_ptr(q), _ptr(k), _ptr(v), q_stride, k_stride, v_stride, _ptr(out), _ptr(dout),
                                           _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), int(workspace_bytes),
                                           _ptr(cu_seqlens), n_seqs, T, Hq, Hkv, d, int(bool(causal)), float(scale), dtype,
                                           _stream(stream)))


def cqsa_kv_cache_write(k, v, k_stride, v_stride, k_cache, v_cache, k_scale, v_scale, block_table, max_pages, cu_seqlens,
                        kv_lens, n_seqs, T, Hkv, d, page_size, n_pages, dtype, cache_dtype, stream=None) -> int:
    return _check(lib.cqsa_kv_cache_write(_ptr(k), _ptr(v), k_stride, v_stride, _ptr(k_cache), _ptr(v_cache),
                                          _ptr(k_scale), _ptr(v_scale), _ptr(block_table), max_pages, _ptr(cu_seqlens),
                                          _ptr(kv_lens), n_seqs, T, Hkv, d, page_size, n_pages, dtype, cache_dtype,
                                          _stream(stream)))


def cqsa_kv_cache_read(k, v, k_cache, v_cache, k_scale, v_scale, block_table, max_pages, cu_seqlens, kv_lens, n_seqs, T,
                       Hkv, d, page_size, n_pages, dtype, cache_dtype, stream=None) -> int:
    return _check(lib.cqsa_kv_cache_read(_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                         _ptr(block_table), max_pages, _ptr(cu_seqlens), _ptr(kv_lens), n_seqs, T, Hkv,
                                         d, page_size, n_pages, dtype, cache_dtype, _stream(stream)))


def cqsa_attn_paged_workspace_size(n_seqs, T, Hq, Hkv, d, page_size, max_q_len, max_kv_len, dtype, cache_dtype) -> int:
    return int(lib.cqsa_attn_paged_workspace_size(n_seqs, T, Hq, Hkv, d, page_size, max_q_len, max_kv_len, dtype,
                                                  cache_dtype))


def cqsa_attn_paged_fwd(q, q_stride, out, lse, k_cache, v_cache, k_scale, v_scale, block_table, max_pages, cu_seqlens,
                        kv_lens, n_seqs, T, max_q_len, max_kv_len, Hq, Hkv, d, page_size, n_pages, causal, scale, dtype,
                        cache_dtype, workspace, workspace_bytes, stream=None) -> int:
    return _check(lib.cqsa_attn_paged_fwd(_ptr(q), q_stride, _ptr(out), _ptr(lse), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(k_scale), _ptr(v_scale), _ptr(block_table), max_pages, _ptr(cu_seqlens),
                                          _ptr(kv_lens), n_seqs, T, max_q_len, max_kv_len, Hq, Hkv, d, page_size,
                                          n_pages, int(bool(causal)), float(scale), dtype, cache_dtype, _ptr(workspace),
                                          int(workspace_bytes), _stream(stream)))


def cqsa_set_stream_kv_resident_bytes(nbytes: int) -> None:
    """K/V of cqsa_stream_attn_fwd stay on the device when they take at most nbytes (< 0: half of the free
    device memory, the default; 0: never, every pair through the fp32 accumulator)."""
    lib.cqsa_set_stream_kv_resident_bytes(int(nbytes))


def cqsa_release_cache() -> int:
    """Free the device buffers, events and streams the host-driven entry points keep between calls."""
    return _check(lib.cqsa_release_cache())


def cqsa_device_error(clear: bool = True):
    """(status, code, block) of the device error word after synchronising the device."""
    code, block = _i(0), _i(0)
    rc = lib.cqsa_device_error(ctypes.byref(code), ctypes.byref(block), int(bool(clear)))
    return rc, code.value, block.value


def cqsa_set_timeout_ms(ms: int) -> None:
    lib.cqsa_set_timeout_ms(ms)


def cqsa_debug_set_fault(kind: int) -> int:
    return _check(lib.cqsa_debug_set_fault(kind))


def cqsa_version() -> str:
    return lib.cqsa_version().decode()


# ---- torch conveniences (marshalling only) --------------------------------------------------------

def attention(q, k, v, *, causal=False, scale=None, return_lse=False, stream=None):
    """SDPA-shaped call on device tensors [B,H,N,d] (fp16/bf16): returns out (and lse [B,H,N] fp32)."""
    import torch
    B, H, N, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or not (q.is_cuda and k.is_cuda and v.is_cuda):
        raise ValueError("q, k, v must be CUDA tensors of one shape [B,H,N,d]")
    q, k, v = (t.contiguous() for t in (q, k, v))
    out = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    cqsa_attn_fwd(q, k, v, out, lse, B, H, N, d, causal, 0.0 if scale is None else scale, dtype_code(q.dtype),
                  stream)
    return (out, lse) if return_lse else out


def attention_backward(q, k, v, out, dout, lse, *, causal=False, scale=None, stream=None):
    """Gradients (dq, dk, dv) of attention on device tensors [B,H,N,d], d = 64 or 128 (fp16/bf16), from
    the forward's out and lse ([B,H,N] fp32) and the upstream gradient dout."""
    import torch
    B, H, N, d = q.shape
    for t in (k, v, out, dout):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_cuda:
            raise ValueError("q, k, v, out, dout must be CUDA tensors of one shape and dtype [B,H,N,d]")
    if lse.shape != (B, H, N) or lse.dtype != torch.float32:
        raise ValueError("lse must be a float32 tensor [B,H,N]")
    q, k, v, out, dout, lse = (t.contiguous() for t in (q, k, v, out, dout, lse))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws_bytes = cqsa_attn_bwd_workspace_size(B, H, N, d)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    cqsa_attn_bwd(q, k, v, out, dout, lse, dq, dk, dv, ws, ws.numel(), B, H, N, d, causal,
                  0.0 if scale is None else scale, dtype_code(q.dtype), stream)
    return dq, dk, dv


# Sequences of different lengths: torch conveniences (checks and marshalling only). They run on the tensors' own
# device, whichever is current, on `stream` (a torch stream or a cudaStream_t value) or that device's current
# stream; what they allocate belongs to that stream. A serving step makes one of these calls per layer, so they look at
# each tensor once and pass addresses straight on.

_torch = None
_codes: dict = {}


def _tc():
    """torch, imported by the first call that needs it."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
        _codes.update({torch.float16: CQSA_F16, torch.bfloat16: CQSA_BF16})
    return _torch


def _elsewhere(device, stream):
    """A context that makes `device` current and `stream` its current stream, or None where they already are."""
    torch = _tc()
    if device.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    here = device.index == torch.cuda.current_device()
    if here and stream is None:
        return None
    import contextlib
    stack = contextlib.ExitStack()
    if not here:
        stack.enter_context(torch.cuda.device(device))
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        stack.enter_context(torch.cuda.stream(stream))
    return stack


def _current(device):
    """The cudaStream_t of the device's current stream."""
    torch = _tc()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return (raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream) or None


def _code(dtype):
    code = _codes.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype} (float16 or bfloat16)")
    return code


def _tokens(name, t, heads, d, like):
    """A [T, heads, d] tensor of like's dtype and device, its heads dense; returns it (a copy if need be) and its token stride."""
    shape = t.shape
    if t is not like and (t.dtype != like.dtype or t.device != like.device) or len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError(f"{name} must be a [T, {heads}, {d}] tensor of {like.dtype} on {like.device}")
    if t.is_contiguous() and not t.data_ptr() & 15:
        return t, heads * d
    T = shape[0]
    s = t.stride()
    if (s[2] != 1 or (s[1] != d and heads > 1) or s[0] < heads * d or s[0] % 8 or t.data_ptr() & 15) and T > 0:
        return _dense(t), heads * d
    return t, (s[0] if T > 1 else heads * d)


def _dense(t):
    """t, or a copy of it where it is not contiguous or not 16-byte aligned."""
    if not t.is_contiguous():
        return t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _ints(name, t, shape, device):
    if t.dtype != _tc().int32 or t.device != device or t.shape != shape:
        raise ValueError(f"{name} must be an int32 tensor of shape {tuple(shape)} on {device}")
    return t if t.is_contiguous() else t.contiguous()


def _out(out, q):
    torch = _tc()
    if out is None:
        return torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if out.shape != q.shape or out.dtype != q.dtype or out.device != q.device or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {tuple(q.shape)} tensor of {q.dtype} on {q.device}")
    return out


def _cache(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, kv_lens, dtype, device):
    """The checks that the calls on a paged cache share; returns the cache's dtype code, n_seqs, max_pages, the three index
    tensors and the scales' addresses."""
    torch = _tc()
    shape, kind = k_cache.shape, k_cache.dtype
    if device.type != "cuda" or k_cache.device != device or v_cache.device != device:
        raise ValueError("k_cache and v_cache must be CUDA tensors on the tokens' device")
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != kind:
        raise ValueError("k_cache and v_cache must be tensors of one shape and dtype [n_pages, Hkv, page_size, d]")
    if not k_cache.is_contiguous() or not v_cache.is_contiguous():
        raise ValueError("k_cache and v_cache must be contiguous")
    ks = vs = None
    if kind == dtype:
        code = _code(dtype)
        if k_scale is not None or v_scale is not None:
            raise ValueError("a 16-bit cache takes no scales")
    elif kind == torch.uint8 or kind == torch.float8_e4m3fn:
        code = CQSA_E4M3
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is None or t.element_size() != 1 or t.shape != shape[:3] or t.device != device or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous byte tensor [n_pages, Hkv, page_size] beside an e4m3 cache")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    else:
        raise ValueError(f"a cache of {kind} does not go with tokens of {dtype}")
    table = block_table.shape
    if len(table) != 2 or kv_lens.shape != table[:1]:
        raise ValueError("block_table must be [n_seqs, max_pages] and kv_lens [n_seqs]")
    n_seqs = table[0]
    return (code, n_seqs, table[1], _ints("block_table", block_table, table, device),
            _ints("cu_seqlens", cu_seqlens, (n_seqs + 1,), device), _ints("kv_lens", kv_lens, (n_seqs,), device), ks, vs)


def _packed(q, k, v, cu_seqlens):
    """The checks that the calls on packed tokens share: (q, k, v) with their strides, cu_seqlens, and the sizes."""
    if len(q.shape) != 3 or len(k.shape) != 3 or not q.is_cuda:
        raise ValueError("q must be a CUDA tensor [T, Hq, d], k and v [T, Hkv, d]")
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    if k.shape[0] != T or v.shape != k.shape:
        raise ValueError("k and v must be [T, Hkv, d] with q's T")
    if len(cu_seqlens.shape) != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be [n_seqs + 1]")
    n_seqs = cu_seqlens.shape[0] - 1
    return (_tokens("q", q, Hq, d, q), _tokens("k", k, Hkv, d, q), _tokens("v", v, Hkv, d, q),
            _ints("cu_seqlens", cu_seqlens, (n_seqs + 1,), q.device), n_seqs, T, Hq, Hkv, d)


def attention_packed(q, k, v, cu_seqlens, *, causal=True, scale=None, return_lse=False, out=None, stream=None):
    """Attention of whole prompts packed end to end: q [T, Hq, d], k, v [T, Hkv, d], cu_seqlens int32 [n_seqs + 1] on the
    device; returns out [T, Hq, d] (and lse [Hq, T] fp32). Rows behind the last sequence are left as they were in `out`."""
    torch = _tc()
    ctx = _elsewhere(q.device, stream)
    if ctx is not None:
        with ctx:
            return attention_packed(q, k, v, cu_seqlens, causal=causal, scale=scale, return_lse=return_lse, out=out)
    (q, qs), (k, ks), (v, vs), cu, n_seqs, T, Hq, Hkv, d = _packed(q, k, v, cu_seqlens)
    out = _out(out, q)
    lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device) if return_lse else None
    _check(lib.cqsa_attn_packed_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, out.data_ptr(),
                                    lse.data_ptr() if return_lse else None, cu.data_ptr(), n_seqs, T, Hq, Hkv, d,
                                    1 if causal else 0, 0.0 if scale is None else scale, _code(q.dtype),
                                    _current(q.device)))
    return (out, lse) if return_lse else out


def attention_packed_backward(q, k, v, out, dout, lse, cu_seqlens, *, causal=True, scale=None, grads=None, stream=None):
    """Gradients (dq, dk, dv) of attention_packed from its out and lse and the upstream gradient dout; dk and dv sum over the
    query heads of a group. Rows behind the last sequence are left as they were in `grads` (three contiguous tensors),
    which are allocated if not given."""
    torch = _tc()
    device, dtype = q.device, q.dtype
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return attention_packed_backward(q, k, v, out, dout, lse, cu_seqlens, causal=causal, scale=scale, grads=grads)
    (q, qs), (k, ks), (v, vs), cu, n_seqs, T, Hq, Hkv, d = _packed(q, k, v, cu_seqlens)
    for name, t in (("out", out), ("dout", dout)):
        if t.shape != q.shape or t.dtype != dtype or t.device != device:
            raise ValueError(f"{name} must be a {tuple(q.shape)} tensor of {dtype} on {device}")
    if lse.shape != (Hq, T) or lse.dtype != torch.float32 or lse.device != device:
        raise ValueError("lse must be a float32 tensor [Hq, T]")
    out, dout, lse = _dense(out), _dense(dout), lse.contiguous()
    if grads is None:
        dq = torch.empty((T, Hq, d), dtype=dtype, device=device)
        dk, dv = (torch.empty((T, Hkv, d), dtype=dtype, device=device) for _ in range(2))
    else:
        dq, dk, dv = grads
        for t, h in ((dq, Hq), (dk, Hkv), (dv, Hkv)):
            if t.shape != (T, h, d) or t.dtype != dtype or t.device != device or not t.is_contiguous():
                raise ValueError("grads must be contiguous tensors of q's, k's and v's shapes and dtype")
    need = lib.cqsa_attn_packed_bwd_workspace_size(n_seqs, T, Hq, Hkv, d)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    _check(lib.cqsa_attn_packed_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, out.data_ptr(), dout.data_ptr(),
                                    lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), need,
                                    cu.data_ptr(), n_seqs, T, Hq, Hkv, d, 1 if causal else 0,
                                    0.0 if scale is None else scale, _code(dtype), _current(device)))
    return dq, dk, dv


def kv_cache_write(k, v, k_cache, v_cache, block_table, cu_seqlens, kv_lens, *, k_scale=None, v_scale=None, stream=None):
    """New tokens k, v [T, Hkv, d] into their pages of the caches [n_pages, Hkv, page_size, d] (k's dtype, or
    uint8 / float8_e4m3fn codes with byte tensors k_scale, v_scale [n_pages, Hkv, page_size])."""
    ctx = _elsewhere(k.device, stream)
    if ctx is not None:
        with ctx:
            return kv_cache_write(k, v, k_cache, v_cache, block_table, cu_seqlens, kv_lens, k_scale=k_scale, v_scale=v_scale)
    code, n_seqs, max_pages, table, cu, lens, ksc, vsc = _cache(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens,
                                                                kv_lens, k.dtype, k.device)
    n_pages, Hkv, page, d = k_cache.shape
    (k, ks), (v, vs) = _tokens("k", k, Hkv, d, k), _tokens("v", v, Hkv, d, k)
    if v.shape != k.shape:
        raise ValueError("k and v must have one shape")
    _check(lib.cqsa_kv_cache_write(k.data_ptr(), v.data_ptr(), ks, vs, k_cache.data_ptr(), v_cache.data_ptr(), ksc, vsc,
                                   table.data_ptr(), max_pages, cu.data_ptr(), lens.data_ptr(), n_seqs, k.shape[0], Hkv, d,
                                   page, n_pages, _code(k.dtype), code, _current(k.device)))


def kv_cache_read(k_cache, v_cache, block_table, cu_seqlens, kv_lens, T, dtype, *, k_scale=None, v_scale=None, out=None,
                  stream=None):
    """The last cu_seqlens[s+1] - cu_seqlens[s] positions of each sequence as (k, v) [T, Hkv, d] of dtype (into `out`, a
    pair of such tensors, if given)."""
    torch = _tc()
    device = k_cache.device
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return kv_cache_read(k_cache, v_cache, block_table, cu_seqlens, kv_lens, T, dtype, k_scale=k_scale,
                                 v_scale=v_scale, out=out)
    code, n_seqs, max_pages, table, cu, lens, ksc, vsc = _cache(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens,
                                                                kv_lens, dtype, device)
    n_pages, Hkv, page, d = k_cache.shape
    if out is None:
        k, v = (torch.empty((T, Hkv, d), dtype=dtype, device=device) for _ in range(2))
    else:
        k, v = out
        for t in (k, v):
            if t.shape != (T, Hkv, d) or t.dtype != dtype or t.device != device or not t.is_contiguous():
                raise ValueError(f"out must be two contiguous [{T}, {Hkv}, {d}] tensors of {dtype}")
    _check(lib.cqsa_kv_cache_read(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ksc, vsc,
                                  table.data_ptr(), max_pages, cu.data_ptr(), lens.data_ptr(), n_seqs, T, Hkv, d, page,
                                  n_pages, _code(dtype), code, _current(device)))
    return k, v


_sizes: dict = {}  # workspace sizes by the arguments that set them


def attention_paged(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, max_q_len, max_kv_len, *, causal=True,
                    scale=None, k_scale=None, v_scale=None, return_lse=False, out=None, workspace=None, stream=None):
    """Attention of each sequence's new tokens q [T, Hq, d] over its positions in the paged cache: out [T, Hq, d] (and
    lse [Hq, T] fp32). max_q_len: at least the most new tokens of a sequence; max_kv_len: about the longest kv_lens.
    `workspace`: a byte tensor of at least cqsa_attn_paged_workspace_size bytes (allocated if not given)."""
    torch = _tc()
    device, dtype = q.device, q.dtype
    ctx = _elsewhere(device, stream)
    if ctx is not None:
        with ctx:
            return attention_paged(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, max_q_len, max_kv_len,
                                   causal=causal, scale=scale, k_scale=k_scale, v_scale=v_scale, return_lse=return_lse,
                                   out=out, workspace=workspace)
    code, n_seqs, max_pages, table, cu, lens, ksc, vsc = _cache(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens,
                                                                kv_lens, dtype, device)
    n_pages, Hkv, page, d = k_cache.shape
    if len(q.shape) != 3:
        raise ValueError("q must be [T, Hq, d]")
    T, Hq = q.shape[:2]
    q, qs = _tokens("q", q, Hq, d, q)
    dt = _code(dtype)
    max_q_len, max_kv_len = min(max_q_len, T), min(max_kv_len, 0x7fffffff)  # (ctypes would cut larger ones down to 32 bits)
    out = _out(out, q)
    lse = torch.empty((Hq, T), dtype=torch.float32, device=device) if return_lse else None
    if workspace is not None and (workspace.device != device or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    if workspace is None:
        key = (n_seqs, T, Hq, Hkv, d, page, max_q_len, max_kv_len, dt, code, device.index)
        size = _sizes.get(key)
        if size is None:
            if len(_sizes) >= 4096:  # (lengths differ from step to step)
                _sizes.clear()
            size = _sizes[key] = lib.cqsa_attn_paged_workspace_size(*key[:-1])
        workspace = torch.empty(max(size, 16), dtype=torch.uint8, device=device)
    else:
        size = workspace.numel() * workspace.element_size()
    _check(lib.cqsa_attn_paged_fwd(q.data_ptr(), qs, out.data_ptr(), lse.data_ptr() if return_lse else None,
                                   k_cache.data_ptr(), v_cache.data_ptr(), ksc, vsc, table.data_ptr(), max_pages,
                                   cu.data_ptr(), lens.data_ptr(), n_seqs, T, max_q_len, max_kv_len, Hq, Hkv, d, page,
                                   n_pages, 1 if causal else 0, 0.0 if scale is None else scale, dt, code,
                                   workspace.data_ptr(), size, _current(device)))
    return (out, lse) if return_lse else out
