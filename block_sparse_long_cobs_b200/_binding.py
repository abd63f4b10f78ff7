"""Thin Python binding of the COBS C ABI (``include/cobs.h``, ``include/cobs_cache.h``).

Argument marshalling only: every function here forwards to the function of
the same name in ``libcobs_b200.so`` (built in-tree by
``python -m block_sparse_long_cobs_b200.build``); all computation happens in
the library's CUDA kernels.  Tensors may be given as torch tensors (their
``data_ptr()`` is passed), integer addresses or ``None`` (NULL).  Streams may
be a ``torch.cuda.Stream``, an integer handle or ``None`` (legacy default
stream).  Importing this module fails if the library has not been built: there
is no fallback path.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "CobsError", "cobs_dims", "LIB_PATH", "lib",
    "cobs_abi_version", "cobs_stats_record_bytes", "cobs_selected_capacity",
    "cobs_workspace_bytes", "COBS_STATS_BF16", "COBS_STATS_FP4", "COBS_STATS_BOX",
    "COBS_STATS_SUBSPACE",
    "cobs_workspace_init", "cobs_build_block_stats", "cobs_select_blocks",
    "cobs_sparse_decode", "cobs_sparse_decode_no_alloc", "cobs_select_blocks_varlen",
    "cobs_sparse_decode_varlen", "cobs_build_block_stats_paged", "cobs_sparse_decode_paged",
    "cobs_select_and_decode", "cobs_read_device_status", "cobs_no_alloc_read_status",
    "cobs_set_wait_limit_ns",
    "cobs_last_error",
    "cobs_status_string",
    "cobs_kv_cache", "cobs_rope", "cobs_rope_init", "cobs_append_tokens", "cobs_read_cache",
    "cobs_prompt_workspace_bytes", "cobs_prompt_attention", "cobs_sparse_decode_cache",
    "COBS_CACHE_BF16", "COBS_CACHE_E4M3", "COBS_ROPE_PLAIN", "COBS_ROPE_LINEAR",
    "COBS_ROPE_BY_PARTS", "COBS_ROPE_CUSTOM",
    "COBS_OK", "COBS_ERR_INVALID_ARG", "COBS_ERR_UNSUPPORTED",
    "COBS_ERR_WORKSPACE", "COBS_ERR_CUDA", "COBS_ERR_TIMEOUT", "COBS_ERR_DEVICE",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcobs_b200.so")

COBS_OK = 0
COBS_ERR_INVALID_ARG = 1
COBS_ERR_UNSUPPORTED = 2
COBS_ERR_WORKSPACE = 3
COBS_ERR_CUDA = 4
COBS_ERR_TIMEOUT = 5
COBS_ERR_DEVICE = 6

COBS_STATS_BF16 = 0     # block records: mu and U in bf16
COBS_STATS_FP4 = 1      # block records: mu in bf16, U in scaled FP4 (E2M1)
COBS_STATS_BOX = 2      # block records: per-dimension min and max of the keys (bf16)
COBS_STATS_SUBSPACE = 3  # block records: mu in bf16, U projected on a query subspace (bf16)

COBS_CACHE_BF16 = 0     # KV cache: keys and values in bf16
COBS_CACHE_E4M3 = 1     # KV cache: E4M3 codes and one fp32 scale per row

COBS_ROPE_PLAIN = 0     # rotary frequencies base^(-2 t / rotary_dim)
COBS_ROPE_LINEAR = 1    # ... divided by factor
COBS_ROPE_BY_PARTS = 2  # ... slow pairs divided by factor, fast ones kept
COBS_ROPE_CUSTOM = 3    # given frequencies


class CobsError(RuntimeError):
    """A COBS call returned a non-OK status."""

    def __init__(self, func: str, status: int, message: str):
        super().__init__(f"{func}: {cobs_status_string(status)}: {message}")
        self.status = status


class cobs_dims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("rank", ctypes.c_int32),
        ("capacity_tokens", ctypes.c_int64),
        ("stats_format", ctypes.c_int32),       # COBS_STATS_BF16 / _FP4 / _BOX / _SUBSPACE
        ("subspace_dim", ctypes.c_int32),       # s of COBS_STATS_SUBSPACE records
        ("subspace_basis", ctypes.c_void_p),    # device [Hkv][s][d] fp32 basis
    ]


class cobs_kv_cache(ctypes.Structure):
    """A KV cache as the cache calls take it (``include/cobs_cache.h``).  Buffers
    are given as in the calls (CUDA tensors, addresses or None); the descriptor
    keeps the tensors alive."""
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("n_pages", ctypes.c_int64),
        ("table_stride", ctypes.c_int32),
        ("format", ctypes.c_int32),             # COBS_CACHE_BF16 / _E4M3
    ]

    def __init__(self, k=None, v=None, k_scale=None, v_scale=None, block_table=None, n_pages=0,
                 table_stride=0, format=COBS_CACHE_BF16):
        super().__init__(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(block_table),
                         n_pages, table_stride, format)
        self._buffers = (k, v, k_scale, v_scale, block_table)


class cobs_rope_params(ctypes.Structure):
    _fields_ = [
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("scaling", ctypes.c_int32),            # COBS_ROPE_*
        ("reserved", ctypes.c_int32),
        ("base", ctypes.c_double),
        ("factor", ctypes.c_double),
        ("original_context", ctypes.c_double),
        ("low", ctypes.c_double),
        ("high", ctypes.c_double),
        ("attention_factor", ctypes.c_double),
        ("frequencies", ctypes.POINTER(ctypes.c_double)),
    ]


class cobs_rope(ctypes.Structure):
    """A rotary table, made by cobs_rope_init."""
    _fields_ = [
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("attention_factor", ctypes.c_float),
        ("reserved", ctypes.c_int32),
        ("turns", ctypes.c_uint64 * 64),        # turns per token of a pair, times 2^64
    ]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"COBS CUDA library not found at {LIB_PATH}; build it with "
            "`python -m block_sparse_long_cobs_b200.build` (needs nvcc)")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ, F32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                            ctypes.c_size_t, ctypes.c_float)
    D, C = ctypes.POINTER(cobs_dims), ctypes.POINTER(cobs_kv_cache)
    sig = {
        "cobs_abi_version": (I32, []),
        "cobs_stats_record_bytes": (I64, [D]),
        "cobs_selected_capacity": (I32, [D, I32, I32, I32]),
        "cobs_workspace_bytes": (SZ, [D, I32, I32, I32]),
        "cobs_workspace_init": (I32, [P, SZ, P]),
        "cobs_build_block_stats": (I32, [D, P, I64, I64, P, P, SZ, P]),
        "cobs_select_blocks": (I32, [D, P, P, I64, I32, I32, I32, P, I32, P, P, P, SZ, P]),
        "cobs_sparse_decode": (I32, [D, P, P, P, P, P, I32, I64, F32, P, P, P, SZ, P]),
        "cobs_sparse_decode_no_alloc": (I32, [D, P, P, P, P, P, I32, I64, F32, P, P, P]),
        "cobs_select_blocks_varlen": (I32, [D, P, P, P, I64, I32, I32, I32, P, I32, P, P, P,
                                            SZ, P]),
        "cobs_sparse_decode_varlen": (I32, [D, P, P, P, P, P, I32, P, I64, F32, P, P, P, SZ, P]),
        "cobs_build_block_stats_paged": (I32, [D, P, I64, P, I32, I64, I64, P, P, SZ, P]),
        "cobs_sparse_decode_paged": (I32, [D, P, P, P, I64, P, I32, P, P, I32, P, I64, F32, P,
                                           P, P, SZ, P]),
        "cobs_select_and_decode": (I32, [D, P, P, P, P, I64, I32, I32, I32, F32, P, I32, P, P,
                                         P, P, P, SZ, P]),
        "cobs_read_device_status": (I32, [P, SZ, ctypes.POINTER(I32), P]),
        "cobs_no_alloc_read_status": (I32, [ctypes.POINTER(I32), P]),
        "cobs_set_wait_limit_ns": (I32, [ctypes.c_uint64]),
        "cobs_rope_init": (I32, [ctypes.POINTER(cobs_rope_params), ctypes.POINTER(cobs_rope)]),
        "cobs_append_tokens": (I32, [D, C, ctypes.POINTER(cobs_rope), P, I64, P, I64, P, I64, P,
                                     I64, P, P, P, SZ, P]),
        "cobs_read_cache": (I32, [D, C, P, I64, I64, P, P, P, SZ, P]),
        "cobs_prompt_workspace_bytes": (SZ, [D, I64, I64]),
        "cobs_prompt_attention": (I32, [D, C, P, P, I64, P, I64, F32, P, P, P, SZ, P]),
        "cobs_sparse_decode_cache": (I32, [D, C, P, P, P, I32, P, I64, F32, P, P, P, SZ, P]),
        "cobs_last_error": (ctypes.c_char_p, []),
        "cobs_status_string": (ctypes.c_char_p, [I32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


lib = _load()


def _ptr(x):
    """Device address of a buffer argument (every pointer of the C ABI is a
    device pointer): an int is taken as is; a torch tensor must be a
    contiguous CUDA tensor (a host or strided tensor would hand the kernels a
    wrong address)."""
    if x is None:
        return None
    if isinstance(x, int):
        return ctypes.c_void_p(x)
    if hasattr(x, "data_ptr"):
        if hasattr(x, "is_cuda") and not x.is_cuda:
            raise TypeError("tensor arguments must be CUDA tensors (got a host tensor)")
        if hasattr(x, "is_contiguous") and not x.is_contiguous():
            raise TypeError("tensor arguments must be contiguous")
        return ctypes.c_void_p(x.data_ptr())
    if hasattr(x, "ctypes"):
        return ctypes.c_void_p(x.ctypes.data)
    raise TypeError(f"cannot pass {type(x).__name__} as a pointer")


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return ctypes.c_void_p(s)
    return ctypes.c_void_p(s.cuda_stream)


def _check(func: str, status: int, check: bool) -> int:
    if check and status != COBS_OK:
        raise CobsError(func, status, cobs_last_error())
    return status


def _dims(d) -> cobs_dims:
    if isinstance(d, cobs_dims):
        return d
    d = dict(d)
    if d.get("subspace_basis") is not None:
        d["subspace_basis"] = _ptr(d["subspace_basis"]).value
    return cobs_dims(**d)


def cobs_abi_version() -> int:
    return lib.cobs_abi_version()


def cobs_stats_record_bytes(dims) -> int:
    """Bytes of one block record for dims' stats_format."""
    n = lib.cobs_stats_record_bytes(ctypes.byref(_dims(dims)))
    if n <= 0:
        raise CobsError("cobs_stats_record_bytes", COBS_ERR_INVALID_ARG, cobs_last_error())
    return n


def cobs_last_error() -> str:
    return lib.cobs_last_error().decode()


def cobs_status_string(status: int) -> str:
    return lib.cobs_status_string(status).decode()


def cobs_selected_capacity(dims, top_k, sink_blocks, local_tokens) -> int:
    n = lib.cobs_selected_capacity(ctypes.byref(_dims(dims)), top_k, sink_blocks,
                                   local_tokens)
    if n < 0:
        raise CobsError("cobs_selected_capacity", COBS_ERR_INVALID_ARG, cobs_last_error())
    return n


def cobs_workspace_bytes(dims, top_k, sink_blocks, local_tokens) -> int:
    n = lib.cobs_workspace_bytes(ctypes.byref(_dims(dims)), top_k, sink_blocks,
                                 local_tokens)
    if n == 0:
        raise CobsError("cobs_workspace_bytes", COBS_ERR_INVALID_ARG, cobs_last_error())
    return n


def cobs_workspace_init(ws, ws_bytes, stream=None, check=True) -> int:
    return _check("cobs_workspace_init",
                  lib.cobs_workspace_init(_ptr(ws), ws_bytes, _stream(stream)), check)


def cobs_build_block_stats(dims, k, block_begin, block_end, stats, ws, ws_bytes,
                           stream=None, check=True) -> int:
    st = lib.cobs_build_block_stats(ctypes.byref(_dims(dims)), _ptr(k), block_begin,
                                    block_end, _ptr(stats), _ptr(ws), ws_bytes,
                                    _stream(stream))
    return _check("cobs_build_block_stats", st, check)


def cobs_select_blocks(dims, q, stats, seq_len, top_k, sink_blocks, local_tokens,
                       idx, idx_stride, n_sel, scores_opt, ws, ws_bytes, stream=None,
                       check=True) -> int:
    st = lib.cobs_select_blocks(ctypes.byref(_dims(dims)), _ptr(q), _ptr(stats), seq_len,
                                top_k, sink_blocks, local_tokens, _ptr(idx), idx_stride,
                                _ptr(n_sel), _ptr(scores_opt), _ptr(ws), ws_bytes,
                                _stream(stream))
    return _check("cobs_select_blocks", st, check)


def cobs_sparse_decode(dims, q, k, v, idx, n_sel, idx_stride, seq_len, softmax_scale,
                       out, lse, ws, ws_bytes, stream=None, check=True) -> int:
    st = lib.cobs_sparse_decode(ctypes.byref(_dims(dims)), _ptr(q), _ptr(k), _ptr(v),
                                _ptr(idx), _ptr(n_sel), idx_stride, seq_len,
                                ctypes.c_float(softmax_scale), _ptr(out), _ptr(lse),
                                _ptr(ws), ws_bytes, _stream(stream))
    return _check("cobs_sparse_decode", st, check)


def cobs_select_and_decode(dims, q, stats, k, v, seq_len, top_k, sink_blocks, local_tokens,
                           softmax_scale, idx, idx_stride, n_sel, scores_opt, out, lse, ws,
                           ws_bytes, stream=None, check=True) -> int:
    st = lib.cobs_select_and_decode(ctypes.byref(_dims(dims)), _ptr(q), _ptr(stats), _ptr(k),
                                    _ptr(v), seq_len, top_k, sink_blocks, local_tokens,
                                    ctypes.c_float(softmax_scale), _ptr(idx), idx_stride,
                                    _ptr(n_sel), _ptr(scores_opt), _ptr(out), _ptr(lse),
                                    _ptr(ws), ws_bytes, _stream(stream))
    return _check("cobs_select_and_decode", st, check)


def cobs_sparse_decode_no_alloc(dims, q, k, v, idx, n_sel, idx_stride, seq_len,
                                softmax_scale, out, lse, stream=None, check=True) -> int:
    """cobs_sparse_decode without a workspace: for callers that cannot give the
    library device memory; it uses the library's own fixed 16 MiB array."""
    st = lib.cobs_sparse_decode_no_alloc(ctypes.byref(_dims(dims)), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(idx), _ptr(n_sel), idx_stride, seq_len,
                                         ctypes.c_float(softmax_scale), _ptr(out), _ptr(lse),
                                         _stream(stream))
    return _check("cobs_sparse_decode_no_alloc", st, check)


def cobs_select_blocks_varlen(dims, q, stats, seq_lens, max_seq_len, top_k, sink_blocks,
                              local_tokens, idx, idx_stride, n_sel, scores_opt, ws, ws_bytes,
                              stream=None, check=True) -> int:
    """cobs_select_blocks with per-sequence lengths (seq_lens: device int64 [batch])."""
    st = lib.cobs_select_blocks_varlen(ctypes.byref(_dims(dims)), _ptr(q), _ptr(stats),
                                       _ptr(seq_lens), max_seq_len, top_k, sink_blocks,
                                       local_tokens, _ptr(idx), idx_stride, _ptr(n_sel),
                                       _ptr(scores_opt), _ptr(ws), ws_bytes, _stream(stream))
    return _check("cobs_select_blocks_varlen", st, check)


def cobs_sparse_decode_varlen(dims, q, k, v, idx, n_sel, idx_stride, seq_lens, max_seq_len,
                              softmax_scale, out, lse, ws, ws_bytes, stream=None,
                              check=True) -> int:
    """cobs_sparse_decode with per-sequence lengths (seq_lens: device int64 [batch])."""
    st = lib.cobs_sparse_decode_varlen(ctypes.byref(_dims(dims)), _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(idx), _ptr(n_sel), idx_stride, _ptr(seq_lens),
                                       max_seq_len, ctypes.c_float(softmax_scale), _ptr(out),
                                       _ptr(lse), _ptr(ws), ws_bytes, _stream(stream))
    return _check("cobs_sparse_decode_varlen", st, check)


def cobs_build_block_stats_paged(dims, k_pool, n_pages, block_table, table_stride,
                                 block_begin, block_end, stats, ws, ws_bytes, stream=None,
                                 check=True) -> int:
    """cobs_build_block_stats over a page pool [n_pages, Hkv, 64, d] addressed through
    block_table (device int32 [batch, table_stride])."""
    st = lib.cobs_build_block_stats_paged(ctypes.byref(_dims(dims)), _ptr(k_pool), n_pages,
                                          _ptr(block_table), table_stride, block_begin,
                                          block_end, _ptr(stats), _ptr(ws), ws_bytes,
                                          _stream(stream))
    return _check("cobs_build_block_stats_paged", st, check)


def cobs_sparse_decode_paged(dims, q, k_pool, v_pool, n_pages, block_table, table_stride,
                             idx, n_sel, idx_stride, seq_lens, max_seq_len, softmax_scale,
                             out, lse, ws, ws_bytes, stream=None, check=True) -> int:
    """cobs_sparse_decode over page pools; seq_lens (device int64 [batch]) or None."""
    st = lib.cobs_sparse_decode_paged(ctypes.byref(_dims(dims)), _ptr(q), _ptr(k_pool),
                                      _ptr(v_pool), n_pages, _ptr(block_table), table_stride,
                                      _ptr(idx), _ptr(n_sel), idx_stride, _ptr(seq_lens),
                                      max_seq_len, ctypes.c_float(softmax_scale), _ptr(out),
                                      _ptr(lse), _ptr(ws), ws_bytes, _stream(stream))
    return _check("cobs_sparse_decode_paged", st, check)


def cobs_read_device_status(ws, ws_bytes, stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    out = ctypes.c_int32(0)
    st = lib.cobs_read_device_status(_ptr(ws), ws_bytes, ctypes.byref(out),
                                     _stream(stream))
    _check("cobs_read_device_status", st, True)
    return out.value


def cobs_no_alloc_read_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the status word of the
    allocation-free decode's fixed array on the current device."""
    out = ctypes.c_int32(0)
    st = lib.cobs_no_alloc_read_status(ctypes.byref(out), _stream(stream))
    _check("cobs_no_alloc_read_status", st, True)
    return out.value


def cobs_set_wait_limit_ns(limit_ns: int) -> int:
    """Limit of the statistics kernel's first bounded device wait (0: the
    default 2 s); a testing and diagnostic knob."""
    return _check("cobs_set_wait_limit_ns", lib.cobs_set_wait_limit_ns(int(limit_ns)), True)


def _addr(x):
    """Like _ptr, as a plain integer or None."""
    if x is None or type(x) is int:
        return x
    try:
        if x.is_cuda and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        pass
    return _ptr(x).value


def _rows_addr(x, stride, name):
    """Address of packed rows that start ``stride`` elements apart: a CUDA
    tensor whose rows are contiguous and lie that far apart (a part of a fused
    projection), an address or None."""
    if x is None or type(x) is int:
        return x
    try:
        st, shape = x.stride(), x.shape
    except AttributeError:
        return _ptr(x).value
    if len(st) == 3 and st[2] == 1 and st[1] == shape[2] and st[0] == stride and x.is_cuda:
        return x.data_ptr()
    if not x.is_cuda:
        raise TypeError("tensor arguments must be CUDA tensors (got a host tensor)")
    row = 1
    for n, s in zip(shape[:0:-1], st[:0:-1]):
        if s != row and n > 1:
            raise TypeError(f"{name}: rows must be contiguous")
        row *= n
    if st[0] != stride and shape[0] > 1:
        raise TypeError(f"{name}: rows must be {name}_stride elements apart")
    return x.data_ptr()


def cobs_rope_init(rotary_dim, interleaved=False, base=10000.0, scaling=COBS_ROPE_PLAIN,
                   factor=1.0, original_context=0.0, low=0.0, high=0.0, attention_factor=1.0,
                   frequencies=None) -> cobs_rope:
    """Rotary table of ``rotary_dim`` leading dimensions (host work only)."""
    f = None
    if frequencies is not None:
        f = [float(x) for x in frequencies]
        if len(f) < rotary_dim // 2:
            raise ValueError("frequencies: one per rotated pair is needed")
        f = (ctypes.c_double * len(f))(*f)
    p = cobs_rope_params(rotary_dim, int(interleaved), scaling, 0, base, factor,
                         original_context, low, high, attention_factor, f)
    rope = cobs_rope()
    _check("cobs_rope_init", lib.cobs_rope_init(ctypes.byref(p), ctypes.byref(rope)), True)
    return rope


def cobs_append_tokens(dims, cache, rope, q, q_stride, k, k_stride, v, v_stride, cu_tokens,
                       n_tokens, start, q_out, ws, ws_bytes, stream=None, check=True) -> int:
    """Rotate the packed new tokens' q and k and store their k and v in the cache.
    q, k and v may be parts of one fused projection (rows q_stride, ... apart);
    rope and q (with q_out) may be None."""
    st = lib.cobs_append_tokens(_dims(dims), cache, rope,
                                _rows_addr(q, q_stride, "q"), q_stride,
                                _rows_addr(k, k_stride, "k"), k_stride,
                                _rows_addr(v, v_stride, "v"), v_stride, _addr(cu_tokens),
                                n_tokens, _addr(start), _addr(q_out), _addr(ws), ws_bytes,
                                _stream(stream))
    return _check("cobs_append_tokens", st, check)


def cobs_read_cache(dims, cache, seq_lens, block_begin, block_end, k_out, v_out, ws, ws_bytes,
                    stream=None, check=True) -> int:
    """Blocks of a cache of either format as bf16 pages (seq_lens, k_out or v_out
    may be None)."""
    st = lib.cobs_read_cache(_dims(dims), cache, _addr(seq_lens),
                             block_begin, block_end, _addr(k_out), _addr(v_out), _addr(ws),
                             ws_bytes, _stream(stream))
    return _check("cobs_read_cache", st, check)


def cobs_prompt_workspace_bytes(dims, n_tokens, max_seq_len) -> int:
    n = lib.cobs_prompt_workspace_bytes(ctypes.byref(_dims(dims)), n_tokens, max_seq_len)
    if n == 0:
        raise CobsError("cobs_prompt_workspace_bytes", COBS_ERR_INVALID_ARG, cobs_last_error())
    return n


def cobs_prompt_attention(dims, cache, q, cu_tokens, n_tokens, seq_lens, max_seq_len,
                          softmax_scale, out, lse, ws, ws_bytes, stream=None,
                          check=True) -> int:
    """Causal attention of the packed new tokens over the bf16 cache that holds
    them (cu_tokens None: one token per sequence; lse may be None)."""
    st = lib.cobs_prompt_attention(_dims(dims), cache, _addr(q),
                                   _addr(cu_tokens), n_tokens, _addr(seq_lens), max_seq_len,
                                   softmax_scale, _addr(out), _addr(lse), _addr(ws), ws_bytes,
                                   _stream(stream))
    return _check("cobs_prompt_attention", st, check)


def cobs_sparse_decode_cache(dims, cache, q, idx, n_sel, idx_stride, seq_lens, max_seq_len,
                             softmax_scale, out, lse, ws, ws_bytes, stream=None,
                             check=True) -> int:
    """cobs_sparse_decode over a cache of either format, contiguous or paged
    (seq_lens None: every sequence is max_seq_len tokens long)."""
    st = lib.cobs_sparse_decode_cache(_dims(dims), cache, _addr(q),
                                      _addr(idx), _addr(n_sel), idx_stride, _addr(seq_lens),
                                      max_seq_len, softmax_scale, _addr(out), _addr(lse),
                                      _addr(ws), ws_bytes, _stream(stream))
    return _check("cobs_sparse_decode_cache", st, check)
