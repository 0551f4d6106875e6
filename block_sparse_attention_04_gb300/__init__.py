"""MiniMax Sparse Attention (MSA) forward on GB300: Python binding of libmsa.

Argument marshalling only.  Every step of the path runs in the CUDA kernels
of libmsa.so (include/msa.h); there is no fallback.  If the library is not
built, loading raises.  Tensors are torch CUDA tensors with 2-byte elements
(bf16, int16 or uint16 holding bf16 bit patterns) in the layouts msa.h
states (the codes and exponents of an 8-bit cache have 1-byte elements);
q_start and kv_len are host sequences of B ints, or positions() of one, which
saves the conversion on every call.
"""
import array
import ctypes
import math
import os

from . import _build

__all__ = ["MsaParams", "MsaError", "params", "load", "msa_workspace_bytes", "msa_index_topk",
           "msa_sparse_attn", "msa_forward", "msa_workspace_status", "msa_status_string",
           "msa_kernel_launch_count", "msa_index_topk_noalloc", "msa_debug_set_wait_polls",
           "msa_debug_delay_copies", "msa_quality_workspace_bytes", "msa_selection_quality",
           "quality_workspace",
           "msa_cache_append", "msa_forward_paged", "msa_dense_workspace_bytes",
           "msa_dense_attn", "dense_workspace", "msa_index_kl_workspace_bytes", "msa_index_kl",
           "kl_workspace", "msa_cache_append_q8", "msa_q8_workspace_bytes", "q8_workspace",
           "msa_sparse_attn_q8", "msa_forward_q8", "msa_window_workspace_bytes",
           "window_workspace", "msa_window_attn", "msa_window_attn_q8", "MsaPool", "pools",
           "msa_pages_workspace_bytes", "pages_workspace", "msa_pages_copy", "msa_pages_fork",
           "msa_pages_free", "msa_pages_alloc", "msa_pages_compact", "positions", "MsaRope",
           "rope", "yarn_mscale", "msa_rope_append", "msa_rope_append_bwd_workspace_bytes",
           "rope_append_bwd_workspace", "msa_rope_append_bwd", "msa_sparse_attn_lse",
           "msa_dense_attn_lse", "msa_sparse_bwd_workspace_bytes", "sparse_bwd_workspace",
           "msa_sparse_attn_bwd", "msa_dense_bwd_workspace_bytes", "dense_bwd_workspace",
           "msa_dense_attn_bwd", "workspace", "BLOCK", "TOPK", "MAX_ROT"]

BLOCK = 128
TOPK = 16
MAX_ROT = 128
KERNELS = {"auto": 0, "streaming": 1, "tensorcore": 2}
EXPORTS = ("msa_workspace_bytes", "msa_index_topk", "msa_sparse_attn", "msa_forward",
           "msa_workspace_status", "msa_status_string", "msa_kernel_launch_count",
           "msa_index_topk_noalloc", "msa_debug_set_wait_polls", "msa_debug_delay_copies",
           "msa_quality_workspace_bytes", "msa_selection_quality", "msa_cache_append",
           "msa_forward_paged",
           "msa_dense_workspace_bytes", "msa_dense_attn", "msa_index_kl_workspace_bytes",
           "msa_index_kl", "msa_cache_append_q8", "msa_q8_workspace_bytes",
           "msa_sparse_attn_q8", "msa_forward_q8", "msa_window_workspace_bytes",
           "msa_window_attn", "msa_window_attn_q8", "msa_pages_workspace_bytes",
           "msa_pages_copy", "msa_pages_fork", "msa_pages_free", "msa_pages_alloc",
           "msa_pages_compact", "msa_rope_append", "msa_rope_append_bwd_workspace_bytes",
           "msa_rope_append_bwd", "msa_sparse_attn_lse", "msa_dense_attn_lse",
           "msa_sparse_bwd_workspace_bytes", "msa_sparse_attn_bwd",
           "msa_dense_bwd_workspace_bytes", "msa_dense_attn_bwd")


class MsaError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (what, msa_status_string(status), status))


class MsaParams(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("G", ctypes.c_int), ("D", ctypes.c_int), ("Di", ctypes.c_int),
                ("block", ctypes.c_int), ("topk", ctypes.c_int), ("max_blocks", ctypes.c_int),
                ("scale", ctypes.c_float), ("kernels", ctypes.c_int)]


class MsaPool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_size_t),
                ("per_token", ctypes.c_int)]


class MsaRope(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int), ("interleaved", ctypes.c_int), ("eps", ctypes.c_float),
                ("mscale", ctypes.c_float), ("inv_freq", ctypes.c_double * (MAX_ROT // 2))]


def params(B, T, H, G, D, Di, max_blocks, scale=None, kernels="auto"):
    return MsaParams(B, T, H, G, D, Di, BLOCK, TOPK, max_blocks,
                     1.0 / math.sqrt(D) if scale is None else scale,
                     KERNELS[kernels] if isinstance(kernels, str) else int(kernels))


_lib = None


def load(path=None):
    """Load libmsa.so (built in-tree by _build.build()); raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or _build.LIBMSA
    if not os.path.exists(path):
        raise RuntimeError("libmsa.so is not built (%s); run __graft_entry__.build()" % path)
    L = ctypes.CDLL(path)
    P, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    PP = ctypes.POINTER(MsaParams)
    L.msa_workspace_bytes.argtypes = [PP]
    L.msa_workspace_bytes.restype = sz
    L.msa_index_topk.argtypes = [PP, P, P, P, P, P, P, sz, P]
    L.msa_sparse_attn.argtypes = [PP, P, P, P, P, P, P, P, P, sz, P]
    L.msa_forward.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, sz, P]
    L.msa_workspace_status.argtypes = [P, P]
    L.msa_index_topk_noalloc.argtypes = [PP, P, P, P, P, P, P]
    L.msa_cache_append.argtypes = [PP, P, ci, P, P, P, P, P, P, P, P, sz, P]
    L.msa_index_kl_workspace_bytes.argtypes = [PP]
    L.msa_index_kl_workspace_bytes.restype = sz
    L.msa_index_kl.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, P, sz, P]
    L.msa_dense_workspace_bytes.argtypes = [PP]
    L.msa_dense_workspace_bytes.restype = sz
    L.msa_dense_attn.argtypes = [PP, P, P, P, P, P, P, P, sz, P]
    L.msa_forward_paged.argtypes = [PP, P, ci, P, P, P, P, P, P, P, P, P, P, sz, P]
    L.msa_quality_workspace_bytes.argtypes = [PP]
    L.msa_quality_workspace_bytes.restype = sz
    L.msa_selection_quality.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, sz, P]
    pool = ctypes.POINTER(MsaPool)
    for name in ("msa_q8_workspace_bytes", "msa_window_workspace_bytes"):
        getattr(L, name).argtypes = [PP]
    L.msa_pages_workspace_bytes.argtypes = [ci]
    L.msa_cache_append_q8.argtypes = [PP, P, ci] + [P] * 10 + [sz, P]
    L.msa_sparse_attn_q8.argtypes = [PP, P, ci] + [P] * 10 + [sz, P]
    L.msa_forward_q8.argtypes = [PP, P, ci] + [P] * 12 + [sz, P]
    L.msa_window_attn.argtypes = [PP, P, ci, ci, ci] + [P] * 7 + [sz, P]
    L.msa_window_attn_q8.argtypes = [PP, P, ci, ci, ci] + [P] * 9 + [sz, P]
    L.msa_pages_copy.argtypes = [pool, ci, ci, P, P, ci, P, sz, P]
    L.msa_pages_fork.argtypes = [pool, ci, ci, P, ci, ci, P, P, P, P, ci, P, sz, P]
    for name in ("msa_pages_free", "msa_pages_alloc"):
        getattr(L, name).argtypes = [ci, P, ci, ci, P, P, P, P, ci, P, sz, P]
    L.msa_pages_compact.argtypes = [pool, ci, ci, P, ci, ci, P, P, P, P, P, sz, P]
    for name in ("msa_q8_workspace_bytes", "msa_window_workspace_bytes",
                 "msa_pages_workspace_bytes"):
        getattr(L, name).restype = sz
    RP, i64 = ctypes.POINTER(MsaRope), ctypes.c_int64
    L.msa_rope_append.argtypes = [PP, RP, P, ci, P, P, P, i64, i64, i64] + [P] * 9 + [sz, P]
    L.msa_rope_append_bwd.argtypes = ([PP, RP, P, P, i64, i64] + [P] * 9 + [i64, i64, i64] +
                                      [P] * 3 + [sz, P])
    L.msa_sparse_attn_lse.argtypes = [PP] + [P] * 9 + [sz, P]
    L.msa_dense_attn_lse.argtypes = [PP] + [P] * 8 + [sz, P]
    L.msa_sparse_attn_bwd.argtypes = [PP] + [P] * 13 + [sz, P]
    L.msa_dense_attn_bwd.argtypes = [PP] + [P] * 12 + [sz, P]
    for name in ("msa_rope_append_bwd_workspace_bytes", "msa_sparse_bwd_workspace_bytes",
                 "msa_dense_bwd_workspace_bytes"):
        getattr(L, name).argtypes = [PP]
        getattr(L, name).restype = sz
    L.msa_debug_set_wait_polls.argtypes = [ctypes.c_uint32]
    L.msa_debug_set_wait_polls.restype = None
    L.msa_debug_delay_copies.argtypes = [ci, ci, ctypes.c_uint32]
    L.msa_debug_delay_copies.restype = None
    L.msa_kernel_launch_count.argtypes = []
    L.msa_kernel_launch_count.restype = ctypes.c_uint64
    L.msa_status_string.argtypes = [ci]
    L.msa_status_string.restype = ctypes.c_char_p
    for f in ("msa_index_topk", "msa_sparse_attn", "msa_forward", "msa_workspace_status",
              "msa_index_topk_noalloc", "msa_selection_quality", "msa_cache_append",
              "msa_forward_paged", "msa_dense_attn", "msa_index_kl", "msa_cache_append_q8",
              "msa_sparse_attn_q8", "msa_forward_q8", "msa_window_attn", "msa_window_attn_q8",
              "msa_pages_copy", "msa_pages_fork", "msa_pages_free", "msa_pages_alloc",
              "msa_pages_compact", "msa_rope_append", "msa_rope_append_bwd", "msa_sparse_attn_lse",
              "msa_dense_attn_lse", "msa_sparse_attn_bwd", "msa_dense_attn_bwd"):
        getattr(L, f).restype = ci
    if path == _build.LIBMSA:
        _lib = L
    return L


def msa_status_string(status):
    return load().msa_status_string(int(status)).decode()


def _ptr(t):
    # the argument types are c_void_p, which takes None and plain ints
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _stream_getter():
    """A function that returns the handle of torch's current stream: the call
    that gives the bare handle where torch has it (0.1 us; a Stream object costs
    3 us, as much as a launch)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    device = torch.cuda.current_device
    return lambda: raw(device())


_current_stream = None


def _stream(stream):
    global _current_stream
    if stream is None:
        if _current_stream is None:
            _current_stream = _stream_getter()
        return _current_stream()
    return getattr(stream, "cuda_stream", stream)


def _int32s(x):
    try:
        if type(x) in (list, tuple) and x:
            try:
                a = array.array("i", x)         # a third of the time of the general form
                return (ctypes.c_int32 * len(a)).from_buffer(a)
            except TypeError:
                pass                            # floats
        x = [int(v) for v in x]
        return (ctypes.c_int32 * len(x))(*array.array("i", x))
    except OverflowError:                       # ctypes alone would wrap it
        raise ValueError("a position, length or row number does not fit 32 bits") from None


def _tokens(n):
    """A count of tokens as the C ABI takes it: past its ends, the end (a window
    longer than any context, or one that the library refuses)."""
    return max(-1, min(int(n), 0x7FFFFFFF))


def positions(x):
    """A host array of ints (positions, lengths, row numbers) in the form that
    the library reads; every call also takes it in place of a sequence."""
    return _int32s(list(x))


def _host_i32(x, B):
    if isinstance(x, ctypes.Array) and x._type_ is ctypes.c_int32:
        if len(x) != B:
            raise ValueError("expected %d positions, got %d" % (B, len(x)))
        return x
    x = x if hasattr(x, "__len__") else [x] * B
    if len(x) != B:
        raise ValueError("expected %d positions, got %d" % (B, len(x)))
    return _int32s(x)


def msa_kernel_launch_count():
    return int(load().msa_kernel_launch_count())


def msa_debug_set_wait_polls(polls):
    """Test-only: cap the tensor-core kernels' pipeline waits at `polls` polls
    (0 restores the default wall-clock bound)."""
    load().msa_debug_set_wait_polls(int(polls))


def msa_debug_delay_copies(kind, at, us):
    """Test-only: the backward attention's CTAs of one kind (1: KV-outer, 2: dQ) wait `us`
    microseconds before their K and V copy number `at` (us 0: none; see msa.h)."""
    load().msa_debug_delay_copies(int(kind), int(at), int(us))


def msa_workspace_bytes(p):
    return int(load().msa_workspace_bytes(ctypes.byref(p)))


def workspace(p, device="cuda"):
    """A device scratch buffer of msa_workspace_bytes(p) bytes."""
    import torch
    n = msa_workspace_bytes(p)
    if n == 0:
        raise MsaError(-2, "msa_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _call(rc, what):
    if rc != 0:
        raise MsaError(rc, what)


def msa_index_topk(p, q_idx, k_idx, q_start, kv_len, sel, ws, stream=None):
    _call(load().msa_index_topk(ctypes.byref(p), _ptr(q_idx), _ptr(k_idx),
                                _host_i32(q_start, p.B), _host_i32(kv_len, p.B), _ptr(sel),
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
          "msa_index_topk")


def msa_index_topk_noalloc(p, q_idx, k_idx, q_start, kv_len, sel, stream=None):
    """msa_index_topk without a workspace: for callers that cannot allocate
    device memory (scratch lives in a static array inside the library)."""
    _call(load().msa_index_topk_noalloc(ctypes.byref(p), _ptr(q_idx), _ptr(k_idx),
                                        _host_i32(q_start, p.B), _host_i32(kv_len, p.B),
                                        _ptr(sel), _stream(stream)), "msa_index_topk_noalloc")


def msa_sparse_attn(p, q, k_cache, v_cache, sel, q_start, kv_len, out, ws, stream=None):
    _call(load().msa_sparse_attn(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(sel), _host_i32(q_start, p.B), _host_i32(kv_len, p.B),
                                 _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                 _stream(stream)), "msa_sparse_attn")


def msa_forward(p, q_idx, k_idx, q, k_cache, v_cache, q_start, kv_len, out, ws, sel_out=None,
                stream=None):
    _call(load().msa_forward(ctypes.byref(p), _ptr(q_idx), _ptr(k_idx), _ptr(q), _ptr(k_cache),
                             _ptr(v_cache), _host_i32(q_start, p.B), _host_i32(kv_len, p.B),
                             _ptr(sel_out), _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                             _stream(stream)), "msa_forward")


def msa_index_kl_workspace_bytes(p):
    return int(load().msa_index_kl_workspace_bytes(ctypes.byref(p)))


def kl_workspace(p, device="cuda"):
    """A device scratch buffer of msa_index_kl_workspace_bytes(p) bytes."""
    import torch
    n = msa_index_kl_workspace_bytes(p)
    if n == 0:
        raise MsaError(-2, "msa_index_kl_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def msa_index_kl(p, q_idx, k_idx, q, k_cache, sel, q_start, kv_len, kl, dq_idx, dk_idx, ws,
                 stream=None):
    """KL(P||Q) of the index branch per (query, group), dQ_idx, and dK_idx
    accumulated into (see msa.h)."""
    _call(load().msa_index_kl(ctypes.byref(p), _ptr(q_idx), _ptr(k_idx), _ptr(q), _ptr(k_cache),
                              _ptr(sel), _host_i32(q_start, p.B), _host_i32(kv_len, p.B),
                              _ptr(kl), _ptr(dq_idx), _ptr(dk_idx), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)), "msa_index_kl")


def msa_dense_workspace_bytes(p):
    return int(load().msa_dense_workspace_bytes(ctypes.byref(p)))


def dense_workspace(p, device="cuda"):
    """A device scratch buffer of msa_dense_workspace_bytes(p) bytes."""
    import torch
    n = msa_dense_workspace_bytes(p)
    if n == 0:
        raise MsaError(-2, "msa_dense_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def msa_dense_attn(p, q, k_cache, v_cache, q_start, kv_len, out, ws, stream=None):
    """Dense causal GQA attention over every token <= t (see msa.h)."""
    _call(load().msa_dense_attn(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                _host_i32(q_start, p.B), _host_i32(kv_len, p.B), _ptr(out),
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
          "msa_dense_attn")


def msa_quality_workspace_bytes(p):
    return int(load().msa_quality_workspace_bytes(ctypes.byref(p)))


def quality_workspace(p, device="cuda"):
    """A device scratch buffer of msa_quality_workspace_bytes(p) bytes."""
    import torch
    n = msa_quality_workspace_bytes(p)
    if n == 0:
        raise MsaError(-2, "msa_quality_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def msa_selection_quality(p, q, k_cache, sel, q_start, kv_len, coverage, best_coverage,
                          dense_sel, hits, ws, stream=None):
    """Attention-mass coverage of sel and of the ideal selection, the ideal
    selection itself and the recall hits (see msa.h)."""
    _call(load().msa_selection_quality(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(sel),
                                       _host_i32(q_start, p.B), _host_i32(kv_len, p.B),
                                       _ptr(coverage), _ptr(best_coverage), _ptr(dense_sel),
                                       _ptr(hits), _ptr(ws), ws.numel() * ws.element_size(),
                                       _stream(stream)), "msa_selection_quality")


def msa_cache_append(p, k_new, v_new, k_idx_new, q_start, k_cache, v_cache, k_idx_cache, ws,
                     block_table=None, num_pool_blocks=0, stream=None):
    """Write p.T new tokens per sequence at positions q_start[b] + i, through
    block_table when the caches are pools (see msa.h)."""
    _call(load().msa_cache_append(ctypes.byref(p), _ptr(block_table), int(num_pool_blocks),
                                  _ptr(k_new), _ptr(v_new), _ptr(k_idx_new),
                                  _host_i32(q_start, p.B), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(k_idx_cache), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)), "msa_cache_append")


def msa_forward_paged(p, block_table, num_pool_blocks, q_idx, k_idx_pool, q, k_pool, v_pool,
                      q_start, kv_len, out, ws, sel_out=None, stream=None):
    _call(load().msa_forward_paged(ctypes.byref(p), _ptr(block_table), int(num_pool_blocks),
                                   _ptr(q_idx), _ptr(k_idx_pool), _ptr(q), _ptr(k_pool),
                                   _ptr(v_pool), _host_i32(q_start, p.B), _host_i32(kv_len, p.B),
                                   _ptr(sel_out), _ptr(out), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)),
          "msa_forward_paged")


def _scratch(n, what, device):
    import torch
    if n == 0:
        raise MsaError(-2, what)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _nbytes(ws):
    return ws.nbytes


def msa_q8_workspace_bytes(p):
    return int(load().msa_q8_workspace_bytes(ctypes.byref(p)))


def q8_workspace(p, device="cuda"):
    """A device scratch buffer of msa_q8_workspace_bytes(p) bytes."""
    return _scratch(msa_q8_workspace_bytes(p), "msa_q8_workspace_bytes", device)


def msa_cache_append_q8(p, k_new, v_new, k_idx_new, q_start, k_cache, v_cache, k_exp, v_exp,
                        k_idx_cache, ws, block_table=None, num_pool_blocks=0, stream=None):
    """msa_cache_append into an 8-bit cache: e4m3 codes and one exponent per
    (block, KV head), see msa.h."""
    _call(load().msa_cache_append_q8(ctypes.byref(p), _ptr(block_table), int(num_pool_blocks),
                                     _ptr(k_new), _ptr(v_new), _ptr(k_idx_new),
                                     _host_i32(q_start, p.B), _ptr(k_cache), _ptr(v_cache),
                                     _ptr(k_exp), _ptr(v_exp), _ptr(k_idx_cache), _ptr(ws),
                                     _nbytes(ws), _stream(stream)), "msa_cache_append_q8")


def msa_sparse_attn_q8(p, q, k_cache, v_cache, k_exp, v_exp, sel, q_start, kv_len, out, ws,
                       block_table=None, num_pool_blocks=0, stream=None):
    """msa_sparse_attn on an 8-bit cache (see msa.h)."""
    _call(load().msa_sparse_attn_q8(ctypes.byref(p), _ptr(block_table), int(num_pool_blocks),
                                    _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_exp),
                                    _ptr(v_exp), _ptr(sel), _host_i32(q_start, p.B),
                                    _host_i32(kv_len, p.B), _ptr(out), _ptr(ws), _nbytes(ws),
                                    _stream(stream)), "msa_sparse_attn_q8")


def msa_forward_q8(p, q_idx, k_idx, q, k_cache, v_cache, k_exp, v_exp, q_start, kv_len, out, ws,
                   sel_out=None, block_table=None, num_pool_blocks=0, stream=None):
    """msa_forward on an 8-bit cache (see msa.h)."""
    _call(load().msa_forward_q8(ctypes.byref(p), _ptr(block_table), int(num_pool_blocks),
                                _ptr(q_idx), _ptr(k_idx), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                _ptr(k_exp), _ptr(v_exp), _host_i32(q_start, p.B),
                                _host_i32(kv_len, p.B), _ptr(sel_out), _ptr(out), _ptr(ws),
                                _nbytes(ws), _stream(stream)), "msa_forward_q8")


def msa_window_workspace_bytes(p):
    return int(load().msa_window_workspace_bytes(ctypes.byref(p)))


def window_workspace(p, device="cuda"):
    """A device scratch buffer of msa_window_workspace_bytes(p) bytes."""
    return _scratch(msa_window_workspace_bytes(p), "msa_window_workspace_bytes", device)


def msa_window_attn(p, window, sinks, q, k_cache, v_cache, q_start, kv_len, out, ws,
                    block_table=None, num_pool_blocks=0, stream=None):
    """GQA attention over the last `window` and the first `sinks` tokens (see msa.h)."""
    _call(load().msa_window_attn(ctypes.byref(p), _ptr(block_table), int(num_pool_blocks),
                                 _tokens(window), _tokens(sinks), _ptr(q), _ptr(k_cache),
                                 _ptr(v_cache), _host_i32(q_start, p.B), _host_i32(kv_len, p.B),
                                 _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)),
          "msa_window_attn")


def msa_window_attn_q8(p, window, sinks, q, k_cache, v_cache, k_exp, v_exp, q_start, kv_len, out,
                       ws, block_table=None, num_pool_blocks=0, stream=None):
    """msa_window_attn on an 8-bit cache (see msa.h)."""
    _call(load().msa_window_attn_q8(ctypes.byref(p), _ptr(block_table), int(num_pool_blocks),
                                    _tokens(window), _tokens(sinks), _ptr(q), _ptr(k_cache),
                                    _ptr(v_cache), _ptr(k_exp), _ptr(v_exp),
                                    _host_i32(q_start, p.B), _host_i32(kv_len, p.B), _ptr(out),
                                    _ptr(ws), _nbytes(ws), _stream(stream)), "msa_window_attn_q8")


def pools(tensors):
    """The pools that move together in a page operation.  Each is a contiguous
    tensor [pages][...]; one of shape [pages][128][...] holds token rows.  Keep
    the tensors alive as long as the result is used."""
    a = (MsaPool * len(tensors))()
    for d, t in zip(a, tensors):
        if not t.is_contiguous():
            raise ValueError("a pool must be contiguous")
        d.base = t.data_ptr()
        d.page_bytes = t[0].numel() * t.element_size()
        d.per_token = int(t.dim() > 2 and t.shape[1] == BLOCK)
    return a


def msa_pages_workspace_bytes(num_pool_blocks):
    return int(load().msa_pages_workspace_bytes(int(num_pool_blocks)))


def pages_workspace(num_pool_blocks, device="cuda"):
    """A device scratch buffer of msa_pages_workspace_bytes(num_pool_blocks) bytes."""
    return _scratch(msa_pages_workspace_bytes(num_pool_blocks), "msa_pages_workspace_bytes", device)


def msa_pages_copy(pools, num_pool_blocks, src, dst, ws, stream=None):
    """Page dst[i] of every pool becomes a copy of page src[i] (device int32 lists)."""
    if dst.numel() != src.numel():
        raise ValueError("expected %d destination pages, got %d" % (src.numel(), dst.numel()))
    _call(load().msa_pages_copy(pools, len(pools), int(num_pool_blocks), _ptr(src), _ptr(dst),
                                src.numel(), _ptr(ws), _nbytes(ws), _stream(stream)),
          "msa_pages_copy")


def msa_pages_fork(pools, num_pool_blocks, block_table, refs, src_rows, dst_rows, lens, ws,
                   stream=None):
    """Rows dst_rows take the first lens tokens of rows src_rows: complete pages
    shared, the last one copied (see msa.h)."""
    n = len(src_rows)
    _call(load().msa_pages_fork(pools, len(pools), int(num_pool_blocks), _ptr(block_table),
                                block_table.shape[0], block_table.shape[1], _ptr(refs),
                                _host_i32(src_rows, n), _host_i32(dst_rows, n),
                                _host_i32(lens, n), n, _ptr(ws), _nbytes(ws), _stream(stream)),
          "msa_pages_fork")


def _ranges(fn, what, num_pool_blocks, block_table, refs, rows, first, last, ws, stream):
    n = len(rows)
    _call(fn(int(num_pool_blocks), _ptr(block_table), block_table.shape[0], block_table.shape[1],
             _ptr(refs), _host_i32(rows, n), _host_i32(first, n), _host_i32(last, n), n, _ptr(ws),
             _nbytes(ws), _stream(stream)), what)


def msa_pages_free(num_pool_blocks, block_table, refs, rows, first, last, ws, stream=None):
    """Unmap blocks [first[j], last[j]) of row rows[j] (see msa.h)."""
    _ranges(load().msa_pages_free, "msa_pages_free", num_pool_blocks, block_table, refs, rows,
            first, last, ws, stream)


def msa_pages_alloc(num_pool_blocks, block_table, refs, rows, first, last, ws, stream=None):
    """Map the unmapped blocks of [first[j], last[j]) of row rows[j] to the lowest
    free pages (see msa.h)."""
    _ranges(load().msa_pages_alloc, "msa_pages_alloc", num_pool_blocks, block_table, refs, rows,
            first, last, ws, stream)


def msa_pages_compact(pools, num_pool_blocks, block_table, refs, table_out, refs_out, live, ws,
                      stream=None):
    """Move the pages in use to the front of the pools (see msa.h)."""
    if table_out.shape != block_table.shape or refs_out.numel() != refs.numel():
        raise ValueError("table_out and refs_out must have the shapes of block_table and refs")
    _call(load().msa_pages_compact(pools, len(pools), int(num_pool_blocks), _ptr(block_table),
                                   block_table.shape[0], block_table.shape[1], _ptr(refs),
                                   _ptr(table_out), _ptr(refs_out), _ptr(live), _ptr(ws),
                                   _nbytes(ws), _stream(stream)), "msa_pages_compact")


def rope(rot, base=10000.0, interleaved=False, eps=1e-6, linear=1.0, yarn=None, mscale=1.0):
    """How positions rotate the first `rot` dims of every head (the library's calls take
    multiples of 16), and the norm's eps (see msa.h).  Frequencies base^(-2i/rot) /
    linear, the position divided by `linear`.  yarn=(factor, trained_length[, beta_fast,
    beta_slow]): each frequency between itself and its `factor`-th part by how often it
    turns within the trained length (all of itself from beta_fast turns on, 32; the part
    below beta_slow, 1); the usual factor of cos and sin goes with it as mscale=yarn_mscale(factor)."""
    if not 0 <= rot <= MAX_ROT or rot % 2:
        raise ValueError("rot must be even and in 0 .. %d" % MAX_ROT)
    f = [base ** (-2.0 * i / rot) / linear for i in range(rot // 2)]
    if yarn is not None:
        factor, trained, fast, slow = (tuple(yarn) + (32.0, 1.0)[len(yarn) - 2:])

        def dim(turns):        # the pair (a fraction) that turns so often in `trained`
            return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(dim(fast)), 0), min(math.ceil(dim(slow)), rot - 1)
        for i, x in enumerate(f):
            part = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f[i] = x * (1 - part) + x / factor * part
    r = MsaRope(rot, int(bool(interleaved)), eps, mscale)
    r.inv_freq[:len(f)] = f
    return r


def yarn_mscale(factor):
    return 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _no_row_ptr(t):
    """The address of an array of the tokens of a call without any: torch gives a tensor
    without elements none, and the library, which asks for one, reads nothing there."""
    a = _ptr(t)
    return a if a != 0 or type(t) is int else 256


def _row_stride(t, p, heads, what):
    """Elements between consecutive tokens of [B][T][heads][D] (a plain address: the
    row itself)."""
    if t is None or type(t) is int:
        return heads * p.D
    B, T, D = p.B, p.T, p.D
    try:
        shape, st = t.shape, t.stride()
    except AttributeError:
        return heads * D
    if shape == (B, T, heads, D):
        ok = heads == 1 or st[2] == D
    elif shape == (B, T, heads * D):
        ok = True
    else:
        raise ValueError("%s must be [B][T][%d][%d], got %s" % (what, heads, D, tuple(shape)))
    if T == 0:
        return heads * D
    step = st[1] if T > 1 else st[0] if B > 1 else heads * D
    if not ok or st[-1] != 1 or (B > 1 and st[0] != T * step):
        raise ValueError("%s: the rows of a token must be contiguous and the tokens evenly "
                         "spaced" % what)
    return step


def msa_rope_append(p, r, q, k, v, k_idx_new, q_weight, k_weight, q_start, q_out, k_cache, v_cache,
                    k_idx_cache, ws, block_table=None, num_pool_blocks=0, stream=None):
    """Norm and rotation of q and k, and the rows of K, V and K_idx into the caches
    (see msa.h).  q, k and v may be parts of one tensor; the weights and k_idx_new
    (with k_idx_cache) may be None."""
    row = _ptr if p.T else _no_row_ptr
    _call(load().msa_rope_append(ctypes.byref(p), ctypes.byref(r), _ptr(block_table),
                                 int(num_pool_blocks), row(q), row(k), row(v),
                                 _row_stride(q, p, p.H, "q"), _row_stride(k, p, p.G, "k"),
                                 _row_stride(v, p, p.G, "v"), _ptr(q_weight), _ptr(k_weight),
                                 row(k_idx_new), _host_i32(q_start, p.B), row(q_out),
                                 _ptr(k_cache), _ptr(v_cache), _ptr(k_idx_cache), _ptr(ws),
                                 _nbytes(ws), _stream(stream)), "msa_rope_append")


def msa_rope_append_bwd_workspace_bytes(p):
    return int(load().msa_rope_append_bwd_workspace_bytes(ctypes.byref(p)))


def rope_append_bwd_workspace(p, device="cuda"):
    """A device scratch buffer of msa_rope_append_bwd_workspace_bytes(p) bytes."""
    return _scratch(msa_rope_append_bwd_workspace_bytes(p), "msa_rope_append_bwd_workspace_bytes",
                    device)


def msa_rope_append_bwd(p, r, q, k, q_weight, k_weight, q_start, dq_out, dk_cache, dv_cache, dq, dk,
                        dv, dq_weight, dk_weight, ws, stream=None):
    """From the gradients of q_out and of the caches to those of the projections and of
    the norms' weights (see msa.h)."""
    row = _ptr if p.T else _no_row_ptr
    _call(load().msa_rope_append_bwd(ctypes.byref(p), ctypes.byref(r), row(q), row(k),
                                     _row_stride(q, p, p.H, "q"), _row_stride(k, p, p.G, "k"),
                                     _ptr(q_weight), _ptr(k_weight), _host_i32(q_start, p.B),
                                     row(dq_out), _ptr(dk_cache), _ptr(dv_cache), row(dq), row(dk),
                                     row(dv), _row_stride(dq, p, p.H, "dq"),
                                     _row_stride(dk, p, p.G, "dk"), _row_stride(dv, p, p.G, "dv"),
                                     _ptr(dq_weight), _ptr(dk_weight), _ptr(ws), _nbytes(ws),
                                     _stream(stream)), "msa_rope_append_bwd")


def msa_sparse_attn_lse(p, q, k_cache, v_cache, sel, q_start, kv_len, out, lse, ws, stream=None):
    """msa_sparse_attn that also writes lse [B][T][H] (see msa.h)."""
    row = _ptr if p.T else _no_row_ptr
    _call(load().msa_sparse_attn_lse(ctypes.byref(p), row(q), _ptr(k_cache), _ptr(v_cache),
                                     row(sel), _host_i32(q_start, p.B), _host_i32(kv_len, p.B),
                                     row(out), row(lse), _ptr(ws), _nbytes(ws), _stream(stream)),
          "msa_sparse_attn_lse")


def msa_dense_attn_lse(p, q, k_cache, v_cache, q_start, kv_len, out, lse, ws, stream=None):
    """msa_dense_attn that also writes lse [B][T][H] (see msa.h)."""
    row = _ptr if p.T else _no_row_ptr
    _call(load().msa_dense_attn_lse(ctypes.byref(p), row(q), _ptr(k_cache), _ptr(v_cache),
                                    _host_i32(q_start, p.B), _host_i32(kv_len, p.B), row(out),
                                    row(lse), _ptr(ws), _nbytes(ws), _stream(stream)),
          "msa_dense_attn_lse")


def msa_sparse_bwd_workspace_bytes(p):
    return int(load().msa_sparse_bwd_workspace_bytes(ctypes.byref(p)))


def sparse_bwd_workspace(p, device="cuda"):
    """A device scratch buffer of msa_sparse_bwd_workspace_bytes(p) bytes."""
    return _scratch(msa_sparse_bwd_workspace_bytes(p), "msa_sparse_bwd_workspace_bytes", device)


def msa_sparse_attn_bwd(p, q, k_cache, v_cache, sel, out, lse, dout, q_start, kv_len, dq, dk, dv, ws,
                        stream=None):
    """dq, and the rows of dk and dv in the caches' layout, of msa_sparse_attn (see msa.h)."""
    row = _ptr if p.T else _no_row_ptr
    _call(load().msa_sparse_attn_bwd(ctypes.byref(p), row(q), _ptr(k_cache), _ptr(v_cache),
                                     row(sel), row(out), row(lse), row(dout),
                                     _host_i32(q_start, p.B), _host_i32(kv_len, p.B), row(dq),
                                     _ptr(dk), _ptr(dv), _ptr(ws), _nbytes(ws), _stream(stream)),
          "msa_sparse_attn_bwd")


def msa_dense_bwd_workspace_bytes(p):
    return int(load().msa_dense_bwd_workspace_bytes(ctypes.byref(p)))


def dense_bwd_workspace(p, device="cuda"):
    """A device scratch buffer of msa_dense_bwd_workspace_bytes(p) bytes."""
    return _scratch(msa_dense_bwd_workspace_bytes(p), "msa_dense_bwd_workspace_bytes", device)


def msa_dense_attn_bwd(p, q, k_cache, v_cache, out, lse, dout, q_start, kv_len, dq, dk, dv, ws,
                       stream=None):
    """dq, and the rows of dk and dv in the caches' layout, of msa_dense_attn (see msa.h)."""
    row = _ptr if p.T else _no_row_ptr
    _call(load().msa_dense_attn_bwd(ctypes.byref(p), row(q), _ptr(k_cache), _ptr(v_cache), row(out),
                                    row(lse), row(dout), _host_i32(q_start, p.B),
                                    _host_i32(kv_len, p.B), row(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                                    _nbytes(ws), _stream(stream)), "msa_dense_attn_bwd")


def msa_workspace_status(ws, stream=None):
    """Waits for the stream; raises MsaError if a kernel recorded an error in ws."""
    _call(load().msa_workspace_status(_ptr(ws), _stream(stream)), "kernel status")
