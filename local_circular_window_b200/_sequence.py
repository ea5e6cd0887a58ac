"""ctypes binding of the token-sequence operators of libclear_attn.so: appending to a paged key/value
cache with the rotary embedding, attention of one new token over that cache, and causal attention over
packed prompts with its gradient (argument marshalling only; see include/clear_attn.h).

Tensors are [heads, tokens, d] views with contiguous rows, e.g. ``x.view(tokens, heads, d).transpose(0, 1)``
of a projection's output. All tensors of a call lie on one CUDA device; the call runs on that device,
on ``stream`` or its current stream.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._binding import CLEAR_OK, ClearError, _lib

_ll, _i, _vp = ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}  # CLEAR_DTYPE_*
_PAIRINGS = {"adjacent": 0, "halves": 1}  # CLEAR_PAIR_*


class ClearSeqParams(ctypes.Structure):
    """Mirror of clear_seq_params_t."""
    _fields_ = [("n_seq", _i), ("n_tok", _i), ("q_heads", _i), ("kv_heads", _i), ("d", _i), ("dtype", _i)]


class ClearSeqView(ctypes.Structure):
    """Mirror of clear_seq_view_t."""
    _fields_ = [("ptr", _vp), ("head_stride", _ll), ("token_stride", _ll)]


class ClearSeqCache(ctypes.Structure):
    """Mirror of clear_seq_cache_t."""
    _fields_ = [("k_pages", _vp), ("v_pages", _vp), ("page_table", _vp), ("k_scale", _vp), ("v_scale", _vp),
                ("k_strides", _ll * 3), ("v_strides", _ll * 3), ("page_table_stride", _ll), ("n_pages", _i),
                ("page_size", _i), ("max_pages", _i), ("dtype", _i)]


class ClearSeqRope(ctypes.Structure):
    """Mirror of clear_seq_rope_t."""
    _fields_ = [("theta", ctypes.c_float), ("ntk", ctypes.c_float), ("rot", _i), ("pairing", _i)]


_PP, _PV, _PC = ctypes.POINTER(ClearSeqParams), ctypes.POINTER(ClearSeqView), ctypes.POINTER(ClearSeqCache)
_lib.clear_attn_cache_append.restype = _i
_lib.clear_attn_cache_append.argtypes = [_PP, _PC, ctypes.POINTER(ClearSeqRope), _vp, _vp, _PV, _PV, _PV, _PV, _PV, _vp]
_lib.clear_attn_decode_workspace_size.restype = ctypes.c_size_t
_lib.clear_attn_decode_workspace_size.argtypes = [_PP, ctypes.POINTER(_i)]
_lib.clear_attn_decode.restype = _i
_lib.clear_attn_decode.argtypes = [_PP, _PC, _vp, _PV, _PV, _vp, _vp, ctypes.c_size_t, _vp]
_lib.clear_attn_prompt_fwd.restype = _i
_lib.clear_attn_prompt_fwd.argtypes = [_PP, _vp, _PV, _PV, _PV, _PV, _vp, _vp]

_lib.clear_attn_prompt_bwd_workspace_size.restype = ctypes.c_size_t
_lib.clear_attn_prompt_bwd_workspace_size.argtypes = [_PP, ctypes.POINTER(_i)]
_lib.clear_attn_prompt_bwd.restype = _i
_lib.clear_attn_prompt_bwd.argtypes = [_PP, _vp, _PV, _PV, _PV, _PV, _vp, _PV, _PV, _PV, _PV, _vp, ctypes.c_size_t, _vp]


def _view(t):
    s = t.stride()
    return ClearSeqView(t.data_ptr(), s[0], s[1])


def _require(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or t.device != device or t.stride(-1) != 1:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} with contiguous rows on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _require_dense(name, t, shape, dtype, device):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _queries(name, q):
    if q.dim() != 3 or q.dtype not in (torch.bfloat16, torch.float16) or not q.is_cuda or q.stride(2) != 1:
        raise ValueError(f"{name} must be a CUDA bf16 or fp16 tensor [heads, tokens, d] with contiguous rows")


@contextlib.contextmanager
def _elsewhere(device, stream):
    """Makes the tensors' device and the given stream current, so that outputs and workspaces allocated in the
    call belong to the stream that uses them."""
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _run(device, stream, body):
    """body(the stream's handle), with the right device and stream current."""
    if stream is None and device.index == torch.cuda.current_device():
        return body(torch.cuda.current_stream(device).cuda_stream)
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream lies on {stream.device}, the tensors on {device}")
    with _elsewhere(device, stream) as handle:
        return body(handle)


def _workspace(workspace, size, device):
    if workspace is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def _cache(k_pages, v_pages, page_table, k_scale, v_scale, kv_heads, d, dtype, device):
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
        raise ValueError("k_pages and v_pages must have one shape [pages, page_size, kv_heads, d] and one dtype")
    n_pages, page_size = k_pages.shape[:2]
    if k_pages.shape[2] != kv_heads or k_pages.shape[3] != d:
        raise ValueError(f"the pages hold {tuple(k_pages.shape[2:])} heads and elements, not {(kv_heads, d)}")
    if k_pages.dtype != dtype and k_pages.dtype != torch.float8_e4m3fn:
        raise ValueError(f"pages must be {dtype} or float8_e4m3fn")
    if k_pages.stride(3) != 1 or v_pages.stride(3) != 1 or k_pages.device != device or v_pages.device != device:
        raise ValueError(f"pages must have contiguous rows and lie on {device}")
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.device != device or (
            page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError(f"page_table must be int32 [sequences, pages] with contiguous rows on {device}")
    ks = vs = None
    if k_pages.dtype == torch.float8_e4m3fn:
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is None:
                raise ValueError(f"an E4M3 cache needs {name}")
            _require_dense(name, s, (kv_heads,), torch.float32, device)
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales belong to an E4M3 cache")
    a, b = k_pages.stride(), v_pages.stride()
    return ClearSeqCache(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), ks, vs, (_ll * 3)(a[0], a[1], a[2]),
                         (_ll * 3)(b[0], b[1], b[2]), page_table.stride(0), n_pages, page_size, page_table.shape[1],
                         _DTYPES[k_pages.dtype])


def clear_attn_cache_append(k, v, k_pages, v_pages, page_table, seq_start, seq_len, q=None, q_out=None, k_out=None, rot=0,
                            theta: float = 10000.0, ntk: float = 1.0, pairing="adjacent", k_scale=None, v_scale=None,
                            stream=None):
    """Appends the packed tokens' keys and values ([kv_heads, n_tok, d]) to the paged cache, rotating the first
    ``rot`` elements of each query and key head by the token's position on the way.

    seq_start: int32 [n_seq + 1], where each sequence's new tokens begin; seq_len: int32 [n_seq], its
    length in the cache after the call. pairing: "adjacent" (elements 2i and 2i + 1 turn together) or "halves"
    (i and i + rot / 2). k_pages and v_pages: [pages, page_size, kv_heads, d], of k's dtype or float8_e4m3fn
    with k_scale and v_scale [kv_heads]; page_table: int32 [n_seq, pages of a sequence]. q_out and k_out may be q and k
    (in place); q_out defaults to a new tensor where q is given. Returns (q_out, k_out)."""
    _queries("k", k)
    device, dtype = k.device, k.dtype
    kv_heads, n_tok, d = k.shape
    _require("v", v, k.shape, dtype, device)
    if q is None and q_out is not None:
        raise ValueError("q_out needs q")
    if q is not None:
        _queries("q", q)
        _require("q", q, (q.shape[0], n_tok, d), dtype, device)
    n_seq = page_table.shape[0]
    _require_dense("seq_start", seq_start, (n_seq + 1,), torch.int32, device)
    _require_dense("seq_len", seq_len, (n_seq,), torch.int32, device)
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {sorted(_PAIRINGS)}")
    cache = _cache(k_pages, v_pages, page_table, k_scale, v_scale, kv_heads, d, dtype, device)
    params = ClearSeqParams(n_seq, n_tok, q.shape[0] if q is not None else kv_heads, kv_heads, d, _DTYPES[dtype])
    rope = ClearSeqRope(theta, ntk, rot, _PAIRINGS[pairing])

    def body(handle):
        qo = torch.empty_like(q) if q is not None and q_out is None else q_out
        if qo is not None:
            _require("q_out", qo, q.shape, dtype, device)
        if k_out is not None:
            _require("k_out", k_out, k.shape, dtype, device)
        st = _lib.clear_attn_cache_append(params, cache, rope, seq_start.data_ptr(), seq_len.data_ptr(),
                                          None if q is None else _view(q), _view(k), _view(v),
                                          None if q is None else _view(qo), None if k_out is None else _view(k_out), handle)
        if st != CLEAR_OK:
            raise ClearError(st, "clear_attn_cache_append")
        return qo, k_out

    return _run(device, stream, body)


def _size(function, params):
    st = _i(0)
    n = function(params, ctypes.byref(st))
    if st.value != CLEAR_OK:
        raise ClearError(st.value, "the workspace size")
    return n


def decode_workspace_size(n_seq: int, q_heads: int, kv_heads: int, d: int) -> int:
    """Bytes of clear_attn_decode's workspace."""
    return _size(_lib.clear_attn_decode_workspace_size, ClearSeqParams(n_seq, n_seq, q_heads, kv_heads, d, 0))


def clear_attn_decode(q, k_pages, v_pages, page_table, seq_len, o=None, lse=None, k_scale=None, v_scale=None, workspace=None,
                      stream=None):
    """Attention of one new token of each sequence (q: [q_heads, n_seq, d]) over the first seq_len rows of its
    cached keys and values. Cache arguments as for clear_attn_cache_append. A sequence of length 0 gets
    o = 0 and lse = -inf. Returns (o, lse)."""
    _queries("q", q)
    device, dtype = q.device, q.dtype
    q_heads, n_seq, d = q.shape
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [pages, page_size, kv_heads, d]")
    kv_heads = k_pages.shape[2]
    cache = _cache(k_pages, v_pages, page_table, k_scale, v_scale, kv_heads, d, dtype, device)
    if page_table.shape[0] != n_seq:
        raise ValueError(f"page_table has {page_table.shape[0]} sequences, q {n_seq}")
    _require_dense("seq_len", seq_len, (n_seq,), torch.int32, device)
    params = ClearSeqParams(n_seq, n_seq, q_heads, kv_heads, d, _DTYPES[dtype])

    def body(handle):
        out = torch.empty_like(q) if o is None else o
        _require("o", out, q.shape, dtype, device)
        ls = torch.empty(q_heads, n_seq, dtype=torch.float32, device=device) if lse is None else lse
        _require_dense("lse", ls, (q_heads, n_seq), torch.float32, device)
        ws = _workspace(workspace, 0 if workspace is not None else _size(_lib.clear_attn_decode_workspace_size, params), device)
        st = _lib.clear_attn_decode(params, cache, seq_len.data_ptr(), _view(q), _view(out), ls.data_ptr(), ws.data_ptr(),
                                    ws.numel() * ws.element_size(), handle)
        if st != CLEAR_OK:
            raise ClearError(st, "clear_attn_decode")
        return out, ls

    return _run(device, stream, body)


def _packed(q, k, v, seq_start):
    _queries("q", q)
    q_heads, n_tok, d = q.shape
    if k.dim() != 3:
        raise ValueError("k must be [kv_heads, tokens, d]")
    _require("k", k, (k.shape[0], n_tok, d), q.dtype, q.device)
    _require("v", v, k.shape, q.dtype, q.device)
    if seq_start.dim() != 1 or seq_start.shape[0] < 2:
        raise ValueError("seq_start must be int32 [sequences + 1]")
    _require_dense("seq_start", seq_start, seq_start.shape, torch.int32, q.device)
    return ClearSeqParams(seq_start.shape[0] - 1, n_tok, q_heads, k.shape[0], d, _DTYPES[q.dtype])


def clear_attn_prompt_fwd(q, k, v, seq_start, o=None, lse=None, stream=None):
    """Causal attention within each sequence of a packed batch: q [q_heads, n_tok, d], k and v
    [kv_heads, n_tok, d] (q_heads a multiple of kv_heads), seq_start int32 [n_seq + 1]. Rows behind the last
    sequence are left as they are. Returns (o, lse)."""
    params = _packed(q, k, v, seq_start)
    device, dtype = q.device, q.dtype

    def body(handle):
        out = torch.empty_like(q) if o is None else o
        _require("o", out, q.shape, dtype, device)
        ls = torch.empty(q.shape[:2], dtype=torch.float32, device=device) if lse is None else lse
        _require_dense("lse", ls, q.shape[:2], torch.float32, device)
        st = _lib.clear_attn_prompt_fwd(params, seq_start.data_ptr(), _view(q), _view(k), _view(v), _view(out), ls.data_ptr(),
                                        handle)
        if st != CLEAR_OK:
            raise ClearError(st, "clear_attn_prompt_fwd")
        return out, ls

    return _run(device, stream, body)


def prompt_bwd_workspace_size(n_tok: int, q_heads: int, kv_heads: int, d: int) -> int:
    """Bytes of clear_attn_prompt_bwd's workspace."""
    return _size(_lib.clear_attn_prompt_bwd_workspace_size, ClearSeqParams(1, n_tok, q_heads, kv_heads, d, 0))


def clear_attn_prompt_bwd(q, k, v, o, lse, dO, seq_start, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of clear_attn_prompt_fwd with respect to q, k and v, given its o and lse and the upstream
    gradient dO; those of k and v are summed over the query heads that share them. Returns (dq, dk, dv)."""
    params = _packed(q, k, v, seq_start)
    device, dtype = q.device, q.dtype
    _require("o", o, q.shape, dtype, device)
    _require("dO", dO, q.shape, dtype, device)
    _require_dense("lse", lse, q.shape[:2], torch.float32, device)

    def body(handle):
        out = [torch.empty_like(x) if y is None else y for x, y in ((q, dq), (k, dk), (v, dv))]
        for name, y, x in (("dq", out[0], q), ("dk", out[1], k), ("dv", out[2], v)):
            _require(name, y, x.shape, dtype, device)
        ws = _workspace(workspace, 0 if workspace is not None else _size(_lib.clear_attn_prompt_bwd_workspace_size, params), device)
        st = _lib.clear_attn_prompt_bwd(params, seq_start.data_ptr(), _view(q), _view(k), _view(v), _view(o), lse.data_ptr(),
                                        _view(dO), _view(out[0]), _view(out[1]), _view(out[2]), ws.data_ptr(),
                                        ws.numel() * ws.element_size(), handle)
        if st != CLEAR_OK:
            raise ClearError(st, "clear_attn_prompt_bwd")
        return tuple(out)

    return _run(device, stream, body)
