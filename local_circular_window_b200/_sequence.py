"""ctypes binding of the token-sequence operators of libclear_attn.so: appending to a paged key/value
cache with the rotary embedding, attention of one new token over that cache, and causal attention over
packed prompts with its gradient (argument marshalling only; see include/clear_attn.h).

Tensors are [heads, tokens, d] views with contiguous rows, e.g. ``x.view(tokens, heads, d).transpose(0, 1)``
of a projection's output. All tensors of a call lie on one CUDA device; the call runs on that device,
on ``stream`` or its current stream.
"""
from __future__ import annotations

import ctypes
import struct

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


# The structures go to the library as packed bytes, in the fields' order: a decoding step is as short as the
# time that its arguments take, and a ctypes structure takes several times as long to fill.
_pack_params = struct.Struct("6i").pack
_pack_view = struct.Struct("P2q").pack
_pack_cache = struct.Struct("5P7q4i").pack
_pack_rope = struct.Struct("2f2i").pack

for _name, _n in (("cache_append", 11), ("decode", 9), ("prompt_fwd", 8), ("prompt_bwd", 14)):
    _f = getattr(_lib, "clear_attn_" + _name)
    _f.restype = _i
    _f.argtypes = [_vp] * _n
_lib.clear_attn_decode.argtypes = [_vp] * 7 + [ctypes.c_size_t, _vp]
_lib.clear_attn_prompt_bwd.argtypes = [_vp] * 12 + [ctypes.c_size_t, _vp]
for _name in ("decode", "prompt_bwd"):
    _f = getattr(_lib, f"clear_attn_{_name}_workspace_size")
    _f.restype = ctypes.c_size_t
    _f.argtypes = [_vp, ctypes.POINTER(_i)]

_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream


def _view(name, t, shape, dtype, device):
    """The packed view of a [heads, tokens, d] tensor, checked."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device.index:
        _wrong(name, t, shape, dtype, device)
    h, n, e = t.stride()
    if e != 1:
        _wrong(name, t, shape, dtype, device)
    return _pack_view(t.data_ptr(), h, n)


def _dense(name, t, shape, dtype, device):
    """The address of a contiguous tensor, checked."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device.index or not t.is_contiguous():
        _wrong(name, t, shape, dtype, device)
    return t.data_ptr()


def _wrong(name, t, shape, dtype, device):
    raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} with contiguous rows on {device}, "
                     f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _queries(name, q):
    if q.dim() != 3 or q.dtype not in (torch.bfloat16, torch.float16) or not q.is_cuda:
        raise ValueError(f"{name} must be a CUDA bf16 or fp16 tensor [heads, tokens, d]")


def _elsewhere(device, stream):
    """Whether a call has to change the current device or stream first. What it allocates then belongs to the
    stream that uses it."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream lies on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    if device.index != _current_device():
        return torch.cuda.device(device)
    return None


def _workspace(workspace, function, params, device):
    if workspace is None:
        return torch.empty(_size(function, params), dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def _size(function, params):
    st = _i(0)
    n = function(params, ctypes.byref(st))
    if st.value != CLEAR_OK:
        raise ClearError(st.value, "the workspace size")
    return n


def _cache(k_pages, v_pages, page_table, k_scale, v_scale, kv_heads, d, dtype, device):
    shape, kind = k_pages.shape, k_pages.dtype
    if len(shape) != 4 or shape != v_pages.shape or kind is not v_pages.dtype:
        raise ValueError("k_pages and v_pages must have one shape [pages, page_size, kv_heads, d] and one dtype")
    n_pages, page_size, heads, e = shape
    if heads != kv_heads or e != d:
        raise ValueError(f"the pages hold {(heads, e)} heads and elements, not {(kv_heads, d)}")
    if kind is not dtype and kind is not torch.float8_e4m3fn:
        raise ValueError(f"pages must be {dtype} or float8_e4m3fn")
    kp, kr, kh, ke = k_pages.stride()
    vp, vr, vh, ve = v_pages.stride()
    if ke != 1 or ve != 1 or k_pages.get_device() != device.index or v_pages.get_device() != device.index:
        raise ValueError(f"pages must have contiguous rows and lie on {device}")
    if page_table.dim() != 2 or page_table.dtype is not torch.int32 or page_table.get_device() != device.index:
        raise ValueError(f"page_table must be int32 [sequences, pages] on {device}")
    max_pages = page_table.shape[1]
    row, step = page_table.stride()
    if step != 1 and max_pages > 1:
        raise ValueError("page_table must have contiguous rows")
    ks = vs = 0
    if kind is torch.float8_e4m3fn:
        if k_scale is None or v_scale is None:
            raise ValueError("an E4M3 cache needs k_scale and v_scale")
        ks = _dense("k_scale", k_scale, (kv_heads,), torch.float32, device)
        vs = _dense("v_scale", v_scale, (kv_heads,), torch.float32, device)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales belong to an E4M3 cache")
    return _pack_cache(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), ks, vs, kp, kr, kh, vp, vr, vh, row, n_pages,
                       page_size, max_pages, _DTYPES[kind])


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
    device, dtype, shape = k.device, k.dtype, k.shape
    there = _elsewhere(device, stream)
    if there is not None:
        with there:
            return clear_attn_cache_append(k, v, k_pages, v_pages, page_table, seq_start, seq_len, q, q_out, k_out, rot, theta, ntk,
                                           pairing, k_scale, v_scale)
    kv_heads, n_tok, d = shape
    n_seq = page_table.shape[0]
    cache = _cache(k_pages, v_pages, page_table, k_scale, v_scale, kv_heads, d, dtype, device)
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {sorted(_PAIRINGS)}")
    vq = vqo = None
    q_heads = kv_heads
    if q is not None:
        _queries("q", q)
        q_heads = q.shape[0]
        vq = _view("q", q, (q_heads, n_tok, d), dtype, device)
        if q_out is None:
            q_out = torch.empty_like(q)
        vqo = _view("q_out", q_out, q.shape, dtype, device)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    st = _lib.clear_attn_cache_append(
        _pack_params(n_seq, n_tok, q_heads, kv_heads, d, _DTYPES[dtype]), cache, _pack_rope(theta, ntk, rot, _PAIRINGS[pairing]),
        _dense("seq_start", seq_start, (n_seq + 1,), torch.int32, device), _dense("seq_len", seq_len, (n_seq,), torch.int32, device),
        vq, _view("k", k, shape, dtype, device), _view("v", v, shape, dtype, device), vqo,
        None if k_out is None else _view("k_out", k_out, shape, dtype, device), _raw_stream(device.index))
    if st != CLEAR_OK:
        raise ClearError(st, "clear_attn_cache_append")
    return q_out, k_out


def decode_workspace_size(n_seq: int, q_heads: int, kv_heads: int, d: int) -> int:
    """Bytes of clear_attn_decode's workspace."""
    return _size(_lib.clear_attn_decode_workspace_size, _pack_params(n_seq, n_seq, q_heads, kv_heads, d, 0))


def clear_attn_decode(q, k_pages, v_pages, page_table, seq_len, o=None, lse=None, k_scale=None, v_scale=None, workspace=None,
                      stream=None):
    """Attention of one new token of each sequence (q: [q_heads, n_seq, d]) over the first seq_len rows of its
    cached keys and values. Cache arguments as for clear_attn_cache_append. A sequence of length 0 gets
    o = 0 and lse = -inf. Returns (o, lse)."""
    _queries("q", q)
    device, dtype, shape = q.device, q.dtype, q.shape
    there = _elsewhere(device, stream)
    if there is not None:
        with there:
            return clear_attn_decode(q, k_pages, v_pages, page_table, seq_len, o, lse, k_scale, v_scale, workspace)
    q_heads, n_seq, d = shape
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [pages, page_size, kv_heads, d]")
    kv_heads = k_pages.shape[2]
    cache = _cache(k_pages, v_pages, page_table, k_scale, v_scale, kv_heads, d, dtype, device)
    if page_table.shape[0] != n_seq:
        raise ValueError(f"page_table has {page_table.shape[0]} sequences, q {n_seq}")
    params = _pack_params(n_seq, n_seq, q_heads, kv_heads, d, _DTYPES[dtype])
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q_heads, n_seq, dtype=torch.float32, device=device)
    workspace = _workspace(workspace, _lib.clear_attn_decode_workspace_size, params, device)
    st = _lib.clear_attn_decode(params, cache, _dense("seq_len", seq_len, (n_seq,), torch.int32, device),
                                _view("q", q, shape, dtype, device), _view("o", o, shape, dtype, device),
                                _dense("lse", lse, (q_heads, n_seq), torch.float32, device), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _raw_stream(device.index))
    if st != CLEAR_OK:
        raise ClearError(st, "clear_attn_decode")
    return o, lse


def _packed(q, k, seq_start):
    q_heads, n_tok, d = q.shape
    if k.dim() != 3:
        raise ValueError("k must be [kv_heads, tokens, d]")
    if seq_start.dim() != 1 or seq_start.shape[0] < 2:
        raise ValueError("seq_start must be int32 [sequences + 1]")
    return _pack_params(seq_start.shape[0] - 1, n_tok, q_heads, k.shape[0], d, _DTYPES[q.dtype])


def clear_attn_prompt_fwd(q, k, v, seq_start, o=None, lse=None, stream=None):
    """Causal attention within each sequence of a packed batch: q [q_heads, n_tok, d], k and v
    [kv_heads, n_tok, d] (q_heads a multiple of kv_heads), seq_start int32 [n_seq + 1]. Rows behind the last
    sequence are left as they are. Returns (o, lse)."""
    _queries("q", q)
    device, dtype, shape = q.device, q.dtype, q.shape
    there = _elsewhere(device, stream)
    if there is not None:
        with there:
            return clear_attn_prompt_fwd(q, k, v, seq_start, o, lse)
    params = _packed(q, k, seq_start)
    shape_kv = (k.shape[0], shape[1], shape[2])
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=device)
    st = _lib.clear_attn_prompt_fwd(params, _dense("seq_start", seq_start, seq_start.shape, torch.int32, device),
                                    _view("q", q, shape, dtype, device), _view("k", k, shape_kv, dtype, device),
                                    _view("v", v, shape_kv, dtype, device), _view("o", o, shape, dtype, device),
                                    _dense("lse", lse, shape[:2], torch.float32, device), _raw_stream(device.index))
    if st != CLEAR_OK:
        raise ClearError(st, "clear_attn_prompt_fwd")
    return o, lse


def prompt_bwd_workspace_size(n_tok: int, q_heads: int, kv_heads: int, d: int) -> int:
    """Bytes of clear_attn_prompt_bwd's workspace, of either type, for n_tok tokens or fewer."""
    return _size(_lib.clear_attn_prompt_bwd_workspace_size, _pack_params(1, n_tok, q_heads, kv_heads, d, 0))


def clear_attn_prompt_bwd(q, k, v, o, lse, dO, seq_start, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of clear_attn_prompt_fwd with respect to q, k and v, given its o and lse and the upstream
    gradient dO; those of k and v are summed over the query heads that share them. Returns (dq, dk, dv)."""
    _queries("q", q)
    device, dtype, shape = q.device, q.dtype, q.shape
    there = _elsewhere(device, stream)
    if there is not None:
        with there:
            return clear_attn_prompt_bwd(q, k, v, o, lse, dO, seq_start, dq, dk, dv, workspace)
    params = _packed(q, k, seq_start)
    shape_kv = (k.shape[0], shape[1], shape[2])
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    workspace = _workspace(workspace, _lib.clear_attn_prompt_bwd_workspace_size, params, device)
    st = _lib.clear_attn_prompt_bwd(params, _dense("seq_start", seq_start, seq_start.shape, torch.int32, device),
                                    _view("q", q, shape, dtype, device), _view("k", k, shape_kv, dtype, device),
                                    _view("v", v, shape_kv, dtype, device), _view("o", o, shape, dtype, device),
                                    _dense("lse", lse, shape[:2], torch.float32, device), _view("dO", dO, shape, dtype, device),
                                    _view("dq", dq, shape, dtype, device), _view("dk", dk, shape_kv, dtype, device),
                                    _view("dv", dv, shape_kv, dtype, device), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), _raw_stream(device.index))
    if st != CLEAR_OK:
        raise ClearError(st, "clear_attn_prompt_bwd")
    return dq, dk, dv
