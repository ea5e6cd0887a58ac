"""Argument checks of the token-sequence operators: found on the host, before any CUDA call, so host
buffers can stand in for device pointers (the canaries prove that nothing was written)."""
import ctypes

import numpy as np
import pytest
import torch

import local_circular_window_b200 as L
from local_circular_window_b200 import _sequence as S

class ByReference:
    """The library with structures passed by reference."""

    def __getattr__(self, name):
        f = getattr(L.lib(), name)
        return lambda *a: f(*(ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in a))


LIB = ByReference()
BUF = np.full(1 << 16, 0x5A, dtype=np.uint8)
PTR = (BUF.ctypes.data + 255) & ~255
OK = dict(n_seq=2, n_tok=2, q_heads=4, kv_heads=2, d=64, dtype=0)


@pytest.fixture(autouse=True)
def untouched():
    yield
    assert (BUF == 0x5A).all()


def params(**kw):
    return S.ClearSeqParams(**{**OK, **kw})


def view(ptr=PTR, head=128, token=512):
    return S.ClearSeqView(ptr, head, token)


def cache(**kw):
    a = dict(k_pages=PTR, v_pages=PTR, page_table=PTR, k_scale=None, v_scale=None, k_strides=(S._ll * 3)(2048, 128, 64),
             v_strides=(S._ll * 3)(2048, 128, 64), page_table_stride=4, n_pages=3, page_size=16, max_pages=4, dtype=0)
    return S.ClearSeqCache(**{**a, **kw})


BAD_PARAMS = [(dict(n_seq=0), 1), (dict(n_seq=-1), 1), (dict(n_seq=(1 << 20) + 1), 1), (dict(n_tok=0), 1), (dict(n_tok=(1 << 30) + 1), 1),
              (dict(q_heads=3), 1), (dict(q_heads=0), 1), (dict(kv_heads=0), 1), (dict(d=96), 2), (dict(d=32), 2), (dict(dtype=2), 2),
              (dict(dtype=-1), 2)]
BAD_VIEWS = [(None, 1), (dict(ptr=None), 1), (dict(ptr=PTR + 8), 1), (dict(head=65), 2), (dict(head=0), 2), (dict(token=-512), 2),
             (dict(token=1 << 40), 2)]
BAD_CACHES = [(None, 1), (dict(k_pages=None), 1), (dict(v_pages=PTR + 2), 1), (dict(page_table=None), 1), (dict(n_pages=0), 1),
              (dict(page_size=0), 1), (dict(page_size=(1 << 20) + 1), 1), (dict(max_pages=0), 1), (dict(page_table_stride=3), 1),
              (dict(dtype=1), 2), (dict(dtype=3), 2), (dict(dtype=2), 1), (dict(k_strides=(S._ll * 3)(2048, 0, 64)), 2),
              (dict(v_strides=(S._ll * 3)(2048, 128, 60)), 2),
              (dict(dtype=2, k_scale=PTR, v_scale=PTR, k_strides=(S._ll * 3)(2048, 128, 72)), 2)]


def append(p=None, c=None, r=None, ss=PTR, sl=PTR, q="same", k="same", v="same", qo="same", ko=None):
    pick = lambda x: view() if x == "same" else x  # noqa: E731
    return LIB.clear_attn_cache_append(p or params(), cache() if c is None else c, r, ss, sl, pick(q), pick(k), pick(v), pick(qo), ko, None)


def decode(p=None, c="same", sl=PTR, q="same", o="same", lse=PTR, ws=PTR, size=1 << 30):
    pick = lambda x: view() if x == "same" else x  # noqa: E731
    return LIB.clear_attn_decode(p or params(), cache() if c == "same" else c, sl, pick(q), pick(o), lse, ws, size, None)


def prompt(p=None, ss=PTR, q="same", k="same", v="same", o="same", lse=PTR):
    pick = lambda x: view() if x == "same" else x  # noqa: E731
    return LIB.clear_attn_prompt_fwd(p or params(), ss, pick(q), pick(k), pick(v), pick(o), lse, None)


def backward(p=None, ss=PTR, lse=PTR, ws=PTR, size=1 << 30, **kw):
    views = [kw.get(n, view()) for n in ("q", "k", "v", "o", "dO", "dq", "dk", "dv")]
    return LIB.clear_attn_prompt_bwd(p or params(), ss, *views[:4], lse, *views[4:], ws, size, None)


@pytest.mark.parametrize("fields,status", BAD_PARAMS)
def test_params(fields, status):
    p = params(**fields)
    assert append(p) == status and decode(p) == status and prompt(p) == status and backward(p) == status
    st = ctypes.c_int(0)
    assert LIB.clear_attn_decode_workspace_size(p, ctypes.byref(st)) == 0 and st.value == status
    assert LIB.clear_attn_prompt_bwd_workspace_size(p, ctypes.byref(st)) == 0 and st.value == status
    assert LIB.clear_attn_decode(None, cache(), PTR, view(), view(), PTR, PTR, 1 << 30, None) == 1


@pytest.mark.parametrize("fields,status", BAD_VIEWS)
def test_views(fields, status):
    v = None if fields is None else view(**fields)
    for name in ("k", "v"):
        assert append(**{name: v}) == status
    if v is not None:
        assert append(q=v) == status and append(qo=v) == status and append(ko=v) == status
    for name in ("q", "o"):
        assert decode(**{name: v}) == status
    for name in ("q", "k", "v", "o"):
        assert prompt(**{name: v}) == status
    for name in ("q", "k", "v", "o", "dO", "dq", "dk", "dv"):
        assert backward(**{name: v}) == status


@pytest.mark.parametrize("fields,status", BAD_CACHES)
def test_caches(fields, status):
    if fields is None:
        assert LIB.clear_attn_cache_append(params(), None, None, PTR, PTR, view(), view(), view(), view(), None, None) == status
        assert decode(c=None) == status
    else:
        assert append(c=cache(**fields)) == status and decode(c=cache(**fields)) == status


def test_indexes_workspace_and_queries():
    assert append(ss=None) == 1 and append(sl=None) == 1 and append(qo=None) == 1 and append(q=None) == 1
    assert decode(sl=None) == 1 and decode(p=params(n_tok=3)) == 1 and prompt(ss=None) == 1
    need = L.decode_workspace_size(2, 4, 2, 64)
    assert backward(ss=None) == 1 and backward(lse=None) == 1
    size = L.prompt_bwd_workspace_size(2, 4, 2, 64)
    assert backward(ws=None) == 3 and backward(size=size - 1) == 3 and backward(ws=PTR + 16) == 3
    assert decode(ws=None) == 3 and decode(size=need - 1) == 3 and decode(ws=PTR + 16) == 3


@pytest.mark.parametrize("fields,status", [
    (dict(theta=1.0), 1), (dict(theta=float("nan")), 1), (dict(theta=float("inf")), 1), (dict(ntk=0.0), 1), (dict(rot=-16), 1),
    (dict(rot=80), 1), (dict(rot=8), 2), (dict(rot=24), 2), (dict(pairing=2), 1)])
def test_rope(fields, status):
    assert append(r=S.ClearSeqRope(**{**dict(theta=1e4, ntk=1.0, rot=64, pairing=0), **fields})) == status


def test_strides_of_single_elements_are_not_used():
    # One head, one token: any stride passes the checks, and the call gets as far as looking for a device.
    if torch.cuda.is_available():
        pytest.skip("would launch on the host buffers")
    one = dict(n_seq=1, n_tok=1, q_heads=1, kv_heads=1)
    assert prompt(params(**one), *[PTR] + [view(head=3, token=-1)] * 4) not in (1, 2, 3)


def test_binding_refuses():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    ss = torch.tensor([0, 2], dtype=torch.int32)
    with pytest.raises(ValueError):
        L.clear_attn_prompt_fwd(q, q[:2], q[:2], ss)
    pages = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        L.clear_attn_decode(q, pages, pages, ss[None], ss)
    with pytest.raises(ValueError):
        L.clear_attn_cache_append(q, q, pages, pages, ss[None], ss, ss[:1])
