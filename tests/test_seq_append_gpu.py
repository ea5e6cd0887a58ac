"""Appending to the paged cache, with the rotation, against its definition in 64 bits."""
import math

import pytest
import torch

import local_circular_window_b200 as L
import seq_util as U

pytestmark = pytest.mark.gpu


def rotated(x, pos, rot, theta, ntk, pairing):
    """x [heads, n, d] turned in 64 bits, and |a| + |b| of each element's pair."""
    x = x.double().clone()
    size = x.abs()
    if rot:
        base = theta * ntk ** (rot / (rot - 2))
        rate = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        angle = pos.double()[:, None] * rate
        c, s = angle.cos(), angle.sin()
        ia = torch.arange(0, rot, 2) if pairing == "adjacent" else torch.arange(rot // 2)
        ib = ia + (1 if pairing == "adjacent" else rot // 2)
        a, b = x[..., ia].clone(), x[..., ib].clone()
        x[..., ia], x[..., ib] = a * c - b * s, a * s + b * c
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return x, size


def close(name, got, ref, size):
    # One rounding to the output's type; the angle's cosine and sine are off by at most 2.2e-7 (the fraction
    # of a turn rounded to fp32: pi 2^-25; two units in the last place of the function) and the products by
    # three roundings: 4e-7 (|a| + |b|) in all.
    U.check(name, got, ref, U.unit(got.dtype) * ref.abs() + 4.5e-7 * size + U.tiny(got.dtype))


CASES = [  # dtype, cache, q_heads, kv_heads, d, page, rot, pairing, new, before
    (torch.bfloat16, None, 6, 2, 128, 16, 128, "adjacent", [1, 1, 1], [0, 15, 16]),
    (torch.float16, None, 3, 3, 64, 7, 32, "halves", [5, 0, 20, 1], [3, 9, 0, 100]),
    (torch.bfloat16, "e4m3", 8, 2, 128, 32, 64, "halves", [33, 2], [31, 5000]),
    (torch.float16, "e4m3", 4, 1, 64, 1, 16, "adjacent", [3, 1], [0, 2]),
    (torch.bfloat16, None, 4, 4, 64, 64, 0, "adjacent", [70], [0]),
    (torch.bfloat16, None, 2, 1, 128, 16, 128, "halves", [4099, 200], [100000, 0]),  # several tokens a block
    (torch.float16, None, 2, 1, 64, 256, 64, "adjacent", [1] * 70, list(range(0, 7000, 100))),  # search over > 32 sequences
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_append(case):
    dtype, cache, hq, hk, d, page, rot, pairing, new, before = case
    gen = torch.Generator().manual_seed(hq * 1000 + d + page)
    theta, ntk = 10000.0, 2.0
    n, behind = sum(new), 5
    lens = [a + b for a, b in zip(new, before)]
    scales = [0.005 + 0.01 * torch.rand(hk, generator=gen) for _ in range(2)] if cache else None
    ctype = torch.float8_e4m3fn if cache else dtype
    kp, vp, table = U.pages(gen, lens, page, hk, d, ctype, scales=scales)
    q, k, v = U.packed(gen, hq, n + behind, d, dtype), U.packed(gen, hk, n + behind, d, dtype), U.packed(gen, hk, n + behind, d, dtype)
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    gk, gv = dev(kp), dev(vp)
    q_out, k_out = torch.full_like(dev(q), 7.0), torch.full_like(dev(k), 7.0)
    L.clear_attn_cache_append(dev(k), dev(v), gk, gv, dev(table), dev(U.starts(new)), torch.tensor(lens, dtype=torch.int32).cuda(),
                              q=dev(q), q_out=q_out, k_out=k_out, rot=rot, theta=theta, ntk=ntk, pairing=pairing,
                              k_scale=dev(scales[0]) if cache else None, v_scale=dev(scales[1]) if cache else None)
    assert L.clear_attn_check() == 0
    pos = torch.cat([torch.arange(b, b + a) for a, b in zip(new, before)])
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    rq, sq = rotated(q[:, :n], pos, rot, theta, ntk, pairing)
    rk, sk = rotated(k[:, :n], pos, rot, theta, ntk, pairing)
    close("q_out", q_out[:, :n].cpu(), rq, sq)
    close("k_out", k_out[:, :n].cpu(), rk, sk)
    assert (q_out[:, n:] == 7).all() and (k_out[:, n:] == 7).all()  # rows behind the last sequence
    page_of = table[seq, pos // page].long()
    for name, got, old, new_rows, size, i in (("k_pages", gk, kp, rk, sk, 0), ("v_pages", gv, vp, v[:, :n].double(), v[:, :n].double().abs() * 0, 1)):
        got = got.cpu()
        rows = got[page_of, pos % page] if not cache else got.float()[page_of, pos % page]
        ref = new_rows.transpose(0, 1)
        if cache:
            x = ref / scales[i].double()[:, None]
            tol = 2.0 ** -4 * x.abs() + 2.0 ** -10 + 5e-7 * (size.transpose(0, 1) + ref.abs()) / scales[i].double()[:, None]
            U.check(name, rows, x.clamp(-448, 448), tol)
        else:
            U.check(name, rows, ref, U.unit(dtype) * ref.abs() + 4.5e-7 * size.transpose(0, 1) + U.tiny(dtype))
        mask = torch.ones(got.shape[:2], dtype=torch.bool)
        mask[page_of, pos % page] = False
        raw = lambda t: t.view(torch.uint8) if cache else t  # noqa: E731
        assert torch.equal(raw(got)[mask], raw(old)[mask])  # nothing else is written


def _small(n=3, d=64, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(5)
    kp, vp, table = U.pages(gen, [20] * n, 16, 2, d, dtype)
    k, v, q = (U.packed(gen, h, n, d, dtype).cuda() for h in (2, 2, 4))
    return q, k, v, kp.cuda(), vp.cuda(), table.cuda(), U.starts([1] * n).cuda(), torch.full((n,), 20, dtype=torch.int32).cuda()


def test_in_place_and_strided_and_heads_first():
    q, k, v, kp, vp, table, ss, sl = _small()
    a = L.clear_attn_cache_append(k, v, kp.clone(), vp.clone(), table, ss, sl, q=q, k_out=torch.empty_like(k), rot=64)
    # in place, from one packed buffer [tokens, heads of q, k, v, d]; the cache as [pages, heads, rows, d]
    buf = torch.cat([q, k, v]).transpose(0, 1).contiguous().transpose(0, 1)
    q2, k2, v2 = buf[:4], buf[4:6], buf[6:]
    kp2, vp2 = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kp, vp))
    L.clear_attn_cache_append(k2, v2, kp2, vp2, table, ss, sl, q=q2, q_out=q2, k_out=k2, rot=64)
    assert torch.equal(q2, a[0]) and torch.equal(k2, a[1])
    kp3, vp3 = kp.clone(), vp.clone()
    L.clear_attn_cache_append(k, v, kp3, vp3, table, ss, sl, rot=64)  # without queries
    assert torch.equal(kp2, kp3) and torch.equal(vp2, vp3)


def test_padding_and_bad_pages_are_left_out():
    q, k, v, kp, vp, table, ss, sl = _small()
    sl[1] = 0  # position -1: padding
    q_out = torch.full_like(q, 7.0)
    a, b = kp.clone(), vp.clone()
    L.clear_attn_cache_append(k, v, a, b, table, ss, sl, q=q, q_out=q_out, rot=64)
    assert L.clear_attn_check() == 0
    assert (q_out[:, 1] == 7).all() and (q_out[:, 0] != 7).any()
    table[2, 1] = kp.shape[0]  # one past the last page
    a2, b2 = kp.clone(), vp.clone()
    L.clear_attn_cache_append(k, v, a2, b2, table, ss, sl, q=q, q_out=q_out, rot=64)
    assert L.clear_attn_check() == 6 and L.clear_attn_check() == 0
    page = int(table[0, 1])
    assert torch.equal(a2[page], a[page])  # the others are stored
    a2[page], b2[page] = kp[page], vp[page]
    assert torch.equal(a2, kp) and torch.equal(b2, vp)
    sl[0] = 16 * table.shape[1] + 1  # past the table's last entry
    L.clear_attn_cache_append(k, v, a2, b2, table, ss, sl, rot=64)
    assert L.clear_attn_check() == 6


def test_e4m3_keeps_nan_and_saturates():
    q, k, v, _, _, table, ss, sl = _small()
    kp = torch.zeros(int(table.max()) + 4, 16, 2, 64, device="cuda").to(torch.float8_e4m3fn)
    vp = kp.clone()
    v[0, 0, 0], v[0, 0, 1], v[0, 0, 2] = math.nan, math.inf, -1e4
    one = torch.ones(2, device="cuda")
    L.clear_attn_cache_append(k, v, kp, vp, table, ss, sl, k_scale=one, v_scale=one)
    row = vp.float()[int(table[0, 1]), 3, 0]
    assert row[0].isnan() and row[1] == 448 and row[2] == -448


def test_captured_graph_follows_lengths():
    q, k, v, kp, vp, table, ss, sl = _small()
    a, b = kp.clone(), vp.clone()
    q_out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.clear_attn_cache_append(k, v, a, b, table, ss, sl, q=q, q_out=q_out, rot=64)
    sl -= 5
    g.replay()
    c, e = kp.clone(), vp.clone()
    want, _ = L.clear_attn_cache_append(k, v, c, e, table, ss, sl, q=q, rot=64)
    assert torch.equal(q_out, want) and torch.equal(a, c) and torch.equal(b, e)
