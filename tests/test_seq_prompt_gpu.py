"""Causal attention over packed prompts with grouped heads, against its definition in 64 bits."""
import math

import pytest
import torch

import local_circular_window_b200 as L
import seq_util as U

pytestmark = pytest.mark.gpu


def make(seed, lens, hq, hk, d, dtype, behind=0, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    n = sum(lens) + behind
    return tuple(U.packed(gen, h, n, d, dtype, scale) for h in (hq, hk, hk)) + (U.starts(lens),)


def verify(o, lse, q, k, v, lens, heads=None):
    hq, hk, at = q.shape[0], k.shape[0], 0
    for s, n in enumerate(lens):
        t = slice(at, at + n)
        keep = torch.ones(n, n, dtype=torch.bool).tril()
        for h in (range(hq) if heads is None else heads):
            if n:
                g = h * hk // hq
                U.check_attention(f"sequence {s} head {h}", o[h, t], lse[h, t], q[h, t], k[g, t], v[g, t], q.dtype, q.dtype, keep)
        at += n


CASES = [  # lens, q_heads, kv_heads, d, dtype
    ([1], 1, 1, 64, torch.bfloat16),
    ([128], 2, 1, 128, torch.bfloat16),
    ([129], 3, 3, 64, torch.float16),
    ([257, 1, 0, 127], 4, 2, 128, torch.float16),
    ([256, 512], 6, 2, 64, torch.bfloat16),
    ([700, 33], 5, 1, 128, torch.bfloat16),
    ([3] * 50 + [300, 0, 0, 2], 2, 2, 64, torch.bfloat16),   # more sequences than lanes
    ([0, 0, 5], 1, 1, 128, torch.float16),
    ([1537], 2, 1, 128, torch.bfloat16),
    # few long sequences: key tiles split between the two halves of a block
    ([513], 1, 1, 64, torch.float16),
    ([600, 1, 1100], 3, 3, 128, torch.bfloat16),
    ([1025, 0, 640], 2, 1, 64, torch.bfloat16),
    ([2300], 9, 3, 128, torch.float16),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_prompt(i):
    lens, hq, hk, d, dtype = CASES[i]
    q, k, v, ss = make(i, lens, hq, hk, d, dtype)
    o, lse = L.clear_attn_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), ss.cuda())
    assert L.clear_attn_check() == 0
    verify(o.cpu(), lse.cpu(), q, k, v, lens)


def test_many_items_for_each_block():
    # More items than SMs, of many lengths, so that every block walks several.
    lens = [260, 1000, 5, 900, 130, 512, 640, 77]
    q, k, v, ss = make(20, lens, 48, 16, 64, torch.float16)
    o, lse = L.clear_attn_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), ss.cuda())
    verify(o.cpu(), lse.cpu(), q, k, v, lens, heads=[0, 1, 17, 46, 47])
    o2, lse2 = L.clear_attn_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), ss.cuda())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("a,b,c", [(100, 200, 60), (700, 100, 1000)])
def test_sequences_do_not_touch_each_other(a, b, c):
    q, k, v, ss = (x.cuda() for x in make(21, [a, b, c], 2, 1, 64, torch.bfloat16, behind=90))
    n = a + b + c
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    L.clear_attn_prompt_fwd(q, k, v, ss, o=o, lse=lse)
    assert (o[:, n:] == 7).all() and (lse[:, n:] == 7).all()  # rows behind the last sequence
    for x in (q, k, v):
        x[:, a:a + b] = math.nan
        x[:, n:] = math.inf
    o2, lse2 = L.clear_attn_prompt_fwd(q, k, v, ss)
    for t in (slice(0, a), slice(a + b, n)):
        assert torch.equal(o2[:, t], o[:, t]) and torch.equal(lse2[:, t], lse[:, t])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[600, 600], [612, 3, 3, 380]])
def test_growing_scores_and_ties(lens, d):
    # Keys that grow along the sequence move the running maximum again and again; equal keys tie everywhere. The second
    # batch's last query tiles stand alone in their items.
    q, k, v, ss = make(22, lens, 2, 1, d, torch.bfloat16)
    n = lens[0]
    # sum |q k| / sqrt(d) is about 0.8 sqrt(d) |k|, 20 at most
    k[0, :n] = (torch.linspace(-1, 1, n)[:, None] * (24 / d ** 0.5) * torch.sign(q[0, :n].float())).to(torch.bfloat16)
    k[0, n:] = k[0, n]
    o, lse = L.clear_attn_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), ss.cuda())
    verify(o.cpu(), lse.cpu(), q, k, v, lens)
    o2, lse2 = L.clear_attn_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), ss.cuda())
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_strided_views_give_the_same_bits():
    lens = [200, 57]
    q, k, v, ss = (x.cuda() for x in make(23, lens, 4, 2, 128, torch.float16))
    o, lse = L.clear_attn_prompt_fwd(q, k, v, ss)
    buf = torch.cat([q, k, v]).transpose(0, 1).contiguous().transpose(0, 1)   # one projection's output
    o2, lse2 = L.clear_attn_prompt_fwd(buf[:4], buf[4:6], buf[6:], ss, o=torch.empty(4, 257, 128, dtype=q.dtype, device="cuda"))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    big = torch.zeros(4, 300, 192, dtype=q.dtype, device="cuda")               # wider rows
    big[:, 40:297, 64:] = q
    o3, _ = L.clear_attn_prompt_fwd(big[:, 40:297, 64:], k, v, ss)
    assert torch.equal(o, o3)


def test_bad_offsets_are_reported():
    q, k, v, ss = (x.cuda() for x in make(24, [50, 60, 40], 2, 1, 64, torch.bfloat16))
    good, _ = L.clear_attn_prompt_fwd(q, k, v, ss)
    for bad in ([0, 50, 110, 151], [0, 50, 40, 150], [-1, 50, 110, 150]):
        o = torch.zeros_like(good)
        L.clear_attn_prompt_fwd(q, k, v, torch.tensor(bad, dtype=torch.int32).cuda(), o=o)
        assert L.clear_attn_check() == 6 and L.clear_attn_check() == 0
        if bad[0] == 0:  # rows 40 to 49 belong to two sequences in the second list
            assert torch.equal(o[:, :40], good[:, :40])


def test_captured_graph_follows_offsets_on_another_stream():
    q, k, v, ss = (x.cuda() for x in make(25, [300, 200, 100], 4, 4, 64, torch.bfloat16))
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.clear_attn_prompt_fwd(q, k, v, ss, o=o, lse=lse)
    ss.copy_(torch.tensor([0, 10, 10, 600], dtype=torch.int32))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    want = L.clear_attn_prompt_fwd(q, k, v, ss, stream=s)
    s.synchronize()
    g.replay()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_thousands_of_sequences():
    gen = torch.Generator().manual_seed(40)
    lens = torch.randint(0, 5, (3000,), generator=gen).tolist()
    lens[1234], lens[2999] = 400, 150
    q, k, v, ss = make(41, lens, 2, 1, 64, torch.bfloat16)
    o, lse = L.clear_attn_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), ss.cuda())
    some = [0, 1, 7, 500, 1234, 1235, 2500, 2998, 2999]
    for s in some:
        t = slice(int(ss[s]), int(ss[s + 1]))
        n = lens[s]
        if n:
            keep = torch.ones(n, n, dtype=torch.bool).tril()
            for h in range(2):
                U.check_attention(f"sequence {s}", o.cpu()[h, t], lse.cpu()[h, t], q[h, t], k[0, t], v[0, t], q.dtype, q.dtype, keep)
    assert not o.isnan().any()
