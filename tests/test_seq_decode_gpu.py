"""Attention of one new token over the paged cache, against its definition in 64 bits."""
import math

import pytest
import torch

import local_circular_window_b200 as L
import seq_util as U

pytestmark = pytest.mark.gpu


def make(seed, lens, hq, hk, d, page, dtype, cache=None, extra=3):
    gen = torch.Generator().manual_seed(seed)
    scales = [0.005 + 0.01 * torch.rand(hk, generator=gen) for _ in range(2)] if cache else None
    kp, vp, table = U.pages(gen, lens, page, hk, d, torch.float8_e4m3fn if cache else dtype, extra=extra, scales=scales)
    q = U.packed(gen, hq, len(lens), d, dtype)
    return q, kp, vp, table, scales


def call(q, kp, vp, table, scales, lens, **kw):
    sc = {} if scales is None else {"k_scale": scales[0].cuda(), "v_scale": scales[1].cuda()}
    return L.clear_attn_decode(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), **sc, **kw)


def verify(o, lse, q, kp, vp, table, scales, lens):
    hq, hk, page = q.shape[0], kp.shape[2], kp.shape[1]
    p_type = torch.float16 if scales is not None else q.dtype
    for s, n in enumerate(lens):
        if n <= 0:
            assert (o[:, s] == 0).all() and (lse[:, s] == -math.inf).all()
            continue
        at = table[s, :-(-n // page)].long()
        k, v = kp.float().double()[at].flatten(0, 1)[:n], vp.float().double()[at].flatten(0, 1)[:n]
        if scales is not None:
            k, v = k * scales[0].double()[:, None], v * scales[1].double()[:, None]
        for h in range(hq):
            g = h * hk // hq
            U.check_attention(f"sequence {s} head {h}", o[h, s:s + 1], lse[h, s:s + 1], q[h, s:s + 1], k[:, g], v[:, g], p_type, q.dtype)


CASES = [  # lens, q_heads, kv_heads, d, page, dtype, cache
    ([1], 1, 1, 64, 1, torch.bfloat16, None),
    ([777], 6, 2, 128, 16, torch.bfloat16, None),
    ([1, 0, 15, 16, 17, 63, 64, 65, 200], 8, 1, 128, 7, torch.float16, None),
    ([300, 5], 17, 1, 64, 64, torch.bfloat16, None),       # 17 rows: a second matrix tile of one row
    ([130, 40], 40, 1, 128, 16, torch.float16, None),
    ([4000, 1, 900], 4, 4, 64, 256, torch.bfloat16, None),
    ([513, 64], 12, 4, 128, 32, torch.bfloat16, "e4m3"),
    ([100, 0, 31], 16, 1, 64, 3, torch.float16, "e4m3"),
    ([2000], 3, 1, 64, 16, torch.bfloat16, "e4m3"),
    ([20] * 140 + [3000], 2, 1, 64, 16, torch.float16, None),  # more sequences than threads
    ([0, 0], 2, 2, 128, 16, torch.bfloat16, None),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_decode(i):
    lens, hq, hk, d, page, dtype, cache = CASES[i]
    a = make(i, lens, hq, hk, d, page, dtype, cache)
    o, lse = call(*a, lens)
    assert L.clear_attn_check() == 0
    verify(o.cpu(), lse.cpu(), *a, lens)


def test_long_sequence_split_over_the_machine():
    lens = [70001]
    a = make(3, lens, 4, 2, 128, 64, torch.bfloat16)
    o, lse = call(*a, lens)
    verify(o.cpu(), lse.cpu(), *a, lens)
    o2, lse2 = call(*a, lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # the same bits on every run


@pytest.mark.parametrize("cache", [None, "e4m3"])
def test_what_lies_behind_the_end_does_not_count(cache):
    lens = [37, 16, 1]
    a = make(4, lens, 4, 2, 64, 16, torch.bfloat16, cache, extra=4)
    o, lse = call(*a, lens)
    q, kp, vp, table, scales = a
    for x in (kp, vp):
        y = x.view(torch.uint8) if cache else x
        used = torch.zeros(x.shape[:2], dtype=torch.bool)
        for s, n in enumerate(lens):
            for p in range(n):
                used[int(table[s, p // 16]), p % 16] = True
        y[~used] = 0x7F if cache else math.nan
    o2, lse2 = call(q, kp, vp, table, scales, lens)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_sharp_and_growing_scores():
    # Scores that grow along the keys, so that the running maximum is followed many times, and one that takes all.
    lens = [1500]
    q, kp, vp, table, _ = make(5, lens, 2, 1, 64, 16, torch.bfloat16)
    order = table[0].long()
    x = torch.linspace(-4, 4, order.numel() * 16).view(-1, 16)
    kp[order] = (x[:, :, None, None] * torch.sign(q[0, 0].float())).to(torch.bfloat16)
    o, lse = call(q, kp, vp, table, None, lens)
    k, v = kp[order].flatten(0, 1)[:1500, 0], vp[order].flatten(0, 1)[:1500, 0]
    for h in range(2):
        # sum |q k| / sqrt(d) reaches 4 * 51 / 8 = 26 here: scores are off by up to 66 * 2^-24 * 26 = 1.1e-4 < SCORE / 2
        U.check_attention(f"head {h}", o[h], lse[h], q[h], k, v, torch.bfloat16, torch.bfloat16)


def test_shared_pages_strides_and_outputs():
    # Two sequences share their first pages; pages laid out [pages, heads, rows, d]; a table with a wider stride.
    lens = [40, 33]
    q, kp, vp, table, _ = make(6, lens, 4, 2, 64, 16, torch.float16)
    table[1, :2] = table[0, :2]
    o, lse = call(q, kp, vp, table, None, lens)
    verify(o.cpu(), lse.cpu(), q, kp, vp, table, None, lens)
    kp2, vp2 = (x.cuda().transpose(1, 2).contiguous().transpose(1, 2) for x in (kp, vp))
    wide = torch.full((2, 9), -7, dtype=torch.int32).cuda()
    wide[:, :table.shape[1]] = table.cuda()
    qq = q.cuda().contiguous()  # heads first
    out = torch.empty_like(q.cuda())
    o2, lse2 = L.clear_attn_decode(qq, kp2, vp2, wide[:, :table.shape[1]], torch.tensor(lens, dtype=torch.int32).cuda(), o=out)
    assert o2 is out and torch.equal(o2, o) and torch.equal(lse2, lse)


def test_cache_offsets_past_32_bits():
    # Pages 3 GB apart in one buffer of 2.2e9 elements and more.
    d, hk, page = 128, 1, 16
    buf = torch.zeros(3 * (1 << 30) + 4 * page * d, dtype=torch.bfloat16, device="cuda")
    kp = torch.as_strided(buf, (3, page, hk, d), (1 << 30, 2 * d, 2 * d, 1))
    vp = torch.as_strided(buf, (3, page, hk, d), (1 << 30, 2 * d, 2 * d, 1), d)
    gen = torch.Generator().manual_seed(8)
    k, v = (torch.randn(3, page, hk, d, generator=gen).to(torch.bfloat16) for _ in range(2))
    kp.copy_(k)
    vp.copy_(v)
    q = U.packed(gen, 2, 1, d, torch.bfloat16)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    o, lse = L.clear_attn_decode(q.cuda(), kp, vp, table.cuda(), torch.tensor([48], dtype=torch.int32).cuda())
    verify(o.cpu(), lse.cpu(), q, k, v, table, None, [48])


def test_bad_pages_are_reported():
    lens = [40, 20]
    q, kp, vp, table, _ = make(7, lens, 2, 1, 64, 16, torch.bfloat16)
    good, _ = call(q, kp, vp, table, None, lens)
    table[0, 1] = 1 << 30
    o, _ = call(q, kp, vp, table, None, lens)
    assert L.clear_attn_check() == 6 and L.clear_attn_check() == 0
    assert torch.equal(o[:, 1], good[:, 1])
    # longer than the table: cut to it, whatever the length says
    table[0, 1] = table[0, 0]
    table[1] = table[0]
    want, _ = call(q, kp, vp, table, None, [0, 16 * table.shape[1]])
    for n in (16 * table.shape[1] + 1, 2 ** 31 - 1):
        o, _ = call(q, kp, vp, table, None, [0, n])
        assert L.clear_attn_check() == 6 and torch.equal(o, want)
    call(q, kp, vp, table, None, [-5, -2 ** 31])
    assert L.clear_attn_check() == 0


def test_many_sequences_and_heads():
    gen = torch.Generator().manual_seed(12)
    lens = torch.randint(0, 40, (1500,), generator=gen).tolist()
    a = make(13, lens, 2, 1, 64, 16, torch.bfloat16)
    o, lse = call(*a, lens)
    q, kp, vp, table, _ = a
    some = [0, 3, 700, 1498, 1499]
    verify(o.cpu()[:, some], lse.cpu()[:, some], q[:, some], kp, vp, table[some], None, [lens[i] for i in some])
    assert not o.isnan().any()


def test_two_calls_at_once():
    # Two streams, a workspace each: neither sees the other.
    cases = [make(30 + i, [3000, 500], 8, 2, 128, 16, torch.bfloat16) for i in range(2)]
    want = [call(*c, [3000, 500]) for c in cases]
    args = [[x.cuda() for x in c[:4]] + [torch.tensor([3000, 500], dtype=torch.int32).cuda()] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i] = L.clear_attn_decode(*args[i], stream=s)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_captured_graph_follows_lengths_and_graphs_share_no_state():
    lens = [700, 40, 0]
    q, kp, vp, table, _ = make(9, [800] * 3, 4, 2, 128, 16, torch.bfloat16)
    q, kp, vp, table = q.cuda(), kp.cuda(), vp.cuda(), table.cuda()
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    ws = torch.full((L.decode_workspace_size(3, 4, 2, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):  # both use one workspace, one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(L.clear_attn_decode(q, kp, vp, table, sl, workspace=ws))
        graphs.append(g)
    sl.copy_(torch.tensor([1, 800, 333], dtype=torch.int32))
    want = L.clear_attn_decode(q, kp, vp, table, sl)
    for g in graphs:
        g.replay()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


def test_other_stream():
    lens = [3000, 12]
    q, kp, vp, table, _ = make(10, lens, 4, 2, 64, 16, torch.bfloat16)
    want = call(q, kp, vp, table, None, lens)
    s = torch.cuda.Stream()
    got = call(q, kp, vp, table, None, lens, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
