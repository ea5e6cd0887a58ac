"""Offsets that decrease or reach outside, held in device memory: their sequences are left out and reported, by every operator,
and the other sequences keep their results."""
import pytest
import torch

import local_circular_window_b200 as L
import seq_util as U

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


BAD = [  # offsets, the sequences that remain
    ([0, 300, 50], [0]),
    ([0, 300, 350, 351], [0, 1]),
    ([-1, 50, 110, 350], [1, 2]),
    ([200, 350, 100, 150], [0, 2]),               # the sequence in front lies behind
    ([340, 350, 260, 300, 10, 200], [0, 2, 4]),
    ([0, 100] + [2 ** 31 - 1, -2 ** 31, 100] * 20 + [350], [0, 61]),   # more of them than lanes
]


@pytest.mark.parametrize("case", range(len(BAD)))
@pytest.mark.parametrize("hq,hk,d,dtype", [(4, 4, 64, torch.bfloat16), (16, 1, 128, torch.float16), (300, 300, 64, torch.float16)],
                         ids=["group1", "parts", "no-parts"])
def test_gradients(case, hq, hk, d, dtype):
    bad, good = BAD[case]
    n = 350
    gen = torch.Generator().manual_seed(case)
    q, k, v, g = (U.packed(gen, h, n, d, dtype).cuda() for h in (hq, hk, hk, hq))
    ws = torch.empty(L.prompt_bwd_workspace_size(n, hq, hk, d), dtype=torch.uint8, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(hq, n, device="cuda")
    L.clear_attn_prompt_fwd(q, k, v, ints(bad), o=o, lse=lse)
    assert L.clear_attn_check() == 6
    got = [torch.full_like(x, 7.0) for x in (q, k, v)]
    ws.fill_(0xFF)
    L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ints(bad), *got, workspace=ws)
    assert L.clear_attn_check() == 6 and L.clear_attn_check() == 0
    seen = torch.zeros(n, dtype=torch.bool)
    for s in good:
        a, b = bad[s], bad[s + 1]
        seen[a:b] = True
        o1, lse1 = L.clear_attn_prompt_fwd(q, k, v, ints([a, b]))
        # the split of the keys goes by the number of sequences, so o need not have the same bits
        for h in (0, hq - 1):
            keep = torch.ones(b - a, b - a, dtype=torch.bool).tril()
            U.check_attention(f"sequence {s}", o[h, a:b].cpu(), lse[h, a:b].cpu(), q[h, a:b].cpu(), k[h * hk // hq, a:b].cpu(),
                              v[h * hk // hq, a:b].cpu(), dtype, dtype, keep)
        want = L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ints([a, b]))
        for x, y in zip(got, want):
            assert torch.equal(x[:, a:b], y[:, a:b])
    for x in got:
        assert (x[:, ~seen.cuda()] == 7).all()  # rows of no sequence


@pytest.mark.parametrize("case", range(len(BAD)))
@pytest.mark.parametrize("hq,hk", [(0, 1), (4, 2)], ids=["one-warp", "warps"])
def test_append(case, hq, hk):
    bad, good = BAD[case]
    n, d, page = 350, 64, 16
    gen = torch.Generator().manual_seed(case)
    lens = [400] * (len(bad) - 1)
    kp, vp, table = (x.cuda() for x in U.pages(gen, lens, page, hk, d, torch.bfloat16))
    k, v = (U.packed(gen, hk, n, d, torch.bfloat16).cuda() for _ in range(2))
    q = U.packed(gen, hq, n, d, torch.bfloat16).cuda() if hq else None
    k_out = torch.full_like(k, 7.0)
    a, b = kp.clone(), vp.clone()
    L.clear_attn_cache_append(k, v, a, b, table, ints(bad), ints(lens), q=q, k_out=k_out, rot=32)
    assert L.clear_attn_check() == 6 and L.clear_attn_check() == 0
    want_k, want_v, want_out = kp.clone(), vp.clone(), torch.full_like(k, 7.0)
    for s in good:  # each alone: its new tokens are the last of 400
        t = slice(bad[s], bad[s + 1])
        part = torch.empty_like(k[:, t])
        L.clear_attn_cache_append(k[:, t], v[:, t], want_k, want_v, table[s:s + 1], ints([0, t.stop - t.start]), ints([400]), k_out=part, rot=32)
        want_out[:, t] = part
    assert L.clear_attn_check() == 0
    assert torch.equal(a, want_k) and torch.equal(b, want_v) and torch.equal(k_out, want_out)


def test_tokens_of_two_sequences_stay_inside():
    # Rows 40 to 49 belong to two sequences: what they get is not defined, all others are.
    n, d = 150, 64
    gen = torch.Generator().manual_seed(3)
    kp, vp, table = (x.cuda() for x in U.pages(gen, [200] * 3, 16, 1, d, torch.bfloat16))
    k, v = (U.packed(gen, 1, n, d, torch.bfloat16).cuda() for _ in range(2))
    a, b = kp.clone(), vp.clone()
    L.clear_attn_cache_append(k, v, a, b, table, ints([0, 50, 40, 150]), ints([200] * 3))
    assert L.clear_attn_check() == 6
    rows = lambda x, s: x[table[s, :13].long()].flatten(0, 1)[:200, 0]  # noqa: E731
    assert torch.equal(rows(a, 0)[150:190], k[0, :40]) and torch.equal(rows(a, 2)[100:], k[0, 50:])
    assert torch.equal(rows(b, 0)[150:190], v[0, :40]) and torch.equal(rows(b, 2)[100:], v[0, 50:])
    assert torch.equal(rows(a, 1), rows(kp, 1))


def test_expired_wait_is_not_hidden_by_a_bad_page():
    # A bad index and an expired wait before one look: the expired wait, whose outputs are invalid, is told first.
    gen = torch.Generator().manual_seed(4)
    q = U.packed(gen, 1, 1, 64, torch.bfloat16).cuda()
    kp, vp, table = (x.cuda() for x in U.pages(gen, [20], 16, 1, 64, torch.bfloat16))
    table[0, 0] = -5
    for first in (False, True):
        if first:
            assert L.selftest_expiry(20) == 0
        L.clear_attn_decode(q, kp, vp, table, ints([20]))
        if not first:
            assert L.selftest_expiry(20) == 0
        assert L.clear_attn_check() == 5 and L.device_diag()[:2] == [5, 31]
        assert L.clear_attn_check() == 6 and L.device_diag()[:2] == [16, 33]
        assert L.clear_attn_check() == 0
