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
                         ids=["few-items", "parts", "many-items"])
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
