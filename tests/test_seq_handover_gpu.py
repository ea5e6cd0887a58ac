"""The prompt kernels where blocks walk several items with d = 128, two buffers of scores and short rings: what one item
leaves behind for the next, against the definition in 64 bits."""
import pytest
import torch

import local_circular_window_b200 as L
import seq_util as U
import test_seq_prompt_bwd_gpu as B
from test_seq_prompt_gpu import make, verify

pytestmark = pytest.mark.gpu

LENS = [260, 1000, 5, 900, 130, 512, 640, 77]  # under 512 tokens a sequence: items are whole


def forward(q, k, v, ss):
    a = [x.cuda() for x in (q, k, v, ss)]
    o, lse = L.clear_attn_prompt_fwd(*a)
    assert L.clear_attn_check() == 0
    for _ in range(3):
        again = L.clear_attn_prompt_fwd(*a)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    return o.cpu(), lse.cpu()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_whole_items(dtype):
    # 864 items with one query tile and with two, about six a block.
    q, k, v, ss = make(50, LENS, 48, 16, 128, dtype)
    o, lse = forward(q, k, v, ss)
    verify(o, lse, q, k, v, LENS, heads=[0, 1, 17, 46, 47])


@pytest.mark.parametrize("group", range(4))
def test_one_warp_moves_its_maximum_late(group):
    # 32 rows of the second item's tile B (rows 384 to 499) meet their largest scores in the key tile before the diagonal's:
    # their warp rescales there, the three others do not.
    lens, d = [500] * 40, 128
    q, k, v, ss = make(51, lens, 8, 2, d, torch.bfloat16)
    u = torch.ones(d) / d ** 0.5
    flat = lambda x: x.float() - (x.float() @ u)[..., None] * u  # noqa: E731
    q, k = flat(q), flat(k)
    for s in range(len(lens)):
        at = 500 * s
        k[:, at + 256:at + 384] += 10 * u
        q[:, at + 384 + 32 * group:at + min(500, 416 + 32 * group)] += 12 * u  # 10 * 12 / sqrt(128) = 10.6: 15 powers of two
    q, k = (x.to(torch.bfloat16) for x in (q, k))
    o, lse = forward(q, k, v, ss)
    # sum |q k| / sqrt(d) is about 19 there, and 130 * 2^-24 of it is 1.5e-4: less than SCORE / 2.
    for s in (0, 7, 39):
        t = slice(500 * s, 500 * s + 500)
        keep = torch.ones(500, 500, dtype=torch.bool).tril()
        for h in (0, 3, 5):
            U.check_attention(f"sequence {s} head {h}", o[h, t], lse[h, t], q[h, t], k[h // 4, t], v[h // 4, t], q.dtype, q.dtype, keep)


@pytest.mark.parametrize("d,heads", [(128, 10), (64, 11)])
def test_split_items_that_end_in_one_tile(d, heads):
    # Key tiles split between the halves (under 300 items of 256 rows, 512 tokens a sequence and more): a block's last
    # items have one key tile, of which the second half has none. Some 600 items, about four a block.
    lens = [128 * 3 + 1] + [640, 1] * 3 + [1300, 2900]
    q, k, v, ss = make(52, lens, heads, heads, d, torch.float16)
    assert sum(lens) >= 512 * len(lens)
    o, lse = forward(q, k, v, ss)
    verify(o, lse, q, k, v, lens, heads=[0, heads - 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hk", [(32, 16), (32, 2)], ids=["whole-groups", "parts"])
def test_gradients(hq, hk, dtype):
    # 1024 items of query tiles, and 512 of key tiles, or 384 where groups are split into six parts.
    q, k, v, g, ss = B.make(53, LENS, hq, hk, 128, dtype)
    got = B.both(q, k, v, g, ss)
    assert L.clear_attn_check() == 0
    B.verify(got, q, k, v, g, LENS, kv_heads=[hk - 1] if hk == 2 else [0, 7, 15])
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(got, B.both(q, k, v, g, ss)))


def test_captured_step_in_fp16():
    # All of a training step's kernels, programmatic dependents among them, in a graph that is replayed with other data.
    q, k, v, g, ss = (x.cuda() for x in B.make(54, [300, 200, 100], 6, 2, 128, torch.float16))
    ws = torch.empty(L.prompt_bwd_workspace_size(600, 6, 2, 128), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = L.clear_attn_prompt_fwd(q, k, v, ss)
        got = L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ss, workspace=ws)
    for i, offsets in enumerate([[0, 10, 10, 600], [0, 599, 600, 600], [0, 200, 400, 600]]):
        ss.copy_(torch.tensor(offsets, dtype=torch.int32))
        g *= 2.0 ** -i
        v *= 2.0
        want = B.both(q, k, v, g, ss)
        ws.fill_(0xFF)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
