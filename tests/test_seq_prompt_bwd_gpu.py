"""Gradients of causal attention over packed prompts, against the formula in 64 bits and against differences."""
import math

import pytest
import torch

import local_circular_window_b200 as L
import seq_util as U

pytestmark = pytest.mark.gpu


def make(seed, lens, hq, hk, d, dtype, behind=0):
    gen = torch.Generator().manual_seed(seed)
    n = sum(lens) + behind
    return tuple(U.packed(gen, h, n, d, dtype) for h in (hq, hk, hk, hq)) + (U.starts(lens),)


def both(q, k, v, g, ss, **kw):
    q, k, v, g, ss = (x.cuda() for x in (q, k, v, g, ss))
    o, lse = L.clear_attn_prompt_fwd(q, k, v, ss)
    return L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ss, **kw)


def verify(got, q, k, v, g, lens, kv_heads=None):
    hq, hk = q.shape[0], k.shape[0]
    group, at = hq // hk, 0
    dq, dk, dv = (x.cpu() for x in got)
    for s, n in enumerate(lens):
        t = slice(at, at + n)
        at += n
        for h in (range(hk) if kv_heads is None else kv_heads) if n else ():
            sums, tols = [0, 0], [0, 0]
            for i in range(h * group, (h + 1) * group):
                (rq, rk, rv), (tq, tk, tv) = U.gradients(q[i, t], k[h, t], v[h, t], g[i, t])
                U.check(f"sequence {s} head {i} dq", dq[i, t], rq, tq + U.unit(q.dtype) * rq.abs() + U.tiny(q.dtype))
                sums = [sums[0] + rk, sums[1] + rv]
                tols = [tols[0] + tk, tols[1] + tv]
            for name, x, ref, tol in (("dk", dk, sums[0], tols[0]), ("dv", dv, sums[1], tols[1])):
                U.check(f"sequence {s} kv head {h} {name}", x[h, t], ref, tol + U.unit(q.dtype) * ref.abs() + U.tiny(q.dtype))


CASES = [  # lens, q_heads, kv_heads, d, dtype
    ([1], 1, 1, 64, torch.bfloat16),
    ([64], 1, 1, 128, torch.bfloat16),
    ([128], 2, 1, 64, torch.float16),
    ([129], 3, 1, 128, torch.bfloat16),
    ([257, 1, 0, 127], 4, 2, 128, torch.float16),
    ([256, 512], 6, 2, 64, torch.bfloat16),
    ([700, 33], 5, 1, 128, torch.bfloat16),
    ([3] * 50 + [300, 0, 0, 2], 2, 2, 64, torch.float16),
    ([0, 0, 5], 1, 1, 128, torch.float16),
    ([1153], 2, 1, 128, torch.bfloat16),
    ([300, 0, 70], 16, 1, 64, torch.bfloat16),   # many heads to one: the group is split and joined
    ([140], 7, 1, 128, torch.float16),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_gradients(i):
    lens, hq, hk, d, dtype = CASES[i]
    q, k, v, g, ss = make(i, lens, hq, hk, d, dtype)
    got = both(q, k, v, g, ss)
    assert L.clear_attn_check() == 0
    verify(got, q, k, v, g, lens)


def test_many_items_for_each_block():
    lens = [260, 1000, 5, 900, 130, 512, 640, 77]
    q, k, v, g, ss = make(20, lens, 32, 16, 64, torch.bfloat16)
    got = both(q, k, v, g, ss)
    verify(got, q, k, v, g, lens, kv_heads=[0, 7, 15])
    again = both(q, k, v, g, ss)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same bits on every run


def test_against_differences():
    # The loss sum(o * g) of the 64-bit definition, moved along a random direction of q, k and v: the kernel's gradients
    # predict the change up to their own rounding (2^-8 of each, of random sign) and the third order of the step.
    n, d = 150, 64
    q, k, v, g, ss = make(30, [n], 2, 1, d, torch.bfloat16)
    dq, dk, dv = (x.double().cpu() for x in both(q, k, v, g, ss))
    gen = torch.Generator().manual_seed(31)
    keep = torch.ones(n, n, dtype=torch.bool).tril()

    def loss(q, k, v):
        return sum((U.attend(q[h], k[0], v[0], keep)[0] * g[h].double()).sum() for h in range(2))

    for which in range(3):
        r = [torch.zeros(x.shape, dtype=torch.float64) for x in (q, k, v)]
        r[which] = torch.randn(r[which].shape, generator=gen, dtype=torch.float64)
        e = 1e-4
        plus = loss(*(x.double() + e * y for x, y in zip((q, k, v), r)))
        minus = loss(*(x.double() - e * y for x, y in zip((q, k, v), r)))
        slope = float((plus - minus) / (2 * e))
        grad = (dq, dk, dv)[which]
        told = float((grad * r[which]).sum())
        # Each product grad * r is off by at most about 3 * 2^-8 of itself, with independent signs: six deviations.
        spread = 3 * 2.0 ** -8 * float((grad * r[which]).norm())
        assert abs(told - slope) <= 6 * spread, (which, told, slope, spread)


def test_sequences_do_not_touch_each_other():
    lens = [100, 200, 60]
    q, k, v, g, ss = (x.cuda() for x in make(21, lens, 2, 1, 64, torch.bfloat16, behind=90))
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    L.clear_attn_prompt_fwd(q, k, v, ss, o=o, lse=lse)
    outs = [torch.full_like(x, 7.0) for x in (q, k, v)]
    L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ss, *outs)
    assert all((x[:, 360:] == 7).all() for x in outs)
    for x in (q, k, v, g, o, lse):
        x[:, 100:300] = math.nan
        x[:, 360:] = math.inf
    outs2 = L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ss)
    for a, b in zip(outs, outs2):
        for t in (slice(0, 100), slice(300, 360)):
            assert torch.equal(a[:, t], b[:, t])


def test_strided_views_and_other_stream_give_the_same_bits():
    lens = [200, 57]
    q, k, v, g, ss = (x.cuda() for x in make(23, lens, 4, 2, 128, torch.float16))
    o, lse = L.clear_attn_prompt_fwd(q, k, v, ss)
    want = L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ss)
    buf = torch.cat([q, k, v]).transpose(0, 1).contiguous().transpose(0, 1)
    grad = torch.zeros_like(buf)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    L.clear_attn_prompt_bwd(buf[:4], buf[4:6], buf[6:], o.contiguous(), lse, g.contiguous(), ss, grad[:4], grad[4:6], grad[6:], stream=s)
    s.synchronize()
    assert torch.equal(grad, torch.cat(want))


def test_captured_graph_follows_offsets():
    q, k, v, g, ss = (x.cuda() for x in make(25, [300, 200, 100], 4, 4, 64, torch.bfloat16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = L.clear_attn_prompt_fwd(q, k, v, ss)
        got = L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ss)
    ss.copy_(torch.tensor([0, 10, 10, 600], dtype=torch.int32))
    want = both(q, k, v, g, ss)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_of_a_group_add_up():
    # The same keys given to each query head apart: their gradients sum to the shared head's, up to rounding.
    q, k, v, g, ss = make(26, [190], 4, 1, 64, torch.float16)
    _, dk, dv = both(q, k, v, g, ss)
    _, dk4, dv4 = both(q, k.expand(4, -1, -1).contiguous(), v.expand(4, -1, -1).contiguous(), g, ss)
    for a, b in ((dk, dk4), (dv, dv4)):
        s = b.double().sum(0, keepdim=True)
        # four roundings of the parts and one of the sum
        tol = U.unit(torch.float16) * (b.double().abs().sum(0, keepdim=True) + s.abs()) + 1e-6
        U.check("shared", a, s.cpu(), tol.cpu())
