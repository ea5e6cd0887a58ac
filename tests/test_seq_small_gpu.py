"""Small values in fp16: many keys of little weight beside a strong one. fp16's steps are absolute below 2^-14, so what lies there
would be lost or doubled with one sign, if it were rounded as it is."""
import math

import pytest
import torch

import local_circular_window_b200 as L
import seq_util as U

pytestmark = pytest.mark.gpu

# Scores of the strong key above the others, in natural units: the others weigh 2^-25.6, 2^-24.4 and 2^-20.4 of it. In fp16 as they
# are the first would be 0, the second 2^-24 and the third off by a thirtieth.
GAPS = [17.75, 16.9375, 14.125]


def weak(gen, n, d, dtype):
    """q, k, v [1, n, d] with scores of 0 but for the first key's, and values of one sign in each column."""
    q, k = torch.zeros(1, n, d), torch.zeros(1, n, d)
    q[..., 0] = d ** 0.5 if d == 64 else 8.0
    sign = torch.randint(0, 2, (d,), generator=gen) * 2.0 - 1.0
    v = (1 + torch.rand(1, n, d, generator=gen)) * sign
    v[:, 0] = 0
    return q.to(dtype), k.to(dtype), v.to(dtype)


def check(name, o, lse, q, k, v, out_type, keep=None):
    ref, rl, av = U.attend(q, k, v, keep)
    u = U.unit(torch.float16)
    # beside the relative half steps, 2^-32 of the strong key's weight for each key (2^-25 in steps of 2^-24, lifted by 2^7)
    lost = 2.0 ** -32 * (v.double().abs().cumsum(0)[-ref.shape[0]:] if keep is not None else v.double().abs().sum(0))
    U.check(name, o, ref, (u + U.SCORE) * av + U.unit(out_type) * ref.abs() + U.tiny(out_type) + lost)
    U.check(name + " lse", lse, rl, torch.full_like(rl, U.LSE_ABS))


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("d,heads", [(64, 2), (64, 20), (128, 2), (128, 20)])  # few heads: split keys
def test_prompt(gap, d, heads):
    n = 4096
    q, k, v = weak(torch.Generator().manual_seed(1), n, d, torch.float16)
    k[0, 0, 0] = gap * d ** 0.5 / float(q[0, 0, 0])
    a = [x.expand(heads, -1, -1).contiguous().cuda() for x in (q, k, v)]
    o, lse = L.clear_attn_prompt_fwd(*a, U.starts([n]).cuda())
    assert L.clear_attn_check() == 0
    t = slice(n - 300, n)
    keep = torch.ones(n, n, dtype=torch.bool).tril()[t]
    for h in (0, heads - 1):
        check(f"head {h}", o[h, t], lse[h, t], q[0, t], k[0], v[0], torch.float16, keep)


@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("dtype,cache", [(torch.float16, None), (torch.float16, "e4m3"), (torch.bfloat16, "e4m3")])
def test_decode(gap, dtype, cache):
    # 640 sequences that share their pages: a block has whole ones, so one warp meets the strong key and a quarter of the others.
    n, d, page, many = 2047, 64, 16, 640
    gen = torch.Generator().manual_seed(2)
    kind = torch.float8_e4m3fn if cache else dtype
    q, k, v = weak(gen, n, d, torch.float16)
    k[0, 0, 0] = 16.0 if cache else gap
    q = q[:, :1].to(dtype)
    pages = -(-n // page)
    order = torch.randperm(pages, generator=gen)
    kp, vp = (torch.zeros(pages, page, 1, d, dtype=kind) for _ in range(2))
    for x, y in ((k, kp), (v, vp)):
        rows = torch.zeros(pages * page, d)
        rows[:n] = x[0].float()
        y[order] = rows.view(pages, page, 1, d).to(kind)
    scales = [torch.tensor([gap / 16.0 if cache else 1.0]), torch.tensor([1.0])]
    kw = {"k_scale": scales[0].cuda(), "v_scale": scales[1].cuda()} if cache else {}
    table = order.to(torch.int32).expand(many, -1).contiguous().cuda()
    o, lse = L.clear_attn_decode(q.expand(1, many, d).contiguous().cuda(), kp.cuda(), vp.cuda(), table, torch.full((many,), n, dtype=torch.int32).cuda(), **kw)
    assert L.clear_attn_check() == 0
    kc, vc = (x.float()[order].flatten(0, 1)[:n, 0].double() * s.double() for x, s in ((kp, scales[0]), (vp, scales[1])))
    for s in (0, 1, 333, many - 1):
        check(f"sequence {s}", o[0, s:s + 1], lse[0, s:s + 1], q[0], kc, vc, dtype)


def gradients(q, k, v, g, lens):
    o, lse = L.clear_attn_prompt_fwd(q.cuda(), k.cuda(), v.cuda(), U.starts(lens).cuda())
    got = L.clear_attn_prompt_bwd(q.cuda(), k.cuda(), v.cuda(), o, lse, g.cuda(), U.starts(lens).cuda())
    assert L.clear_attn_check() == 0
    return [x.cpu() for x in got]


def check_gradients(got, q, k, v, g, at=0):
    """One kv head and its group of query heads, one sequence."""
    n, d = k.shape[1:]
    t = slice(at, at + n)
    keep = torch.ones(n, n, dtype=torch.bool).tril()
    dk = dv = tk = tv = 0
    for h in range(q.shape[0]):
        (rq, rk, rv), (eq, ek, ev) = U.gradients(q[h], k[0], v[0], g[h])
        # D reaches the key gradients as three 16-bit parts, to 2^-38: at most 2^-37 of each P
        p = torch.exp((q[h].double() @ k[0].double().T / math.sqrt(d)).masked_fill(~keep, -math.inf) -
                      U.attend(q[h], k[0], v[0], keep)[1][:, None])
        ek = ek + 2.0 ** -37 / math.sqrt(d) * (p.T @ q[h].double().abs())
        U.check(f"head {h} dq", got[0][h, t], rq, eq + U.unit(q.dtype) * rq.abs() + U.tiny(q.dtype))
        dk, dv, tk, tv = dk + rk, dv + rv, tk + ek, tv + ev
    U.check("dk", got[1][0, t], dk, tk + U.unit(q.dtype) * dk.abs() + U.tiny(q.dtype))
    U.check("dv", got[2][0, t], dv, tv + U.unit(q.dtype) * dv.abs() + U.tiny(q.dtype))


@pytest.mark.parametrize("d,group", [(64, 1), (64, 3), (128, 16)])
@pytest.mark.parametrize("which", ["dq", "dk"])
def test_small_upstream_gradients(which, d, group):
    # dS is about 2^-25 here, a step of fp16 in all; the other factor of dq or dk is large, so that the result is not.
    gen = torch.Generator().manual_seed(10)
    n = 600
    q, k, v, g = (U.packed(gen, h, n, d, torch.float16) for h in (group, 1, 1, group))
    q, k = (q / 1024, k * 64) if which == "dq" else (q * 64, k / 1024)
    g = (g.float() * 2.0 ** -20).half()
    check_gradients(gradients(q, k, v, g, [n]), q, k, v, g)


@pytest.mark.parametrize("gap", GAPS)
def test_gradients_of_weak_keys(gap):
    n, d = 2048, 64
    gen = torch.Generator().manual_seed(11)
    q, k, v = weak(gen, n, d, torch.float16)
    k[0, 0, 0] = gap
    g = (1 + torch.rand(1, n, d, generator=gen)).half()
    check_gradients(gradients(q, k, v, g, [n]), q, k, v, g)


@pytest.mark.parametrize("d,group", [(64, 1), (128, 4)])
def test_large_upstream_gradients(d, group):
    # dP is about 4e5, out of fp16's range; dq, dk and dv are in it.
    gen = torch.Generator().manual_seed(12)
    n = 300
    q, k, v, g = (U.packed(gen, h, n, d, torch.float16) for h in (group, 1, 1, group))
    q, k, v, g = q / 4096, k / 4096, v * 200, g * 200
    check_gradients(gradients(q, k, v, g, [n]), q, k, v, g)


def test_sequences_of_unlike_size():
    gen = torch.Generator().manual_seed(13)
    lens, d = [200, 140, 300], 128
    q, k, v, g = (U.packed(gen, h, sum(lens), d, torch.float16) for h in (2, 1, 1, 2))
    g[:, :200] *= 100
    g[:, 200:340] *= 1e-4
    got = gradients(q, k, v, g, lens)
    for at, n in ((0, 200), (200, 140), (340, 300)):
        t = slice(at, at + n)
        check_gradients(got, q[:, t], k[:, t], v[:, t], g[:, t], at)
    for x in (q, k, v, g):  # what one of them holds is nothing to the others
        x[:, 200:340] = math.inf
    v[:, 250] = math.nan
    again = gradients(q, k, v, g, lens)
    for t in (slice(0, 200), slice(340, 640)):
        assert all(torch.equal(a[:, t], b[:, t]) for a, b in zip(got, again))


def test_zero_gradients_and_rows():
    gen = torch.Generator().manual_seed(14)
    q, k, v, g = (U.packed(gen, h, 200, 64, torch.float16) for h in (2, 1, 1, 2))
    assert all((x == 0).all() for x in gradients(q, k, v, torch.zeros_like(g), [200])[:2])
    g[:, ::3] = 0
    check_gradients(gradients(q, k, v, g, [200]), q, k, v, g)
    v[:] = 0
    check_gradients(gradients(q, k, v, g, [200]), q, k, v, g)


def test_gradients_of_far_scores():
    # Scores of a million: each key is its own query's only one. q k is exact (multiples of 90000 under 2^24); its
    # logarithm to base 2 in fp32 has steps of 1/8, and lse, a natural one, of 1/16. The forward rounds to them twice
    # (2 * 1/16 in base 2) and lse once, the gradients lse sqrt(d) (steps of 1: 0.5 / sqrt(d)) or lse log2 e (1/16 in base 2), and the scale's
    # own rounding (2^-24 of a million: 0.06) does not cancel between base 2 and lse: P = 1 is off by e^0.3 at most.
    n, d = 300, 128
    gen = torch.Generator().manual_seed(15)
    q = (300.0 * (torch.randint(0, 2, (1, n, d), generator=gen) * 2 - 1)).half()
    q[:, 100:200] /= 16  # and rows with ordinary statistics between them
    v, g = (U.packed(gen, 1, n, d, torch.float16) for _ in range(2))
    dq, dk, dv = (x[0].double() for x in gradients(q, q, v, g, [n]))
    own = torch.ones(n, dtype=torch.bool)
    own[100:200] = False  # their own key is not their largest: another's is
    x = (q[0].double() @ q[0].double().T / math.sqrt(d)).masked_fill(~torch.ones(n, n, dtype=torch.bool).tril(), -math.inf)
    p = torch.softmax(x, -1)
    assert (p[own].amax(-1) == 1).all() and (p[own].argmax(-1) == torch.arange(n)[own]).all()
    off = math.exp(0.3) - 1
    ref, size = p.T @ g[0].double(), p.T @ g[0].double().abs()
    U.check("dv", dv, ref, off * size + 2.0 ** -9 * size + U.tiny(torch.float16))
    # dP and D are equal up to o's rounding: dq and dk are no more than that leaves
    left = math.exp(0.3) * (g[0].double().abs() * v[0].double().abs()).sum(-1) * 2.0 ** -10
    scale = 300 / math.sqrt(d)
    assert (dq[own].abs() <= (left * scale)[own][:, None]).all()
    assert not dk.isnan().any() and not dk.isinf().any()
    later = torch.arange(n) >= 200  # keys that only their own rows read
    assert (dk[later].abs() <= (left * scale)[later][:, None]).all()


@pytest.mark.parametrize("d,group", [(64, 2), (128, 1)])
def test_gradients_of_far_sums(d, group):
    # D = dO o is about 4e7 in the first rows, and less further on.
    gen = torch.Generator().manual_seed(16)
    n = 260
    q, k, v, g = (U.packed(gen, h, n, d, torch.float16) for h in (group, 1, 1, group))
    q, k, v, g = q / 8192, k / 8192, v * 4000, g * 1000
    assert (g[0].double() * v[0].double()).sum(-1)[0].abs() > 8e6 or d == 64
    check_gradients(gradients(q, k, v, g, [n]), q, k, v, g)
