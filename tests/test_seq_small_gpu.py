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
    n, d, page = 8191, 64, 16
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
    o, lse = L.clear_attn_decode(q.cuda(), kp.cuda(), vp.cuda(), order[None].to(torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda(), **kw)
    assert L.clear_attn_check() == 0
    kc, vc = (x.float()[order].flatten(0, 1)[:n, 0].double() * s.double() for x, s in ((kp, scales[0]), (vp, scales[1])))
    check("decode", o[0], lse[0], q[0], kc, vc, dtype)
    assert not math.isnan(float(o.float().sum()))
