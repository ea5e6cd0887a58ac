"""The token-sequence operators in 64 bits, from their definitions, and the error bounds that their
arithmetic allows.

Bounds. u = torch.finfo(t).eps / 2 bounds the relative error of one rounding to type t. The kernels round
probabilities (and, in the backward pass, P and dS) once to a 16-bit type and the result once to the
output's type; everything else is fp32. An fp32 score is off by at most (d + 2) 2^-24 sum |q k| / sqrt(d): with
standard normal q and k of d = 128, sum |q k| / sqrt(d) is about 7, and 20 at most here, so by less than 1.6e-4.
That moves a probability by as much, relative, and its normalised form by twice that: SCORE = 3.2e-4."""
import math

import torch

SCORE = 3.2e-4
LSE_ABS = 2e-4   # the score's error, and the logarithm's and the sum's roundings behind it


def unit(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half of the smallest step of t: what rounding may move a value below the normal range."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def packed(gen, heads, n, d, dtype, scale=1.0):
    """[heads, n, d] as a view of [n, heads, d] memory."""
    return (scale * torch.randn(n, heads, d, generator=gen)).to(dtype).transpose(0, 1)


def starts(lens):
    s = [0]
    for x in lens:
        s.append(s[-1] + x)
    return torch.tensor(s, dtype=torch.int32)


def pages(gen, lens, page, kv_heads, d, dtype, extra=3, scales=None):
    """(k_pages, v_pages, page_table) on the CPU: pages in random order, unused entries -1."""
    need = [-(-x // page) for x in lens]
    total = sum(need) + extra
    order = torch.randperm(total, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    out = []
    for i in range(2):
        x = torch.randn(total, page, kv_heads, d, generator=gen)
        if scales is not None:
            x = (x / scales[i][:, None]).clamp(-448, 448)
        out.append(x.to(dtype))
    return out[0], out[1], table


def attend(q, k, v, keep=None):
    """One head in 64 bits: (o, lse, sum_j a_j |v_j|) for q [m, d], k, v [n, d]; keep [m, n]."""
    q, k, v = q.double(), k.double(), v.double()
    x = q @ k.T / math.sqrt(q.shape[1])
    if keep is not None:
        x = x.masked_fill(~keep, -math.inf)
    lse = torch.logsumexp(x, -1)
    a = torch.exp(x - lse[:, None])
    return a @ v, lse, a @ v.abs()


def check(name, got, ref, tol):
    got, ref = got.double().cpu(), ref.double()
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got {got[i]:.6g}, "
                             f"expected {ref[i]:.6g}, allowed {tol[i]:.3g}")


def check_attention(name, o, lse, q, k, v, p_type, out_type, keep=None):
    """o and lse of one head against the definition."""
    ref, rl, av = attend(q, k, v, keep)
    check(name + " o", o, ref, (unit(p_type) + SCORE) * av + unit(out_type) * ref.abs() + tiny(out_type))
    check(name + " lse", lse, rl, torch.full_like(rl, LSE_ABS))


def gradients(q, k, v, g):
    """Gradients of causal attention of one head (q, k, v, g [n, d]) in 64 bits, and the error that the kernels'
    arithmetic allows each, for element type q.dtype: ((dq, dk, dv), (tolerances)) without the final
    rounding's part, which the caller adds once the shared heads are summed.

    P: half a step when rounded, and EP relative: the score's error and that of the given lse. dP: fp32, (d + 1) roundings
    of sum |g v|. D = sum g o from the rounded o. dS = P (dP - D): half a step when rounded, and what its
    factors are off by. Sums in fp32 add at most 2e-5 of the sum of magnitudes."""
    u, d = unit(q.dtype), q.shape[1]
    q, k, v, g = (x.double() for x in (q, k, v, g))
    n, s = q.shape[0], 1 / math.sqrt(d)
    keep = torch.ones(n, n, dtype=torch.bool).tril()
    o, lse, av = attend(q, k, v, keep)
    p = torch.exp((q @ k.T * s).masked_fill(~keep, -math.inf) - lse[:, None])
    dp = g @ v.T
    dd = (g * o).sum(-1, keepdim=True)
    ds = p * (dp - dd)
    ep = SCORE / 2 + LSE_ABS + 1e-6
    o_err = (u + SCORE) * av + u * o.abs()
    d_err = (g.abs() * o_err).sum(-1, keepdim=True)
    dp_err = (d + 1) * 2.0 ** -24 * (g.abs() @ v.abs().T)
    ds_err = (u + ep) * ds.abs() + p * (dp_err + d_err) * (1 + u + ep)
    more = 2e-5
    tol = (s * ((ds_err + more * ds.abs()) @ k.abs()), s * ((ds_err + more * ds.abs()).T @ q.abs()), (u + ep + more) * (p.T @ g.abs()))
    return (s * (ds @ k), s * (ds.T @ q), p.T @ g), tol
