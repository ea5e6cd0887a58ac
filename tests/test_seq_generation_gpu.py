"""The token-sequence operators together, as a program that generates text uses them: prompts are rotated and
appended to the cache and attended to in one pass, then each step appends one token per sequence and attends over the cache."""
import math

import pytest
import torch

import local_circular_window_b200 as L
import seq_util as U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cache,hq,hk,d,page", [
    (torch.bfloat16, None, 6, 2, 128, 16), (torch.float16, None, 4, 4, 64, 7), (torch.bfloat16, "e4m3", 8, 1, 128, 48)])
def test_prompt_then_steps(dtype, cache, hq, hk, d, page):
    prompts, steps = [37, 1, 200, 0], 5
    total = [n + steps for n in prompts]
    gen = torch.Generator().manual_seed(77)
    seqs = [[U.packed(gen, h, n, d, dtype) for h in (hq, hk, hk)] for n in total]
    scales = [torch.full((hk,), 5.0 / 448).cuda() for _ in range(2)] if cache else [None, None]
    kp, vp, table = U.pages(gen, total, page, hk, d, torch.float8_e4m3fn if cache else dtype,
                            scales=[s.cpu() for s in scales] if cache else None)
    kp, vp, table = kp.cuda(), vp.cuda(), table.cuda()
    kw = dict(rot=d, theta=10000.0, pairing="halves", k_scale=scales[0], v_scale=scales[1])
    sc = dict(k_scale=scales[0], v_scale=scales[1])

    # the prompts, in one packed batch
    q, k, v = (torch.cat([s[i][:, :n] for s, n in zip(seqs, prompts)], 1).cuda() for i in range(3))
    ss = U.starts(prompts).cuda()
    seq_len = torch.tensor(prompts, dtype=torch.int32).cuda()
    k_rot = torch.empty_like(k)
    q_rot, _ = L.clear_attn_cache_append(k, v, kp, vp, table, ss, seq_len, q=q, k_out=k_rot, **kw)
    o, lse = L.clear_attn_prompt_fwd(q_rot, k_rot, v, ss)
    at = 0
    for n in prompts:
        t = slice(at, at + n)
        at += n
        keep = torch.ones(n, n, dtype=torch.bool).tril()
        for h in range(hq if n else 0):
            g = h * hk // hq
            U.check_attention("prompt", o[h, t], lse[h, t], q_rot[h, t].cpu(), k_rot[g, t].cpu(), v[g, t].cpu(), dtype, dtype, keep)

    # the steps: one captured graph, replayed with new tokens and lengths
    one = U.starts([1] * len(prompts)).cuda()
    q1, k1, v1 = (torch.empty(h, len(prompts), d, dtype=dtype, device="cuda") for h in (hq, hk, hk))
    q1r, out = torch.empty_like(q1), torch.empty_like(q1)
    lse1 = torch.empty(hq, len(prompts), device="cuda")
    ws = torch.empty(L.decode_workspace_size(len(prompts), hq, hk, d), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        seq_len += 1
        L.clear_attn_cache_append(k1, v1, kp, vp, table, one, seq_len, q=q1, q_out=q1r, **kw)
        L.clear_attn_decode(q1r, kp, vp, table, seq_len, o=out, lse=lse1, workspace=ws, **sc)
    p_type = torch.float16 if cache else dtype
    for step in range(steps):
        for x, i in ((q1, 0), (k1, 1), (v1, 2)):
            x.copy_(torch.stack([s[i][:, n + step] for s, n in zip(seqs, prompts)], 1))
        graph.replay()
        assert L.clear_attn_check() == 0
        for s, n in enumerate(prompts):
            m = n + step + 1
            pages = table[s, :-(-m // page)].long()
            kc, vc = (x.float()[pages].flatten(0, 1)[:m].double().cpu() for x in (kp, vp))
            if cache:
                kc, vc = kc * scales[0].double().cpu()[:, None], vc * scales[1].double().cpu()[:, None]
            for h in range(hq):
                g = h * hk // hq
                U.check_attention(f"step {step} sequence {s}", out[h, s:s + 1], lse1[h, s:s + 1], q1r[h, s:s + 1].cpu(), kc[:, g], vc[:, g],
                                  p_type, dtype)
            if not cache:  # the cache holds what the packed keys and values were
                assert torch.equal(vc[:, 0], seqs[s][2][0, :m].double())


def test_decode_step_is_the_prompts_last_row():
    # Attention over the cache gives the last row of causal attention over the same tokens.
    n, hq, hk, d = 300, 4, 2, 64
    gen = torch.Generator().manual_seed(78)
    q, k, v = (U.packed(gen, h, n, d, torch.bfloat16).cuda() for h in (hq, hk, hk))
    kp, vp, table = (x.cuda() for x in U.pages(gen, [n], 16, hk, d, torch.bfloat16))
    ss, sl = U.starts([n]).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    k_rot = torch.empty_like(k)
    q_rot, _ = L.clear_attn_cache_append(k, v, kp, vp, table, ss, sl, q=q, k_out=k_rot, rot=d)
    o, lse = L.clear_attn_prompt_fwd(q_rot, k_rot, v, ss)
    o1, lse1 = L.clear_attn_decode(q_rot[:, -1:].contiguous(), kp, vp, table, sl)
    # Both are within these of the definition (the bound of each, twice).
    for h in range(hq):
        g = h * hk // hq
        ref, _, av = U.attend(q_rot[h, -1:].cpu(), k_rot[g].cpu(), v[g].cpu())
        u = U.unit(torch.bfloat16)
        U.check("o", o1[h], o[h, -1:].double().cpu(), 2 * ((u + U.SCORE) * av + u * ref.abs()))
        assert abs(float(lse1[h, 0] - lse[h, -1])) <= 2 * U.LSE_ABS
    assert not math.isnan(float(lse1.sum()))
