"""One workspace for batches of many sizes: what the size query gives for the largest serves every smaller one."""
import pytest
import torch

import local_circular_window_b200 as L
import seq_util as U
from test_seq_abi import backward, params

HEADS = [(16, 1, 128), (16, 1, 64), (8, 2, 64), (4, 4, 128), (30, 10, 64), (1, 1, 64)]


@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_size_holds_for_smaller_batches(hq, hk, d):
    last = 0
    for n in [1, 2, 100, 127, 128, 129, 640, 1000, 2048, 4736, 4737, 20000, 37888, 37889, 40000, 300000]:
        size = L.prompt_bwd_workspace_size(n, hq, hk, d)
        assert size >= last, (n, size, last)
        last = size


@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_calls_accept_the_largest_batchs_workspace(hq, hk, d):
    # Up to the check of the workspace, which comes last before the device is asked for.
    if torch.cuda.is_available():
        pytest.skip("would launch on the host buffers")
    size = L.prompt_bwd_workspace_size(40000, hq, hk, d)
    for n in (1, 128, 2048, 5000, 38000, 40000):
        p = params(n_seq=1, n_tok=n, q_heads=hq, kv_heads=hk, d=d)
        assert backward(p, size=size) not in (1, 2, 3), n
        assert backward(p, size=min(size, 255)) == 3


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_one_workspace_for_all(dtype):
    hq, hk, d = 16, 1, 64
    ws = torch.empty(L.prompt_bwd_workspace_size(40000, hq, hk, d), dtype=torch.uint8, device="cuda")
    gen = torch.Generator().manual_seed(1)
    for lens in ([1500, 548], [130], [3000, 20, 2000]):
        n = sum(lens)
        q, k, v, g = (U.packed(gen, h, n, d, dtype).cuda() for h in (hq, hk, hk, hq))
        ss = U.starts(lens).cuda()
        o, lse = L.clear_attn_prompt_fwd(q, k, v, ss)
        ws.fill_(0xFF)
        got = L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ss, workspace=ws)
        want = L.clear_attn_prompt_bwd(q, k, v, o, lse, g, ss)
        assert L.clear_attn_check() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
