"""Cases of the token-sequence attention operators, with each operator in its plain form.

Four operators share one picture of a batch. The tokens of all sequences lie one after another
along one axis; seq_start (int32 [n_seq + 1]) says where each sequence's begin and end. A paged
cache holds keys and values of earlier tokens: page_table (int32 [n_seq, max_pages]) names the pages
of each sequence, seq_len (int32 [n_seq]) how many tokens it has in all.

  append   rotates new queries and keys by their positions and stores keys and values in the cache
  decode   attention of one new token of each sequence over its cached keys and values
  prompt   causal attention within each sequence of a packed batch, with grouped key/value heads
  train    the same attention forward, then its gradients

Tensors are [heads, tokens, d]; they are views of [tokens, heads, d] memory, as a projection's output is.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One decoding step of a small batch: sixteen sequences get one token each. Latency counts.
        {"name": "append-step-16", "op": "append", "dtype": "bf16", "cache": "bf16", "q_heads": 24, "kv_heads": 8, "d": 128,
         "page": 16, "rot": 128, "pairing": "halves", "theta": 10000.0, "new": ",".join(["1"] * 16),
         "before": "511,0,77,1023,300,16,15,640,31,900,128,5,255,256,257,700"},
        # Prompts of a mixed batch as they arrive, two of them continuing an earlier turn.
        {"name": "append-prompts-ragged", "op": "append", "dtype": "bf16", "cache": "bf16", "q_heads": 32, "kv_heads": 8,
         "d": 128, "page": 64, "rot": 128, "pairing": "adjacent", "theta": 500000.0, "new": "4608,1,777,2048,513,130,1000",
         "before": "0,4607,0,1500,0,33,0"},
        # A long prompt into an 8-bit cache; a quarter of each head is rotated, at far positions.
        {"name": "append-prompt-e4m3", "op": "append", "dtype": "fp16", "cache": "e4m3", "q_heads": 32, "kv_heads": 8, "d": 128,
         "page": 32, "rot": 32, "pairing": "halves", "theta": 10000.0, "new": "16384", "before": "4321"},
        # A single user's next token over a short history: the smallest call.
        {"name": "decode-one-777", "op": "decode", "dtype": "bf16", "cache": "bf16", "q_heads": 24, "kv_heads": 8, "d": 128,
         "page": 16, "len": "777"},
        # A serving batch of many lengths, one of them just begun and one slot empty.
        {"name": "decode-ragged-48", "op": "decode", "dtype": "bf16", "cache": "bf16", "q_heads": 32, "kv_heads": 8, "d": 128,
         "page": 16, "len": _ragged(46, 8192) + ",1,0"},
        # One very long context alone: all of the machine works on one sequence.
        {"name": "decode-long-131072", "op": "decode", "dtype": "fp16", "cache": "fp16", "q_heads": 32, "kv_heads": 4, "d": 128,
         "page": 64, "len": "131071"},
        # A large batch over an 8-bit cache.
        {"name": "decode-e4m3-96", "op": "decode", "dtype": "bf16", "cache": "e4m3", "q_heads": 24, "kv_heads": 8, "d": 128,
         "page": 32, "len": _ragged(96, 6000)},
        # Short prompts packed together, every head with its own keys: latency counts.
        {"name": "prompt-short-packed", "op": "prompt", "dtype": "fp16", "q_heads": 16, "kv_heads": 16, "d": 64,
         "len": "77,1,130,512,33,256,200,64"},
        # A mixed batch of prompts.
        {"name": "prompt-ragged", "op": "prompt", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "d": 128,
         "len": "4608,777,2049,130,1000,513"},
        # One long prompt.
        {"name": "prompt-long-16896", "op": "prompt", "dtype": "bf16", "q_heads": 24, "kv_heads": 8, "d": 128, "len": "16896"},
        # A training step on packed samples with narrow heads.
        {"name": "train-packed-d64", "op": "train", "dtype": "fp16", "q_heads": 16, "kv_heads": 16, "d": 64,
         "len": "1024,512,300,1,2000,259"},
        # A training step on two full samples and a short one.
        {"name": "train-4608", "op": "train", "dtype": "bf16", "q_heads": 24, "kv_heads": 8, "d": 128, "len": "4608,4608,1001"},
    ]


def _ragged(n, longest):
    """n lengths between longest/64 and longest, spread by the golden ratio over the logarithm."""
    return ",".join(str(max(1, int(longest * 64.0 ** -((i * 0.6180339887498949) % 1.0)))) for i in range(n))


def _ints(text):
    return [int(x) for x in text.split(",")]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prompt", "train"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    kv_heads = rng.choice([1, 2, 4, 8, 16] if op in ("prompt", "train") else [1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if g * kv_heads <= (24 if op == "train" else 32)])
    c = {"op": op, "dtype": dtype, "q_heads": kv_heads * group, "kv_heads": kv_heads, "d": d}
    if op in ("append", "decode"):
        c["cache"] = rng.choice([dtype, dtype, "e4m3"])
        c["page"] = rng.choice([1, 7, 16, 16, 32, 64, 128, 256])
    if op == "append":
        n = _log(rng, 1, 128)
        step = rng.random() < 0.4
        new = [1 if step else _log(rng, 1, max(1, 8000 // n)) for _ in range(n)]
        before = [rng.choice([0, _log(rng, 1, 2000)]) for _ in range(n)]
        if n == 1:
            before = [rng.choice([0, _log(rng, 1, 30000)])]
        c |= {"rot": rng.choice([0, d // 4, d // 2, d, d]), "pairing": rng.choice(["adjacent", "halves"]),
              "theta": rng.choice([10000.0, 500000.0]), "new": ",".join(map(str, new)), "before": ",".join(map(str, before))}
    elif op == "decode":
        n = _log(rng, 1, 128)
        c["len"] = ",".join(str(_log(rng, 1, max(2, min(131072, 150000 // n)))) for _ in range(n))
    elif op == "prompt":
        n = _log(rng, 1, 40)
        c["len"] = ",".join(str(_log(rng, 1, int(14000 / math.sqrt(n)))) for _ in range(n))
    else:
        n = _log(rng, 1, 24)
        c["len"] = ",".join(str(_log(rng, 1, int(6000 / math.sqrt(n)))) for _ in range(n))
    return c


# ------------------------------------------------------------------------------------------- work
def work(case):
    hq, hk, d, e = case["q_heads"], case["kv_heads"], case["d"], _BYTES[case["dtype"]]
    if case["op"] == "append":
        n, ec = sum(_ints(case["new"])), _BYTES[case["cache"]]
        # q, k, v read; rotated q and k written, and the cache's new rows
        return {"bytes": n * d * (e * (2 * hq + 3 * hk) + ec * 2 * hk), "flops": 3 * n * case["rot"] * (hq + hk)}
    lens = _ints(case["len"])
    n = sum(lens)
    if case["op"] == "decode":
        ec, s = _BYTES[case["cache"]], len(lens)
        return {"bytes": 2 * n * hk * d * ec + s * hq * (2 * d * e + 4) + 4 * sum(-(-x // case["page"]) for x in lens),
                "flops": 4 * n * hq * d}
    pairs = sum(x * (x + 1) // 2 for x in lens)
    if case["op"] == "prompt":
        return {"bytes": n * (e * d * 2 * (hq + hk) + 4 * hq), "flops": 4 * d * hq * pairs}
    # forward and backward: q, k, v, dO read; o, lse, dq, dk, dv written; 2 + 5 products
    return {"bytes": n * (e * d * (4 * hq + 4 * hk) + 4 * hq), "flops": 14 * d * hq * pairs}


# ----------------------------------------------------------------------------------------- inputs
def _starts(lens):
    s = [0]
    for x in lens:
        s.append(s[-1] + x)
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def _normal(gen, heads, n, d, dtype):
    return torch.randn(n, heads, d, generator=gen, device="cuda").to(dtype).transpose(0, 1)


def _pages(case, lens, gen):
    """A cache of random contents, and a page table whose pages lie in random order; unused entries are -1."""
    page, hk, d = case["page"], case["kv_heads"], case["d"]
    need = [-(-x // page) for x in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    order_h, at = order.cpu(), 0
    for i, m in enumerate(need):
        table[i, :m] = order_h[at:at + m]
        at += m
    st = {"page_table": table.cuda(), "k_scale": None, "v_scale": None}
    for name in ("k", "v"):
        x = torch.randn(total, page, hk, d, generator=gen, device="cuda")
        if case["cache"] == "e4m3":
            scale = (0.5 + torch.rand(hk, generator=gen, device="cuda")) / 64.0
            st[name + "_scale"] = scale
            x = (x / scale[:, None]).clamp(-448.0, 448.0)
        st[name + "_pages"] = x.to(_TYPES[case["cache"]])
    return st


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    dtype, hq, hk, d = _TYPES[case["dtype"]], case["q_heads"], case["kv_heads"], case["d"]
    st = {"case": dict(case)}
    if case["op"] == "append":
        new, before = _ints(case["new"]), _ints(case["before"])
        n = sum(new)
        st |= _pages(case, [a + b for a, b in zip(new, before)], gen)
        st |= {"q": _normal(gen, hq, n, d, dtype), "k": _normal(gen, hk, n, d, dtype), "v": _normal(gen, hk, n, d, dtype)}
        st |= {"q_out": torch.empty_like(st["q"]), "k_out": torch.empty_like(st["k"]), "seq_start": _starts(new),
               "seq_len": torch.tensor([a + b for a, b in zip(new, before)], dtype=torch.int32, device="cuda")}
        return st
    lens = _ints(case["len"])
    if case["op"] == "decode":
        st |= _pages(case, lens, gen)
        st["q"] = _normal(gen, hq, len(lens), d, dtype)
        st["o"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(hq, len(lens), dtype=torch.float32, device="cuda")
        st["seq_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        return st
    n = sum(lens)
    st |= {"lens": lens, "seq_start": _starts(lens), "q": _normal(gen, hq, n, d, dtype), "k": _normal(gen, hk, n, d, dtype),
           "v": _normal(gen, hk, n, d, dtype)}
    st["o"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(hq, n, dtype=torch.float32, device="cuda")
    if case["op"] == "train":
        st["dO"] = _normal(gen, hq, n, d, dtype)
        st |= {"dq": torch.empty_like(st["q"]), "dk": torch.empty_like(st["k"]), "dv": torch.empty_like(st["v"])}
    return st


# -------------------------------------------------------------------------------------------- run
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _raw(x):
    """8-bit values as bytes, which every indexing operation takes; others as they are."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _append_plain(st):
    c = st["case"]
    n, start, page = st["q"].shape[1], st["seq_start"].long(), c["page"]
    tok = torch.arange(n, device="cuda")
    seq = torch.searchsorted(start, tok, right=True) - 1
    pos = tok - start[seq + 1] + st["seq_len"].long()[seq]
    out = {}
    rot = c["rot"]
    if rot:
        freq = c["theta"] ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = pos.double()[:, None] * freq
        cos, sin = angle.cos().float(), angle.sin().float()
    for name in ("q", "k"):
        x = st[name].float()
        if rot:
            if c["pairing"] == "adjacent":
                a, b = x[..., 0:rot:2], x[..., 1:rot:2]
                turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
            else:
                a, b = x[..., :rot // 2], x[..., rot // 2:rot]
                turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
            x = torch.cat((turned, x[..., rot:]), -1)
        out[name] = x
    where = st["page_table"][seq, pos // page].long(), pos % page
    for name, x in (("k", out["k"]), ("v", st["v"].float())):
        x = x.transpose(0, 1)
        if c["cache"] == "e4m3":
            x = (x / st[name + "_scale"][:, None]).clamp(-448.0, 448.0)
        pages = st[name + "_pages"]
        _raw(pages)[where] = _raw(x.to(pages.dtype))
    return [out["q"].to(st["q"].dtype), out["k"].to(st["k"].dtype), st["k_pages"], st["v_pages"]]


def _decode_plain(st):
    c = st["case"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["d"]
    s, m = st["page_table"].shape
    table = st["page_table"].long().clamp(min=0)
    # [sequences, kv heads, keys, d]; what lies behind a sequence's end does not count
    k, v = (_raw(st[x + "_pages"])[table].view(_TYPES[c["cache"]]).float().reshape(s, m * c["page"], hk, d).transpose(1, 2)
            for x in ("k", "v"))
    if c["cache"] == "e4m3":
        k, v = k * st["k_scale"][:, None, None], v * st["v_scale"][:, None, None]
    kept = torch.arange(m * c["page"], device="cuda") < st["seq_len"][:, None]
    v = v * kept[:, None, :, None]
    q = st["q"].float().transpose(0, 1).reshape(s, hk, hq // hk, d)
    x = (q @ k.transpose(-1, -2)) / math.sqrt(d)
    x = torch.where(kept[:, None, None], x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)  # a row with no key keeps no infinity
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total.clamp(min=torch.finfo(torch.float32).tiny)
    lse = (top + torch.log(total)).reshape(s, hq).transpose(0, 1)
    return [o.reshape(s, hq, d).transpose(0, 1).to(st["q"].dtype), lse]


def _blocks(st):
    """The parts of a packed batch, one sequence and as many key/value heads at a time as two gigabytes of scores allow:
    the query heads, the key/value heads and the tokens of each, and the pairs that come later."""
    hk, at = st["case"]["kv_heads"], 0
    group = st["case"]["q_heads"] // hk
    for n in st["lens"]:
        t = slice(at, at + n)
        later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        step = max(1, (1 << 29) // (group * n * n))
        for h in range(0, hk, step):
            hs = slice(h, min(hk, h + step))
            yield slice(h * group, hs.stop * group), hs, t, later
        at += n


def _grouped(x, like):
    """[query heads, n, d] as [key/value heads, heads of each, n, d]."""
    return x.float().unflatten(0, (like.shape[0], -1))


def _prompt_plain(st):
    scale = 1.0 / math.sqrt(st["case"]["d"])
    o, lse = torch.empty_like(st["o"]), torch.empty_like(st["lse"])
    for qs, hs, t, later in _blocks(st):
        k, v = st["k"][hs, t].float()[:, None], st["v"][hs, t].float()[:, None]
        x = (_grouped(st["q"][qs, t], k) @ k.transpose(-1, -2)).mul_(scale).masked_fill_(later, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o[qs, t] = ((p @ v) / total).flatten(0, 1).to(o.dtype)
        lse[qs, t] = (top + torch.log(total)).squeeze(-1).flatten(0, 1)
    return [o, lse]


def _train_plain(st):
    scale = 1.0 / math.sqrt(st["case"]["d"])
    o, lse = torch.empty_like(st["o"]), torch.empty_like(st["lse"])
    dq, dk, dv = torch.empty_like(st["dq"]), torch.empty_like(st["dk"]), torch.empty_like(st["dv"])
    for qs, hs, t, later in _blocks(st):
        k, v = st["k"][hs, t].float()[:, None], st["v"][hs, t].float()[:, None]
        q, g = _grouped(st["q"][qs, t], k), _grouped(st["dO"][qs, t], k)
        x = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(later, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        p /= total
        out = p @ v
        o[qs, t] = out.flatten(0, 1).to(o.dtype)
        lse[qs, t] = (top + torch.log(total)).squeeze(-1).flatten(0, 1)
        dv[hs, t] = (p.transpose(-1, -2) @ g).sum(1).to(dv.dtype)
        ds = (g @ v.transpose(-1, -2)).sub_((g * out).sum(-1, keepdim=True)).mul_(p)
        dq[qs, t] = (ds @ k).mul_(scale).flatten(0, 1).to(dq.dtype)
        dk[hs, t] = (ds.transpose(-1, -2) @ q).sum(1).mul_(scale).to(dk.dtype)
    return [o, lse, dq, dk, dv]


_plain = {"append": _append_plain, "decode": _decode_plain, "prompt": _prompt_plain, "train": _train_plain}


def _append_own(st):
    import local_circular_window_b200 as L

    c = st["case"]
    L.clear_attn_cache_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["page_table"], st["seq_start"], st["seq_len"],
                              q=st["q"], q_out=st["q_out"], k_out=st["k_out"], rot=c["rot"], theta=c["theta"],
                              pairing=c["pairing"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return [st["q_out"], st["k_out"], st["k_pages"], st["v_pages"]]


def _decode_own(st):
    import local_circular_window_b200 as L

    if "workspace" not in st:  # kept from step to step, as a program that decodes keeps it
        st["workspace"] = torch.empty(L.decode_workspace_size(st["q"].shape[1], st["case"]["q_heads"], st["case"]["kv_heads"], st["case"]["d"]),
                                      dtype=torch.uint8, device="cuda")
    L.clear_attn_decode(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["seq_len"], o=st["o"], lse=st["lse"],
                        k_scale=st["k_scale"], v_scale=st["v_scale"], workspace=st["workspace"])
    return [st["o"], st["lse"]]



def _prompt_own(st):
    import local_circular_window_b200 as L

    L.clear_attn_prompt_fwd(st["q"], st["k"], st["v"], st["seq_start"], o=st["o"], lse=st["lse"])
    return [st["o"], st["lse"]]


def _train_own(st):
    import local_circular_window_b200 as L

    L.clear_attn_prompt_fwd(st["q"], st["k"], st["v"], st["seq_start"], o=st["o"], lse=st["lse"])
    L.clear_attn_prompt_bwd(st["q"], st["k"], st["v"], st["o"], st["lse"], st["dO"], st["seq_start"], dq=st["dq"],
                            dk=st["dk"], dv=st["dv"])
    return [st["o"], st["lse"], st["dq"], st["dk"], st["dv"]]


_own = {"append": _append_own, "decode": _decode_own, "prompt": _prompt_own, "train": _train_own}


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _append_exact, "decode": _decode_exact, "prompt": _packed_exact, "train": _packed_exact}[case["op"]](st)


def _append_exact(st):
    # Each pair is a complex number, turned by a unit complex number, sequence by sequence.
    c = st["case"]
    rot, page = c["rot"], c["page"]
    q, k, v = st["q"].double().clone(), st["k"].double().clone(), st["v"].double()
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    start, lens = st["seq_start"].tolist(), st["seq_len"].tolist()
    for s, total in enumerate(lens):
        a, b = start[s], start[s + 1]
        pos = torch.arange(total - (b - a), total, device="cuda", dtype=torch.float64)
        if rot:
            rate = torch.exp(-math.log(c["theta"]) * 2.0 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / rot)
            turn = torch.polar(torch.ones(b - a, rot // 2, device="cuda", dtype=torch.float64), torch.outer(pos, rate))
            for x in (q, k):
                y = x[:, a:b, :rot]
                y = y.unflatten(-1, (rot // 2, 2)) if c["pairing"] == "adjacent" else torch.stack(y.split(rot // 2, -1), -1)
                z = torch.view_as_real(torch.view_as_complex(y.contiguous()) * turn)
                x[:, a:b, :rot] = z.flatten(-2) if c["pairing"] == "adjacent" else torch.cat((z[..., 0], z[..., 1]), -1)
        at = pos.long()
        pages = st["page_table"][s].long()[torch.div(at, page, rounding_mode="floor")]
        for store, x, scale in ((kp, k, st["k_scale"]), (vp, v, st["v_scale"])):
            new = x[:, a:b].transpose(0, 1)
            store[pages, at % page] = new if scale is None else (new / scale.double()[:, None]).clamp(-448.0, 448.0)
    return [q, k, kp, vp]


def _decode_exact(st):
    c = st["case"]
    hq, hk, d, page = c["q_heads"], c["kv_heads"], c["d"], c["page"]
    o = torch.zeros(hq, st["q"].shape[1], d, dtype=torch.float64, device="cuda")
    lse = torch.full(o.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for s, n in enumerate(st["seq_len"].tolist()):
        if n == 0:
            continue
        pages = st["page_table"][s, :-(-n // page)].long()
        k, v = (st[x + "_pages"].double()[pages].flatten(0, 1)[:n] for x in ("k", "v"))
        if c["cache"] == "e4m3":
            k, v = k * st["k_scale"].double()[:, None], v * st["v_scale"].double()[:, None]
        for h in range(hq):
            x = (k[:, h * hk // hq] @ st["q"][h, s].double()) * d ** -0.5
            lse[h, s] = torch.logsumexp(x, 0)
            o[h, s] = torch.softmax(x, 0) @ v[:, h * hk // hq]
    return [o, lse]


def _packed_exact(st):
    # One head at a time; the gradients come from automatic differentiation in 64 bits.
    c = st["case"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["d"]
    train = c["op"] == "train"
    outs = {n: torch.zeros(st[m].shape, dtype=torch.float64, device="cuda") for n, m in
            (("o", "o"), ("lse", "lse"), ("q", "q"), ("k", "k"), ("v", "v"))}
    at = 0
    for n in st["lens"]:
        t = slice(at, at + n)
        keep = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        for h in range(hq):
            g = h * hk // hq
            q, k, v = (st[x][i, t].double().requires_grad_(train) for x, i in (("q", h), ("k", g), ("v", g)))
            x = torch.einsum("id,jd->ij", q, k) * d ** -0.5
            x = x.masked_fill(~keep, -math.inf)
            o = torch.softmax(x, -1) @ v
            outs["o"][h, t] = o.detach()
            outs["lse"][h, t] = torch.logsumexp(x.detach(), -1)
            if train:
                for name, i, grad in zip("qkv", (h, g, g), torch.autograd.grad(o, (q, k, v), st["dO"][h, t].double())):
                    outs[name][i, t] += grad
        at += n
    return [outs[x] for x in (("o", "lse", "q", "k", "v") if train else ("o", "lse"))]
