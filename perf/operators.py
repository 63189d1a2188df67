"""The operators of a serving step over the paged KV cache, in their plain form and as calls of the library.

A step takes a batch of sequences that each bring some new tokens (a chunk of a prompt, one token, or
one token and the drafts behind it):

  plan     block tables and slot maps from the requests' lengths          llama_paged_plan
  append   RoPE at per-token positions, K and V written into their pages  llama_rope_append_paged
  chunk    causal attention of the new tokens over the paged cache        llama_gqa_attention_chunk_paged
  verify   drafted tokens against the target's probabilities              llama_verify_drafts

New tokens are packed one sequence after the other: sequence b owns rows cu[b] .. cu[b+1]-1.
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 128            # positions per cache page
THETA = 5e5           # RoPE base of the 8B configuration
EPS = 1e-5


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # planning a decode step that verifies four drafts for each of 64 requests: latency
        dict(name="plan-b64-drafts", op="plan", B=64, new_lo=1, new_hi=5, cached_lo=0, cached_hi=8192, lead=0,
             max_pages=128),
        # planning a large mixed batch: prompt chunks of all lengths among running requests
        dict(name="plan-b1024-mixed", op="plan", B=1024, new_lo=0, new_hi=101, cached_lo=0, cached_hi=32000,
             lead=8192, max_pages=512),
        # the 8B heads, a decode step with drafts, q/k/v views of one fused projection
        dict(name="append-8b-300", op="append", T=300, n_q=32, n_kv=8, hd=128, far=131000, fused=True),
        # the 8B heads, a whole prefill batch
        dict(name="append-8b-8192", op="append", T=8192, n_q=32, n_kv=8, hd=128, far=8192, fused=True),
        # the smallest attention call: one token for each of three short sequences
        dict(name="chunk-b3-one-token", op="chunk", B=3, new_lo=1, new_hi=1, cached_lo=100, cached_hi=900, lead=0,
             n_q=32, n_kv=8, hd=128),
        # four drafts and the last accepted token for 64 running sequences (8B heads): K/V streaming
        dict(name="chunk-b64-drafts", op="chunk", B=64, new_lo=3, new_hi=5, cached_lo=2000, cached_hi=8187, lead=0,
             n_q=32, n_kv=8, hd=128),
        # the small block's heads, ragged prompts from an empty cache
        dict(name="chunk-small-ragged", op="chunk", B=9, new_lo=1, new_hi=777, cached_lo=0, cached_hi=0, lead=0,
             n_q=8, n_kv=2, hd=64),
        # one prompt chunk among 40 decoding sequences (8B heads)
        dict(name="chunk-mixed", op="chunk", B=41, new_lo=1, new_hi=1, cached_lo=30, cached_hi=5000, lead=1500,
             n_q=32, n_kv=8, hd=128),
        # a chunk of a long prompt: 2048 tokens after 30720 cached (8B heads): tensor cores
        dict(name="chunk-8b-2048-after-30720", op="chunk", B=1, new_lo=2048, new_hi=2048, cached_lo=30720,
             cached_hi=30720, lead=0, n_q=32, n_kv=8, hd=128),
        # one request, three drafts, against the 7B vocabulary: latency
        dict(name="verify-b1-v32000", op="verify", B=1, new_lo=4, new_hi=4, V=32000, temperature=1.0, drafts=True),
        # 64 requests with four drafts each, the 8B vocabulary
        dict(name="verify-b64-v128256", op="verify", B=64, new_lo=2, new_hi=5, V=128256, temperature=0.8, drafts=True),
        # 48 requests whose drafts come from a lookup (no draft distribution), the 8B vocabulary
        dict(name="verify-b48-lookup", op="verify", B=48, new_lo=1, new_hi=9, V=128256, temperature=1.0, drafts=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = [(32, 8, 128), (32, 32, 128), (8, 2, 64), (8, 1, 128), (28, 4, 128), (16, 2, 64), (12, 4, 128), (16, 1, 128)]


def draw(rng):
    op = rng.choice(["plan", "append", "chunk", "chunk", "chunk", "verify", "verify"])
    if op == "plan":
        B = _log_int(rng, 1, 1024)
        cached_hi = _log_int(rng, 1, 32000)
        lead = rng.choice([0, _log_int(rng, 1, 8192)])
        new_hi = _log_int(rng, 1, 101)
        need = (max(cached_hi + max(new_hi, lead), 1) + PAGE - 1) // PAGE
        return dict(op=op, B=B, new_lo=rng.choice([0, 1]), new_hi=new_hi, cached_lo=0, cached_hi=cached_hi, lead=lead,
                    max_pages=need + rng.randrange(0, 40))
    if op == "append":
        n_q, n_kv, hd = rng.choice(_HEADS)
        T = _log_int(rng, 1, 8192 * 48 // (n_q + 2 * n_kv) if n_q == n_kv else 8192)
        return dict(op=op, T=T, n_q=n_q, n_kv=n_kv, hd=hd, far=_log_int(rng, T + 1, 200000), fused=rng.random() < 0.7)
    if op == "chunk":
        n_q, n_kv, hd = rng.choice(_HEADS)
        kind = rng.choice(["decode", "drafts", "prompts", "mixed", "long"])
        if kind in ("decode", "drafts"):
            B = _log_int(rng, 1, 64)
            hi = _log_int(rng, 2, 8187 if n_kv <= 8 else 4000)
            c = dict(B=B, new_lo=1, new_hi=1 if kind == "decode" else rng.randrange(2, 10), cached_lo=hi // 4,
                     cached_hi=hi, lead=0)
        elif kind == "prompts":
            c = dict(B=rng.randrange(1, 12), new_lo=1, new_hi=_log_int(rng, 2, 1200), cached_lo=0,
                     cached_hi=rng.choice([0, 0, _log_int(rng, 1, 2000)]), lead=0)
        elif kind == "mixed":
            c = dict(B=rng.randrange(2, 49), new_lo=rng.choice([0, 1]), new_hi=rng.randrange(1, 6), cached_lo=0,
                     cached_hi=_log_int(rng, 1, 5000), lead=_log_int(rng, 64, 2000))
        else:
            hi = _log_int(rng, 1000, 30000)
            n = _log_int(rng, 16, 2000)
            c = dict(B=1, new_lo=n, new_hi=n, cached_lo=hi, cached_hi=hi, lead=0)
        return dict(op=op, n_q=n_q, n_kv=n_kv, hd=hd, **c)
    V = rng.choice([32000, 128256, _log_int(rng, 50, 128256)])
    drafts = rng.random() < 0.7
    return dict(op="verify", B=_log_int(rng, 1, 64), new_lo=1, new_hi=rng.randrange(1, 6), V=V,
                temperature=rng.choice([0.0, 1.0, round(rng.uniform(0.3, 1.5), 2)]), drafts=drafts)


# ------------------------------------------------------------------------------------------ lengths
def _spread(lo, hi, i, salt):
    """A fixed, scattered choice in [lo, hi] (lengths belong to the case, values to the seed)."""
    x = (i * 2654435761 + salt * 40503 + 12345) & 0xFFFFFFFF
    x ^= x >> 15
    x = (x * 2246822519) & 0xFFFFFFFF
    x ^= x >> 13
    return lo + x % (hi - lo + 1)


def _lengths(case):
    """(new tokens, cached positions) of every sequence; the middle one brings `lead` tokens if set."""
    B = case["B"]
    new = [_spread(case["new_lo"], case["new_hi"], b, 1) for b in range(B)]
    cached = [_spread(case.get("cached_lo", 0), case.get("cached_hi", 0), b, 2) for b in range(B)]
    if case.get("lead"):
        new[B // 2] = case["lead"]
    if sum(new) == 0:
        new[0] = 1
    return new, cached


def _ceil_page(n):
    return (n + PAGE - 1) // PAGE


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed, device):
    return torch.Generator(device=device).manual_seed(seed)


def _i32(values, device):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _cumulative(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    return {"plan": _prepare_plan, "append": _prepare_append, "chunk": _prepare_chunk,
            "verify": _prepare_verify}[case["op"]](case, g, dev)


def _prepare_plan(case, g, dev):
    new, cached = _lengths(case)
    B, P = case["B"], case["max_pages"]
    have = [_ceil_page(c) for c in cached]
    take = [_ceil_page(c + n) - h for c, n, h in zip(cached, new, have)]
    n_pages = sum(have) + sum(take) + 17
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, P), -1, dtype=torch.int32, device=dev)
    have_t = _i32(have, dev)
    held = torch.arange(P, device=dev)[None] < have_t[:, None]
    table[held] = perm[:sum(have)]
    T = sum(new) + 5                                  # a few rows of padding, as a captured step has
    return dict(case=case, n_cached=_i32(cached, dev), n_new=_i32(new, dev), free=perm[sum(have):].contiguous(),
                n_pages=n_pages, table=table, T=T,
                cu=torch.empty(B + 1, dtype=torch.int32, device=dev),
                positions=torch.empty(T, dtype=torch.int32, device=dev),
                slots=torch.empty(T, dtype=torch.int32, device=dev),
                used=torch.empty(1, dtype=torch.int32, device=dev))


def _prepare_append(case, g, dev):
    T, n_q, n_kv, hd = case["T"], case["n_q"], case["n_kv"], case["hd"]
    if case["fused"]:                                 # views of one projection's output
        qkv = torch.randn(T, n_q + 2 * n_kv, hd, generator=g, device=dev).to(torch.bfloat16)
        q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    else:
        q = torch.randn(T, n_q, hd, generator=g, device=dev).to(torch.bfloat16)
        k = torch.randn(T, n_kv, hd, generator=g, device=dev).to(torch.bfloat16)
        v = torch.randn(T, n_kv, hd, generator=g, device=dev).to(torch.bfloat16)
    n_pages = _ceil_page(T) + 3
    k_pool = torch.randn(n_pages, PAGE, n_kv, hd, generator=g, device=dev).to(torch.bfloat16)
    v_pool = torch.randn(n_pages, PAGE, n_kv, hd, generator=g, device=dev).to(torch.bfloat16)
    first = case["far"] - T
    positions = (first + torch.arange(T, device=dev)).to(torch.int32)
    pages = torch.randperm(n_pages, generator=g, device=dev)[:_ceil_page(T + PAGE - 1)]
    row = first % PAGE + torch.arange(T, device=dev)
    slots = (pages[row // PAGE] * PAGE + row % PAGE).to(torch.int32)
    return dict(case=case, q=q, k=k, v=v, positions=positions, slots=slots, k_pool=k_pool, v_pool=v_pool,
                q_out=torch.empty(T, n_q, hd, dtype=torch.bfloat16, device=dev))


def _prepare_chunk(case, g, dev):
    new, cached = _lengths(case)
    n_q, n_kv, hd, B = case["n_q"], case["n_kv"], case["hd"], case["B"]
    pages = [_ceil_page(c + n) for c, n in zip(cached, new)]
    P, n_pages = max(max(pages), 1), sum(pages) + 2
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, P), -1, dtype=torch.int32, device=dev)
    held = torch.arange(P, device=dev)[None] < _i32(pages, dev)[:, None]
    table[held] = perm[:sum(pages)]
    k_pool = torch.empty(n_pages, PAGE, n_kv, hd, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    v_pool = torch.empty(n_pages, PAGE, n_kv, hd, dtype=torch.bfloat16, device=dev).normal_(generator=g)
    T = sum(new)
    # queries of twice the keys' scale: rows whose weight sits on a few keys, as trained heads have
    q = torch.empty(T, n_q, hd, dtype=torch.bfloat16, device=dev).normal_(std=2.0, generator=g)
    max_pos = max([c + n for c, n in zip(cached, new)] + [1]) - 1
    st = dict(case=case, q=q, k_pool=k_pool, v_pool=v_pool, table=table, cu=_i32(_cumulative(new), dev),
              n_cached=_i32(cached, dev), new=new, cached=cached, max_pos=max_pos,
              o=torch.empty(T, n_q, hd, dtype=torch.bfloat16, device=dev))
    if own:
        import llama_decoder_block_fwd_gb300 as L
        st["dims"] = L.dims_of(B, T, n_q * hd, n_q, n_kv, hd, 128, THETA, EPS)
        st["ws"] = torch.empty(L.llama_workspace_bytes(L.OP_GQA_ATTENTION_CHUNK_PAGED, st["dims"], L.BF16,
                                                       kv_capacity=max_pos + 1), dtype=torch.uint8, device=dev)
    return st


def _prepare_verify(case, g, dev):
    new, _ = _lengths(case)
    B, V, T, temp = case["B"], case["V"], sum(new), case["temperature"]
    cu = _cumulative(new)
    z = torch.randn(T, V, generator=g, device=dev).mul_(2.5)
    # the draft model: the target's logits with an error of its own; drafts drawn from it
    y = torch.randn(T, V, generator=g, device=dev).mul_(0.6).add_(z)
    tokens = torch.randint(V, (T,), generator=g, device=dev, dtype=torch.int32)
    race = torch.empty(1, V, device=dev)
    for b in range(B):
        for j in range(cu[b], cu[b + 1] - 1):
            race.exponential_(generator=g)
            tokens[j + 1] = (torch.softmax(y[j] / max(temp, 0.05), 0) / race[0]).argmax().to(torch.int32)
    noise = torch.empty(B, V, device=dev).exponential_(generator=g).clamp_min_(1e-30)
    u = torch.rand(T, generator=g, device=dev)
    st = dict(case=case, z=z, y=y if case["drafts"] else None, tokens=tokens, noise=noise, u=u, cu=_i32(cu, dev),
              n_acc=torch.empty(B, dtype=torch.int32, device=dev), out=torch.empty(T, dtype=torch.int32, device=dev))
    if own:
        import llama_decoder_block_fwd_gb300 as L
        dims = L.dims_of(B, T, 128, 1, 1, 128, 128, THETA, EPS)
        st["ws"] = torch.empty(L.llama_workspace_bytes(L.OP_VERIFY_DRAFTS, dims, L.F32, vocab=V), dtype=torch.uint8,
                               device=dev)
    return st


# ------------------------------------------------------------------------------------------ the pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "chunk": _own_chunk, "verify": _own_verify}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "chunk": _plain_chunk, "verify": _plain_verify}[op](state)


def _own_plan(s):
    import llama_decoder_block_fwd_gb300 as L
    L.llama_paged_plan(s["n_cached"], s["n_new"], s["free"], s["n_pages"], s["table"], s["cu"], s["positions"],
                       s["slots"], s["used"])
    return s["table"], s["cu"], s["positions"], s["slots"], s["used"]


def _own_append(s):
    import llama_decoder_block_fwd_gb300 as L
    c = s["case"]
    dims = L.dims_of(1, c["T"], c["n_q"] * c["hd"], c["n_q"], c["n_kv"], c["hd"], 128, THETA, EPS)
    L.llama_rope_append_paged(dims, s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], s["k_pool"],
                              s["v_pool"])
    return s["q_out"], s["k_pool"], s["v_pool"]


def _own_chunk(s):
    import llama_decoder_block_fwd_gb300 as L
    L.llama_gqa_attention_chunk_paged(s["dims"], s["q"], s["k_pool"], s["v_pool"], s["table"], s["cu"], s["n_cached"],
                                      s["max_pos"], s["o"], s["ws"])
    return s["o"]


def _own_verify(s):
    import llama_decoder_block_fwd_gb300 as L
    L.llama_verify_drafts(s["z"], s["y"], s["case"]["temperature"], s["cu"], s["tokens"], s["u"], s["noise"],
                          s["n_acc"], s["out"], s["ws"])
    return s["n_acc"], s["out"]


def _plain_plan(s):
    cached, new, table, T = s["n_cached"].long(), s["n_new"].long(), s["table"], s["T"]
    dev, P = table.device, table.shape[1]
    have = (cached + PAGE - 1) // PAGE
    need = (cached + new + PAGE - 1) // PAGE
    take = need - have
    zero = torch.zeros(1, dtype=torch.long, device=dev)
    cu = torch.cat([zero, new.cumsum(0)])
    base = torch.cat([zero, take.cumsum(0)])
    col = torch.arange(P, device=dev)[None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    src = (base[:-1, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][src], table))
    row = torch.arange(T, device=dev)
    b = torch.searchsorted(cu, row, right=True) - 1
    live = row < cu[-1]
    b = b.clamp_max(new.numel() - 1)
    pos = cached[b] + row - cu[b]
    slot = table[b, (pos // PAGE).clamp(0, P - 1)].long() * PAGE + pos % PAGE
    s["cu"].copy_(cu)
    s["positions"].copy_(torch.where(live, pos, -1))
    s["slots"].copy_(torch.where(live, slot, -1))
    s["used"].copy_(base[-1:])
    return table, s["cu"], s["positions"], s["slots"], s["used"]


def _plain_append(s):
    hd = s["case"]["hd"]
    k = torch.arange(hd // 2, device=s["q"].device, dtype=torch.float64)
    angle = s["positions"].double()[:, None] * THETA ** (-2.0 * k / hd)      # 64 bits: far positions
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        a, b = x.float()[..., 0::2], x.float()[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2).to(torch.bfloat16)

    s["q_out"].copy_(turn(s["q"]))
    at = s["slots"].long()
    s["k_pool"].view(-1, *s["k_pool"].shape[2:])[at] = turn(s["k"])
    s["v_pool"].view(-1, *s["v_pool"].shape[2:])[at] = s["v"]
    return s["q_out"], s["k_pool"], s["v_pool"]


def _plain_chunk(s):
    c = s["case"]
    n_q, n_kv, hd = c["n_q"], c["n_kv"], c["hd"]
    r, at = n_q // n_kv, 0
    for b, (n, past) in enumerate(zip(s["new"], s["cached"])):
        if n == 0:
            continue
        keys = past + n
        pages = s["table"][b, :_ceil_page(keys)].long()
        k = s["k_pool"][pages].reshape(-1, n_kv, hd)[:keys].float().permute(1, 2, 0)       # [n_kv, hd, keys]
        v = s["v_pool"][pages].reshape(-1, n_kv, hd)[:keys].float().permute(1, 0, 2)       # [n_kv, keys, hd]
        step = max(1, (1 << 28) // (n_q * keys))                                           # rows at a time
        for t in range(0, n, step):
            m = min(step, n - t)
            q = s["q"][at + t:at + t + m].float().view(m, n_kv, r, hd).permute(1, 0, 2, 3).reshape(n_kv, m * r, hd)
            x = torch.matmul(q, k).view(n_kv, m, r, keys) / math.sqrt(hd)
            seen = torch.arange(keys, device=q.device)[None] <= past + t + torch.arange(m, device=q.device)[:, None]
            x = x.masked_fill(~seen[None, :, None], -math.inf)
            x = (x - x.amax(-1, keepdim=True)).exp()
            x = x / x.sum(-1, keepdim=True)
            o = torch.matmul(x.view(n_kv, m * r, keys), v).view(n_kv, m, r, hd)
            s["o"][at + t:at + t + m] = o.permute(1, 0, 2, 3).reshape(m, n_q, hd).to(torch.bfloat16)
        at += n
    return s["o"]


def _plain_verify(s):
    z, y, temp, cu = s["z"], s["y"], s["case"]["temperature"], s["cu"].long()
    T, V = z.shape
    dev = z.device
    first, last = cu[:-1], cu[1:] - 1                       # every sequence has at least one row
    row = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu, row, right=True) - 1
    drafted = row < last[seq]                               # row j judges the token of row j + 1
    d = s["tokens"].long()[(row + 1).clamp_max(T - 1)]
    if temp <= 0:
        best = z.argmax(-1)
        ok = best == d
    else:
        p = torch.softmax(z.double() / temp, -1)            # 64 bits: u and the race sit next to borders
        pd = p.gather(1, d[:, None])[:, 0]
        if y is None:
            q, qd = None, 1.0
        else:
            q = torch.softmax(y.double() / temp, -1)
            qd = q.gather(1, d[:, None])[:, 0]
        ok = s["u"].double() * qd < pd
    refused = torch.where(drafted & ~ok, row, T)
    stop = torch.full_like(last, T).scatter_reduce(0, seq, refused, "amin")
    stop = torch.minimum(stop, last)                        # the row that gives the new token
    if temp <= 0:
        token = best[stop]
    else:
        w = p[stop]
        rejected = stop < last
        if q is None:
            rest = w.scatter(1, d[stop][:, None], 0.0)
        else:
            rest = (w - q[stop]).clamp_min(0.0)
        use = rejected & (rest.sum(-1) > 0)
        w = torch.where(use[:, None], rest, w)
        token = (w / s["noise"].double()).argmax(-1)
    out = torch.where(row < stop[seq], d, -1)
    out[stop] = token
    s["n_acc"].copy_(stop - first)
    s["out"].copy_(out)
    return s["n_acc"], s["out"]


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "chunk":
        return _exact_chunk(s) if work(case)["flops"] < 3e12 else None
    return _exact_verify(s)


def _exact_plan(s):
    """Page by page and token by token on the host."""
    dev = s["table"].device
    table = s["table"].cpu().numpy().copy()
    cached, new, free = s["n_cached"].tolist(), s["n_new"].tolist(), s["free"].tolist()
    cu, positions, slots, taken = [0], [], [], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        for page in range((c + 127) // 128, (c + n + 127) // 128):
            table[b, page] = free[taken]
            taken += 1
        for p in range(c, c + n):
            positions.append(p)
            slots.append(int(table[b, p // 128]) * 128 + p % 128)
        cu.append(cu[-1] + n)
    pad = s["T"] - len(slots)
    return (torch.from_numpy(table).to(dev), _i32(cu, dev), _i32(positions + [-1] * pad, dev),
            _i32(slots + [-1] * pad, dev), _i32([taken], dev))


def _exact_append(s):
    hd = s["case"]["hd"]
    j = torch.arange(0, hd, 2, device=s["q"].device, dtype=torch.float64)
    turn = torch.polar(torch.ones_like(j), torch.zeros_like(j))[None] * torch.exp(
        1j * s["positions"].double()[:, None] * torch.exp(-j / hd * math.log(THETA)))

    def rotate(x):
        w = torch.view_as_complex(x.double().reshape(*x.shape[:-1], hd // 2, 2).contiguous())
        return torch.view_as_real(w * turn[:, None]).reshape(x.shape)

    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    at = s["slots"].long()
    k_pool[at // PAGE, at % PAGE] = rotate(s["k"])
    v_pool[at // PAGE, at % PAGE] = s["v"].double()
    return rotate(s["q"]), k_pool, v_pool


def _exact_chunk(s):
    c = s["case"]
    r, hd = c["n_q"] // c["n_kv"], c["hd"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    cu = s["cu"].tolist()
    for b, past in enumerate(s["cached"]):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        keys = past + hi - lo
        where = torch.arange(keys, device=out.device)
        page = s["table"][b].long()[where // PAGE]
        position = past + torch.arange(hi - lo, device=out.device)
        hidden = where[None] > position[:, None]
        for g in range(c["n_kv"]):
            k = s["k_pool"][page, where % PAGE, g].double()
            v = s["v_pool"][page, where % PAGE, g].double()
            for h in range(g * r, (g + 1) * r):
                x = s["q"][lo:hi, h].double() @ k.T * hd ** -0.5
                x[hidden] = -math.inf
                out[lo:hi, h] = torch.exp(x - torch.logsumexp(x, -1, keepdim=True)) @ v
    return out


def _exact_verify(s):
    """One sequence after the other, stopping at the first draft that is turned down."""
    temp, cu, tokens = s["case"]["temperature"], s["cu"].tolist(), s["tokens"].tolist()
    u = s["u"].double().tolist()
    n_acc, out = [], []
    for b in range(len(cu) - 1):
        lo, n = cu[b], cu[b + 1] - cu[b]
        row = [-1] * n
        for i in range(n):
            z = s["z"][lo + i].double()
            if temp <= 0:
                top = int(torch.nonzero(z == z.max())[0])
                row[i] = top
                if i < n - 1 and top == tokens[lo + i + 1]:
                    continue
                break
            w = torch.exp(z / temp - torch.logsumexp(z / temp, 0))
            if i < n - 1:
                d = tokens[lo + i + 1]
                q = torch.zeros_like(w)
                if s["y"] is None:
                    q[d] = 1.0
                else:
                    y = s["y"][lo + i].double() / temp
                    q = torch.exp(y - torch.logsumexp(y, 0))
                if u[lo + i] * float(q[d]) < float(w[d]):
                    row[i] = d
                    continue
                rest = torch.relu(w - q)
                w = rest if float(rest.sum()) > 0 else w
            row[i] = int(torch.argmax(w / s["noise"][b].double()))
            break
        n_acc.append(i)
        out += row
    dev = s["z"].device
    return _i32(n_acc, dev), _i32(out, dev)


# ------------------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "plan":
        new, cached = _lengths(case)
        fresh = sum(_ceil_page(c + n) - _ceil_page(c) for c, n in zip(cached, new))
        # lengths in, offsets out, new pages in and out, one partly filled page per sequence, tokens out
        return {"bytes": 8 * case["B"] + 4 * (case["B"] + 1) + 8 * fresh + 4 * case["B"] + 8 * (sum(new) + 5) + 4,
                "flops": 4 * sum(new)}
    if op == "append":
        n = case["T"] * (case["n_q"] + 2 * case["n_kv"]) * case["hd"]
        return {"bytes": 4 * n + 8 * case["T"], "flops": 3 * case["T"] * (case["n_q"] + case["n_kv"]) * case["hd"]}
    if op == "chunk":
        new, cached = _lengths(case)
        n_q, n_kv, hd = case["n_q"], case["n_kv"], case["hd"]
        kv = sum(c + n for c, n in zip(cached, new) if n)
        pages = sum(_ceil_page(c + n) for c, n in zip(cached, new) if n)
        seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
        return {"bytes": 4 * sum(new) * n_q * hd + 4 * kv * n_kv * hd + 4 * pages + 8 * case["B"],
                "flops": 4 * n_q * hd * seen}
    new, _ = _lengths(case)
    T, B, V = sum(new), case["B"], case["V"]
    if case["temperature"] <= 0:
        return {"bytes": 4 * V * T + 12 * T, "flops": V * T}
    rows = T + (T - B if case["drafts"] else 0)
    return {"bytes": 4 * V * (rows + B) + 16 * T, "flops": 4 * V * rows + 6 * V * B}
