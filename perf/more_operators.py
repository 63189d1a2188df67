"""An 8-bit paged KV cache and beam search over it, in plain form and as calls of the library.

  append8   RoPE, then K and V written into their pages as E4M3 codes       llama_rope_append_paged_kv8
  readback  codes back to bf16 pages, for the calls that read bf16          llama_kv_dequantize_paged
  attn8     one new token per sequence over the 8-bit pages                 llama_gqa_attention_decode_paged_kv8
  select    the best (beam, token) pairs over all beams of a request        llama_beam_select
  reorder   block tables and pages follow the beams that were kept          llama_beam_reorder_paged

Codes are [n_pages, 128, n_kv, hd] bytes, their scales [n_pages, n_kv, 128] fp32: one power of two per token
and KV head, the smallest 2^e (e in -100 .. 100) with u <= 448 * 2^e, where u is the row's largest
magnitude for V and its largest |a| + |b| over the rotated pairs (a, b) for K, which no rotation exceeds.
"""
from __future__ import annotations

import math
import random

import torch

own = False

PAGE = 128            # positions per cache page
THETA = 5e5           # RoPE base of the 8B configuration
EPS = 1e-5
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step with drafts (8B heads), q/k/v views of one fused projection: latency
        dict(name="append8-8b-300", op="append8", T=300, n_q=32, n_kv=8, hd=128, far=131000, fused=True),
        # a whole prefill batch (8B heads)
        dict(name="append8-8b-8192", op="append8", T=8192, n_q=32, n_kv=8, hd=128, far=8192, fused=True),
        # one request of the small block's heads is read back: latency
        dict(name="readback-small-b1", op="readback", B=1, lo=700, hi=700, n_kv=2, hd=64),
        # sixteen ragged requests (8B heads) before a chunk of their prompts
        dict(name="readback-8b-b16", op="readback", B=16, lo=1000, hi=6000, n_kv=8, hd=128),
        # the smallest attention call: three short sequences (8B heads)
        dict(name="attn8-8b-b3-short", op="attn8", B=3, lo=100, hi=900, n_q=32, n_kv=8, hd=128),
        # a ragged decode batch (8B heads): K/V streaming
        dict(name="attn8-8b-b64", op="attn8", B=64, lo=2000, hi=8187, n_q=32, n_kv=8, hd=128),
        # one long sequence: the split over its length
        dict(name="attn8-8b-b1-131000", op="attn8", B=1, lo=131000, hi=131000, n_q=32, n_kv=8, hd=128),
        # the small block's heads, ragged, some sequences of a few tokens
        dict(name="attn8-small-b24", op="attn8", B=24, lo=1, hi=2500, n_q=8, n_kv=2, hd=64),
        # one request, four beams, the 7B vocabulary: latency
        dict(name="select-b1-w4-v32000", op="select", B=1, W=4, V=32000, K=4, done=False),
        # 48 requests of eight beams, the 8B vocabulary, twice as many candidates as beams are kept
        dict(name="select-b48-w8-v128256", op="select", B=48, W=8, V=128256, K=16, done=True),
        # one request of four beams over a bf16 cache of the small block's heads: latency
        dict(name="reorder-bf16-b1-w4", op="reorder", B=1, W=4, prompt=300, grown=90, n_kv=2, hd=64, layers=2, bits=16),
        # sixteen requests of eight beams over an 8-bit cache (8B heads, eight layers)
        dict(name="reorder-8bit-b16-w8", op="reorder", B=16, W=8, prompt=700, grown=250, n_kv=8, hd=128, layers=8,
             bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = [(32, 8, 128), (32, 32, 128), (8, 2, 64), (8, 1, 128), (28, 4, 128), (16, 2, 64), (12, 4, 128), (16, 1, 128),
          (24, 1, 128), (6, 3, 64)]


def draw(rng):
    op = rng.choice(["append8", "readback", "attn8", "attn8", "attn8", "select", "select", "reorder"])
    n_q, n_kv, hd = rng.choice(_HEADS)
    if op == "append8":
        T = _log_int(rng, 1, 8192 * 48 // (n_q + 2 * n_kv) if n_q == n_kv else 8192)
        return dict(op=op, T=T, n_q=n_q, n_kv=n_kv, hd=hd, far=_log_int(rng, T + 1, 200000), fused=rng.random() < 0.7)
    if op == "readback":
        hi = _log_int(rng, 2, 6000 if n_kv <= 8 else 1500)
        return dict(op=op, B=_log_int(rng, 1, 16), lo=rng.choice([1, hi // 2 + 1]), hi=hi, n_kv=n_kv, hd=hd)
    if op == "attn8":
        if rng.random() < 0.25:
            n = _log_int(rng, 8000, 131000 if n_kv <= 8 else 60000)
            return dict(op=op, B=1, lo=n, hi=n, n_q=n_q, n_kv=n_kv, hd=hd)
        hi = _log_int(rng, 2, 8187 if n_kv <= 8 else 2000)
        return dict(op=op, B=_log_int(rng, 1, 64), lo=rng.choice([1, hi // 4 + 1]), hi=hi, n_q=n_q, n_kv=n_kv, hd=hd)
    if op == "select":
        W = _log_int(rng, 1, 16)
        B = _log_int(rng, 1, 384 // W)
        V = rng.choice([32000, 128256, _log_int(rng, 50, 128256)])
        return dict(op=op, B=B, W=W, V=V, K=min(V, rng.choice([W, 2 * W, rng.randrange(1, 2 * W + 1)])),
                    done=rng.random() < 0.5)
    return dict(op=op, B=_log_int(rng, 1, 16), W=rng.randrange(2, 9), prompt=_log_int(rng, 1, 900),
                grown=_log_int(rng, 1, 250), n_kv=min(n_kv, 8), hd=hd, layers=rng.randrange(1, 9 if hd * n_kv <= 512 else 5),
                bits=rng.choice([8, 16]))


def _spread(lo, hi, i, salt):
    """A fixed, scattered choice in [lo, hi] (lengths belong to the case, values to the seed)."""
    x = (i * 2654435761 + salt * 40503 + 12345) & 0xFFFFFFFF
    x ^= x >> 15
    x = (x * 2246822519) & 0xFFFFFFFF
    x ^= x >> 13
    return lo + x % (hi - lo + 1)


def _lengths(case):
    return [_spread(case["lo"], case["hi"], b, 3) for b in range(case["B"])]


def _beams(case):
    """Per request (prompt, positions held by each of its beams), and each new beam's parent: a few good
    beams have most of the children, as in a search."""
    B, W = case["B"], case["W"]
    prompt = [_spread(case["prompt"] // 2 + 1, case["prompt"], b, 6) for b in range(B)]
    held = [p + _spread(case["grown"] // 2 + 1, case["grown"], b, 7) for b, p in enumerate(prompt)]
    return list(zip(prompt, held)), [[_spread(0, W - 1, b * W + w, 8) ** 2 // W for w in range(W)] for b in range(B)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


# ------------------------------------------------------------------------------------------ inputs
def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _row_scale(u):
    """The smallest power of two 2^e, e in -100 .. 100, with u <= 448 * 2^e (exact: exponents only)."""
    m, x = torch.frexp(u)                               # u = m * 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, x - 8, x - 9)
    e = torch.where(u > 0, e, torch.full_like(e, -100)).clamp(-100, 100)
    return torch.ldexp(torch.ones_like(u), e)


def _random_cache(g, dev, n_pages, n_kv, hd):
    """Codes and scales of rows whose size varies from token to token, as K and V rows do."""
    x = torch.empty(n_pages, PAGE, n_kv, hd, device=dev).normal_(generator=g)
    x *= torch.empty(n_pages, PAGE, n_kv, 1, device=dev).normal_(std=0.6, generator=g).exp_()
    s = _row_scale(x.abs().amax(-1))
    return (x / s[..., None]).to(F8), s.transpose(1, 2).contiguous()


def _random_table(g, dev, lengths, more):
    """A block table over a shuffled pool: (table [B, P], pages in the pool)."""
    pages = [_pages(n) for n in lengths]
    n_pages, P = sum(pages) + more, max(max(pages), 1)
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lengths), P), -1, dtype=torch.int32, device=dev)
    held = torch.arange(P, device=dev)[None] < _i32(pages, dev)[:, None]
    table[held] = perm[:sum(pages)]
    return table, n_pages


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    make = {"append8": _prepare_append, "readback": _prepare_readback, "attn8": _prepare_attn,
            "select": _prepare_select, "reorder": _prepare_reorder}[case["op"]]
    return dict(make(case, g, dev, seed), case=case)


def _prepare_append(case, g, dev, seed):
    T, n_q, n_kv, hd = case["T"], case["n_q"], case["n_kv"], case["hd"]
    if case["fused"]:                                 # views of one projection's output
        x = torch.randn(T, n_q + 2 * n_kv, hd, generator=g, device=dev).to(torch.bfloat16)
        q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    else:
        q = torch.randn(T, n_q, hd, generator=g, device=dev).to(torch.bfloat16)
        k = torch.randn(T, n_kv, hd, generator=g, device=dev).to(torch.bfloat16)
        v = torch.randn(T, n_kv, hd, generator=g, device=dev).to(torch.bfloat16)
    n_pages = _pages(T) + 3
    kc, ks = _random_cache(g, dev, n_pages, n_kv, hd)
    vc, vs = _random_cache(g, dev, n_pages, n_kv, hd)
    first = case["far"] - T
    positions = (first + torch.arange(T, device=dev)).to(torch.int32)
    pages = torch.randperm(n_pages, generator=g, device=dev)[:_pages(T + PAGE - 1)]
    row = first % PAGE + torch.arange(T, device=dev)
    slots = (pages[row // PAGE] * PAGE + row % PAGE).to(torch.int32)
    return dict(q=q, k=k, v=v, positions=positions, slots=slots, kc=kc, ks=ks, vc=vc, vs=vs,
                q_out=torch.empty(T, n_q, hd, dtype=torch.bfloat16, device=dev))


def _prepare_readback(case, g, dev, seed):
    lengths = _lengths(case)
    table, n_pages = _random_table(g, dev, lengths, 2)
    kc, ks = _random_cache(g, dev, n_pages, case["n_kv"], case["hd"])
    vc, vs = _random_cache(g, dev, n_pages, case["n_kv"], case["hd"])
    shape = (n_pages, PAGE, case["n_kv"], case["hd"])
    return dict(table=table, n_pos=_i32(lengths, dev), kc=kc, ks=ks, vc=vc, vs=vs,
                k_pool=torch.zeros(shape, dtype=torch.bfloat16, device=dev),
                v_pool=torch.zeros(shape, dtype=torch.bfloat16, device=dev))


def _prepare_attn(case, g, dev, seed):
    lengths = _lengths(case)
    n_q, n_kv, hd, B = case["n_q"], case["n_kv"], case["hd"], case["B"]
    table, n_pages = _random_table(g, dev, lengths, 2)
    kc, ks = _random_cache(g, dev, n_pages, n_kv, hd)
    vc, vs = _random_cache(g, dev, n_pages, n_kv, hd)
    # queries of twice the keys' scale: rows whose weight sits on a few keys, as trained heads have
    q = torch.empty(B, n_q, hd, device=dev).normal_(std=2.0, generator=g).to(torch.bfloat16)
    return dict(table=table, seq_pos=_i32([n - 1 for n in lengths], dev), max_pos=max(lengths) - 1, q=q, kc=kc, ks=ks,
                vc=vc, vs=vs, o=torch.empty(B, n_q, hd, dtype=torch.bfloat16, device=dev))


def _prepare_select(case, g, dev, seed):
    B, W, V, K = case["B"], case["W"], case["V"], case["K"]
    z = torch.empty(B * W, V, device=dev).normal_(std=2.5, generator=g)
    # sums of log-probabilities some ten tokens into the search, beams close to one another
    scores = -20.0 - 3.0 * torch.rand(B, 1, generator=g, device=dev) - 4.0 * torch.rand(B, W, generator=g, device=dev)
    done = (torch.rand(B, W, generator=g, device=dev) < 0.15).to(torch.int32) if case["done"] else None
    return dict(z=z, scores=scores, done=done, parents=torch.empty(B, K, dtype=torch.int32, device=dev),
                tokens=torch.empty(B, K, dtype=torch.int32, device=dev), out=torch.empty(B, K, device=dev))


def _prepare_reorder(case, g, dev, seed):
    B, W, layers, n_kv, hd = case["B"], case["W"], case["layers"], case["n_kv"], case["hd"]
    rng = random.Random(seed)
    every, parents = _beams(case)
    most = _pages(case["prompt"] + case["grown"]) + 1
    n_pages = B * (most + W * (_pages(case["grown"]) + 2)) + B * W
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, n_cached = [], []
    for prompt, n in every:
        cols = _pages(n)
        shared = prompt // PAGE                       # the prompt's full pages: one copy for all beams
        rows = [[-1] * most for _ in range(W)]
        for j in range(cols):
            for w in range(W):
                # behind the prompt some beams still share their ancestors' full pages
                full = (j + 1) * PAGE <= n
                same = j < shared or (full and rng.random() < 0.4)
                rows[w][j] = rows[w - 1][j] if w and same else ids.pop()
        table += rows
        n_cached += [n] * W

    def pool(*shape):
        if case["bits"] == 16:
            return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g)
        return torch.randint(0, 120, shape, dtype=torch.uint8, generator=g, device=dev).view(F8)

    kv = [pool(layers, n_pages, PAGE, n_kv, hd) for _ in range(2)]
    sc = [torch.exp2(torch.randint(-9, 3, (layers, n_pages, n_kv, PAGE), generator=g, device=dev).float())
          for _ in range(2 if case["bits"] == 8 else 0)]
    return dict(parents=_i32(parents, dev), n_cached=_i32(n_cached, dev), n_out=_i32([0] * (B * W), dev),
                table=_i32(table, dev), table_out=torch.full((B * W, most), -1, dtype=torch.int32, device=dev),
                free=_i32(ids, dev), n_pages=n_pages, kv=kv, sc=sc,
                freed=torch.full((B * W * 8,), -1, dtype=torch.int32, device=dev),
                counts=torch.zeros(2, dtype=torch.int32, device=dev))


# ------------------------------------------------------------------------------------------ the pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append8": _own_append, "readback": _own_readback, "attn8": _own_attn, "select": _own_select,
                "reorder": _own_reorder}[op](state)
    return {"append8": _plain_append, "readback": _plain_readback, "attn8": _plain_attn, "select": _plain_select,
            "reorder": _plain_reorder}[op](state)


def _own_append(s):
    import llama_decoder_block_fwd_gb300 as L
    c = s["case"]
    dims = L.dims_of(1, c["T"], c["n_q"] * c["hd"], c["n_q"], c["n_kv"], c["hd"], 128, THETA, EPS)
    L.llama_rope_append_paged_kv8(dims, s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], s["kc"], s["ks"],
                                  s["vc"], s["vs"])
    return s["q_out"], s["kc"], s["ks"], s["vc"], s["vs"]


def _own_readback(s):
    import llama_decoder_block_fwd_gb300 as L
    L.llama_kv_dequantize_paged(s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["n_pos"], s["k_pool"], s["v_pool"])
    return s["k_pool"], s["v_pool"]


def _workspace(s, op, dims, dtype, **more):
    """Allocated by the first call, kept with the state as a serving program keeps it."""
    import llama_decoder_block_fwd_gb300 as L
    if "ws" not in s:
        s["ws"] = torch.empty(L.llama_workspace_bytes(op, dims, dtype, **more), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own_attn(s):
    import llama_decoder_block_fwd_gb300 as L
    c = s["case"]
    dims = L.dims_of(c["B"], 1, c["n_q"] * c["hd"], c["n_q"], c["n_kv"], c["hd"], 128, THETA, EPS)
    ws = _workspace(s, L.OP_GQA_ATTENTION_DECODE_PAGED_KV8, dims, L.BF16, kv_capacity=s["max_pos"] + 1)
    L.llama_gqa_attention_decode_paged_kv8(dims, s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["seq_pos"],
                                           s["max_pos"], s["o"], ws)
    return s["o"]


def _own_select(s):
    import llama_decoder_block_fwd_gb300 as L
    c = s["case"]
    dims = L.dims_of(c["B"], c["W"], 128, 1, 1, 128, 128, THETA, EPS)
    ws = _workspace(s, L.OP_BEAM_SELECT, dims, L.F32, vocab=c["V"])
    L.llama_beam_select(s["z"], s["scores"], s["done"], 0, s["parents"], s["tokens"], s["out"], ws)
    return s["parents"], s["tokens"], s["out"]


def _own_reorder(s):
    import llama_decoder_block_fwd_gb300 as L
    c = s["case"]
    dims = L.dims_of(c["B"], c["W"], 128, 1, 1, 128, 128, THETA, EPS)
    ws = _workspace(s, L.OP_BEAM_REORDER_PAGED, dims, L.BF16, kv_capacity=PAGE * s["table"].shape[1])
    L.llama_beam_reorder_paged(s["parents"], s["n_cached"], s["n_out"], s["table"], s["table_out"], s["free"], s["n_pages"],
                               s["kv"], s["sc"], s["freed"], s["counts"], ws)
    return s["table_out"], s["n_out"], s["freed"], s["counts"], s["kv"], s["sc"]


def _plain_append(s):
    hd, n_kv = s["case"]["hd"], s["case"]["n_kv"]
    j = torch.arange(hd // 2, device=s["q"].device, dtype=torch.float64)
    angle = s["positions"].double()[:, None] * THETA ** (-2.0 * j / hd)      # 64 bits: far positions
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        a, b = x.float()[..., 0::2], x.float()[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)

    k, v = s["k"].float(), s["v"].float()
    at = s["slots"].long()
    rows = (-1, n_kv, hd)
    for x, u, codes, scales in ((turn(k), k.abs().unflatten(-1, (-1, 2)).sum(-1).amax(-1), s["kc"], s["ks"]),
                                (v, v.abs().amax(-1), s["vc"], s["vs"])):
        scale = _row_scale(u)
        codes.view(torch.uint8).view(rows)[at] = (x / scale[..., None]).to(F8).view(torch.uint8)
        scales[at // PAGE, :, at % PAGE] = scale
    s["q_out"].copy_(turn(s["q"]))
    return s["q_out"], s["kc"], s["ks"], s["vc"], s["vs"]


def _values(codes, scales, pages):
    """The rows [.., 128, n_kv, hd] in 32 bits that the listed pages stand for."""
    return codes.view(torch.uint8)[pages].view(F8).float() * scales[pages].transpose(-1, -2)[..., None]


def _plain_readback(s):
    table, n = s["table"], s["n_pos"]
    where = torch.arange(table.shape[1] * PAGE, device=n.device)
    b, pos = (where[None] < n[:, None]).nonzero(as_tuple=True)
    page, row = table[b, pos // PAGE].long(), pos % PAGE
    for codes, scales, pool in ((s["kc"], s["ks"], s["k_pool"]), (s["vc"], s["vs"], s["v_pool"])):
        x = codes.view(torch.uint8)[page, row].view(F8).float() * scales[page, :, row][..., None]
        pool[page, row] = x.to(torch.bfloat16)
    return s["k_pool"], s["v_pool"]


def _plain_attn(s):
    c = s["case"]
    n_q, n_kv, hd, B = c["n_q"], c["n_kv"], c["hd"], c["B"]
    pages = s["table"].clamp_min(0).long()
    seen = torch.arange(pages.shape[1] * PAGE, device=pages.device)[None] <= s["seq_pos"][:, None]    # [B, keys]
    k = _values(s["kc"], s["ks"], pages).flatten(1, 2).permute(0, 2, 3, 1)                            # [B, n_kv, hd, keys]
    v = _values(s["vc"], s["vs"], pages).flatten(1, 2).permute(0, 2, 1, 3)
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    q = s["q"].float().view(B, n_kv, n_q // n_kv, hd)
    x = torch.matmul(q, k) / math.sqrt(hd)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp()
    x = x / x.sum(-1, keepdim=True)
    s["o"].copy_(torch.matmul(x, v).view(B, n_q, hd))
    return s["o"]


def _plain_select(s):
    c = s["case"]
    B, W, V, K = c["B"], c["W"], c["V"], c["K"]
    z = s["z"].double().view(B, W, V)                    # 64 bits: scores of different beams lie close
    m = z.amax(-1, keepdim=True)
    score = s["scores"].double()[..., None] + (z - m - (z - m).exp().sum(-1, keepdim=True).log())
    if s["done"] is not None:                            # a finished beam stays as it is, once
        done = s["done"].bool()[..., None]
        pad = torch.arange(V, device=z.device) == 0
        score = torch.where(done, torch.where(pad, s["scores"].double()[..., None], -math.inf), score)
    best, at = score.view(B, W * V).sort(dim=-1, descending=True, stable=True)     # ties: the lower index first
    best, at = best[:, :K], at[:, :K]
    none = best == -math.inf
    s["parents"].copy_(torch.where(none, -1, at // V))
    s["tokens"].copy_(torch.where(none, -1, at % V))
    s["out"].copy_(best)
    return s["parents"], s["tokens"], s["out"]


def _plain_reorder(s):
    c = s["case"]
    B, W = c["B"], c["W"]
    old = s["table"].long().view(B, W, -1)
    P = old.shape[-1]
    n, par = s["n_cached"].long().view(B, W), s["parents"].long()
    col = torch.arange(P, device=old.device)
    held = col < ((n + PAGE - 1) // PAGE)[..., None]                                   # [B, W, P]
    kept = (par[:, None, :] == torch.arange(W, device=old.device)[None, :, None]).any(-1)  # beams with children
    same = (old[:, :, None] == old[:, None]) & held[:, :, None] & held[:, None]           # [B, W, W, P]: one page
    stays = (same & kept[:, None, :, None]).any(2)
    lower = torch.ones(W, W, dtype=torch.bool, device=old.device).tril(-1)[None, :, :, None]
    dead = (held & ~stays & ~(same & lower).any(2)).transpose(1, 2).reshape(B, P * W)     # by column, then beam
    n_new = n.gather(1, par)
    new = old.gather(1, par[..., None].expand(-1, -1, P))
    last = n_new // PAGE
    open_ = n_new % PAGE != 0                            # the last page is not full: its holder will write to it
    page = new.gather(2, last.clamp_max(P - 1)[..., None])[..., 0]
    lower = torch.ones(W, W, dtype=torch.bool, device=old.device).tril(-1)
    again = ((page[:, :, None] == page[:, None]) & open_[:, None] & lower).any(-1)
    copy = open_ & again                                 # all children but the first need a page of their own
    n_dead, n_copy = dead.sum(-1), copy.sum(-1)
    short, spare = (n_copy - n_dead).clamp_min(0), (n_dead - n_copy).clamp_min(0)
    rank = copy.cumsum(-1) - 1
    b, w = copy.nonzero(as_tuple=True)
    i = rank[b, w]
    dead_at = dead.nonzero()                             # in order: request, column, beam
    dead_page = old.transpose(1, 2).reshape(B, P * W)[dead_at[:, 0], dead_at[:, 1]]
    first_dead = n_dead.cumsum(0) - n_dead
    reuse = i < n_dead[b]
    pad = torch.cat([dead_page, dead_page.new_zeros(1)])
    free = torch.cat([s["free"].long(), dead_page.new_zeros(1)])
    none = torch.zeros_like(i)
    dst = torch.where(reuse, pad[torch.where(reuse, first_dead[b] + i, none)],
                      free[torch.where(reuse, none, (short.cumsum(0) - short)[b] + i - n_dead[b])])
    src, rows = page[b, w], n_new[b, w] % PAGE
    new[b, w, last[b, w]] = dst
    table = s["table_out"].view(B, W, P)
    table.copy_(torch.where(held.gather(1, par[..., None].expand(-1, -1, P)), new, table.long()))
    s["n_out"].copy_(n_new.view(-1))
    rest = torch.arange(len(dead_page), device=old.device) - first_dead[dead_at[:, 0]] >= n_copy[dead_at[:, 0]]
    gone = dead_page[rest]
    s["freed"][:len(gone)] = gone.to(torch.int32)
    s["counts"].copy_(torch.stack([short.sum(), spare.sum()]))
    live = torch.arange(PAGE, device=old.device)[None] < rows[:, None]
    for pool in s["kv"]:
        x = pool.view(torch.uint8) if c["bits"] == 8 else pool
        x[:, dst] = torch.where(live[None, :, :, None, None], x[:, src], x[:, dst])
    for pool in s["sc"]:
        pool[:, dst] = torch.where(live[None, :, None], pool[:, src], pool[:, dst])
    return s["table_out"], s["n_out"], s["freed"], s["counts"], s["kv"], s["sc"]


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append8": _exact_append, "readback": _exact_readback, "attn8": _exact_attn, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](s)


def _exact_append(s):
    hd, n_kv = s["case"]["hd"], s["case"]["n_kv"]
    j = torch.arange(0, hd, 2, device=s["q"].device, dtype=torch.float64)
    phase = torch.exp(1j * s["positions"].double()[:, None] * torch.exp(-j / hd * math.log(THETA)))[:, None]
    at = s["slots"].long()
    page, row = at // PAGE, at % PAGE

    def rotate(x):
        w = torch.view_as_complex(x.double().reshape(*x.shape[:-1], hd // 2, 2).contiguous())
        return torch.view_as_real(w * phase).reshape(x.shape)

    def stored(codes, scales, x, u):
        # 2^e >= u / 448: from the logarithm, then put right by the comparison itself
        e = torch.ceil(torch.log2(u / 448))
        e = torch.where(u <= 448 * torch.exp2(e - 1), e - 1, e)
        e = torch.where(u > 448 * torch.exp2(e), e + 1, e)
        scale = torch.exp2(e.clamp(-100, 100))
        codes, scales = codes.double(), scales.double()
        codes[page, row] = x / scale[..., None]
        for h in range(n_kv):
            scales[page, h, row] = scale[:, h]
        return codes, scales

    k, v = s["k"].double(), s["v"].double()
    kc, ks = stored(s["kc"], s["ks"], rotate(k), (k[..., 0::2].abs() + k[..., 1::2].abs()).max(-1)[0])
    vc, vs = stored(s["vc"], s["vs"], v, torch.maximum(v.max(-1)[0], -v.min(-1)[0]))
    return rotate(s["q"]), kc, ks, vc, vs


def _rows64(codes, scales, table_row, n, h):
    """Positions 0 .. n-1 of KV head h of one sequence."""
    where = torch.arange(n, device=codes.device)
    page = table_row.long()[where // PAGE]
    return codes.view(torch.uint8)[page, where % PAGE, h].view(F8).double() * scales[page, h, where % PAGE].double()[:, None]


def _exact_readback(s):
    out = []
    for codes, scales, pool in ((s["kc"], s["ks"], s["k_pool"]), (s["vc"], s["vs"], s["v_pool"])):
        pool = pool.double()
        for row, n in zip(s["table"], s["n_pos"].tolist()):
            where = torch.arange(n, device=pool.device)
            page = row.long()[where // PAGE]
            for h in range(pool.shape[2]):
                pool[page, where % PAGE, h] = _rows64(codes, scales, row, n, h)
        out.append(pool)
    return tuple(out)


def _exact_attn(s):
    c = s["case"]
    r, hd = c["n_q"] // c["n_kv"], c["hd"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b, pos in enumerate(s["seq_pos"].tolist()):
        for g in range(c["n_kv"]):
            k = _rows64(s["kc"], s["ks"], s["table"][b], pos + 1, g)
            v = _rows64(s["vc"], s["vs"], s["table"][b], pos + 1, g)
            x = s["q"][b, g * r:(g + 1) * r].double() @ k.T * hd ** -0.5
            out[b, g * r:(g + 1) * r] = torch.exp(x - torch.logsumexp(x, -1, keepdim=True)) @ v
    return out


def _exact_select(s):
    """One request after the other: the candidates of each beam, then those of all beams in order."""
    c = s["case"]
    W, V, K = c["W"], c["V"], c["K"]
    parents, tokens, out = [], [], []
    for b in range(c["B"]):
        found = []
        for w in range(W):
            base = float(s["scores"][b, w])
            if s["done"] is not None and int(s["done"][b, w]):
                found.append((-base, w, 0))
                continue
            z = s["z"][b * W + w].double()
            norm = float(torch.logsumexp(z, 0))
            floor = float(torch.topk(z, min(K, V))[0][-1])
            at = torch.nonzero(z >= floor)[:, 0]           # ties of the last one too
            found += [(-(base + x - norm), w, t) for x, t in zip(z[at].tolist(), at.tolist())]
        found = sorted(found)[:K]
        found += [(math.inf, -1, -1)] * (K - len(found))
        parents.append([f[1] for f in found])
        tokens.append([f[2] for f in found])
        out.append([-f[0] for f in found])
    dev = s["z"].device
    return _i32(parents, dev), _i32(tokens, dev), torch.tensor(out, dtype=torch.float64, device=dev)


def _exact_reorder(s):
    """Page by page on the host."""
    c = s["case"]
    B, W, dev = c["B"], c["W"], s["table"].device
    old, n, par = s["table"].tolist(), s["n_cached"].tolist(), s["parents"].tolist()
    free, out = s["free"].tolist(), s["table_out"].tolist()
    n_out, freed, moves, taken = [], [], [], 0
    for b in range(B):
        alive = [b * W + p for p in sorted(set(par[b]))]
        dead = []
        for j in range(len(old[0])):
            holds = [q for q in range(b * W, b * W + W) if j * PAGE < n[q]]
            stay = {old[q][j] for q in alive if q in holds}
            for q in holds:
                if old[q][j] not in stay and old[q][j] not in dead:
                    dead.append(old[q][j])
        claimed = set()
        for w in range(W):
            p = b * W + par[b][w]
            n_out.append(n[p])
            for j in range(-(-n[p] // PAGE)):
                page = old[p][j]
                if j == n[p] // PAGE:                     # not full
                    if page in claimed:
                        if dead:
                            page = dead.pop(0)
                        else:
                            page, taken = free[taken], taken + 1
                        moves.append((old[p][j], page, n[p] % PAGE))
                    claimed.add(old[p][j])
                out[b * W + w][j] = page
        freed += dead
    kv, sc = [x.double() for x in s["kv"]], [x.double() for x in s["sc"]]
    for src, dst, rows in moves:
        for x in kv:
            x[:, dst, :rows] = x[:, src, :rows]
        for x in sc:
            x[:, dst, :, :rows] = x[:, src, :, :rows]
    rest = [-1] * (s["freed"].numel() - len(freed))
    return _i32(out, dev), _i32(n_out, dev), _i32(freed + rest, dev), _i32([taken, len(freed)], dev), kv, sc


# ------------------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "append8":
        T, n_q, n_kv, hd = case["T"], case["n_q"], case["n_kv"], case["hd"]
        return {"bytes": T * (4 * n_q * hd + 2 * n_kv * (2 * hd + hd + 4) + 8),
                "flops": 3 * T * (n_q + n_kv) * hd + 2 * T * n_kv * hd}
    if op == "readback":
        n = sum(_lengths(case)) * case["n_kv"]
        return {"bytes": 2 * n * (3 * case["hd"] + 4), "flops": 2 * n * case["hd"]}
    if op == "attn8":
        n, hd = sum(_lengths(case)), case["hd"]
        return {"bytes": 2 * n * case["n_kv"] * (hd + 4) + 4 * case["B"] * case["n_q"] * hd + 4 * sum(map(_pages, _lengths(case))),
                "flops": 4 * n * case["n_q"] * hd}
    if op == "select":
        rows = case["B"] * case["W"]
        return {"bytes": 4 * rows * case["V"] + 4 * rows + 12 * case["B"] * case["K"], "flops": 4 * rows * case["V"]}
    # tables in and out; of children that share a parent all but one copy its open page
    B, W = case["B"], case["W"]
    every, parents = _beams(case)
    rows = sum((n % PAGE) * (W - len(set(p))) for (_, n), p in zip(every, parents))
    row = case["n_kv"] * (case["hd"] + 4 if case["bits"] == 8 else 2 * case["hd"])
    return {"bytes": 8 * W * sum(_pages(n) + 1 for _, n in every) + 4 * B * W + 2 * 2 * rows * case["layers"] * row,
            "flops": B * W * W}
