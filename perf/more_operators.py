"""Cases for long contexts in the softmax-attention layers: a cache in 8 bits, and attention
over selected blocks.

A hybrid stack's few softmax-attention layers keep every row of the context, so at long
contexts their caches are what a decode step reads and what bounds the batch.  Two means
against that, as a serving program calls them:

  append8  norm and rotation of new tokens, queries out, keys and values into cache pages in
           8 bits (e4m3) with a power-of-two scale for 16 rows of a key head
  attend8  attention of each sequence's new tokens over such a cache
  scores   a cheap score of every page for every new token: its queries with the mean key of
           the page (the means of the pages that the new tokens lie in are formed anew)
  select   the pages that each token reads: its first and last ones and the best by score
  blocks   attention of each token over its selected pages, of a cache in 16 or in 8 bits

`own` chooses between the library's calls and the plain form of the same operators.
Caches: [pages][kv heads][page rows][head size]; scales: [pages][kv heads][page rows / 16];
means: [pages][kv heads][head size]; page_table [sequence][page].
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------ cases


def listed():
    """The 2B/4B head layouts (12 or 16 query heads on 2 key heads of 128) at the lengths of
    the framework's own workloads (contexts of 64K rows, chunks of 2K, 64 decode steps), and
    odd small shapes of the fp32 mode."""
    return [
        # one token of one request in the middle of 16 rows: the latency of a step's first launch
        _case("append8", name="append8 step 1", B=1, T=1, ctx=4103),
        # a prefill step of 32 requests, chunks of many lengths (packed), 4B heads
        _case("append8", name="append8 chunks", B=32, T=1024, ctx=1024, H=16, packed=True),
        # a decode batch with contexts up to 64K
        _case("attend8", name="attend8 step 64", B=64, T=1, ctx=65535, ragged=True, lse=True),
        # chunked prefill: 2K new tokens at the end of a 64K context
        _case("attend8", name="attend8 chunk at 64K", B=1, T=2048, ctx=65536 - 2048),
        # odd lengths in the fp32 mode, small pages
        _case("attend8", name="attend8 f32 odd", B=3, T=77, ctx=423, H=6, Hkv=3, D=64, page=16, packed=True, lse=True,
              dtype="f32"),
        # scores of a decode batch, contexts up to 64K
        _case("scores", name="scores step 64", B=64, T=1, ctx=65535, ragged=True),
        # scores of a chunk of 2K tokens at the end of a 64K context, cache in 8 bits
        _case("scores", name="scores chunk at 64K", B=1, T=2048, ctx=65536 - 2048, bits=8),
        # one request's selection among the 1024 pages of a 64K context
        _case("select", name="select step 1", B=1, T=1, ctx=65535, count=32),
        # a chunk's selection
        _case("select", name="select chunk at 64K", B=1, T=2048, ctx=65536 - 2048, count=32),
        # a decode batch over 32 pages each, cache in 8 bits
        _case("blocks", name="blocks step 64", B=64, T=1, ctx=65535, ragged=True, count=32, bits=8),
        # one request's decode step at 64K over 16 pages, cache in 16 bits
        _case("blocks", name="blocks step 1", B=1, T=1, ctx=65535, count=16, lse=True),
        # a chunk of 500 tokens, each over its own 32 pages
        _case("blocks", name="blocks chunk at 32K", B=1, T=500, ctx=32000, H=16, count=32),
    ]


def _case(op, **kw):
    c = dict(op=op, B=1, T=1, ctx=0, H=12, Hkv=2, D=128, rot=kw.get("D", 128), pairs=False, page=64, window=0,
             packed=False, ragged=False, lse=False, dtype="bf16", bits=16, count=0)
    c.update(kw)
    return c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Another case of the same ranges: one token to chunks of 4K, caches of 0 to 64K rows, 1 to
    8 queries to a key head, three head sizes, both types, 4 to 64 pages of 16 to 128 rows."""
    op = rng.choice(["append8", "attend8", "attend8", "scores", "select", "blocks", "blocks"])
    f32 = rng.random() < 0.2
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 2, 3, 4])
    G = rng.choice([1, 2, 4, 5, 6, 8]) if D < 256 else rng.choice([1, 2, 4])
    kw = dict(H=Hkv * G, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2]), pairs=rng.random() < 0.3,
              dtype="f32" if f32 else "bf16", page=rng.choice([16, 32, 64, 128]))
    if op == "append8":
        B = _log(rng, 1, 64)
        return _case(op, B=B, T=_log(rng, 1, max(1, 16384 // (B * max(1, Hkv * G // 16)))), ctx=_log(rng, 1, 1024),
                     packed=rng.random() < 0.5, **kw)
    if op == "select":
        n, page, count = _log(rng, 1, 4096), kw["page"], _log(rng, 4, 64)
        # of more pages than are selected
        pages = _log(rng, 2 * count, max(2 * count, min(8192, 8 * 1024 * 1024 // (n * Hkv))))
        ctx = pages * page - 1 - rng.randrange(page)
        if rng.random() < 0.5:
            return _case(op, B=1, T=n, ctx=ctx, count=count, **kw)
        return _case(op, B=n, T=1, ctx=ctx, ragged=True, count=count, **kw)
    kw["bits"] = rng.choice([8, 16])
    if op == "scores":
        if rng.random() < 0.5:
            return _case(op, B=_log(rng, 1, 64), T=1, ctx=_log(rng, 1, 65000 * 2 // max(2, Hkv)), ragged=True, **kw)
        T = _log(rng, 2, 2048)
        return _case(op, B=rng.choice([1, 1, 2, 3]), T=T, ctx=_log(rng, 1, min(60000, 65536 * 2 * kw["page"] // (64 * Hkv))),
                     packed=rng.random() < 0.5, **kw)
    kw["lse"] = rng.random() < 0.5
    if op == "blocks":
        count = _log(rng, 4, 64)
        rows = count * kw["page"]
        most = 500 * 2 * 2048 * 128 // (Hkv * rows * D * (2 if f32 else 1))
        if rng.random() < 0.5:
            B = _log(rng, 1, max(1, min(64, most)))
            return _case(op, B=B, T=1, ctx=_log(rng, 1, min(65000, 64 * 65536 * 256 // (B * Hkv * D * (2 if f32 else 1)))),
                         ragged=True, count=count, **kw)
        B = rng.choice([1, 1, 2])
        return _case(op, B=B, T=_log(rng, 2, max(2, most // B)), ctx=_log(rng, 1, 32000), packed=rng.random() < 0.5,
                     count=count, **kw)
    kw["bits"], kw["window"] = 8, rng.choice([0, 0, 0, 1152, 2048, 100])
    if rng.random() < 0.5:  # a decode step
        B = _log(rng, 1, 64)
        rows = 64 * 65536 * 256 // (B * Hkv * D * (2 if f32 else 1))
        return _case(op, B=B, T=rng.choice([1, 1, 1, 2, 3]), ctx=_log(rng, 1, min(65000, rows)), ragged=True, **kw)
    B = _log(rng, 1, 16)
    pairs = 2048 * 65536 * 12 // (B * Hkv * G * (D // 64) * (6 if f32 else 1))
    T = _log(rng, 2, min(4096, int(math.sqrt(pairs))))
    return _case(op, B=B, T=T, ctx=_log(rng, 1, max(1, min(60000, pairs // T))) - 1, packed=rng.random() < 0.5, **kw)


def _lengths(c):
    """New tokens and cached rows (the new ones among them) of every sequence: all alike, or
    (packed, ragged) spread over the range by a fixed rule, the first one the longest."""
    new, kv = [], []
    for b in range(c["B"]):
        u = ((b * 0.6180339887498949) % 1.0)
        n = c["T"] if not c["packed"] or b == 0 else (1 if b % 4 == 3 else max(1, int(c["T"] * (1 - u))))
        old = c["ctx"] if not (c["packed"] or c["ragged"]) or b == 0 else int(c["ctx"] * (1 - u))
        new.append(n)
        kv.append(n + old)
    return new, kv


def _cells(c):
    """Pairs of a new token and a page that it sees, over all sequences."""
    new, kv = _lengths(c)
    total = 0
    for t, l in zip(new, kv):
        upto = lambda n: (n // c["page"]) * (n // c["page"] + 1) // 2 * c["page"] + (n // c["page"] + 1) * (n % c["page"])  # noqa: E731
        total += upto(l) - upto(l - t)
    return total


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    ce = 1 + 1 / (16 * c["D"]) if c["bits"] == 8 or c["op"] in ("append8", "attend8") else e
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]
    new, kv = _lengths(c)
    n = sum(new)
    if c["op"] == "append8":
        return {"bytes": n * (2 * H + 2 * Hkv) * D * e + 2 * n * Hkv * D * ce, "flops": n * (H + Hkv) * D * 8}
    if c["op"] == "scores":
        rows = sum(l - (l - t) // page * page for t, l in zip(new, kv))  # of the pages with new tokens
        pages = sum(-(-l // page) for l in kv)
        width = max(-(-l // page) for l in kv)
        return {"bytes": n * H * D * e + rows * Hkv * D * ce + pages * Hkv * D * 4 + n * Hkv * width * 4,
                "flops": 2 * _cells(c) * H * D}
    if c["op"] == "select":
        return {"bytes": Hkv * (_cells(c) * 4 + n * c["count"] * 4), "flops": 0}
    if c["op"] == "blocks":
        rows = [[min(c["count"] * page, l - t + i + 1) for i in range(t)] for t, l in zip(new, kv)]
        seen = sum(min(l, sum(r)) for r, l in zip(rows, kv))
        return {"bytes": 2 * n * H * D * e + n * Hkv * c["count"] * 4 + 2 * seen * Hkv * D * ce,
                "flops": 4 * sum(map(sum, rows)) * H * D}
    seen = pairs = 0
    for t, l in zip(new, kv):
        w = c["window"] or l
        first = l - t  # position of the first new token
        seen += l - max(0, first - w + 1)
        full = max(0, min(t, w - first))  # queries whose window reaches back to row 0
        pairs += full * first + full * (full + 1) // 2 + (t - full) * w
    return {"bytes": 2 * n * H * D * e + 2 * seen * Hkv * D * ce, "flops": 4 * pairs * H * D}


# ----------------------------------------------------------------- inputs


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _DT[c["dtype"]]
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]

    def randn(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    new, kv = _lengths(c)
    s = {"c": c, "max_seqlen": max(new), "max_kv": max(kv)}
    s["kv_lens"] = torch.tensor(kv, device="cuda", dtype=torch.int32)
    s["cu"] = None
    if c["packed"]:
        s["cu"] = torch.tensor([0] + [sum(new[:i + 1]) for i in range(len(new))], device="cuda", dtype=torch.int32)
    n = sum(new)
    lead = (n,) if c["packed"] else (c["B"], c["T"])
    need = [-(-l // page) for l in kv]
    if c["op"] == "select":
        s["scores"] = randn(*lead, Hkv, max(need), dtype=torch.float32)
        s["q"] = torch.empty(*lead, 0, device="cuda")
        _hide(c, s)
        return s
    # every sequence's pages lie anywhere in the pool; 3 pages stay free
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(kv), max(need), device="cuda", dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    s["table"] = table
    s["q"] = randn(*lead, H, D)  # [sequences, new tokens, heads, D] (dense) or [all new tokens, heads, D]
    if c["op"] in ("append8", "attend8") or c["bits"] == 8:
        for x in ("k", "v"):
            s[x + "_cache"], s[x + "_scales"] = _in8(randn(pool, Hkv, page // 16, 16, D, dtype=torch.float32))
            s[x + "_cache"] = s[x + "_cache"].view(pool, Hkv, page, D)
    else:
        s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"] = randn(pool, Hkv, page, D), randn(pool, Hkv, page, D), None, None
    if c["op"] == "append8":
        rot = c["rot"]
        s["inv_freq"] = (1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        s["wq"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt)
        s["wk"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dt)
        s["k"], s["v"] = randn(*lead, Hkv, D), randn(*lead, Hkv, D)
    if c["op"] == "scores":
        s["means"] = _values(s["k_cache"], s["k_scales"]).mean(2)
    if c["op"] == "blocks":
        # neighbouring tokens want much the same pages
        base = randn(len(kv), 1, Hkv, max(need), dtype=torch.float32)
        seq, row, _ = _places(s, c)
        s["scores"] = (base[seq, 0] + 0.5 * randn(n, Hkv, max(need), dtype=torch.float32)).view(*lead, Hkv, max(need))
        s["blocks"] = _select(c, s)["blocks"]
        del s["scores"]
    return s


def _hide(c, s):
    """Scores of pages that a token does not see are -inf."""
    _, row, _ = _places(s, c)
    x = s["scores"].view(len(row), c["Hkv"], -1)
    x.masked_fill_((torch.arange(x.shape[2], device="cuda") > (row // c["page"])[:, None])[:, None], -math.inf)


def _exponent(most):
    """k of the smallest scale 2^k with most <= 448 * 2^k, -126 at least, as int32."""
    m, p = torch.frexp(most)
    return (p - 9 + (m > 0.875)).masked_fill(most == 0, -126).clamp(min=-126)


def _in8(x):
    """[..., 16, D] fp32 in e4m3 with a power-of-two scale for each 16 rows."""
    k = _exponent(x.abs().amax((-2, -1)))
    return torch.ldexp(x, -k[..., None, None]).to(E4M3), (k + 127).to(torch.uint8).view(E8M0)


def _values(cache, scales):
    """What a cache [..., page, D] holds, in fp32."""
    if scales is None:
        return cache.float()
    x = cache.float().unflatten(-2, (-1, 16))
    return x.mul_(scales.float()[..., None, None]).flatten(-3, -2)


# -------------------------------------------------------------------- run


def run(state):
    c = state["c"]
    if own:
        return _own(c, state)
    return {"append8": _append8, "attend8": _attend8, "scores": _scores, "select": _select, "blocks": _blocks}[c["op"]](c, state)


def _own(c, s):
    from gated_delta_rule_jetblock_amd import jetblock as jb
    if c["op"] == "append8":
        return jb.qk_norm_rope_paged8(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                      s["table"], s["kv_lens"], s["inv_freq"], s["wq"], s["wk"], cu_seqlens=s["cu"],
                                      max_seqlen=s["max_seqlen"], interleaved=c["pairs"])
    if c["op"] == "attend8":
        r = jb.attn_paged8(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"], s["kv_lens"],
                           cu_seqlens=s["cu"], max_seqlen=s["max_seqlen"], max_kv=s["max_kv"], window=c["window"],
                           want_lse=c["lse"])
        return r if c["lse"] else {"o": r["o"]}
    if c["op"] == "scores":
        return jb.block_scores(s["q"], s["k_cache"], s["means"], s["table"], s["kv_lens"], k_scales=s["k_scales"],
                               cu_seqlens=s["cu"], max_seqlen=s["max_seqlen"])
    if c["op"] == "select":
        return {"blocks": jb.block_select(s["scores"], s["kv_lens"], c["count"], c["page"], cu_seqlens=s["cu"])}
    r = jb.attn_blocks(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["blocks"], k_scales=s["k_scales"],
                       v_scales=s["v_scales"], cu_seqlens=s["cu"], max_seqlen=s["max_seqlen"], want_lse=c["lse"])
    return r if c["lse"] else {"o": r["o"]}


# ------------------------------------------------------------- plain forms


def _places(s, c):
    """Of every new token: its sequence, its row in the sequence's cache, its place among the new."""
    kv = s["kv_lens"].long()
    if s["cu"] is None:
        seq = torch.arange(c["B"], device=kv.device).repeat_interleave(c["T"])
        i = torch.arange(c["T"], device=kv.device).repeat(c["B"])
        return seq, kv[seq] - c["T"] + i, i
    cu = s["cu"].long()
    n = s["q"].shape[0]
    t = torch.arange(n, device=kv.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[seq]
    return seq, kv[seq] - (cu[seq + 1] - cu[seq]) + i, i


def _norm_rope(x, w, cos, sin, c, eps=1e-6):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()
    rot = c["rot"]
    if c["pairs"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, y[..., rot:]), -1)


def _append8(c, s):
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]
    seq, row, _ = _places(s, c)
    # cos and sin of position times frequency, formed in 64 bits
    a = row.double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
    q = _norm_rope(s["q"].view(-1, H, D), s["wq"], cos, sin, c).to(s["q"].dtype)
    k = _norm_rope(s["k"].view(-1, Hkv, D), s["wk"], cos, sin, c)
    # the 16-row blocks that hold new rows, each once, and every new row's place among them
    part = seq * (s["table"].shape[1] * page // 16) + row // 16
    cells, inverse = torch.unique_consecutive(part, return_inverse=True)
    per = page // 16
    cell_seq, cell = cells // (s["table"].shape[1] * per), cells % (s["table"].shape[1] * per)
    where = s["table"][cell_seq, cell // per].long()
    is_new = torch.zeros(len(cells), 16, device=row.device, dtype=torch.bool)
    is_new[inverse, row % 16] = True
    old = (is_new.int().cumsum(1) == 0)  # rows before the first new one
    out = {"q": q.view(s["q"].shape)}
    for x, fresh in (("k", k), ("v", s["v"].view(-1, Hkv, D).float())):
        cache, scales = s[x + "_cache"].view(-1, Hkv, per, 16, D), s[x + "_scales"].view(torch.uint8)
        new = torch.zeros(len(cells), Hkv, 16, D, device=row.device)
        new[inverse, :, row % 16] = fresh
        was = cache.view(torch.uint8)[where, :, cell % per]
        e_was = scales[where, :, cell % per].int() - 127
        e = _exponent(torch.where(is_new[:, None, :, None], new.abs(), 0.0).amax((-2, -1)))
        e = torch.where(old.any(1)[:, None], torch.maximum(e, e_was), e)
        kept = torch.ldexp(was.view(E4M3).float(), (e_was - e)[..., None, None])
        codes = torch.where(is_new[:, None, :, None], torch.ldexp(new, -e[..., None, None]), kept).to(E4M3)
        codes = torch.where((is_new | old)[:, None, :, None], codes.view(torch.uint8), was)
        cache.view(torch.uint8)[where, :, cell % per] = codes
        scales[where, :, cell % per] = (e + 127).to(torch.uint8)
        out[x + "_cache"], out[x + "_scales"] = s[x + "_cache"], s[x + "_scales"]
    return out


def _softmax(x, v):
    """Weights of x [..., rows] over v [..., rows, D] and the logarithm of their sum."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    return torch.matmul(x, v) / torch.where(total == 0, 1.0, total), (m + total.log()).squeeze(-1)


def _attend8(c, s):
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    G, B, T, L = H // Hkv, c["B"], s["max_seqlen"], s["max_kv"]
    dt = s["q"].dtype
    seq, row, i = _places(s, c)
    # caches by sequence, padded to the longest; queries likewise
    where = s["table"].long()
    k, v = (_values(s[x + "_cache"].view(torch.uint8)[where].view(E4M3), s[x + "_scales"].view(torch.uint8)[where].view(E8M0))
            .permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)[:, :, :L] for x in ("k", "v"))
    q = torch.zeros(B, T, H, D, device=k.device)
    q[seq, i] = s["q"].view(-1, H, D).float()
    q = q.view(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, T, L)
    at = torch.full((B, T), -1, device=k.device, dtype=torch.long)
    at[seq, i] = row
    j = torch.arange(L, device=k.device)
    seen = j <= at[:, :, None]
    if c["window"]:
        seen &= j > at[:, :, None] - c["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    o, lse = _softmax(x.view(B, Hkv, G * T, L), v)
    o = o.view(B, Hkv, G, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, H, D)[seq, i].to(dt).view(s["q"].shape)
    if not c["lse"]:
        return {"o": o}
    lse = lse.view(B, Hkv, G, T).permute(0, 3, 1, 2).reshape(B, T, H)[seq, i]
    return {"o": o, "lse": lse.view(s["q"].shape[:-1])}


def _scores(c, s):
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]
    G, B, T = H // Hkv, c["B"], s["max_seqlen"]
    seq, row, i = _places(s, c)
    width = s["table"].shape[1]
    # the pages with new tokens, each once: the mean of the rows that they hold by now
    cells = torch.unique_consecutive(seq * width + row // page)
    where = s["table"].view(-1)[cells].long()
    held = (s["kv_lens"].long()[cells // width] - cells % width * page).clamp(max=page)
    rows = _values(s["k_cache"].view(torch.uint8)[where].view(E4M3), s["k_scales"].view(torch.uint8)[where].view(E8M0)) \
        if c["bits"] == 8 else s["k_cache"][where].float()
    rows = torch.where((torch.arange(page, device=row.device) < held[:, None])[:, None, :, None], rows, 0.0)
    s["means"][where] = rows.sum(2) / held[:, None, None]
    q = torch.zeros(B, T, H, D, device=row.device)
    q[seq, i] = s["q"].view(-1, H, D).float()
    q = q.view(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    means = s["means"][s["table"].long()].permute(0, 2, 3, 1).contiguous()  # [B, Hkv, D, pages]
    x = torch.matmul(q, means).view(B, Hkv, G, T, width).amax(2).permute(0, 2, 1, 3)[seq, i]
    x = x.masked_fill((torch.arange(width, device=row.device) > (row // page)[:, None])[:, None], -math.inf)
    return {"scores": x.view(*s["q"].shape[:-2], Hkv, width), "means": s["means"]}


def _select(c, s, first=1, recent=1):
    _, row, _ = _places(s, c)
    width, count = s["scores"].shape[-1], c["count"]
    x = s["scores"].view(len(row), c["Hkv"], width)
    j, mine = torch.arange(width, device=row.device), (row // c["page"])[:, None, None]
    x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=torch.finfo(torch.float32).max)
    x = torch.where((j < first) | (j > mine - recent), math.inf, x)
    x = torch.where(j > mine, -math.inf, x)
    best = x.sort(dim=-1, descending=True, stable=True).indices[..., :count]  # ties: the lowest index first
    best = torch.where(best > mine, width, best).sort(-1).values
    out = torch.full((*x.shape[:2], count), -1, device=row.device, dtype=torch.int32)
    out[..., :best.shape[-1]] = torch.where(best == width, -1, best).int()
    return {"blocks": out.view(*s["scores"].shape[:-1], count)}


def _blocks(c, s):
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]
    G, count = H // Hkv, c["count"]
    seq, row, _ = _places(s, c)
    n = len(row)
    at = s["blocks"].view(n, Hkv, count).long()
    where = s["table"].long()[seq[:, None, None], at.clamp(min=0)]
    head = torch.arange(Hkv, device=row.device)[None, :, None]
    if c["bits"] == 8:
        k, v = (_values(s[x + "_cache"].view(torch.uint8)[where, head].view(E4M3),
                        s[x + "_scales"].view(torch.uint8)[where, head].view(E8M0)) for x in ("k", "v"))
    else:
        k, v = s["k_cache"][where, head].float(), s["v_cache"][where, head].float()
    k, v = k.view(n, Hkv, count * page, D), v.view(n, Hkv, count * page, D)
    x = torch.matmul(s["q"].view(n, Hkv, G, D).float(), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    j = at[..., None] * page + torch.arange(page, device=row.device)
    seen = (at[..., None] >= 0) & (j <= row[:, None, None, None])
    x.masked_fill_(~seen.view(n, Hkv, 1, count * page), -math.inf)
    o, lse = _softmax(x, v)
    o = o.reshape(s["q"].shape).to(s["q"].dtype)
    return {"o": o, "lse": lse.reshape(s["q"].shape[:-1])} if c["lse"] else {"o": o}


# ------------------------------------------------- from the definition, 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "select":
        return None  # whole numbers
    H, Hkv, D, page = c["H"], c["Hkv"], c["D"], c["page"]
    G = H // Hkv
    new, kv = _lengths(c)
    q = s["q"].double().reshape(-1, H, D)
    at = 0
    if c["op"] == "append8":
        codes = {x: s[x + "_cache"].double().reshape(-1, Hkv, page // 16, 16, D) for x in ("k", "v")}
        scales = {x: s[x + "_scales"].double() for x in ("k", "v")}
        fresh = {x: s[x].double().reshape(-1, Hkv, D) for x in ("k", "v")}
        for b, (t, l) in enumerate(zip(new, kv)):
            turn = torch.polar(torch.ones(1, device="cuda", dtype=torch.float64),
                               torch.arange(l - t, l, device="cuda").double()[:, None, None] * s["inv_freq"].double())
            here = slice(at, at + t)
            q[here] = _turned(q[here] / (q[here].square().sum(-1, keepdim=True) / D + 1e-6).sqrt() * s["wq"].double(), turn, c)
            y = fresh["k"][here]
            fresh["k"][here] = _turned(y / (y.square().sum(-1, keepdim=True) / D + 1e-6).sqrt() * s["wk"].double(), turn, c)
            # 16 rows at a time, all blocks of the sequence at once: rows before the first new one stay, rescaled
            low, high = (l - t) // 16, (l - 1) // 16
            cell = torch.arange(low, high + 1, device="cuda")
            page_of = s["table"][b].long()[cell * 16 // page]
            slot = cell % (page // 16)
            r = cell[:, None] * 16 + torch.arange(16, device="cuda")
            mine, before = ((r >= l - t) & (r < l))[:, None, :, None], (r < l - t)[:, None, :, None]
            for x in ("k", "v"):
                rows = torch.zeros((high - low + 1) * 16, Hkv, D, device="cuda", dtype=torch.float64)
                rows[l - t - 16 * low:l - 16 * low] = fresh[x][here]
                rows = rows.view(-1, 16, Hkv, D).transpose(1, 2)
                most = rows.abs().amax((2, 3))
                scale = torch.exp2(torch.ceil(torch.log2(most / 448)).clamp(min=-126))
                scale = torch.where(448 * scale / 2 >= most, scale / 2, scale)  # (a logarithm next to a whole number)
                was = scales[x][page_of, :, slot]
                scale[0] = torch.where(before[0].any(), torch.maximum(scale[0], was[0]), scale[0])
                old = codes[x][page_of, :, slot]
                put = torch.where(mine, _e4m3(rows / scale[..., None, None]),
                                  torch.where(before, _e4m3(old * (was / scale)[..., None, None]), old))
                codes[x][page_of, :, slot], scales[x][page_of, :, slot] = put, scale
            at += t
        out = {"q": q.view(s["q"].shape)}
        for x in ("k", "v"):
            out[x + "_cache"], out[x + "_scales"] = codes[x].view(s[x + "_cache"].shape), scales[x]
        return out
    if c["op"] == "scores":
        width = s["table"].shape[1]
        means = s["means"].double()
        scores = torch.full((q.shape[0], Hkv, width), -math.inf, device="cuda", dtype=torch.float64)
        for b, (t, l) in enumerate(zip(new, kv)):
            table = s["table"][b].long()
            for blk in range((l - t) // page, (l - 1) // page + 1):
                m = min(page, l - blk * page)
                means[table[blk]] = _held(s, "k", table[blk][None], c)[0, :, :m].sum(1) / m
            for h in range(H):
                x = q[at:at + t, h] @ means[table, h // G].t().contiguous()
                p = torch.arange(l - t, l, device="cuda")[:, None] // page
                x[torch.arange(width, device="cuda")[None] > p] = -math.inf
                scores[at:at + t, h // G] = torch.maximum(scores[at:at + t, h // G], x)
            at += t
        return {"scores": scores.view(*s["q"].shape[:-2], Hkv, width), "means": means}
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda", dtype=torch.float64)
    for b, (t, l) in enumerate(zip(new, kv)):
        p = torch.arange(l - t, l, device="cuda")[:, None]
        table = s["table"][b, :-(-l // page)].long()
        k, v = (_held(s, x, table, c).transpose(0, 1).reshape(Hkv, -1, D)[:, :l] for x in ("k", "v"))
        j = torch.arange(l, device="cuda")
        for h in range(H):
            g = h // G
            hidden = j[None] > p
            if c["op"] == "blocks":
                chosen = torch.zeros(t, len(table) + 1, device="cuda", dtype=torch.bool)
                chosen.scatter_(1, s["blocks"].view(-1, Hkv, c["count"])[at:at + t, g].long() % (len(table) + 1), True)
                hidden |= ~chosen[:, j // page]
            elif c["window"]:
                hidden |= j[None] <= p - c["window"]
            x = q[at:at + t, h] @ k[g].t().contiguous() / D ** 0.5
            x[hidden] = -math.inf
            lse[at:at + t, h] = torch.logsumexp(x, -1)
            o[at:at + t, h] = torch.exp(x - lse[at:at + t, h, None]) @ v[g]
            del x
        at += t
    return {"o": o.view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])} if c["lse"] else {"o": o.view(s["q"].shape)}


def _held(s, x, pages, c):
    """[pages, Hkv, page, D] of a cache in 64 bits."""
    if s[x + "_scales"] is None:
        return s[x + "_cache"][pages].double()
    code = s[x + "_cache"].view(torch.uint8)[pages].long()
    sign, e, f = 1.0 - 2.0 * (code >> 7), (code >> 3) & 15, (code & 7).double()
    v = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2(e.double() - 7)) * sign
    scale = torch.exp2(s[x + "_scales"].view(torch.uint8)[pages].double() - 127)
    return v * scale.repeat_interleave(16, -1)[..., None]


def _e4m3(x):
    """The nearest e4m3 value (ties to even), |x| at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs())).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _turned(x, turn, c):
    """Every pair as a complex number, times e^(i angle)."""
    rot = c["rot"]
    first = torch.arange(0, rot, 2, device=x.device) if c["pairs"] else torch.arange(rot // 2, device=x.device)
    second = first + (1 if c["pairs"] else rot // 2)
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y
