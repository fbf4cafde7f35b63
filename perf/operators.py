"""Workloads of the attention-side operators of a decoder layer's serving step.

Four operators, which share one paged K/V cache (pages of `page` tokens, each
[kv heads, page, head dim], bf16 or e4m3 codes with one scale per kv head):

  rope     rotary positions on q and k of the step's new tokens, k and v stored
           into the cache's pages
  attn     attention of the step's new tokens (single tokens, verify blocks of
           up to 8 rows, prefill chunks) over the cache, with the log-sum-exp
  weights  the attention weight every cached key received in the step, added to
           the running scores that eviction goes by
  evict    per kv head the keys with the largest scores and the most recent
           ones kept, their K and V rows moved together into other pages

`run` computes them in elementary fp32 torch operations, or (own) through the
framework's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
# rotary scaling for long contexts used by the cases that say so: the by-parts
# ramp between 1 and 32 turns over an original length of 4096, factor 8
RAMP = {"factor": 8.0, "orig": 4096, "fast": 32.0, "slow": 1.0}


def _c(name, op, seqs, ctx_lo, ctx_hi, new, ragged, hq, hkv, dim, page, kv, **more):
    return dict(name=name, op=op, seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new=new, ragged=ragged,
                hq=hq, hkv=hkv, dim=dim, page=page, kv=kv, **{**_MORE, **more})


# layout: order of a page's axes (hnd: head, token; nhd: token, head); rot: rotated
# part of the head; window: sliding window (0: none); tree: draft masks; budget/recent: eviction
_MORE = dict(layout="hnd", rot=0, inter=False, ramp=False, window=0, tree=False, budget=0, recent=0)


def listed():
    return [
        # one 8-row verify block of a single user: the smallest call, all latency
        _c("rope_verify8", "rope", 1, 4097, 4097, 8, False, 64, 8, 128, 64, "bf16", rot=128),
        # a ragged mixed batch into an e4m3 cache: odd counts, small pages, part of the
        # head rotated in the interleaved layout with long-context scaling
        _c("rope_mixed_e4m3", "rope", 37, 100, 20011, 19, True, 24, 3, 64, 16, "e4m3", rot=32, inter=True,
           ramp=True, layout="nhd"),
        # a prefill chunk of the most rows a layer call takes
        _c("rope_chunk4096", "rope", 1, 4096, 4096, 4096, False, 64, 8, 128, 64, "bf16", rot=128, ramp=True),
        # single-user speculative verify: one committed token and 7 drafts
        _c("attn_verify8", "attn", 1, 6011, 6011, 8, False, 64, 8, 128, 64, "bf16"),
        # continuous batching: single tokens at lengths spread over 1:128
        _c("attn_decode48", "attn", 48, 251, 32011, 1, False, 64, 8, 128, 64, "bf16"),
        # batched verify blocks over an e4m3 cache, ragged block lengths
        _c("attn_verify16_e4m3", "attn", 16, 4099, 16411, 8, True, 64, 8, 128, 64, "e4m3", tree=True),
        # a prefill chunk over a long cached prefix: the largest call
        _c("attn_chunk2048", "attn", 1, 16384, 16384, 2048, False, 64, 8, 128, 64, "bf16"),
        # weights of a decode batch
        _c("weights_decode8", "weights", 8, 1021, 8209, 1, False, 64, 8, 128, 64, "bf16"),
        # weights of batched verify blocks over an e4m3 cache
        _c("weights_verify16_e4m3", "weights", 16, 4099, 16411, 8, True, 64, 8, 128, 64, "e4m3"),
        # weights of a prefill chunk
        _c("weights_chunk1024", "weights", 1, 8192, 8192, 1024, False, 64, 8, 128, 64, "bf16"),
        # one user's cache halved
        _c("evict_one", "evict", 1, 8191, 8191, 1, False, 64, 8, 128, 64, "bf16", budget=4096, recent=256),
        # a batch of long e4m3 caches cut to a fixed budget (one of them is under it already)
        _c("evict_batch16_e4m3", "evict", 16, 5003, 32003, 1, False, 64, 8, 128, 64, "e4m3", budget=8000,
           recent=1000),
    ]


HEADS = [(64, 8, 128), (32, 8, 128), (24, 3, 64), (16, 16, 128), (40, 8, 128), (12, 1, 64), (8, 8, 64), (48, 4, 128)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "attn", "attn", "weights", "evict"])
        hq, hkv, dim = rng.choice(HEADS)
        page = rng.choice([16, 32, 64, 128])
        kv = rng.choice(["bf16", "e4m3"])
        layout = rng.choice(["hnd", "nhd"])
        hi = _log(rng, 1, 32768)
        lo = _log(rng, 1, hi)
        form = rng.choice(["single", "verify", "chunk"])
        new = 1 if form == "single" else rng.randint(2, 8) if form == "verify" else _log(rng, 9, 2048)
        seqs = _log(rng, 1, 64) if form != "chunk" else _log(rng, 1, 6)
        c = _c(None, op, seqs, lo, hi, new, rng.random() < 0.5, hq, hkv, dim, page, kv, layout=layout)
        del c["name"]
        if op == "rope":
            c["rot"] = rng.choice([dim, dim // 2, dim // 4])
            c["inter"] = rng.random() < 0.5
            c["ramp"] = rng.random() < 0.5
        elif op == "evict":
            if hi < 16:
                continue
            c["new"], c["ragged"] = 1, False
            c["budget"] = _log(rng, 8, hi)
            c["recent"] = rng.randint(0, c["budget"])
        else:
            c["window"] = _log(rng, 1, hi) if rng.random() < 0.25 else 0
            c["tree"] = form == "verify" and rng.random() < 0.5
        # no drawn case costs more than the largest listed one, nor holds more than a few times its memory
        cells = seqs * (hi + new) * hkv
        if cells * dim > 640e6 or seqs * hi * new * hq > 2.4e9 or work(c)["flops"] > 1.1e12 or work(c)["bytes"] > 2.5e9:
            continue
        if work(c)["bytes"] < 20000:
            continue
        return c


# ---------------------------------------------------------------- geometry --
def _lens(case):
    """New tokens and total cache lengths of the sequences; by the case alone."""
    news, lens = [], []
    for b in range(case["seqs"]):
        u = 1.0 - math.modf(b * 0.6180339887498949)[0]
        ctx = int(round(case["ctx_lo"] * (case["ctx_hi"] / case["ctx_lo"]) ** u))
        n = case["new"] - (b * 5) % case["new"] if case["ragged"] else case["new"]
        news.append(n)
        lens.append(ctx + n)
    return news, lens


def _pairs(case):
    """(query, key) pairs that attention computes, and keys that some query of their sequence sees."""
    news, lens = _lens(case)
    pairs = keys = 0
    w = case["window"] or 1 << 60
    for n, length in zip(news, lens):
        first = length - n + 1                       # keys up to the first query, itself included
        full = max(0, min(n, w - first + 1))         # queries whose window reaches the start
        pairs += full * first + full * (full - 1) // 2 + (n - full) * min(w, length)
        keys += min(length, first - 1 + n - max(0, first - w))
    return pairs, keys


def work(case):
    news, lens = _lens(case)
    t, hq, hkv, d = sum(news), case["hq"], case["hkv"], case["dim"]
    e = 2 if case["kv"] == "bf16" else 1
    if case["op"] == "rope":      # q, k, v read; q, k, v written; the angles' cos and sin
        return {"bytes": t * d * (4 * hq + (4 + 2 * e) * hkv) + 4 * t, "flops": t * case["rot"] * (hq + hkv) * 3}
    if case["op"] == "attn":
        pairs, keys = _pairs(case)
        return {"bytes": keys * hkv * d * 2 * e + t * hq * (4 * d + 4), "flops": 4 * pairs * hq * d}
    if case["op"] == "weights":
        pairs, keys = _pairs(case)
        return {"bytes": keys * hkv * d * e + sum(lens) * hkv * 8 + t * hq * (2 * d + 4), "flops": 2 * pairs * hq * d}
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": sum(lens) * hkv * 4 + kept * hkv * (4 * d * e + 8) + 4 * case["seqs"], "flops": 0}


# ------------------------------------------------------------------ inputs --
def _freqs(case):
    """Turns per position of each rotated pair as two fp32 (their sum is it to 48 bits), and the magnitude."""
    half = case["rot"] // 2
    i = torch.arange(half, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / case["rot"])
    mag = 1.0
    if case["ramp"]:
        at = lambda turns: case["rot"] * math.log(RAMP["orig"] / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
        lo, hi = max(math.floor(at(RAMP["fast"])), 0), min(math.ceil(at(RAMP["slow"])), case["rot"] - 1)
        r = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - r) + f / RAMP["factor"] * r
        mag = 0.1 * math.log(RAMP["factor"]) + 1.0
    f = f / (2 * math.pi)
    hi32 = f.float()
    return torch.stack([hi32, (f - hi32.double()).float()], 1), mag


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16)
    news, lens = _lens(case)
    hq, hkv, d, page, n = case["hq"], case["hkv"], case["dim"], case["page"], case["seqs"]
    need = [-(-x // page) for x in lens]
    after = [-(-min(x, case["budget"]) // page) for x in lens]
    total = sum(need) + sum(after) + 3
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()

    def table(counts, at):
        t = torch.full((n, max(max(counts), 1)), -1, dtype=torch.int32)
        for b, c in enumerate(counts):
            t[b, :c] = perm[at:at + c]
            at += c
        return t.to(DEV)

    shape = (total, hkv, page, d) if case["layout"] == "hnd" else (total, page, hkv, d)
    k, v = rnd(*shape), rnd(*shape)
    s = {"case": case, "lens": lens}
    if case["kv"] == "e4m3":      # codes of values of unit size: the largest of them near the codes' end
        s["k_scale"] = 0.011 * (1 + torch.rand(hkv, generator=g, device=DEV))
        s["v_scale"] = 0.011 * (1 + torch.rand(hkv, generator=g, device=DEV))
        k = (k * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        v = (v * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    if case["layout"] == "nhd":
        k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    s["k"], s["v"] = k, v
    t = sum(news)
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    s["cu"], s["kv_len"], s["table"] = i32(cu), i32(lens), table(need, 0)
    s["max_q"] = max(news)
    # the projections' output: q, k and v heads of a token side by side
    qkv = rnd(t, hq + 2 * hkv, d)
    s["q"], s["nk"], s["nv"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["scale"] = d ** -0.5
    cap = max(need) * page
    if case["op"] == "rope":
        s["pos"] = i32([lens[b] - news[b] + i for b in range(n) for i in range(news[b])])
        s["freqs"], s["mag"] = _freqs(case)
        s["freqs"] = s["freqs"].to(DEV)
        s["q_out"] = torch.zeros(t, hq, d, dtype=torch.bfloat16, device=DEV)
    else:
        s["q"] = (s["q"] * 1.5).contiguous() if case["op"] != "evict" else s["q"]   # scores spread as in earnest
        s["tree"] = None
        if case["tree"]:          # each draft sees itself, its parent's path, a random parent a draft
            bits = []
            for x in news:
                par = torch.randint(0, 1 << 20, (x,), generator=g, device=DEV).cpu().tolist()
                seen = []
                for i in range(x):
                    seen.append((1 << i) | (seen[par[i] % i] if i else 0))
                bits += seen
            s["tree"] = torch.tensor(bits, dtype=torch.int64, device=DEV)
    if case["op"] == "attn":
        s["out"] = torch.zeros(t, hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(t, hq, dtype=torch.float32, device=DEV)
    if case["op"] in ("weights", "evict"):
        # running scores: a few keys carry most of the weight
        s["scores"] = torch.rand(n, hkv, cap, generator=g, device=DEV).pow_(-0.7)
        s["scores_out"] = torch.zeros_like(s["scores"])
    if case["op"] == "weights":
        s["decay"] = 0.98
        s["lse"] = _attend(s)[1]
    if case["op"] == "evict":
        s["to"] = table(after, sum(need))
        s["kept"] = torch.zeros(n, hkv, case["budget"], dtype=torch.int32, device=DEV)
        s["new_len"] = torch.zeros(n, dtype=torch.int32, device=DEV)
    if own:                       # the handles that a program builds once for its cache and its batch
        import moe_speculative_verify_gb300 as m
        m.load()
        s["h_cache"] = m.KVCache.from_tensors(k, v, s.get("k_scale"), s.get("v_scale"))
        s["h_seqs"] = m.Seqs.from_tensors(s["cu"], s["kv_len"], s["table"], s["max_q"])
        if case["op"] == "rope":
            s["h_rope"] = m.Rope.from_freqs(s["freqs"], case["inter"], s["mag"])
        else:
            s["h_attn"] = m.Attn(hq, s["scale"], True, case["window"])
            s["ws"] = torch.zeros(m.moe_attn_workspace_bytes(s["h_attn"], s["h_cache"]), dtype=torch.uint8, device=DEV)
    return s


# -------------------------------------------------------------- plain forms --
def _gather(s, x, scale):
    """The sequences' cached rows, fp32 [seqs, kv heads, keys, dim]; places past a sequence's end hold some page's rows."""
    x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
    y = x[s["table"].clamp(min=0).long()]                       # [seqs, pages, heads, page, dim]
    n, p, h, t, d = y.shape
    y = y.permute(0, 2, 1, 3, 4).reshape(n, h, p * t, d)
    if scale is None:
        return y.float()
    return y.view(torch.float8_e4m3fn).float() * scale[:, None, None]


def _rows(s):
    """Token index of query i of every sequence [seqs, new], and which of them exist."""
    i = torch.arange(s["max_q"], device=DEV)
    cu = s["cu"].long()
    live = i[None] < (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + i[None]).clamp(max=int(s["q"].shape[0]) - 1), live


def _seen(s, keys):
    """Which keys each query sees: [seqs, new, keys]."""
    cu, length = s["cu"].long(), s["kv_len"].long()
    first = (length - (cu[1:] - cu[:-1]))[:, None, None]        # cache place of the first new token
    i = torch.arange(s["max_q"], device=DEV)[None, :, None]
    j = torch.arange(keys, device=DEV)[None, None, :]
    if s["tree"] is None:
        seen = j <= first + i
    else:
        bits = s["tree"][_rows(s)[0]][:, :, None]
        at = (j - first).clamp(0, 63)
        seen = (j < first) | ((j - first < 64) & ((bits >> at) & 1 == 1))
    seen = seen & (j < length[:, None, None]) & _rows(s)[1][:, :, None]
    if s["case"]["window"]:
        seen = seen & (j > first + i - s["case"]["window"])
    return seen


def _scores(s):
    c = s["case"]
    kk = _gather(s, s["k"], s.get("k_scale"))
    rows, _ = _rows(s)
    n, g = c["seqs"], c["hq"] // c["hkv"]
    q = s["q"][rows].float().view(n, -1, c["hkv"], g, c["dim"]).permute(0, 2, 1, 3, 4)
    x = q.reshape(n, c["hkv"], -1, c["dim"]) @ kk.transpose(2, 3)
    x = x.mul_(s["scale"])                                      # [seqs, kv heads, new x group, keys]
    seen = _seen(s, x.shape[3]).repeat_interleave(g, 1)[:, None]
    return x.masked_fill_(~seen, -math.inf)


def _tokens(s, x):
    """[seqs, kv heads, new x group, ...] to [tokens, heads, ...]."""
    c = s["case"]
    g = c["hq"] // c["hkv"]
    x = x.view(c["seqs"], c["hkv"], -1, g, x.shape[3]).permute(0, 2, 1, 3, 4)
    return x[_rows(s)[1]].reshape(-1, c["hq"], x.shape[4])


def _attend(s):
    x = _scores(s)
    top = x.amax(3, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = x.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    lse = _tokens(s, top + total.log())[:, :, 0]
    vv = _gather(s, s["v"], s.get("v_scale"))
    past = torch.arange(vv.shape[2], device=DEV)[None, :] >= s["kv_len"][:, None]
    y = p @ vv.masked_fill_(past[:, None, :, None], 0.0)
    return _tokens(s, torch.where(total > 0, y / total, 0.0)).to(torch.bfloat16), lse


def _weights(s):
    x = _scores(s)
    rows, _ = _rows(s)
    c = s["case"]
    n, g = c["seqs"], c["hq"] // c["hkv"]
    lse = s["lse"][rows].view(n, -1, c["hkv"], g).permute(0, 2, 1, 3).reshape(n, c["hkv"], -1, 1)
    w = x.sub_(torch.where(lse > -math.inf, lse, 0.0)).exp_().sum(2)     # [seqs, kv heads, keys]
    cu, j = s["cu"], torch.arange(w.shape[2], device=DEV)[None, None]
    length = s["kv_len"][:, None, None]
    old = j < length - (cu[1:] - cu[:-1])[:, None, None]
    w = w + torch.where(old, s["scores"] * s["decay"], 0.0)
    return torch.where(j < length, w, s["scores_out"])


def _rotate(s, x):
    """Rotary positions of [tokens, heads, dim], fp32."""
    c = s["case"]
    half = c["rot"] // 2
    pos = s["pos"].float()[:, None]
    hi, lo = s["freqs"][:, 0][None], s["freqs"][:, 1][None]
    # pos * hi in fp32 without a rounding: both split into 12-bit halves, whole turns dropped from each product
    ph = torch.floor(pos / 4096) * 4096
    big = hi * 4097
    hh = big - (big - hi)
    part = [a * b for a in (ph, pos - ph) for b in (hh, hi - hh)]
    part = [a - torch.round(a) for a in part]
    turn = part[0] + part[1] + part[2] + part[3] + pos * lo
    a = (turn - torch.round(turn)) * (2 * math.pi)
    cos, sin = (a.cos() * s["mag"])[:, None], (a.sin() * s["mag"])[:, None]
    x = x.float()
    r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    x1, x2 = (r[..., 0::2], r[..., 1::2]) if c["inter"] else (r[..., :half], r[..., half:])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack([y1, y2], -1).flatten(-2) if c["inter"] else torch.cat([y1, y2], -1)
    return torch.cat([y, rest], -1)


def _store(s, cache, x, scale):
    cu, length = s["cu"].long(), s["kv_len"].long()
    rows, live = _rows(s)
    at = ((length - (cu[1:] - cu[:-1]))[:, None] + torch.arange(s["max_q"], device=DEV)[None])[live]
    seq = torch.arange(cu.numel() - 1, device=DEV)[:, None].expand_as(live)[live]
    page = s["table"][seq, at // s["case"]["page"]].long()
    if scale is None:
        cache[page, :, at % s["case"]["page"]] = x.to(cache.dtype)
    else:
        codes = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache.view(torch.uint8)[page, :, at % s["case"]["page"]] = codes


def _append(s):
    s["q_out"].copy_(_rotate(s, s["q"]))
    _store(s, s["k"], _rotate(s, s["nk"]), s.get("k_scale"))
    _store(s, s["v"], s["nv"].float(), s.get("v_scale"))
    return s["q_out"], s["k"], s["v"]


def _evict(s):
    c = s["case"]
    x, length = s["scores"], s["kv_len"].long()[:, None, None]
    j = torch.arange(x.shape[2], device=DEV)[None, None]
    x = torch.where(j >= length - c["recent"], math.inf, x)
    x = torch.where(j < length, x, -math.inf)
    order = torch.sort(x, dim=2, descending=True, stable=True)[1][:, :, :c["budget"]]
    if order.shape[2] < c["budget"]:
        order = torch.nn.functional.pad(order, (0, c["budget"] - order.shape[2]))
    left = length.clamp(max=c["budget"])
    r = torch.arange(c["budget"], device=DEV)[None, None]
    kept = torch.where(r < left, order, 1 << 40).sort(dim=2)[0]
    live = r < left
    kept = torch.where(live, kept, -1)
    s["kept"].copy_(kept)
    b, h, r = live.expand_as(kept).nonzero(as_tuple=True)
    j = kept[b, h, r]
    page = c["page"]
    src, dst = s["table"][b, j // page].long(), s["to"][b, r // page].long()
    for cache in (s["k"], s["v"]):
        cache = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        cache[dst, h, r % page] = cache[src, h, j % page]
    s["scores_out"][b, h, r] = s["scores"][b, h, j]
    s["new_len"].copy_(left[:, 0, 0])
    return s["kept"], s["new_len"], s["scores_out"], s["k"], s["v"]


def run(s):
    c = s["case"]
    if own:
        import moe_speculative_verify_gb300 as m
        if c["op"] == "rope":
            m.moe_rope_append(s["h_rope"], s["h_cache"], s["h_seqs"], s["q"], s["nk"], s["nv"], s["pos"], s["q_out"])
            return s["q_out"], s["k"], s["v"]
        if c["op"] == "attn":
            m.moe_paged_attention(s["h_attn"], s["h_cache"], s["h_seqs"], s["q"], s["out"], s["ws"], lse=s["lse"],
                                  draft_mask=s["tree"])
            return s["out"], s["lse"]
        if c["op"] == "weights":
            m.moe_key_weights(s["h_attn"], s["h_cache"], s["h_seqs"], s["q"], s["lse"], s["scores"], s["scores_out"],
                              s["ws"], decay=s["decay"], draft_mask=s["tree"])
            return s["scores_out"]
        m.moe_cache_evict(s["h_cache"], s["h_seqs"], s["scores"], c["budget"], c["recent"], s["to"], s["kept"],
                          s["scores_out"], s["new_len"], s["ws"])
        return s["kept"], s["new_len"], s["scores_out"], s["k"], s["v"]
    with torch.no_grad():
        return {"rope": _append, "attn": _attend, "weights": _weights, "evict": _evict}[c["op"]](s)


# ------------------------------------------------------- 64-bit definition --
def exact(case, seed):
    if case["op"] == "evict":     # chosen and moved values only
        return None
    news, lens = _lens(case)
    if _pairs(case)[0] * case["hq"] * case["dim"] > 4e11:
        return None
    s = prepare(case, seed)
    hq, hkv, d, page = case["hq"], case["hkv"], case["dim"], case["page"]
    g = hq // hkv
    f64 = torch.float64
    table = s["table"].cpu().tolist()
    if case["op"] == "rope":
        fr = s["freqs"].double().sum(1)
        half = case["rot"] // 2
        ang = s["pos"].double()[:, None] * fr[None]
        ang = (ang - ang.floor()) * (2 * math.pi)
        z = torch.polar(torch.full_like(ang, s["mag"]), ang)[:, None]

        def turn(x):
            x = x.double().clone()
            a, b = (slice(0, case["rot"], 2), slice(1, case["rot"], 2)) if case["inter"] else (
                slice(0, half), slice(half, case["rot"]))
            y = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * z
            x[..., a], x[..., b] = y.real, y.imag
            return x

        k, v = s["k"].float().double(), s["v"].float().double()
        nk, nv = turn(s["nk"]), s["nv"].double()
        if case["kv"] == "e4m3":
            nk = (nk / s["k_scale"].double()[:, None]).clamp(-448, 448)
            nv = (nv / s["v_scale"].double()[:, None]).clamp(-448, 448)
        t = 0
        for b, n in enumerate(news):
            at = torch.arange(lens[b] - n, lens[b], device=DEV)
            pages = s["table"][b].long()[at // page]
            k[pages, :, at % page] = nk[t:t + n]
            v[pages, :, at % page] = nv[t:t + n]
            t += n
        return turn(s["q"]), k, v
    out = torch.zeros(s["q"].shape, dtype=f64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=f64, device=DEV)
    if case["op"] == "weights":
        new = s["scores_out"].double().clone()
    t = 0
    for b, n in enumerate(news):
        length = lens[b]
        idx = torch.tensor(table[b][:-(-length // page)], device=DEV)
        seen = torch.zeros(n, length, dtype=torch.bool, device=DEV)
        place = torch.arange(length, device=DEV)
        for i in range(n) if s["tree"] is not None else ():
            m = int(s["tree"][t + i])
            seen[i, :length - n] = True
            for c in range(n):
                seen[i, length - n + c] = bool((m >> c) & 1)
        if s["tree"] is None:
            seen = place[None] <= (length - n + torch.arange(n, device=DEV))[:, None]
        if case["window"]:
            seen &= place[None] > (length - n - case["window"] + torch.arange(n, device=DEV))[:, None]
        for h in range(hkv):
            kh = s["k"][idx, h].reshape(-1, d)[:length].float().double()
            if case["kv"] == "e4m3":
                kh = kh * s["k_scale"][h].double()
            q = s["q"][t:t + n, h * g:(h + 1) * g].double()
            x = torch.einsum("igd,jd->gij", q, kh) * s["scale"]
            x.masked_fill_(~seen[None], -math.inf)
            if case["op"] == "attn":
                z = torch.logsumexp(x, 2)
                p = torch.exp(x - z[:, :, None]).nan_to_num_(0.0)
                vh = s["v"][idx, h].reshape(-1, d)[:length].float().double()
                if case["kv"] == "e4m3":
                    vh = vh * s["v_scale"][h].double()
                out[t:t + n, h * g:(h + 1) * g] = (p @ vh).transpose(0, 1)
                lse[t:t + n, h * g:(h + 1) * g] = z.t()
            else:
                z = s["lse"][t:t + n, h * g:(h + 1) * g].double().t()
                w = torch.exp(x - z[:, :, None]).nan_to_num_(0.0).sum((0, 1))
                w[:length - n] += s["scores"][b, h, :length - n].double() * s["decay"]
                new[b, h, :length] = w
            del x
        t += n
    return (out, lse) if case["op"] == "attn" else new
