"""Workloads of attention through a latent cache.

Such a layer caches one row a token for all of its heads: a latent vector, of
which every head's keys and values are linear maps, and a rotary key that the
heads share.  Pages of `page` tokens, each [page, latent] (bf16, or e4m3 codes
times a power of two) and [page, 64] (bf16).  Four operators:

  append   the step's new tokens: latents normalised (RMS), rotary positions on
           the shared keys and on the queries' rotary parts, rows stored
  attend   absorbed form: queries in latent space (one row of latent + 64 a
           head) over the cached rows, whose latent parts are keys and values
  gather   cached rows read back as bf16 rows, one sequence after another
  expand   expanded form: attention over keys (a part of each head's own beside
           the shared rotary one) and values made from such rows

`run` computes them in elementary fp32 torch operations, or (own) through the
framework's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
ROT = 64                                  # rotary part of a row
# rotary scaling for long contexts used by the cases that say so: the by-parts
# ramp between 1 and 32 turns over an original length of 4096, factor 8
RAMP = {"factor": 8.0, "orig": 4096, "fast": 32.0, "slow": 1.0}
EPS = 1e-6


def _c(name, op, seqs, ctx_lo, ctx_hi, new, ragged, heads, latent, page, kv, **more):
    return dict(name=name, op=op, seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new=new, ragged=ragged, heads=heads,
                latent=latent, page=page, kv=kv, **{**_MORE, **more})


# dim: a head's own part of keys, and its values (expand); norm: latents arrive before their
# normalisation; inter, ramp: rotary pairs and scaling; window: sliding window (0: none); tree: draft masks
_MORE = dict(dim=128, norm=True, inter=True, ramp=False, window=0, tree=False)


def listed():
    return [
        # one 8-row verify block of a single user: the smallest call, all latency
        _c("append_verify8", "append", 1, 4097, 4097, 8, False, 64, 512, 64, "bf16"),
        # a ragged mixed batch into an e4m3 cache: odd counts, small pages, halves rotated, long-context scaling
        _c("append_mixed_e4m3", "append", 37, 100, 20011, 19, True, 24, 256, 16, "e4m3", inter=False, ramp=True),
        # a prefill chunk of the most rows a layer call takes
        _c("append_chunk4096", "append", 1, 4096, 4096, 4096, False, 64, 512, 64, "bf16"),
        # single-user speculative verify: one committed token and 7 drafts
        _c("attend_verify8", "attend", 1, 6011, 6011, 8, False, 64, 512, 64, "bf16"),
        # a share of the heads of one token: the fewest rows
        _c("attend_decode1", "attend", 1, 1021, 1021, 1, False, 16, 512, 64, "bf16"),
        # continuous batching: single tokens at lengths spread over 1:128
        _c("attend_decode48", "attend", 48, 251, 32011, 1, False, 64, 512, 64, "bf16"),
        # batched verify blocks over an e4m3 cache, ragged block lengths, draft trees
        _c("attend_verify16_e4m3", "attend", 16, 4099, 16411, 8, True, 64, 512, 64, "e4m3", tree=True),
        # a prefill chunk over a long cached prefix: the largest call
        _c("attend_chunk512", "attend", 1, 16384, 16384, 512, False, 64, 512, 64, "bf16"),
        # one user's rows before their expansion
        _c("gather_one", "gather", 1, 8191, 8191, 1, False, 64, 512, 64, "bf16"),
        # a batch of long e4m3 caches
        _c("gather_batch16_e4m3", "gather", 16, 5003, 32003, 1, False, 64, 512, 64, "e4m3"),
        # a prompt of odd length without a prefix
        _c("expand_prompt1000", "expand", 1, 1, 1, 1000, False, 16, 512, 64, "bf16"),
        # ragged prompts and chunks behind a prefix
        _c("expand_batch4", "expand", 4, 300, 9001, 1024, True, 64, 512, 64, "bf16"),
    ]


HEADS = [1, 8, 12, 16, 24, 32, 40, 64, 128]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attend", "attend", "attend", "gather", "expand"])
        heads, page = rng.choice(HEADS), rng.choice([16, 32, 64, 128])
        latent, kv = rng.choice([256, 512, 512]), rng.choice(["bf16", "e4m3"])
        hi = _log(rng, 1, 32768)
        lo = _log(rng, 1, hi)
        form = rng.choice(["single", "verify", "chunk"]) if op != "expand" else "chunk"
        new = 1 if form == "single" else rng.randint(2, 8) if form == "verify" else _log(rng, 9, 2048)
        seqs = _log(rng, 1, 64) if form != "chunk" else _log(rng, 1, 6)
        c = _c(None, op, seqs, lo, hi, new, rng.random() < 0.5, heads, latent, page, kv)
        del c["name"]
        if op == "append":
            c["norm"] = rng.random() < 0.7
            c["inter"] = rng.random() < 0.5
            c["ramp"] = rng.random() < 0.5
        elif op == "gather":
            c["new"], c["ragged"] = 1, False
        else:
            c["window"] = _log(rng, 1, hi) if rng.random() < 0.25 else 0
            c["tree"] = op == "attend" and form == "verify" and rng.random() < 0.5
            c["dim"] = rng.choice([64, 128, 128])
            if op == "expand":
                c["kv"] = "bf16"
        # no drawn case costs more than the largest listed one, nor holds more than a few times its memory
        if seqs * (hi + new) * latent > 8e8 or seqs * hi * new * heads > 1.2e9:
            continue
        if op == "expand" and seqs * (hi + new) * heads * c["dim"] > 4e8:
            continue
        if work(c)["flops"] > 1.1e12 or work(c)["bytes"] > 1.2e9 or work(c)["bytes"] < 20000:
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
    t, h, c, d = sum(news), case["heads"], case["latent"], case["dim"]
    row = c * (2 if case["kv"] == "bf16" else 1) + 2 * ROT
    if case["op"] == "append":    # rows read and stored, the queries' rotary parts read and written
        return {"bytes": t * (2 * (c + ROT) + row + 4 * h * ROT + 4), "flops": t * (5 * c + 3 * ROT * (h + 1))}
    if case["op"] == "gather":
        return {"bytes": sum(lens) * (row + 2 * (c + ROT)), "flops": 0}
    pairs, keys = _pairs(case)
    if case["op"] == "attend":
        return {"bytes": keys * row + t * h * (4 * c + 2 * ROT + 4), "flops": 2 * pairs * h * (2 * c + ROT)}
    return {"bytes": keys * (4 * h * d + 2 * ROT) + t * h * (4 * d + 2 * ROT + 4), "flops": 2 * pairs * h * (2 * d + ROT)}


# ------------------------------------------------------------------ inputs --
def _freqs(case):
    """Turns per position of each rotated pair as two fp32 (their sum is it to 48 bits), and the magnitude."""
    half = ROT // 2
    i = torch.arange(half, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / ROT)
    mag = 1.0
    if case["ramp"]:
        at = lambda turns: ROT * math.log(RAMP["orig"] / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
        lo, hi = max(math.floor(at(RAMP["fast"])), 0), min(math.ceil(at(RAMP["slow"])), ROT - 1)
        r = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - r) + f / RAMP["factor"] * r
        mag = 0.1 * math.log(RAMP["factor"]) + 1.0
    f = f / (2 * math.pi)
    hi32 = f.float()
    return torch.stack([hi32, (f - hi32.double()).float()], 1), mag


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    news, lens = _lens(case)
    h, c, d, page, n, t = case["heads"], case["latent"], case["dim"], case["page"], case["seqs"], sum(news)
    s = {"case": case, "lens": lens, "max_q": max(news)}
    cu, ck = [0], [0]
    for x, y in zip(news, lens):
        cu.append(cu[-1] + x)
        ck.append(ck[-1] + y)
    s["cu"], s["kv_len"], s["cu_k"] = i32(cu), i32(lens), i32(ck)
    # a head's scores as the layer scales them: by its own part and the rotary one, with scores spread as in earnest
    s["scale"] = (d + ROT) ** -0.5
    if case["op"] == "expand":
        kv = rnd(ck[-1], h, 2 * d)                     # the expansion's output: a head's key part and values side by side
        s["k"], s["v"] = kv[..., :d], kv[..., d:]
        s["k_rope"] = rnd(ck[-1], c + ROT)[:, c:]      # the rotary keys as they lie in the rows
        s["q"] = (rnd(t, h, d + ROT) * 1.5).contiguous()
        s["out"] = torch.zeros(t, h, d, dtype=torch.bfloat16, device=DEV)
        s["table"] = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    else:
        need = [-(-x // page) for x in lens]
        total = sum(need) + 3
        perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32).cpu()
        table, at = torch.full((n, max(need)), -1, dtype=torch.int32), 0
        for b, x in enumerate(need):
            table[b, :x] = perm[at:at + x]
            at += x
        s["table"] = table.to(DEV)
        s["exp"] = 0
        if case["kv"] == "bf16":                       # a row's two parts side by side in one allocation
            rows = rnd(total, page, c + ROT)
            s["latent"], s["rope"] = rows[..., :c], rows[..., c:]
        else:
            s["exp"] = -4                              # values of unit size: codes up to a few dozen
            s["latent"] = (rnd(total, page, c) * 16).clamp(-448, 448).to(torch.float8_e4m3fn)
            s["rope"] = rnd(total, page, ROT)
    if case["op"] == "append":
        s["kv"] = rnd(t, c + ROT + 64)[:, :c + ROT]    # a slice of the projection's output
        s["gamma"] = (1 + 0.2 * torch.randn(c, generator=g, device=DEV)) if case["norm"] else None
        s["q_rope"] = rnd(t, h, 128 + ROT)[..., 128:]  # behind the heads' own parts
        s["q"] = torch.zeros(t, h, c + ROT, dtype=torch.bfloat16, device=DEV)
        s["q_out"] = s["q"][..., c:]                   # behind the queries' latent parts
        s["pos"] = i32([lens[b] - news[b] + i for b in range(n) for i in range(news[b])])
        s["freqs"], s["mag"] = _freqs(case)
        s["freqs"] = s["freqs"].to(DEV)
    if case["op"] == "gather":
        s["out"] = torch.zeros(ck[-1], c + ROT, dtype=torch.bfloat16, device=DEV)
    if case["op"] == "attend":
        s["q"] = (rnd(t, h, c + ROT)).contiguous()
        s["out"] = torch.zeros(t, h, c, dtype=torch.bfloat16, device=DEV)
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
    if case["op"] in ("attend", "expand"):
        s["lse"] = torch.zeros(t, h, dtype=torch.float32, device=DEV)
    if own:                       # the handles that a program builds once for its cache and its batch
        import moe_speculative_verify_gb300 as m
        m.load()
        s["h_seqs"] = m.Seqs.from_tensors(s["cu"], s["kv_len"], s["table"], s["max_q"])
        if case["op"] != "expand":
            s["h_cache"] = m.LatentCache.from_tensors(s["latent"], s["rope"], s["exp"])
        if case["op"] == "append":
            s["h_rope"] = m.Rope.from_freqs(s["freqs"], case["inter"], s["mag"])
        elif case["op"] == "gather":
            s["ws"] = torch.zeros(256, dtype=torch.uint8, device=DEV)
        else:
            s["h_attn"] = m.Attn(h, s["scale"], True, case["window"])
            need = (m.moe_latent_workspace_bytes(s["h_attn"], s["h_cache"]) if case["op"] == "attend"
                    else m.moe_expanded_workspace_bytes(s["h_attn"], d))
            s["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    return s


# -------------------------------------------------------------- plain forms --
def _rows_of(s):
    """The sequences' cached rows, fp32 [seqs, places, latent + 64]; places past a sequence's end hold some page's rows."""
    at = s["table"].clamp(min=0).long()
    x = s["latent"]
    x = (x.view(torch.uint8)[at].view(torch.float8_e4m3fn) if x.dtype == torch.float8_e4m3fn else x[at]).float()
    x = torch.cat([x * 2.0 ** s["exp"], s["rope"][at].float()], -1)
    return x.flatten(1, 2)


def _tokens(s):
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
    if s.get("tree") is None:
        seen = j <= first + i
    else:
        bits = s["tree"][_tokens(s)[0]][:, :, None]
        at = (j - first).clamp(0, 63)
        seen = (j < first) | ((j - first < 64) & ((bits >> at) & 1 == 1))
    seen = seen & (j < length[:, None, None]) & _tokens(s)[1][:, :, None]
    if s["case"]["window"]:
        seen = seen & (j > first + i - s["case"]["window"])
    return seen


def _soften(x, seen):
    """Powers, their sums and the log-sum-exp of scores [..., keys]."""
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return p, total, top + total.log()


def _attend(s):
    rows = _rows_of(s)                                           # [seqs, places, latent + 64]
    past = torch.arange(rows.shape[1], device=DEV)[None, :] >= s["kv_len"][:, None]
    rows = rows.masked_fill_(past[:, :, None], 0.0)
    at, live = _tokens(s)
    n, h, c = s["case"]["seqs"], s["case"]["heads"], s["case"]["latent"]
    q = s["q"][at].float().flatten(1, 2)                         # [seqs, new x heads, latent + 64]
    x = (q @ rows.transpose(1, 2)).mul_(s["scale"])
    p, total, z = _soften(x, _seen(s, rows.shape[1]).repeat_interleave(h, 1))
    y = p @ rows[..., :c]
    y = torch.where(total > 0, y / total, 0.0).view(n, -1, h, c)
    return y[live].to(torch.bfloat16), z.view(n, -1, h)[live]


def _expand(s):
    cu, longest = s["cu_k"].long(), max(s["lens"])
    j = torch.arange(longest, device=DEV)
    at = (cu[:-1, None] + j[None]).clamp(max=int(s["k"].shape[0]) - 1)
    past = (j[None] >= s["kv_len"][:, None])[:, None, :, None]
    tok, live = _tokens(s)
    d = s["case"]["dim"]
    q = s["q"][tok].float().transpose(1, 2)                      # [seqs, heads, new, dim + 64]
    k, v = s["k"][at].float().transpose(1, 2), s["v"][at].float().transpose(1, 2)
    x = q[..., :d] @ k.transpose(2, 3)
    x += q[..., d:] @ s["k_rope"][at].float()[:, None].transpose(2, 3)
    p, total, z = _soften(x.mul_(s["scale"]), _seen(s, longest)[:, None])
    y = p @ v.masked_fill_(past, 0.0)
    y = torch.where(total > 0, y / total, 0.0).transpose(1, 2)[live]
    return y.to(torch.bfloat16), z[..., 0].transpose(1, 2)[live]


def _rotate(s, x):
    """Rotary positions of [tokens, heads, 64], fp32."""
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
    half = ROT // 2
    x1, x2 = (x[..., 0::2], x[..., 1::2]) if s["case"]["inter"] else (x[..., :half], x[..., half:])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return torch.stack([y1, y2], -1).flatten(-2) if s["case"]["inter"] else torch.cat([y1, y2], -1)


def _append(s):
    c, page = s["case"]["latent"], s["case"]["page"]
    s["q_out"].copy_(_rotate(s, s["q_rope"]))
    x = s["kv"][:, :c].float()
    if s["gamma"] is not None:
        x = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * s["gamma"]
    length, cu = s["kv_len"].long(), s["cu"].long()
    at, live = _tokens(s)
    at = ((length - (cu[1:] - cu[:-1]))[:, None] + torch.arange(s["max_q"], device=DEV)[None])[live]
    seq = torch.arange(cu.numel() - 1, device=DEV)[:, None].expand_as(live)[live]
    where = s["table"][seq, at // page].long(), at % page
    if s["latent"].dtype == torch.float8_e4m3fn:
        x = (x * 2.0 ** -s["exp"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["latent"].view(torch.uint8)[where] = x.view(torch.uint8)
    else:
        s["latent"][where] = x.to(torch.bfloat16)
    s["rope"][where] = _rotate(s, s["kv"][:, None, c:])[:, 0].to(torch.bfloat16)
    return s["q_out"], s["latent"], s["rope"]


def _gather(s):
    rows = _rows_of(s)
    live = torch.arange(rows.shape[1], device=DEV)[None] < s["kv_len"][:, None]
    s["out"].copy_(rows[live])
    return s["out"]


def run(s):
    op = s["case"]["op"]
    if own:
        import moe_speculative_verify_gb300 as m
        if op == "append":
            m.moe_latent_append(s["h_rope"], s["h_cache"], s["h_seqs"], s["kv"], s["q_rope"], s["pos"], s["q_out"],
                                gamma=s["gamma"], eps=EPS)
            return s["q_out"], s["latent"], s["rope"]
        if op == "attend":
            m.moe_latent_attention(s["h_attn"], s["h_cache"], s["h_seqs"], s["q"], s["out"], s["ws"], lse=s["lse"],
                                   draft_mask=s["tree"])
            return s["out"], s["lse"]
        if op == "gather":
            m.moe_latent_gather(s["h_cache"], s["h_seqs"], s["cu_k"], s["out"], s["ws"])
            return s["out"]
        m.moe_expanded_attention(s["h_attn"], s["h_seqs"], s["cu_k"], s["q"], s["k"], s["k_rope"], s["v"], s["out"],
                                 s["ws"], lse=s["lse"])
        return s["out"], s["lse"]
    with torch.no_grad():
        return {"append": _append, "attend": _attend, "gather": _gather, "expand": _expand}[op](s)


# ------------------------------------------------------- 64-bit definition --
def exact(case, seed):
    news, lens = _lens(case)
    h, c, d, page = case["heads"], case["latent"], case["dim"], case["page"]
    if case["op"] in ("attend", "expand") and work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "append":
        fr = s["freqs"].double().sum(1)
        ang = s["pos"].double()[:, None] * fr[None]
        z = torch.polar(torch.full_like(ang, s["mag"]), (ang - ang.floor()) * (2 * math.pi))[:, None]

        def turn(x):
            x = x.double().clone()
            a, b = (slice(0, ROT, 2), slice(1, ROT, 2)) if case["inter"] else (slice(0, ROT // 2), slice(ROT // 2, ROT))
            y = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * z
            x[..., a], x[..., b] = y.real, y.imag
            return x

        new = s["kv"][:, :c].double()
        if case["norm"]:
            new = new / torch.sqrt((new * new).sum(1, keepdim=True) / c + EPS) * s["gamma"].double()
        if case["kv"] == "e4m3":
            new = (new / 2.0 ** s["exp"]).clamp(-448, 448)
        key = turn(s["kv"][:, None, c:])[:, 0]
        latent, rope = s["latent"].float().double(), s["rope"].double()
        t = 0
        for b, n in enumerate(news):
            at = torch.arange(lens[b] - n, lens[b], device=DEV)
            pages = s["table"][b].long()[at // page]
            latent[pages, at % page] = new[t:t + n]
            rope[pages, at % page] = key[t:t + n]
            t += n
        return turn(s["q_rope"]), latent, rope
    if case["op"] == "gather":    # moved values only
        return None
    t, at = sum(news), 0
    width = c if case["op"] == "attend" else d
    out = torch.zeros(t, h, width, dtype=f64, device=DEV)
    lse = torch.full((t, h), -math.inf, dtype=f64, device=DEV)
    for b, n in enumerate(news):
        length = lens[b]
        place = torch.arange(length, device=DEV)
        seen = place[None] <= (length - n + torch.arange(n, device=DEV))[:, None]
        for i in range(n) if s.get("tree") is not None else ():
            m = int(s["tree"][at + i])
            seen[i, :length - n] = True
            for x in range(n):
                seen[i, length - n + x] = bool((m >> x) & 1)
        if case["window"]:
            seen &= place[None] > (length - n - case["window"] + torch.arange(n, device=DEV))[:, None]
        if case["op"] == "attend":
            pages = s["table"][b, :-(-length // page)].long()
            lat = s["latent"][pages].float().double().reshape(-1, c)[:length] * 2.0 ** s["exp"]
            rot = s["rope"][pages].double().reshape(-1, ROT)[:length]
        else:
            r = slice(int(s["cu_k"][b]), int(s["cu_k"][b]) + length)
            rot = s["k_rope"][r].double()
        for a in range(h):
            q = s["q"][at:at + n, a].double()
            own_k, val = (lat, lat) if case["op"] == "attend" else (s["k"][r, a].double(), s["v"][r, a].double())
            x = torch.einsum("id,jd->ij", q[:, :own_k.shape[1]], own_k)
            x += torch.einsum("id,jd->ij", q[:, own_k.shape[1]:], rot)
            x = (x * s["scale"]).masked_fill_(~seen, -math.inf)
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None]).nan_to_num_(0.0)
            out[at:at + n, a] = p @ val
            lse[at:at + n, a] = z
        at += n
    return out, lse
