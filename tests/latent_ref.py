"""Plain 64-bit implementations of the operators over a latent cache, and random
problems for their tests.  Tolerances of the attention calls, from the
arithmetic: a probability rounded to bf16 (2^-8) moves the output by at most
2^-8 sum p|v| / sum p, a score's fp32 error e (at most D 2^-23 sum |q||k| scale
over D elements) by 2 e times that, the exponential's 2^-21 alike, the output's own
rounding by 2^-8 |out|; the log-sum-exp moves by e and its fp32 roundings."""
import torch

import moe_speculative_verify_gb300 as m

ROT = 64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Problem:
    """A random paged batch.  lens: cached rows of each sequence, new tokens
    included; news: new tokens of each; pads: token rows before and after them.
    Slots that no sequence owns hold NaN, block-table entries past a sequence's
    end wild indices.  store: 'rows' (both parts of a row side by side) or 'split'."""

    def __init__(self, lens, news, heads, latent, page, dtype="bf16", store="rows", pads=(0, 0), seed=0, q_scale=1.0,
                 scale_log2=-4, fill=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.news, self.heads, self.c, self.page, self.dtype = list(lens), list(news), heads, latent, page, dtype
        n = len(lens)
        need = [-(-x // page) for x in lens]
        total = sum(need) + 4
        perm = torch.randperm(total, generator=g)
        self.exp = scale_log2 if dtype == "e4m3" else 0
        lat = torch.randn(total, page, latent, generator=g) if fill is None else fill(total, page, latent, g)
        rot = torch.randn(total, page, ROT, generator=g).bfloat16()
        if dtype == "e4m3":
            lat = (lat * 2.0 ** -self.exp).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            lat = lat.bfloat16()
        self.table = torch.full((n, max(max(need), 1) + 2), 1 << 30, dtype=torch.int32)
        owned, at = torch.zeros(total, page, dtype=torch.bool), 0
        for b in range(n):
            self.table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            for j in range(lens[b]):
                owned[self.table[b, j // page], j % page] = True
        if dtype == "e4m3":
            lat.view(torch.uint8)[~owned] = 0x7F
        else:
            lat[~owned] = float("nan")
        rot[~owned] = float("nan")
        if store == "rows" and dtype == "bf16":
            rows = torch.cat([lat, rot], -1).cuda()
            self.latent, self.rope = rows[..., :latent], rows[..., latent:]
        else:                                          # token-major, pages of both parts strided apart
            self.latent = lat.transpose(0, 1).contiguous().cuda().transpose(0, 1) if store == "split" else lat.cuda()
            self.rope = rot.cuda()
        self.cache = m.LatentCache.from_tensors(self.latent, self.rope, self.exp)
        self.t = sum(news) + sum(pads)
        cu = [pads[0]]
        for x in news:
            cu.append(cu[-1] + x)
        self.cu = cu
        self.d_cu, self.kv_len, self.d_table = i32(cu), i32(self.lens), self.table.cuda()
        self.seqs = m.Seqs.from_tensors(self.d_cu, self.kv_len, self.d_table, max(self.news + [1]))
        self.scale = (128 + ROT) ** -0.5
        self.q = (torch.randn(self.t, heads, latent + ROT, generator=g) * q_scale).bfloat16().cuda()

    def rows(self, b):
        """(latents, rotary keys) of sequence b, float64."""
        j = torch.arange(self.lens[b], device="cuda")
        pg = self.d_table[b][j // self.page].long()
        lat = self.latent.view(torch.uint8)[pg, j % self.page].view(torch.float8_e4m3fn) if self.dtype == "e4m3" else \
            self.latent[pg, j % self.page]
        return lat.float().double() * 2.0 ** self.exp, self.rope[pg, j % self.page].double()


def sees(length, n, causal, window, draft):
    """[n, length]: which cache places each of a sequence's n queries sees; draft: its rows' masks (ints) or None."""
    j = torch.arange(length, device="cuda")[None]
    i = torch.arange(n, device="cuda")[:, None]
    first = length - n
    ok = torch.ones(n, length, dtype=torch.bool, device="cuda")
    if draft is not None:
        c = (j - first).expand(n, length)
        bit = torch.zeros(n, length, dtype=torch.bool)
        for a in range(n):
            for k in range(max(first, 0), min(length, first + 64)):
                bit[a, k] = bool((draft[a] >> (k - first)) & 1)
        ok = (c < 0) | bit.cuda()
    elif causal:
        ok = j <= first + i
    if window > 0:
        ok = ok & (j > first + i - window)
    return ok


def attend(q, keys, vals, seen, scale):
    """(out, lse, mag, err) of one sequence and head set in float64: q [n, H, D], keys [L, D] or [L, H, D], vals alike."""
    per = keys.dim() == 3
    s = torch.einsum("ihd,jhd->hij" if per else "ihd,jd->hij", q, keys) * scale
    e = torch.einsum("ihd,jhd->hij" if per else "ihd,jd->hij", q.abs(), keys.abs()) * (abs(scale) * q.shape[2] * 2.0 ** -23)
    s = s.masked_fill(~seen[None], float("-inf"))
    e = e.masked_fill(~seen[None], 0.0).amax(2) if keys.shape[0] else torch.zeros(q.shape[1], q.shape[0], device="cuda").double()
    z = torch.logsumexp(s, 2) if keys.shape[0] else torch.full((q.shape[1], q.shape[0]), float("-inf"), device="cuda").double()
    p = torch.where(seen[None], torch.exp(s - z.masked_fill(z.isneginf(), 0)[..., None]), torch.zeros((), device="cuda").double())
    out = torch.einsum("hij,jhd->ihd" if per else "hij,jd->ihd", p, vals)
    mag = torch.einsum("hij,jhd->ihd" if per else "hij,jd->ihd", p, vals.abs())
    return out, z.t(), mag, e.t()


def check(got, lse, want, z, mag, err):
    """Every element within the module's tolerances; rows that see nothing +0 and -inf."""
    tol = mag * (2.0 ** -8 + 2 * err[..., None] + 2.0 ** -20) + 2.0 ** -8 * want.abs() + 1e-30
    d = (got.double() - want).abs()
    assert bool((d <= tol).all()), (float((d / tol).nan_to_num(1e9).max()), int((~(d <= tol)).sum()))
    empty = z.isneginf()
    assert bool(torch.all(got[empty].contiguous().view(torch.int16) == 0))
    assert torch.equal(lse.isneginf(), empty)
    dz = (lse.double() - z).abs()[~empty]
    assert bool((dz <= (err + 2.0 ** -20 * (1 + z.abs().nan_to_num(0, 0, 0)))[~empty]).all())


def latent_attention(p, causal=True, window=0, draft=None):
    """(out, lse, mag, err) over all token rows."""
    d = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")
    out, mag, err = d(p.t, p.heads, p.c), d(p.t, p.heads, p.c), d(p.t, p.heads)
    z = torch.full((p.t, p.heads), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(p.news):
        if not n or not p.lens[b]:
            continue
        r = slice(p.cu[b], p.cu[b] + n)
        lat, rot = p.rows(b)
        seen = sees(p.lens[b], n, causal, window, None if draft is None else [int(x) for x in draft[r]])
        out[r], z[r], mag[r], err[r] = attend(p.q[r].double(), torch.cat([lat, rot], 1), lat, seen, p.scale)
    return out, z, mag, err


def turn(x, pos, freqs, magnitude, interleaved):
    """float64 rotary positions of [T, heads, 64]; the angles in exact rationals."""
    import math
    from fractions import Fraction
    x = x.double().cpu().clone()
    half = ROT // 2
    for t in range(x.shape[0]):
        for i in range(half):
            a = Fraction(int(pos[t])) * (Fraction(float(freqs[i, 0])) + Fraction(float(freqs[i, 1])))
            a = 2.0 * math.pi * float(a - math.floor(a))
            c, s = math.cos(a) * magnitude, math.sin(a) * magnitude
            i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            x1, x2 = x[t, :, i1].clone(), x[t, :, i2].clone()
            x[t, :, i1], x[t, :, i2] = x1 * c - x2 * s, x2 * c + x1 * s
    return x
