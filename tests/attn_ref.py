"""Plain 64-bit implementations of the attention-side operators, and random
problems for their tests (numpy and torch on the CPU, one loop per row)."""
import math

import numpy as np
import torch

import moe_speculative_verify_gb300 as m


class Problem:
    """A random paged batch on the CPU.  lens: cached keys of each sequence,
    new ones included; news: new tokens of each; pad rows before and after.
    Cache slots that no sequence owns, and block-table entries past a
    sequence's end, hold NaN and wild indices."""

    def __init__(self, lens, news, hq, hkv, dim, page, dtype="bf16", layout="hnd", pads=(0, 0), seed=0,
                 q_scale=1.5, shared_pages=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.news = list(lens), list(news)
        self.hq, self.hkv, self.dim, self.page, self.dtype = hq, hkv, dim, page, dtype
        n = len(lens)
        need = [-(-x // page) for x in lens]
        total = sum(need) + 5
        perm = torch.randperm(total, generator=g)
        shape = (total, hkv, page, dim) if layout == "hnd" else (total, page, hkv, dim)
        k = torch.randn(shape, generator=g)
        v = torch.randn(shape, generator=g)
        self.k_scale = self.v_scale = None
        if dtype == "e4m3":
            self.k_scale = 0.01 + 0.02 * torch.rand(hkv, generator=g)
            self.v_scale = 0.01 + 0.02 * torch.rand(hkv, generator=g)
            k, v = (k * 50).clamp(-448, 448).to(torch.float8_e4m3fn), (v * 50).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            k, v = k.bfloat16(), v.bfloat16()
        if layout == "nhd":
            k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
        width = max(max(need), 1) + 2
        self.table = torch.full((n, width), 1 << 30, dtype=torch.int32)
        at = 0
        owned = torch.zeros(total, page, dtype=torch.bool)
        for b in range(n):
            if shared_pages and b and need[b] and need[0]:
                self.table[b, :need[b]] = perm[at:at + need[b]]
                self.table[b, 0] = self.table[0, 0]
            else:
                self.table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            for j in range(lens[b]):
                owned[self.table[b, j // page], j % page] = True
        nan_code = torch.tensor(0x7F, dtype=torch.uint8)
        for c in (k, v):
            for pg in range(total):
                for t in range(page):
                    if not owned[pg, t]:
                        if dtype == "e4m3":
                            c.view(torch.uint8)[pg, :, t] = nan_code
                        else:
                            c[pg, :, t] = float("nan")
        self.k, self.v = k, v
        self.t = sum(news) + sum(pads)
        cu = [pads[0]]
        for x in news:
            cu.append(cu[-1] + x)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.kv_len = torch.tensor(self.lens, dtype=torch.int32)
        # q, k, v heads side by side, as one projection writes them
        self.qkv = torch.randn(self.t, hq + 2 * hkv, dim, generator=g)
        self.qkv[:, :hq] *= q_scale
        self.qkv = self.qkv.bfloat16()
        self.scale = dim ** -0.5

    def cuda(self):
        for name in ("k", "v", "k_scale", "v_scale", "table", "cu", "kv_len", "qkv"):
            x = getattr(self, name)
            if x is not None:
                setattr(self, "d_" + name, x.cuda())
        self.d_k, self.d_v = _same_strides(self.d_k, self.k), _same_strides(self.d_v, self.v)
        self.cache = m.KVCache.from_tensors(self.d_k, self.d_v, getattr(self, "d_k_scale", None),
                                            getattr(self, "d_v_scale", None))
        self.seqs = m.Seqs.from_tensors(self.d_cu, self.d_kv_len, self.d_table, max(self.news + [1]))
        return self

    def q(self):
        return self.qkv[:, :self.hq]

    def d_q(self):
        return self.d_qkv[:, :self.hq]

    def rows(self, x, scale, b, h, upto=None):
        """Cached rows of a sequence and kv head, float64."""
        n = self.lens[b] if upto is None else upto
        out = np.zeros((n, self.dim))
        for j in range(n):
            out[j] = x[int(self.table[b, j // self.page]), h, j % self.page].float().numpy()
        return out * (1.0 if scale is None else float(scale[h]))


def _same_strides(d, x):
    assert d.stride() == x.stride()
    return d


def sees(p, b, i, causal, window, draft):
    """Cache places that query i of sequence b sees."""
    length, first = p.lens[b], p.lens[b] - p.news[b]
    out = np.zeros(length, bool)
    for j in range(length):
        ok = True
        if draft is not None:
            c = j - first
            ok = c < 0 or (c < 64 and bool((int(draft[int(p.cu[b]) + i]) >> c) & 1))
        elif causal:
            ok = j <= first + i
        if window > 0:
            ok = ok and j > first + i - window
        out[j] = ok
    return out


def attention(p, causal=True, window=0, draft=None):
    """(out, lse, mag, err): the definition's results [T, Hq(, D)], sum p|v| / sum p, and the bound
    D 2^-23 sum |q||k| scale on a score's fp32 error, per row the largest."""
    g = p.hq // p.hkv
    out = np.zeros((p.t, p.hq, p.dim))
    mag = np.zeros((p.t, p.hq, p.dim))
    lse = np.full((p.t, p.hq), -np.inf)
    err = np.zeros((p.t, p.hq))
    q = p.q().float().numpy().astype(np.float64)
    for b in range(len(p.lens)):
        vis = [sees(p, b, i, causal, window, draft) for i in range(p.news[b])]
        for h in range(p.hkv):
            kk, vv = p.rows(p.k, p.k_scale, b, h), p.rows(p.v, p.v_scale, b, h)
            for i in range(p.news[b]):
                if not vis[i].any():
                    continue
                t = int(p.cu[b]) + i
                for hd in range(h * g, (h + 1) * g):
                    s = (kk[vis[i]] @ q[t, hd]) * p.scale
                    top = s.max()
                    e = np.exp(s - top)
                    out[t, hd] = e @ vv[vis[i]] / e.sum()
                    mag[t, hd] = e @ np.abs(vv[vis[i]]) / e.sum()
                    lse[t, hd] = top + math.log(e.sum())
                    err[t, hd] = p.dim * 2.0 ** -23 * (np.abs(kk[vis[i]]) @ np.abs(q[t, hd])).max() * p.scale
    return out, lse, mag, err


def key_weights(p, lse, scores, decay, causal=True, window=0, draft=None):
    """(new scores, bound): [B, Hkv, places]; places past a sequence's end as in scores."""
    g = p.hq // p.hkv
    out = scores.numpy().astype(np.float64).copy()
    tol = np.zeros_like(out)
    q = p.q().float().numpy().astype(np.float64)
    for b in range(len(p.lens)):
        length, first = p.lens[b], p.lens[b] - p.news[b]
        for h in range(p.hkv):
            kk = p.rows(p.k, p.k_scale, b, h)
            w, e = np.zeros(length), np.zeros(length)
            for i in range(p.news[b]):
                vis = sees(p, b, i, causal, window, draft)
                t = int(p.cu[b]) + i
                for hd in range(h * g, (h + 1) * g):
                    z = float(lse[t, hd])
                    if math.isinf(z):
                        continue
                    s = (kk @ q[t, hd]) * p.scale
                    x = np.where(vis, np.exp(np.where(vis, s - z, 0.0)), 0.0)
                    w += x
                    # a score's fp32 sum, its and the offset's rounding in log2 units, the power's own error
                    e += x * (p.dim * 2.0 ** -23 * (np.abs(kk) @ np.abs(q[t, hd])) * p.scale
                              + 2.0 ** -22 * (np.abs(s) + abs(z) + 2))
            old = np.where(np.arange(length) < first, decay * out[b, h, :length], 0.0)
            out[b, h, :length] = old + w
            tol[b, h, :length] = e + 2.0 ** -21 * np.abs(out[b, h, :length])
    return out, tol


def evict(scores, lens, budget, recent):
    """kept [B][H] lists."""
    out = []
    for b, n in enumerate(lens):
        per = []
        for h in range(scores.shape[1]):
            x = scores[b, h, :n].numpy().astype(np.float64)
            rank = sorted(range(n), key=lambda j: (0 if j >= n - recent else (2 if math.isnan(x[j]) else 1),
                                                   0.0 if math.isnan(x[j]) or j >= n - recent else -(x[j] + 0.0), j))
            per.append(sorted(rank[:budget]))
        out.append(per)
    return out


def rope(x, pos, freqs, magnitude, interleaved):
    """float64 rotary positions of [T, heads, dim]."""
    x = x.float().numpy().astype(np.float64).copy()
    f = freqs.double().sum(1).numpy()
    half = f.shape[0]
    for t in range(x.shape[0]):
        # whole turns leave the product exactly only in integers: use Python's exact rationals
        from fractions import Fraction
        for i in range(half):
            turn = Fraction(int(pos[t])) * (Fraction(float(freqs[i, 0])) + Fraction(float(freqs[i, 1])))
            turn -= math.floor(turn)
            a = 2.0 * math.pi * float(turn)
            c, s = math.cos(a) * magnitude, math.sin(a) * magnitude
            i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            x1, x2 = x[t, :, i1].copy(), x[t, :, i2].copy()
            x[t, :, i1], x[t, :, i2] = x1 * c - x2 * s, x2 * c + x1 * s
    return x
