"""One long sequence on the GPU, for tests of attention over many keys: inputs
as fp32 values that the types hold, results against 64 bits.  The bounds are those of
test_gpu_attn.py: a probability rounded to 16 bits moves the output by at most
2^-8 sum p|v| / sum p, a score's fp32 error e by 2 e times that, the output's own
rounding by 2^-8 |out|."""
import torch

import moe_speculative_verify_gb300 as m

PAGE = 64


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


class One:
    """One sequence of `keys` cached keys, the last `news` of them new; k and v
    [keys, hkv, dim] and q [news, hq, dim] hold fp32 values that the types hold
    (k, v: multiples of 1/16 in e4m3's range)."""

    def __init__(self, k, v, q, dtype, scale, k_scale=None, v_scale=None):
        keys, hkv, dim = k.shape
        self.k, self.v, self.q, self.scale = k, v, q, scale
        pages = -(-keys // PAGE)
        one = torch.full((hkv,), 1 / 16, device="cuda")
        self.k_scale = one if k_scale is None else k_scale
        self.v_scale = one if v_scale is None else v_scale

        def paged(x, s):
            full = torch.zeros(pages * PAGE, hkv, dim, device="cuda")
            full[:keys] = x if dtype == "bf16" else x / s[:, None]
            full = full.view(pages, PAGE, hkv, dim).permute(0, 2, 1, 3).contiguous()
            return full.to(torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn)

        self.dk, self.dv = paged(k, self.k_scale), paged(v, self.v_scale)
        self.dtype = dtype
        scales = (self.k_scale, self.v_scale) if dtype == "e4m3" else (None, None)
        self.cache = m.KVCache.from_tensors(self.dk, self.dv, *scales)
        news = q.shape[0]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.seqs = m.Seqs.from_tensors(i32([0, news]), i32([keys]), torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                                        news)
        # the values the cache holds
        back = lambda c, s: (c.double() * (s.double()[:, None, None] if dtype == "e4m3" else 1)).permute(0, 2, 1, 3).reshape(
            -1, hkv, dim)[:keys]
        self.k64, self.v64 = back(self.dk, self.k_scale), back(self.dv, self.v_scale)

    def run(self):
        news, hq, dim = self.q.shape
        attn = m.Attn(hq, self.scale)
        ws = torch.zeros(m.moe_attn_workspace_bytes(attn, self.cache), dtype=torch.uint8, device="cuda")
        out = torch.full((news, hq, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((news, hq), float("nan"), device="cuda")
        m.moe_paged_attention(attn, self.cache, self.seqs, self.q.bfloat16(), out, ws, lse=lse)
        assert m.moe_get_device_error(ws) == 0
        return out, lse

    def check(self):
        out, lse = self.run()
        news, hq, dim = self.q.shape
        keys, hkv = self.k64.shape[:2]
        q = self.q.bfloat16().double()
        for h in range(hkv):
            heads = slice(h * hq // hkv, (h + 1) * hq // hkv)
            qh, kk, vv = q[:, heads], self.k64[:, h], self.v64[:, h]
            s = torch.einsum("igd,jd->igj", qh, kk) * self.scale
            seen = torch.arange(keys, device="cuda")[None] <= (keys - news + torch.arange(news, device="cuda"))[:, None]
            s.masked_fill_(~seen[:, None], float("-inf"))
            z = torch.logsumexp(s, 2)
            p = torch.exp(s - z[..., None])
            want, mag = p @ vv, p @ vv.abs()
            err = dim * 2.0 ** -23 * abs(self.scale) * torch.einsum("igd,jd->igj", qh.abs(), kk.abs()).amax(2)
            tol = mag * (2.0 ** -8 + 2 * err[..., None] + 2.0 ** -20) + 2.0 ** -8 * want.abs() + 1e-30
            d = (out[:, heads].double() - want).abs()
            assert bool((d <= tol).all()), float((d / tol).nan_to_num(1e9).max())
            dz = (lse[:, heads].double() - z).abs()
            assert bool((dz <= err + 2.0 ** -20 * (1 + z.abs())).all()), float(dz.max())
