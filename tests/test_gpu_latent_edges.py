"""Attention through a latent cache where it can go wrong: kernels that follow one
another at once, numbers that are not finite in cached rows, every number of pieces."""
import pytest
import torch

import latent_ref as ref
import moe_speculative_verify_gb300 as m
from latent_ref import i32
from test_gpu_latent import Expanded, attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    m.build()
    m.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_kernels_that_follow_one_another(dtype):
    """Short calls of both attention kernels in turn, without a pause: a CTA's barriers lie where those of the kernel before
    lay, so an arrival of that one which came after its CTA's end would be counted here."""
    p = ref.Problem([70, 3], [2, 1], 16, 256, 32, dtype, seed=41)
    x = Expanded([40, 300], [9, 2], 2, 64, seed=42)
    attn, xa = m.Attn(16, p.scale), m.Attn(2, x.scale)
    ws = torch.zeros(m.moe_latent_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
    wx = torch.zeros(m.moe_expanded_workspace_bytes(xa, 64), dtype=torch.uint8, device="cuda")
    outs = torch.zeros(200, p.t, 16, 256, dtype=torch.bfloat16, device="cuda")
    xouts = torch.zeros(200, x.t, 2, 64, dtype=torch.bfloat16, device="cuda")
    lse, xl = torch.zeros(p.t, 16, device="cuda"), torch.zeros(x.t, 2, device="cuda")
    for k in range(200):
        m.moe_latent_attention(attn, p.cache, p.seqs, p.q, outs[k], ws, lse=lse)
        m.moe_expanded_attention(xa, x.seqs, x.d_ck, x.q, x.k, x.rope, x.v, xouts[k], wx, lse=xl)
    assert m.moe_get_device_error(ws) == 0 and m.moe_get_device_error(wx) == 0
    ref.check(outs[0], lse, *ref.latent_attention(p))
    ref.check(xouts[0], xl, *x.want())
    assert torch.equal(outs, outs[:1].expand_as(outs)) and torch.equal(xouts, xouts[:1].expand_as(xouts))


def infinite_latent(p, value, place, part, causal=True, window=0, draft=None):
    """Puts `value` into element 3 of a cached row of sequence 0 and calls: rows that do not see it are as without it; a row
    that scores it +inf is NaN; where the score is -inf the row has no weight, but 0 times an infinite value is NaN in that one
    element.  Returns what was called for, for a check of its own."""
    n, first = p.news[0], p.lens[0] - p.news[0]
    lat, rot = p.rows(0)
    q, keys = p.q[p.cu[0]:p.cu[0] + n].double(), torch.cat([lat, rot], 1)
    seen = ref.sees(p.lens[0], n, causal, window, None if draft is None else [int(x) for x in draft.cpu()[p.cu[0]:p.cu[0] + n]])
    apart = seen.clone()
    apart[:, place] = False
    whole, less = ref.attend(q, keys, lat, seen, p.scale), ref.attend(q, keys, lat, apart, p.scale)
    (p.latent if part == "latent" else p.rope)[int(p.table[0, place // p.page]), place % p.page, 3] = value
    out, lse = (x[p.cu[0]:p.cu[0] + n] for x in attend(p, causal, window, draft))
    sign = (p.q[p.cu[0]:p.cu[0] + n, :, 3 if part == "latent" else p.c + 3].double() * value * p.scale).sign()
    sees_it = seen[:, place, None].expand(n, p.heads)
    up, down = sees_it & (sign > 0), sees_it & (sign < 0)
    assert bool((sees_it == (up | down)).all())
    assert bool(torch.isnan(out[up]).all()) and not bool(torch.isfinite(lse[up]).any())
    if bool((~sees_it).any()):
        ref.check(out[~sees_it], lse[~sees_it], *(x[~sees_it] for x in whole))
    if bool(down.any()):
        got, want = out[down].clone(), [x[down] for x in less]
        if part == "latent":
            live = ~want[1].isneginf()                        # (a row with no other key: nothing has weight)
            assert bool(torch.isnan(got[live][:, 3]).all())
            got[live, 3] = want[0][live, 3].to(got.dtype)
        ref.check(got, lse[down], *want)
    return int(up.sum()), int(down.sum())


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("part", ["latent", "rope"])
@pytest.mark.parametrize("heads,latent,news,page", [(8, 512, 8, 64), (16, 512, 8, 16), (5, 256, 40, 128)])   # items of 64 rows, of 128, several
@pytest.mark.parametrize("place", ["old", "beside", "new", "last"])
def test_infinite_latents_in_whole_and_cut_tiles(value, part, heads, latent, news, page, place):
    """In a tile that all rows see, among the old keys of one that the causal mask cuts, and in new tokens' rows."""
    p = ref.Problem([420 + news], [news], heads, latent, page, seed=43)
    infinite_latent(p, value, {"old": 70, "beside": 418, "new": 420 + news // 2, "last": 419 + news}[place], part)


@pytest.mark.parametrize("mask", ["window", "draft", "full", "negative", "long"])
@pytest.mark.parametrize("heads", [8, 32])
def test_infinite_latents_under_other_masks(mask, heads):
    news = 8
    p = ref.Problem([20000 if mask == "long" else 200], [news], heads, 512, 32, seed=44)
    draft = None
    if mask == "draft":
        draft = torch.tensor([0b1, 0b11, 0b101, 0b1001, 0b10011, 0b100101, 0b1000001, 0b10000011], device="cuda")
    if mask == "negative":
        p.scale = -p.scale
    n = p.lens[0]
    up, down = infinite_latent(p, float("-inf"), {"window": n - 45, "draft": n - 7, "long": n - 10}.get(mask, n - 3), "latent", mask != "full",
                               40 if mask == "window" else 0, draft)
    assert up > 0 and down > 0


@pytest.mark.parametrize("lens", [[400] * 100, [20000]])       # several tiles a pair of SMs; one sequence over all of them
@pytest.mark.parametrize("bad", [1, 64, 300])
@pytest.mark.parametrize("heads", [8, 96])
def test_infinite_latents_before_a_heavy_key(lens, bad, heads):
    """Rows of weight 0 whose element 3 is infinite, alone in their tiles or not, and then a key beside which all before it has
    no weight in fp32: 0 times an infinite value is NaN, wherever the row lies."""
    p = ref.Problem(lens, [1] * len(lens), heads, 512, 64, seed=45)
    p.q[:] = p.q[:1, :1]
    p.q[..., 3] = 1.0
    flat = lambda j: (p.d_table[:, j // 64].long(), j % 64)
    heavy = lens[0] - 80
    p.latent[flat(heavy)] = (p.q[0, 0, :512].float() * (300.0 / p.scale / float(p.q[0, 0, :512].float().square().sum()))).bfloat16()
    want = None
    for b in range(len(lens)):
        lat, rot = p.rows(b)
        seen = ref.sees(lens[b], 1, True, 0, None)
        seen[:, :bad] = False
        w = ref.attend(p.q[b:b + 1].double(), torch.cat([lat, rot], 1), lat, seen, p.scale)
        want = w if want is None else [torch.cat(x) for x in zip(want, w)]
    for j in range(bad):
        pg, sl = flat(j)
        p.latent[pg, sl, 3] = float("-inf")
    out, lse = attend(p)
    assert bool(torch.isnan(out[..., 3]).all())
    out[..., 3] = want[0][..., 3].to(out.dtype)
    ref.check(out, lse, *want)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads,seqs", [(16, 8), (1, 1)])
def test_expanded_infinite_values_before_a_heavy_key(heads, seqs, value):
    """The same of the expanded form, whose values are apart from its keys: not finite, wherever the key lies."""
    p = Expanded([900] * seqs, [200] * seqs, heads, 128, seed=46)
    p.q[:] = p.q[:1, :1]
    at = i32(p.ck[:-1]).long()
    p.k[at + 650] = p.q[0, 0, :128] * (300.0 / p.scale / float(p.q[0, 0, :128].float().square().sum()))
    want = p.want()
    p.v[at + 5, :, 3] = value
    out, lse = p.run()
    assert not bool(torch.isfinite(out[..., 3]).any())
    out[..., 3] = want[0][..., 3].to(out.dtype)
    ref.check(out, lse, *want)
