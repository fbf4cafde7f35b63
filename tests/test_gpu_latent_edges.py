"""The operators over a latent cache where they can go wrong: kernels that follow one another at once, numbers that are
not finite in cached rows, magnitudes near the ends of bf16, every number of pieces."""
import pytest
import torch

import latent_ref as ref
import moe_speculative_verify_gb300 as m
from latent_ref import ROT, i32
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


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("which", ["v", "k", "rope"])
@pytest.mark.parametrize("shape", [([300, 700], [150, 130], 2, 128), ([600], [600], 3, 64), ([2000], [9], 1, 128)])
def test_expanded_bad_rows_reach_those_that_see_them(shape, which, value):
    """A value that is not finite comes out in its element of every row that sees its key, an infinite score as NaN or as no
    weight; all else is as it was.  In the tiles that the causal mask cuts, with items of one pair of SMs and of several."""
    p = Expanded(*shape, seed=47)
    b, h, new = len(p.lens) - 1, p.heads - 1, p.news[-1] // 2
    key = p.lens[b] - p.news[b] + new                         # of token `new`
    row, tok = p.ck[b] + key, p.cu[b] + new
    want, sign = p.want(), torch.zeros(p.t, p.heads, device="cuda", dtype=torch.float64)
    hit = torch.zeros(p.t, p.heads, dtype=torch.bool, device="cuda")
    if which == "v":
        p.v[row, h, 3] = value
        hit[tok:p.cu[b + 1], h] = True
    else:
        d = 3 if which == "k" else p.dim + 3
        sign[tok:p.cu[b + 1]] = (p.q[tok:p.cu[b + 1], :, d].double() * value).sign()
        hit[tok:p.cu[b + 1], h if which == "k" else slice(None)] = True
        (p.k[row, h] if which == "k" else p.rope[row])[3] = value
    out, lse = p.run()
    ref.check(out[~hit], lse[~hit], *(x[~hit] for x in want))
    if which == "v":
        got = out[hit].clone()
        assert bool((torch.isnan(got[:, 3]) if value != value else got[:, 3] == value).all())
        got[:, 3] = want[0][hit][:, 3].to(got.dtype)
        ref.check(got, lse[hit], *(x[hit] for x in want))
        return
    up, down = hit & ~(sign < 0), hit & (sign < 0)
    assert bool(torch.isnan(out[up]).all()) and not bool(torch.isfinite(lse[up]).any())
    if bool(down.any()):
        # without that key: as if its own part were so small that it had no weight
        heads = [h] if which == "k" else range(p.heads)
        kr = slice(p.ck[b], p.ck[b] + p.lens[b])
        (p.k[row, h] if which == "k" else p.rope[row])[3] = 0.0
        keys = torch.cat([p.k[kr].double(), p.rope[kr].double()[:, None].expand(-1, p.heads, -1)], 2)
        seen = ref.sees(p.lens[b], p.news[b], True, 0, None)
        seen[:, key] = False
        r = slice(p.cu[b], p.cu[b + 1])
        less = ref.attend(p.q[r].double(), keys, p.v[kr].double(), seen, p.scale)
        ref.check(out[r][down[r]], lse[r][down[r]], *(x[down[r]] for x in less))


def test_a_bad_value_costs_its_own_item_only():
    """One value that is not finite, in one head of many items: the others do not pay for it (1.4 times the call's time; 47 times
    where every item after it did)."""
    p = Expanded([1500] * 8, [1024] * 8, 32, 128, seed=48)
    attn = m.Attn(p.heads, p.scale, wait_timeout_us=200000)
    ws = torch.zeros(m.moe_expanded_workspace_bytes(attn, 128), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(p.t, p.heads, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    t = []
    for k in range(2):
        if k:
            p.v[p.ck[0] + 600, 0, 3] = float("inf")
        runs = []
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            m.moe_expanded_attention(attn, p.seqs, p.d_ck, p.q, p.k, p.rope, p.v, outs[k], ws)
            b.record()
            torch.cuda.synchronize()
            runs.append(a.elapsed_time(b))
        t.append(min(runs))
    print("ms clean, one bad value:", t)
    assert m.moe_get_device_error(ws) == 0
    hit = torch.zeros(p.t, p.heads, 128, dtype=torch.bool, device="cuda")
    hit[1024 - 900:1024, 0, 3] = True                         # tokens at places from 600 on
    assert torch.equal(outs[0][~hit], outs[1][~hit]) and bool(torch.isposinf(outs[1][hit]).all())
    assert t[1] < 4 * t[0]


def test_expanded_values_that_are_all_nan():
    """Nothing finite in any value: every row that sees a key is NaN, with its log-sum-exp as ever."""
    p = Expanded([700, 90], [600, 90], 8, 128, seed=49)
    p.v.fill_(float("nan"))
    _, want, _, err = p.want()
    out, lse = p.run()
    assert bool(torch.isnan(out).all())
    assert bool(((lse.double() - want).abs() <= err + 2.0 ** -20 * (1 + want.abs())).all())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("latent", [256, 512])
@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e30])
@pytest.mark.parametrize("size", ["lone", 3e38, 1e25, 2e19, 1e-15, 1e-25, 1e-38, 1e-40])
def test_append_normalises_rows_of_any_size(dtype, latent, eps, size):
    """Rows whose squares pass the end of fp32, or lose their bits below it.  Tolerances as test_gpu_latent_rows.py's, and half the
    least bf16 (2^-134) for each of the result's two roundings where it is that small: a product's fp32 and the bf16."""
    p = ref.Problem([64], [3], 1, latent, 64, dtype, seed=50)
    freqs, mag = m.moe_rope_freqs(ROT)
    g = torch.Generator().manual_seed(latent)
    kv = torch.randn(3, latent + ROT, generator=g)
    if size == "lone":
        kv[1, 7] = 3e38
    else:
        kv[1, :latent] = kv[1, :latent].clamp(-1, 1) * size
    kv = kv.bfloat16().cuda()
    q = torch.zeros(3, 1, ROT, dtype=torch.bfloat16, device="cuda")
    gamma = (1 + 0.3 * torch.randn(latent, generator=g)).cuda()
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    m.moe_latent_append(m.Rope.from_freqs(freqs.cuda(), False, mag), p.cache, p.seqs, kv, q, pos, torch.empty_like(q), gamma=gamma, eps=eps)
    x = kv[:, :latent].double()
    eps = float(torch.tensor(eps))                              # as fp32 has it
    want = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * gamma.double()
    got = p.latent[int(p.table[0, 0]), 61:64].float().double() * 2.0 ** p.exp
    tol, floor = (2.0 ** -8, 2.0 ** -133) if dtype == "bf16" else (2.0 ** -4, 2.0 ** (p.exp - 10))
    if dtype == "e4m3":
        want = want.clamp(-448 * 2.0 ** p.exp, 448 * 2.0 ** p.exp)
    bad = ~((got - want).abs() <= (tol + 2.0 ** -18) * want.abs() + floor)
    assert not bool(bad.any()), (got[bad][:4], want[bad][:4])


def tiles_of(count, tile, rest):
    """Keys that make so many tiles, `pairs` of them or so where it is a text; with the last of one key alone or whole."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    n = eval(count, {"pairs": pairs}) if isinstance(count, str) else count
    return tile * (n - 1) + (rest or tile)


@pytest.mark.parametrize("rest", [0, 1])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 31, 33, "pairs-1", "pairs", "pairs+1", "2*pairs+1"])
@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_every_number_of_tiles(form, tiles, rest):
    """One item cut into as many pieces as it has tiles of keys (64 and 128), one a pair of SMs, and past that in runs."""
    if form == "absorbed":
        p = ref.Problem([tiles_of(tiles, 64, rest)], [1], 5, 512, 128, seed=51)
        out, lse = attend(p)
        ref.check(out, lse, *ref.latent_attention(p))
    else:
        x = Expanded([tiles_of(tiles, 128, rest)], [1], 1, 128, seed=52)
        out, lse = x.run()
        ref.check(out, lse, *x.want())
