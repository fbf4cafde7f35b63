"""Absorbed and expanded attention through a latent cache against 64 bits."""
import pytest
import torch

import latent_ref as ref
import moe_speculative_verify_gb300 as m
from latent_ref import ROT, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    m.build()
    m.load()
    torch.cuda.set_device(0)


def attend(p, causal=True, window=0, draft=None, stream=None, error=0, q=None):
    attn = m.Attn(p.heads, p.scale, causal, window, wait_timeout_us=200000)
    # beyond its error word a workspace may hold anything
    ws = torch.full((m.moe_latent_workspace_bytes(attn, p.cache),), 255, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    out = torch.full((p.t, p.heads, p.c), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.t, p.heads), float("nan"), device="cuda")
    m.moe_latent_attention(attn, p.cache, p.seqs, p.q if q is None else q, out, ws, lse=lse, draft_mask=draft, stream=stream)
    torch.cuda.synchronize()
    assert m.moe_get_device_error(ws) == error
    return out, lse


SHAPES = [
    # lens, news, heads, latent, page, dtype, store, pads
    ([1], [1], 8, 512, 16, "bf16", "rows", (0, 0)),                       # one token over itself
    ([1, 2, 63, 64, 65], [1] * 5, 16, 512, 64, "bf16", "rows", (0, 0)),   # halves of a tile
    ([127, 128, 129, 255, 257], [1] * 5, 64, 256, 32, "bf16", "split", (0, 0)),   # tile edges
    ([130, 0, 700, 17], [1, 0, 1, 1], 128, 512, 64, "bf16", "split", (2, 3)),
    ([300, 9, 4], [8, 8, 8], 32, 512, 32, "bf16", "rows", (0, 1)),        # verify blocks; more new tokens than keys
    ([77, 400], [5, 3], 24, 256, 16, "bf16", "rows", (1, 0)),
    ([129, 128, 127], [7, 1, 3], 12, 512, 128, "bf16", "split", (0, 0)),  # tiles across tokens
    ([257], [40], 16, 512, 64, "bf16", "rows", (0, 0)),
    ([333, 150], [150, 150], 3, 512, 64, "bf16", "rows", (3, 3)),         # chunks, one without a prefix
    ([500, 100], [11, 10], 1, 256, 16, "bf16", "rows", (0, 0)),           # one head
    ([900], [130], 40, 512, 32, "bf16", "split", (1, 1)),                 # thousands of rows over many tiles
    ([200], [3], 256, 512, 128, "bf16", "rows", (0, 0)),                  # the most heads
    ([1, 2, 63, 64, 65], [1] * 5, 16, 512, 64, "e4m3", "rows", (0, 0)),
    ([127, 128, 129, 255, 257], [1] * 5, 64, 256, 32, "e4m3", "split", (0, 0)),
    ([300, 9, 4], [8, 8, 8], 32, 512, 32, "e4m3", "split", (0, 1)),
    ([77, 400], [5, 3], 24, 256, 16, "e4m3", "rows", (1, 0)),
    ([333, 150], [150, 150], 3, 512, 64, "e4m3", "rows", (3, 3)),
    ([900], [130], 40, 512, 128, "e4m3", "split", (1, 1)),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[5]}-{s[6]}-c{s[3]}-p{s[4]}-h{s[2]}-{s[0]}-{s[1]}")
@pytest.mark.parametrize("mask", ["causal", "full", "window", "window1", "draft"])
def test_attention(shape, mask):
    p = ref.Problem(*shape[:5], shape[5], shape[6], shape[7], seed=len(shape[0]) + shape[4])
    causal, window, draft = mask != "full", {"window": 50, "window1": 1}.get(mask, 0), None
    if mask == "draft":
        draft = torch.randint(-2 ** 62, 2 ** 62, (p.t,), generator=torch.Generator().manual_seed(5)) * 2 + 1
        draft[p.t // 2] = 0                  # sees no new key
        draft = draft.cuda()
    out, lse = attend(p, causal, window, draft)
    ref.check(out, lse, *ref.latent_attention(p, causal, window, None if draft is None else draft.cpu()))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,news,heads", [([9000], [1], 64), ([20000], [1], 8), ([5000, 3, 2000], [8, 2, 8], 64),
                                             ([3000, 2900], [1, 1], 128)])
def test_long_split(lens, news, heads, dtype):
    """A long sequence cut over the card; equal calls give equal bits."""
    p = ref.Problem(lens, news, heads, 512, 64, dtype, seed=3)
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))
    for _ in range(3):
        o2, l2 = attend(p)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("keys", [128 * k for k in (2, 3, 7, 8, 29, 32, 61, 64, 75, 76, 77)])
def test_every_number_of_pieces(keys):
    """One row tile cut into as many pieces as it has key tiles, up to one a pair of SMs and past it."""
    p = ref.Problem([keys], [1], 5, 512, 128, seed=keys)
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 3])
def test_many_items(news, dtype):
    """Many short sequences: several items a pair of SMs, some without new tokens."""
    lens = [1 + (37 * b) % 131 for b in range(400)]
    p = ref.Problem(lens, [0 if b % 11 == 5 else min(news, n) for b, n in enumerate(lens)], 20, 256, 16, dtype, seed=17)
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_peaked_scores(dtype):
    """Scores of +-100s: the running maximum moves and most probabilities vanish."""
    p = ref.Problem([700, 90], [8, 3], 16, 512, 64, dtype, seed=4, q_scale=60.0)
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_small_probabilities_behind_a_heavy_key(dtype):
    """A first key that takes most of the weight, and many whose little each has to be kept."""
    def fill(total, page, c, g):
        x = torch.randn(total, page, c, generator=g)
        return (x * 16).round().clamp(-240, 240) / 16
    p = ref.Problem([3000], [2], 16, 512, 64, dtype, seed=8, fill=fill)
    p.q[:, :, :] = 0
    lat, rot = p.rows(0)
    # the first key scores 12 above the others, which score about 0
    p.q[:, :, :p.c] = (lat[0] / lat[0].norm() ** 2 * 12 / p.scale).bfloat16()
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))


@pytest.mark.parametrize("scale", [0.0, -0.07])
def test_zero_and_negative_scale(scale):
    p = ref.Problem([200, 31], [2, 5], 8, 256, 32, seed=9)
    p.scale = scale
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))


@pytest.mark.parametrize("exp", [-64, -9, 0, 7])
def test_e4m3_scales(exp):
    """Every size of the codes' power of two; queries to match."""
    p = ref.Problem([150], [2], 8, 256, 16, "e4m3", seed=10, scale_log2=exp, fill=lambda n, pg, c, g: torch.randn(
        n, pg, c, generator=g) * 2.0 ** (exp + 4))
    p.q[..., :p.c] = (p.q[..., :p.c].float() * 2.0 ** -(exp + 4)).bfloat16()
    out, lse = attend(p)
    want = ref.latent_attention(p)
    ref.check(out, lse, *want)


def test_query_rows_with_a_stride_and_another_stream():
    p = ref.Problem([300, 90], [5, 2], 6, 512, 64, seed=11)
    wide = torch.full((p.t, p.heads * (p.c + ROT) + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[:, :p.heads * (p.c + ROT)].view(p.t, p.heads, p.c + ROT)
    q.copy_(p.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = attend(p, q=q, stream=s)
    ref.check(out, lse, *ref.latent_attention(p))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 8, 40])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_query_stays_in_its_row(dtype, news, value):
    p = ref.Problem([300], [news], 8, 512, 64, dtype, seed=7)
    want = ref.latent_attention(p)
    p.q[news // 2, 3, 5] = value
    out, lse = attend(p)
    assert bool(torch.isnan(out[news // 2, 3]).all()) and bool(torch.isnan(lse[news // 2, 3]))
    rest = torch.ones(news, 8, dtype=torch.bool, device="cuda")
    rest[news // 2, 3] = False
    ref.check(out[rest], lse[rest], *(x[rest] for x in want))


@pytest.mark.parametrize("dtype,value", [("bf16", float("nan")), ("bf16", float("inf")), ("bf16", float("-inf")), ("e4m3", float("nan"))])
@pytest.mark.parametrize("place", [0, 299, 303, 307])
@pytest.mark.parametrize("part", ["latent", "rope"])
def test_a_bad_cached_row_reaches_only_the_rows_that_see_it(dtype, value, place, part):
    """8 new tokens at places 300 .. 307: a row that is not finite in a new token's place leaves the earlier tokens' outputs
    as they are; tokens that see a NaN have NaN throughout."""
    p = ref.Problem([308], [8], 8, 512, 64, dtype, seed=12)
    want = ref.latent_attention(p)
    pg, sl = int(p.table[0, place // 64]), place % 64
    if part == "rope":
        p.rope[pg, sl, 3] = value
    elif dtype == "e4m3":
        p.latent.view(torch.uint8)[pg, sl, 3] = 0x7F
    else:
        p.latent[pg, sl, 3] = value
    out, lse = attend(p)
    clear = max(place - 300, 0) if place >= 300 else 0
    if clear:
        ref.check(out[:clear], lse[:clear], *(x[:clear] for x in want))
    if value != value:
        assert bool(torch.isnan(out[clear:]).all()) and bool(torch.isnan(lse[clear:]).all())


def test_tables_that_do_not_fit():
    """A page outside the cache reads as zeros, a length past the table as what the table holds; both are recorded."""
    p = ref.Problem([200, 100], [2, 1], 8, 256, 32, seed=13)
    p.d_table[0, 1], p.d_table[1, 0] = -7, p.cache.n_pages
    out, lse = attend(p, error=1)
    j0 = torch.arange(200, device="cuda")
    tab = p.d_table.clone()
    tab[0, 1] = tab[1, 0] = 0
    keep, p.d_table = p.d_table, tab
    rows = [p.rows(b) for b in range(2)]
    p.d_table = keep
    for b, hole in ((0, (j0 >= 32) & (j0 < 64)), (1, j0[:100] < 32)):
        lat, rot = (x.masked_fill(hole[:, None], 0.0) for x in rows[b])
        r = slice(p.cu[b], p.cu[b + 1])
        ref.check(out[r], lse[r], *ref.attend(p.q[r].double(), torch.cat([lat, rot], 1), lat,
                                              ref.sees(p.lens[b], p.news[b], True, 0, None), p.scale))


@pytest.mark.parametrize("news", [1, 6])
@pytest.mark.parametrize("cu", ["past", "back", "first", "negative"])
def test_rows_of_a_bad_sequence_are_pad_rows(news, cu):
    p = ref.Problem([70, 50, 90], [news] * 3, 8, 256, 16, seed=31)
    good_out, good_lse = attend(p)
    offs = {"past": [0, news, 3 * news + 1, 3 * news], "back": [0, news, news - 1, news - 1],
            "first": [3 * news + 4, 3 * news + 5, 3 * news + 6, 3 * news + 7], "negative": [-2, -1, 0, 1]}[cu]
    good = {"past": 1, "back": 1, "first": 0, "negative": 0}[cu] * news
    p.seqs = m.Seqs.from_tensors(i32(offs), p.kv_len, p.d_table, news)
    out, lse = attend(p, error=1)
    assert torch.equal(out[:good], good_out[:good]) and torch.equal(lse[:good], good_lse[:good])
    assert bool(torch.all(out[good:].view(torch.int16) == 0) and torch.all(torch.isneginf(lse[good:])))


def test_graph_of_two_steps_follows_the_lengths():
    """One captured graph, replayed with other lengths, tables and queries; two graphs share a workspace on one stream."""
    p = ref.Problem([500, 130], [4, 2], 16, 512, 64, seed=21)
    attn = m.Attn(p.heads, p.scale)
    ws = torch.zeros(m.moe_latent_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(p.t, p.heads, p.c, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.zeros(p.t, p.heads, device="cuda") for _ in range(2)]
    call = lambda k: m.moe_latent_attention(attn, p.cache, p.seqs, p.q, outs[k], ws, lse=lses[k])
    call(0)
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(k)
        graphs.append(g)
    for lens in ([500, 130], [260, 64], [444, 2]):
        p.lens = lens
        p.kv_len.copy_(i32(lens))
        p.q.copy_(torch.randn(p.q.shape, device="cuda"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = ref.latent_attention(p)
        for k in range(2):
            ref.check(outs[k], lses[k], *want)
    assert m.moe_get_device_error(ws) == 0


# ------------------------------------------------------------ expanded form --
class Expanded:
    def __init__(self, lens, news, heads, dim, pads=(0, 0), seed=0, gaps=False, apart=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.news, self.heads, self.dim = lens, news, heads, dim
        ck, cu = [5 if gaps else 0], [pads[0]]
        for x, y in zip(lens, news):
            ck.append(ck[-1] + x)
            cu.append(cu[-1] + y)
        self.ck, self.cu, self.n, self.t = ck, cu, ck[-1] + (7 if gaps else 0), cu[-1] + pads[1]
        kv = torch.randn(self.n, heads, 2 * dim, generator=g).bfloat16().cuda()
        self.k, self.v = kv[..., :dim], kv[..., dim:]
        if apart:                                      # head-major storage
            self.k = self.k.transpose(0, 1).contiguous().transpose(0, 1)
        row = torch.randn(self.n, 512 + ROT, generator=g).bfloat16().cuda()
        self.rope = row[:, 512:]
        if gaps:                                       # rows of no sequence hold NaN
            for x in (self.k, self.v, self.rope):
                x[:5] = float("nan")
                x[ck[-1]:] = float("nan")
        self.q = (torch.randn(self.t, heads, dim + ROT, generator=g) * 1.5).bfloat16().cuda()
        self.scale = (dim + ROT) ** -0.5
        self.seqs = m.Seqs.from_tensors(i32(cu), i32(lens), torch.zeros(len(lens), 0, dtype=torch.int32, device="cuda"),
                                        max(news + [1]))
        self.d_ck = i32(ck)

    def run(self, causal=True, window=0, error=0):
        attn = m.Attn(self.heads, self.scale, causal, window, wait_timeout_us=200000)
        ws = torch.full((m.moe_expanded_workspace_bytes(attn, self.dim),), 255, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        out = torch.full((self.t, self.heads, self.dim), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.t, self.heads), float("nan"), device="cuda")
        m.moe_expanded_attention(attn, self.seqs, self.d_ck, self.q, self.k, self.rope, self.v, out, ws, lse=lse)
        torch.cuda.synchronize()
        assert m.moe_get_device_error(ws) == error
        return out, lse

    def want(self, causal=True, window=0):
        d = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")
        out, mag, err = d(self.t, self.heads, self.dim), d(self.t, self.heads, self.dim), d(self.t, self.heads)
        z = torch.full((self.t, self.heads), float("-inf"), dtype=torch.float64, device="cuda")
        for b, n in enumerate(self.news):
            if not n or not self.lens[b]:
                continue
            r, kr = slice(self.cu[b], self.cu[b] + n), slice(self.ck[b], self.ck[b] + self.lens[b])
            keys = torch.cat([self.k[kr].double(), self.rope[kr].double()[:, None].expand(-1, self.heads, -1)], 2)
            out[r], z[r], mag[r], err[r] = ref.attend(self.q[r].double(), keys, self.v[kr].double(),
                                                      ref.sees(self.lens[b], n, causal, window, None), self.scale)
        return out, z, mag, err


EXPANDED = [
    ([1], [1], 1, 128, (0, 0)),
    ([127, 128, 129], [127, 128, 129], 3, 128, (0, 0)),       # tile edges, no prefix
    ([300, 0, 40], [257, 0, 1], 2, 128, (2, 3)),
    ([700, 5], [100, 9], 4, 128, (0, 1)),                     # the second has more queries than keys
    ([1000], [1000], 2, 64, (0, 0)),
    ([90, 513], [33, 500], 5, 64, (1, 0)),
    ([2000], [3], 1, 128, (0, 0)),                            # few rows over many keys: split and joined
]


@pytest.mark.parametrize("shape", EXPANDED, ids=lambda s: f"d{s[3]}-h{s[2]}-{s[0]}-{s[1]}")
@pytest.mark.parametrize("mask", ["causal", "full", "window", "window1"])
@pytest.mark.parametrize("layout", ["side", "gaps", "apart"])
def test_expanded(shape, mask, layout):
    p = Expanded(*shape, seed=shape[2], gaps=layout == "gaps", apart=layout == "apart")
    causal, window = mask != "full", {"window": 70, "window1": 1}.get(mask, 0)
    out, lse = p.run(causal, window)
    ref.check(out, lse, *p.want(causal, window))
    o2, l2 = p.run(causal, window)
    assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_expanded_many_items():
    lens = [1 + (53 * b) % 200 for b in range(60)]
    p = Expanded(lens, [min(1 + (7 * b) % 90, n) for b, n in enumerate(lens)], 16, 128, seed=2)
    out, lse = p.run()
    ref.check(out, lse, *p.want())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["q", "k", "v", "rope"])
def test_expanded_bad_rows(which, value):
    """What is not finite in a new token's row leaves the tokens before it as they are."""
    p = Expanded([300], [150], 2, 128, seed=5)
    want = p.want()
    at = 60                                                   # token 60, key 210
    {"q": lambda: p.q[at].__setitem__((1, 3), value), "k": lambda: p.k[210, 1].__setitem__(3, value),
     "v": lambda: p.v[210, 1].__setitem__(3, value), "rope": lambda: p.rope[210].__setitem__(3, value)}[which]()
    out, lse = p.run()
    ref.check(out[:at], lse[:at], *(x[:at] for x in want))
    ref.check(out[:, :1], lse[:, :1], *(x[:, :1] for x in want)) if which != "rope" else None
    if value != value and which in ("k", "rope"):
        assert bool(torch.isnan(out[at:, 1]).all()) and bool(torch.isnan(lse[at:, 1]).all())
    if value != value and which == "v":
        assert bool(torch.isnan(out[at:, 1, 3]).all())
    if which == "q":
        assert bool(torch.isnan(out[at, 1]).all())
        ref.check(out[at + 1:], lse[at + 1:], *(x[at + 1:] for x in want))


def test_expanded_rows_outside():
    """Rows past the last one read as zeros and are recorded; a length past the rows there are is cut."""
    p = Expanded([100, 60], [10, 4], 2, 128, seed=6)
    p.d_ck = i32([0, 110, 170])                               # the second sequence's last ten rows lie outside
    out, lse = p.run(error=1)
    zero = lambda x: torch.cat([x, torch.zeros(10, *x.shape[1:], dtype=x.dtype, device="cuda")])
    p.k, p.v, p.rope, p.ck = zero(p.k), zero(p.v), zero(p.rope), [0, 110, 170]
    ref.check(out, lse, *p.want())


# ------------------------------------------------------------------ together --
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prompt_expanded_then_verify_absorbed(dtype):
    """The four operators as a layer runs them: a prompt appended, gathered, expanded and attended to; then a verify block
    through the cache in absorbed form, which has to agree with the expanded form over the same rows."""
    g = torch.Generator().manual_seed(3)
    H, C, D, page, n = 4, 512, 128, 64, 300
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()
    wk, wv = rnd(H, D, C) * C ** -0.5, rnd(H, D, C) * C ** -0.5
    lat = torch.zeros(8, page, C, dtype=torch.bfloat16, device="cuda")
    lat = lat if dtype == "bf16" else lat.to(torch.float8_e4m3fn)
    rot = torch.zeros(8, page, ROT, dtype=torch.bfloat16, device="cuda")
    cache = m.LatentCache.from_tensors(lat, rot, -4)
    attn = m.Attn(H, (D + ROT) ** -0.5)
    ws = torch.zeros(m.moe_latent_workspace_bytes(attn, cache), dtype=torch.uint8, device="cuda")
    ws2 = torch.zeros(m.moe_expanded_workspace_bytes(attn, D), dtype=torch.uint8, device="cuda")
    freqs, mag = m.moe_rope_freqs(ROT)
    rope = m.Rope.from_freqs(freqs.cuda(), True, mag, ws)
    gamma = 1 + 0.1 * rnd(C)
    table = i32([[5, 0, 3, 1, 7, 2]])
    cached = 0
    for new in (n, 8):
        cached += new
        seqs = m.Seqs.from_tensors(i32([0, new]), i32([cached]), table, new)
        kv, q = rnd(new, C + ROT).bfloat16(), rnd(new, H, D + ROT).bfloat16()
        ql = torch.zeros(new, H, C + ROT, dtype=torch.bfloat16, device="cuda")
        m.moe_latent_append(rope, cache, seqs, kv, q[..., D:], torch.arange(cached - new, cached, dtype=torch.int32, device="cuda"),
                            ql[..., C:], gamma=gamma)
        rows = torch.full((cached, C + ROT), float("nan"), dtype=torch.bfloat16, device="cuda")
        m.moe_latent_gather(cache, seqs, i32([0, cached]), rows, ws)
        k = torch.einsum("jc,hdc->jhd", rows[:, :C].float(), wk).bfloat16()
        v = torch.einsum("jc,hdc->jhd", rows[:, :C].float(), wv).bfloat16()
        qe = torch.cat([q[..., :D], ql[..., C:]], 2)
        out = torch.zeros(new, H, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(new, H, device="cuda")
        m.moe_expanded_attention(attn, seqs, i32([0, cached]), qe, k, rows[:, C:], v, out, ws2, lse=lse)
        ql[..., :C] = torch.einsum("ihd,hdc->ihc", q[..., :D].float(), wk).bfloat16()
        ol, lsel = torch.zeros(new, H, C, dtype=torch.bfloat16, device="cuda"), torch.zeros(new, H, device="cuda")
        m.moe_latent_attention(attn, cache, seqs, ql, ol, ws, lse=lsel)
        got = torch.einsum("ihc,hdc->ihd", ol.float(), wv)
        assert m.moe_get_device_error(ws) == 0 and m.moe_get_device_error(ws2) == 0
        # k rounded per head on one side, q on the other: scores differ by 2^-8 of sums of random signs, outputs by a few bf16 steps
        assert float((got - out.float()).norm() / out.float().norm()) < 0.02
        assert float((lse - lsel).abs().max()) < 0.05
