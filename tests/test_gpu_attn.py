"""Paged attention and key weights against a 64-bit implementation.

Tolerances, from the arithmetic: a probability is rounded to bf16 (8 significant
bits: relative 2^-8) or, beside e4m3 codes, to f16 or a pair of 8-bit codes (at
most 2^-8), so the output's sum moves by at most 2^-8 sum p|v| / sum p; its own rounding to bf16 adds as much of |out|; a score's
fp32 error (at most D 2^-23 sum |q||k| scale) and the exponential's (2^-21)
move both sums alike, at most twice that times sum p|v| / sum p.  The
log-sum-exp moves by the score's error, and by its fp32 roundings."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import moe_speculative_verify_gb300 as m

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    m.build()
    m.load()
    torch.cuda.set_device(0)


def attend(p, causal=True, window=0, draft=None, stream=None):
    attn = m.Attn(p.hq, p.scale, causal, window, wait_timeout_us=200000)
    # beyond its error word a workspace may hold anything
    ws = torch.full((m.moe_attn_workspace_bytes(attn, p.cache),), 255, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    out = torch.full((p.t, p.hq, p.dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.t, p.hq), float("nan"), device="cuda")
    d = None if draft is None else draft.cuda()
    m.moe_paged_attention(attn, p.cache, p.seqs, p.d_q(), out, ws, lse=lse, draft_mask=d, stream=stream)
    torch.cuda.synchronize()
    assert m.moe_get_device_error(ws) == 0
    return out, lse, ws


def check(p, out, lse, causal=True, window=0, draft=None):
    want, z, mag, err = ref.attention(p, causal, window, draft)
    got = out.float().cpu().numpy().astype(np.float64)
    tol = mag * (2.0 ** -8 + 2 * err[..., None] + 2.0 ** -20) + 2.0 ** -8 * np.abs(want) + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
    empty = np.isneginf(z)
    assert np.all(got[empty] == 0) and not np.signbit(got[empty]).any()
    zl = lse.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(zl), empty)
    d = np.abs(zl[~empty] - z[~empty])
    assert np.all(d <= (err + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, z))))[~empty])


SHAPES = [
    # lens, news, hq, hkv, dim, page, dtype, layout, pads
    ([1], [1], 8, 8, 128, 16, "bf16", "hnd", (0, 0)),                       # one token over itself
    ([1, 2, 63, 64, 65], [1] * 5, 16, 2, 128, 64, "bf16", "hnd", (0, 0)),   # tile edges
    ([130, 0, 700, 17], [1, 0, 1, 1], 64, 8, 128, 64, "bf16", "nhd", (2, 3)),
    ([300, 9, 4], [8, 8, 8], 32, 4, 128, 32, "bf16", "hnd", (0, 1)),        # verify blocks; more new tokens than keys
    ([77, 400], [5, 3], 24, 3, 64, 16, "bf16", "nhd", (1, 0)),              # odd group of 8 heads, small head
    ([129, 128, 127], [7, 1, 3], 12, 1, 64, 128, "bf16", "hnd", (0, 0)),    # group of 12: tiles across tokens
    ([200, 33], [4, 2], 14, 2, 128, 128, "bf16", "hnd", (0, 0)),            # group of 7
    ([257], [40], 16, 16, 128, 64, "bf16", "hnd", (0, 0)),                  # no sharing of heads
    ([333, 150], [150, 150], 16, 2, 128, 64, "bf16", "hnd", (3, 3)),        # chunks, one without a prefix
    ([300], [200], 20, 4, 64, 32, "bf16", "nhd", (0, 0)),
    ([500, 100], [11, 10], 16, 2, 128, 16, "bf16", "hnd", (0, 0)),          # 88 rows a kv head
    ([900], [130], 8, 1, 64, 32, "bf16", "nhd", (1, 1)),                    # 1040 rows over many key tiles
    ([500, 100], [11, 10], 16, 2, 128, 16, "e4m3", "nhd", (0, 0)),
    ([900], [130], 8, 1, 64, 32, "e4m3", "hnd", (1, 1)),
    ([1, 2, 63, 64, 65], [1] * 5, 16, 2, 128, 64, "e4m3", "hnd", (0, 0)),
    ([300, 9, 4], [8, 8, 8], 32, 4, 128, 32, "e4m3", "nhd", (0, 1)),
    ([77, 400], [5, 3], 24, 3, 64, 16, "e4m3", "hnd", (1, 0)),
    ([129, 128, 127], [7, 1, 3], 12, 1, 64, 128, "e4m3", "nhd", (0, 0)),
    ([333, 150], [150, 150], 16, 2, 128, 64, "e4m3", "hnd", (3, 3)),
    ([300], [200], 20, 4, 64, 32, "e4m3", "hnd", (0, 0)),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[6]}-{s[7]}-d{s[4]}-p{s[5]}-{s[2]}x{s[3]}-{s[0]}-{s[1]}")
@pytest.mark.parametrize("mask", ["causal", "full", "window", "window1", "draft"])
def test_attention(shape, mask):
    p = ref.Problem(*shape[:6], shape[6], shape[7], shape[8], seed=len(shape[0]) + shape[5]).cuda()
    causal, window, draft = mask != "full", {"window": 50, "window1": 1}.get(mask, 0), None
    if mask == "draft":
        g = torch.Generator().manual_seed(5)
        draft = torch.randint(-2 ** 62, 2 ** 62, (p.t,), generator=g) * 2 + 1
        draft[p.t // 2] = 0                  # sees no new key
    out, lse, _ = attend(p, causal, window, draft)
    check(p, out, lse, causal, window, draft)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,news,hq,hkv", [([9000], [1], 8, 1), ([5000, 3, 2000], [8, 2, 8], 16, 2),
                                              ([3000, 2900], [1, 1], 32, 32)])
def test_long_split(lens, news, hq, hkv, dtype):
    """One long sequence cut over many CTAs; equal calls give equal bits."""
    p = ref.Problem(lens, news, hq, hkv, 128, 64, dtype, seed=3).cuda()
    out, lse, _ = attend(p)
    check(p, out, lse)
    for _ in range(3):
        o2, l2, _ = attend(p)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 3])
def test_many_items(news, dtype):
    """Many short sequences: dozens of items a CTA, some without new tokens."""
    lens = [1 + (37 * b) % 131 for b in range(500)]
    p = ref.Problem(lens, [0 if b % 11 == 5 else min(news, n) for b, n in enumerate(lens)], 32, 4, 64, 16, dtype,
                    seed=17).cuda()
    out, lse, _ = attend(p)
    check(p, out, lse)


def test_peaked_scores():
    """Scores of +-100s: the running maximum moves and most probabilities vanish."""
    p = ref.Problem([700, 90], [8, 3], 16, 2, 128, 64, seed=4, q_scale=80.0).cuda()
    out, lse, _ = attend(p)
    check(p, out, lse)


@pytest.mark.parametrize("factor", [1e-30, 1e30])
def test_e4m3_query_range(factor):
    """Queries far outside f16's range beside e4m3 codes."""
    p = ref.Problem([200], [4], 8, 1, 128, 64, "e4m3", seed=6)
    p.qkv = (p.qkv.float() * factor).bfloat16()
    p.scale = p.scale / factor
    p.cuda()
    out, lse, _ = attend(p)
    check(p, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [1, 8, 40])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_query_stays_in_its_row(dtype, news, value):
    """A NaN or infinite query gives NaN in its own row and head, and there alone."""
    p = ref.Problem([300], [news], 8, 1, 128, 64, dtype, seed=7)
    clean = ref.attention(p)
    p.qkv[news // 2, 3, 5] = value
    p.cuda()
    out, lse, _ = attend(p)
    assert torch.isnan(out[news // 2, 3]).all() and torch.isnan(lse[news // 2, 3])
    x, z = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    rest = np.ones((news, 8), bool)
    rest[news // 2, 3] = False
    tol = clean[2] * (2.0 ** -8 + 2 * clean[3][..., None] + 2.0 ** -20) + 2.0 ** -8 * np.abs(clean[0]) + 1e-30
    assert np.all(np.abs(x - clean[0])[rest] <= tol[rest])
    assert np.all(np.abs(z - clean[1])[rest] <= (clean[3] + 2.0 ** -20 * (1 + np.abs(clean[1])))[rest])


def test_page_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32."""
    p = ref.Problem([150], [3], 8, 2, 128, 64, seed=8)
    small_k, small_v = p.k, p.v
    pages = 2 ** 32 // (2 * 64 * 128 * 2) + 40
    big = torch.empty(2, pages, 2, 64, 128, dtype=torch.bfloat16, device="cuda")
    used = p.table[0, :3].long()
    far = torch.tensor([pages - 1, pages - 3, 7])
    big[0][far.cuda()] = small_k[used].cuda()
    big[1][far.cuda()] = small_v[used].cuda()
    p.cuda()
    p.d_table[0, :3] = far.int().cuda()
    p.cache = m.KVCache.from_tensors(big[0], big[1])
    out, lse, _ = attend(p)
    check(p, out, lse)
    sc = torch.zeros(1, 2, 192, device="cuda")
    ws = torch.zeros(m.moe_attn_workspace_bytes(m.Attn(8, p.scale), p.cache), dtype=torch.uint8, device="cuda")
    m.moe_key_weights(m.Attn(8, p.scale), p.cache, p.seqs, p.d_q(), lse, sc, sc, ws)
    want, tol = ref.key_weights(p, lse.cpu(), torch.zeros(1, 2, 192), 1.0)
    assert np.all(np.abs(sc.cpu().numpy() - want) <= tol)


def test_other_stream_and_graph():
    p = ref.Problem([500, 70], [8, 1], 16, 2, 128, 64, seed=9).cuda()
    want, lse0, _ = attend(p)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        out, lse, _ = attend(p)
    assert torch.equal(out, want) and torch.equal(lse, lse0)
    attn = m.Attn(p.hq, p.scale)
    ws = torch.zeros(m.moe_attn_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_paged_attention(attn, p.cache, p.seqs, p.d_q(), out, ws)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # the lengths are read on the device: a shorter sequence replays rightly
    p.lens[0] = 301
    p.d_kv_len[0] = 301
    g.replay()
    torch.cuda.synchronize()
    check(p, out, torch.from_numpy(ref.attention(p)[1]))


def test_bad_numbers_are_recorded():
    """A page index outside the cache reads as zeros, a length past the table is
    cut; both recorded, neither followed."""
    p = ref.Problem([130, 40], [1, 1], 8, 2, 128, 64, seed=10).cuda()
    attn = m.Attn(p.hq, p.scale)
    for wreck in ("page", "len", "cu"):
        ws = torch.zeros(m.moe_attn_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
        table, kv_len, cu = p.d_table.clone(), p.d_kv_len.clone(), p.d_cu.clone()
        if wreck == "page":
            table[0, 1] = -7
            table[1, 0] = 1 << 30
        elif wreck == "len":
            table[:] = 0
            kv_len[0] = 1 << 30
        else:
            cu[1] = 9
        seqs = m.Seqs.from_tensors(cu, kv_len, table, 1)
        out = torch.empty((p.t, p.hq, p.dim), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((p.t, p.hq), device="cuda")
        m.moe_paged_attention(attn, p.cache, seqs, p.d_q(), out, ws, lse=lse)
        assert m.moe_get_device_error(ws) == 1, wreck
        sc = torch.zeros(2, 2, 512, device="cuda")
        m.moe_key_weights(attn, p.cache, seqs, p.d_q(), lse, sc, sc, ws)
        assert m.moe_get_device_error(ws) == 1, wreck


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[6]}-{s[7]}-d{s[4]}-p{s[5]}-{s[2]}x{s[3]}-{s[0]}-{s[1]}")
@pytest.mark.parametrize("mask", ["causal", "full", "window", "draft"])
def test_key_weights(shape, mask):
    p = ref.Problem(*shape[:6], shape[6], shape[7], shape[8], seed=len(shape[0]) + shape[5]).cuda()
    causal, window, draft = mask != "full", 50 if mask == "window" else 0, None
    if mask == "draft":
        g = torch.Generator().manual_seed(5)
        draft = torch.randint(-2 ** 62, 2 ** 62, (p.t,), generator=g) * 2 + 1
        draft[p.t // 2] = 0
    lse = torch.from_numpy(ref.attention(p, causal, window, draft)[1]).float()
    lse[p.t // 3] = float("inf")             # a row that is left out
    g = torch.Generator().manual_seed(6)
    scores = torch.rand(len(p.lens), p.hkv, max(p.lens) + 3, generator=g)
    attn = m.Attn(p.hq, p.scale, causal, window, wait_timeout_us=200000)
    ws = torch.zeros(m.moe_attn_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
    want, tol = ref.key_weights(p, lse, scores, 0.75, causal, window, draft)
    d = None if draft is None else draft.cuda()
    got = scores.cuda()
    other = got.clone()
    m.moe_key_weights(attn, p.cache, p.seqs, p.d_q(), lse.cuda(), got, got, ws, decay=0.75, draft_mask=d)
    m.moe_key_weights(attn, p.cache, p.seqs, p.d_q(), lse.cuda(), scores.cuda(), other, ws, decay=0.75, draft_mask=d)
    assert m.moe_get_device_error(ws) == 0
    assert torch.equal(got, other)           # in place or not, the same bits
    x = got.cpu().numpy().astype(np.float64)
    bad = ~(np.abs(x - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], x[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_key_weights_many_items(dtype):
    """More items than SMs, many row tiles an item, and rows of other sequences
    that hold NaN beside those that count."""
    p = ref.Problem([2600, 900, 1, 257], [40, 3, 1, 9], 64, 16, 64, 32, dtype, seed=21, pads=(2, 2))
    p.qkv[0], p.qkv[-1] = float("nan"), float("nan")
    p.cuda()
    lse = torch.from_numpy(ref.attention(p)[1]).float()
    scores = torch.rand(4, 16, 2600, generator=torch.Generator().manual_seed(3))
    want, tol = ref.key_weights(p, lse, scores, 1.0)
    attn = m.Attn(p.hq, p.scale, wait_timeout_us=200000)
    ws = torch.zeros(m.moe_attn_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
    got = scores.cuda()
    m.moe_key_weights(attn, p.cache, p.seqs, p.d_q(), lse.cuda(), got, got, ws)
    assert m.moe_get_device_error(ws) == 0
    x = got.cpu().numpy().astype(np.float64)
    bad = ~(np.abs(x - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], x[bad][:4], want[bad][:4])


@pytest.mark.parametrize("hq,hkv", [(160, 1), (130, 1), (256, 2), (15, 5)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_wide_groups(hq, hkv, dtype):
    """More query heads a kv head than a row tile holds, and odd groups."""
    p = ref.Problem([200, 70], [3, 2], hq, hkv, 64, 64, dtype, seed=22).cuda()
    out, lse, _ = attend(p)
    check(p, out, lse)
    z = torch.from_numpy(ref.attention(p)[1]).float()
    scores = torch.zeros(2, hkv, 200)
    want, tol = ref.key_weights(p, z, scores, 1.0)
    attn = m.Attn(p.hq, p.scale, wait_timeout_us=200000)
    ws = torch.zeros(m.moe_attn_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
    got = scores.cuda()
    m.moe_key_weights(attn, p.cache, p.seqs, p.d_q(), z.cuda(), got, got, ws)
    assert m.moe_get_device_error(ws) == 0
    assert np.all(np.abs(got.cpu().numpy().astype(np.float64) - want) <= tol)


def test_key_weights_without_new_tokens():
    """Sequences without new tokens only decay."""
    p = ref.Problem([300, 20], [0, 0], 8, 2, 128, 64, seed=23).cuda()
    attn = m.Attn(p.hq, p.scale, wait_timeout_us=200000)
    ws = torch.zeros(m.moe_attn_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
    scores = torch.rand(2, 2, 300, device="cuda")
    got = scores.clone()
    m.moe_key_weights(attn, p.cache, p.seqs, p.d_q(), torch.zeros(0, 8, device="cuda"), got, got, ws, decay=0.5)
    assert m.moe_get_device_error(ws) == 0
    for b, n in enumerate(p.lens):
        assert torch.equal(got[b, :, :n], scores[b, :, :n] * 0.5) and torch.equal(got[b, :, n:], scores[b, :, n:])


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_key_weights_all_codes_and_nan(dtype):
    """Every finite e4m3 code (subnormals too) counts with its value, and a NaN
    key makes its own weight NaN and no other."""
    p = ref.Problem([256], [1], 8, 1, 128, 64, dtype, seed=24, q_scale=0.2)
    codes = torch.arange(256, dtype=torch.uint8)
    codes[[0x7F, 0xFF]] = 0
    grid = codes[(torch.arange(256)[:, None] + 7 * torch.arange(128)[None]) % 256]
    vals = grid.view(torch.float8_e4m3fn).float() / 64
    for j in range(256):
        pg, o = int(p.table[0, j // 64]), j % 64
        if dtype == "e4m3":
            p.k.view(torch.uint8)[pg, 0, o] = grid[j]
        else:
            p.k[pg, 0, o] = vals[j].bfloat16()
    if dtype == "e4m3":
        p.k_scale[:] = 1 / 64
    lse = torch.from_numpy(ref.attention(p)[1]).float()
    scores = torch.zeros(1, 1, 256)
    want, tol = ref.key_weights(p, lse, scores, 1.0)
    pg, o = int(p.table[0, 1]), 9
    if dtype == "e4m3":
        p.k.view(torch.uint8)[pg, 0, o, 77] = 0xFF
    else:
        p.k[pg, 0, o, 77] = float("nan")
    p.cuda()
    attn = m.Attn(p.hq, p.scale, wait_timeout_us=200000)
    ws = torch.zeros(m.moe_attn_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
    got = scores.cuda()
    m.moe_key_weights(attn, p.cache, p.seqs, p.d_q(), lse.cuda(), got, got, ws)
    x = got.cpu().numpy().astype(np.float64)[0, 0]
    assert np.isnan(x[64 + 9])
    keep = np.arange(256) != 64 + 9
    assert np.all(np.abs(x - want[0, 0])[keep] <= tol[0, 0][keep])
