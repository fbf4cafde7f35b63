"""Rows of a latent cache written and read back, against 64 bits.

Tolerances: a bf16 store is within 2^-8 of the value, an e4m3 code within 2^-4
(2^-10 below the normal codes); the normalisation's fp32 sum, root and products
add less than 2^-18 of the value (512 squares summed in pieces: 2^-24 each of at most
80 additions in a row, halved by the root); rotary parts as in test_gpu_rope_evict.py."""
import numpy as np
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


def raw(x):
    return x.contiguous().view(torch.uint8).cpu()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("latent,inter,kind", [(512, True, m.ROPE_PLAIN), (256, False, m.ROPE_RAMP)])
@pytest.mark.parametrize("lens,news,heads,page,store,pads", [
    ([1], [1], 8, 16, "rows", (0, 0)),
    ([40, 3, 0, 130], [8, 1, 0, 5], 24, 32, "split", (1, 2)),
    ([70, 5], [70, 9], 12, 64, "rows", (0, 0)),               # the second holds fewer rows than new tokens
    ([200], [200], 3, 128, "split", (3, 0)),
])
def test_append(dtype, norm, latent, inter, kind, lens, news, heads, page, store, pads):
    p = ref.Problem(lens, news, heads, latent, page, dtype, store, pads, seed=latent + heads)
    freqs, mag = m.moe_rope_freqs(ROT, kind=kind, factor=4.0, original_len=64)
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(0, 1 << 24, (p.t,), generator=g, dtype=torch.int32)
    pos[0] = (1 << 24) - 1
    kv = torch.randn(p.t, latent + ROT + 8, generator=g).bfloat16().cuda()[:, :latent + ROT]
    gamma = (1 + 0.3 * torch.randn(latent, generator=g)).cuda() if norm else None
    q = torch.randn(p.t, heads, 32 + ROT, generator=g).bfloat16().cuda()[..., 32:]
    wide = torch.full((p.t, heads, latent + ROT), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    rope = m.Rope.from_freqs(freqs.cuda(), inter, mag, ws)
    before = p.latent.clone(), p.rope.clone()
    m.moe_latent_append(rope, p.cache, p.seqs, kv, q, pos.cuda(), wide[..., latent:], gamma=gamma, eps=1e-5)
    assert m.moe_get_device_error(ws) == 0
    assert torch.isnan(wide[..., :latent]).all()              # beside the rotary parts nothing is written

    def near(got, want, spread, eps, floor=0.0):
        bad = ~((got - want).abs() <= eps * want.abs() + floor + spread * 2.0 ** -20)
        assert not bad.any(), (got[bad][:4], want[bad][:4])

    spread = lambda x: x.double().cpu().abs().amax(2, keepdim=True) * 2 * mag
    wq, live = ref.turn(q, pos, freqs, mag, inter), torch.zeros(p.t, dtype=torch.bool)
    for b, n in enumerate(news):
        live[p.cu[b]:p.cu[b] + n] = True
    near(wide[live.cuda()][..., latent:].double().cpu(), wq[live], spread(q)[live], 2.0 ** -8)
    assert bool(torch.all(wide[~live.cuda()][..., latent:].contiguous().view(torch.int16) == 0))
    x = kv[:, :latent].double().cpu()
    if norm:
        x = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5) * gamma.double().cpu()
    key = ref.turn(kv[:, None, latent:], pos, freqs, mag, inter)[:, 0]
    ks = spread(kv[:, None, latent:])[:, 0]
    stored = torch.zeros(p.latent.shape[:2], dtype=torch.bool)
    gl, gr = p.latent.float().double().cpu() * 2.0 ** p.exp, p.rope.double().cpu()
    for b, n in enumerate(news):
        for i in range(n):
            j = lens[b] - n + i
            if j < 0:
                continue
            pg, sl, t = int(p.table[b, j // page]), j % page, p.cu[b] + i
            stored[pg, sl] = True
            eps, floor = (2.0 ** -8, 0.0) if dtype == "bf16" else (2.0 ** -4, 2.0 ** (p.exp - 10))
            near(gl[pg, sl], x[t].clamp(-448 * 2.0 ** p.exp, 448 * 2.0 ** p.exp) if dtype == "e4m3" else x[t],
                 x[t].abs(), eps + 2.0 ** -18, floor)
            near(gr[pg, sl], key[t], ks[t], 2.0 ** -8)
    for now, old in zip((p.latent, p.rope), before):          # every other slot keeps its bytes
        assert torch.equal(raw(now[~stored.cuda()]), raw(old[~stored.cuda()]))


def test_append_in_place_and_bad_places():
    """q_out may be q_rope itself; tokens without a place are recorded, and the others stored."""
    p = ref.Problem([40, 100], [3, 2], 5, 256, 32, seed=4)
    freqs, mag = m.moe_rope_freqs(ROT)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    rope = m.Rope.from_freqs(freqs.cuda(), False, mag, ws)
    kv = torch.randn(p.t, 256 + ROT, device="cuda").bfloat16()
    q = torch.randn(p.t, 5, ROT, device="cuda").bfloat16()
    pos = torch.arange(p.t, dtype=torch.int32, device="cuda") * 1000
    apart = torch.empty_like(q)
    p.d_table[1, 3] = -1                                      # the page of the second sequence's new tokens
    before = p.latent.clone()
    m.moe_latent_append(rope, p.cache, p.seqs, kv, q, pos, apart)
    assert m.moe_get_device_error(ws) == 1
    m.moe_latent_append(rope, p.cache, p.seqs, kv, q, pos, q)
    assert m.moe_get_device_error(ws) == 1 and torch.equal(q, apart)
    j = torch.arange(37, 40, device="cuda")
    pg = p.d_table[0][j // 32].long()
    assert torch.equal(p.latent[pg, j % 32], kv[:3, :256])    # without gamma latents are stored as they are
    rest = torch.ones(p.latent.shape[:2], dtype=torch.bool, device="cuda")
    rest[pg, j % 32] = False
    assert torch.equal(raw(p.latent[rest]), raw(before[rest]))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 0.0, 3e38])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_append_of_extreme_rows(dtype, value):
    """A row of zeros stays zeros, one with NaN is NaN under the norm, and no row reaches another."""
    p = ref.Problem([64], [3], 1, 256, 64, dtype, seed=5)
    freqs, mag = m.moe_rope_freqs(ROT)
    rope = m.Rope.from_freqs(freqs.cuda(), False, mag)
    kv = torch.randn(3, 256 + ROT, device="cuda").bfloat16()
    clean = kv.clone()
    kv[1, :256] = 0.0
    if value:
        kv[1, 7] = value
    q = torch.randn(3, 1, ROT, device="cuda").bfloat16()
    pos, gamma = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(256, device="cuda")
    m.moe_latent_append(rope, p.cache, p.seqs, clean, q, pos, torch.empty_like(q), gamma=gamma)
    pg = int(p.table[0, 0])
    want = raw(p.latent[pg, 61:64])
    m.moe_latent_append(rope, p.cache, p.seqs, kv, q, pos, torch.empty_like(q), gamma=gamma)
    got = p.latent[pg, 61:64].float()
    assert torch.equal(raw(p.latent[pg, 61:64])[[0, 2]], want[[0, 2]])
    if value == 0.0:
        assert bool(torch.all(got[1] == 0))
    elif value != value:
        assert bool(torch.isnan(got[1]).all())
    # (an infinite sum of squares makes finite elements 0; infinite ones NaN)
    else:
        assert bool(torch.all(got[1][torch.arange(256) != 7] == 0))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,latent,page,store", [([1], 512, 16, "rows"), ([63, 0, 130, 5], 256, 32, "split"),
                                                    ([700, 1, 333], 512, 64, "split"), ([2000], 512, 128, "rows")])
@pytest.mark.parametrize("form", ["tight", "gaps", "short"])
def test_gather(dtype, lens, latent, page, store, form):
    """Exactly the values cached; rows of no sequence, and rows past a sequence's length, are +0."""
    p = ref.Problem(lens, [0] * len(lens), 1, latent, page, dtype, store, seed=sum(lens), scale_log2=-7)
    at, rows = [4 if form == "gaps" else 0], 0
    for n in lens:
        at.append(at[-1] + (n + 3 if form == "gaps" else max(n - 2, 0) if form == "short" else n))
    rows = at[-1] + (6 if form == "gaps" else 0)
    wide = torch.full((rows, latent + ROT + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    m.moe_latent_gather(p.cache, p.seqs, i32(at), wide[:, :latent + ROT], ws)
    assert m.moe_get_device_error(ws) == 0
    assert bool(torch.isnan(wide[:, latent + ROT:]).all())
    want = torch.zeros(rows, latent + ROT, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        k = min(n, at[b + 1] - at[b])
        lat, rot = p.rows(b)
        want[at[b]:at[b] + k] = torch.cat([lat, rot], 1)[:k]
    got = wide[:, :latent + ROT]
    assert torch.equal(got.double(), want)


def test_gather_of_numbers_that_do_not_fit():
    p = ref.Problem([100, 70, 40], [0] * 3, 1, 256, 32, seed=6)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.full((210, 256 + ROT), float("nan"), dtype=torch.bfloat16, device="cuda")
    m.moe_latent_gather(p.cache, p.seqs, i32([0, 100, 170, 210]), out, ws)
    good = out.clone()
    assert m.moe_get_device_error(ws) == 0
    for cu, rows in (([0, 100, 90, 130], 100), ([0, 100, 211, 211], 100), ([-1, 100, 170, 210], 0)):
        out.fill_(float("nan"))
        m.moe_latent_gather(p.cache, p.seqs, i32(cu), out, ws)
        assert m.moe_get_device_error(ws) == 1
        assert torch.equal(out[:rows], good[:rows]) and torch.all(out[rows:].view(torch.int16) == 0)
    p.d_table[1, 1] = 1 << 29                                 # a page outside the cache reads as zeros
    m.moe_latent_gather(p.cache, p.seqs, i32([0, 100, 170, 210]), out, ws)
    assert m.moe_get_device_error(ws) == 1
    good[132:164] = 0
    assert torch.equal(out, good)
    # NaN codes read back as NaN
    q = ref.Problem([20], [0], 1, 256, 32, "e4m3", seed=6)
    q.latent.view(torch.uint8)[int(q.table[0, 0]), 3, 9] = 0x7F
    o = torch.zeros(20, 256 + ROT, dtype=torch.bfloat16, device="cuda")
    m.moe_latent_gather(q.cache, q.seqs, i32([0, 20]), o, ws)
    assert torch.isnan(o[3, 9]) and int(torch.isnan(o).sum()) == 1
