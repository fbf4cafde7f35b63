"""Rotary append and eviction against 64-bit (exact) implementations.

Rotary tolerances: bf16 stores within half a unit (8 significant bits: 2^-8 relative) of the exact
value, e4m3 codes within half a code step (2^-4 relative, 2^-10 below the
normal codes), plus the fp32 arithmetic: the angle's error (2^-23 turns, the
fraction's two roundings) and cos, sin, products and sum at 2^-22 of |x1| + |x2|."""
import math

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


def _bytes(x):
    return x.contiguous().view(torch.uint8).cpu()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,rot,inter,kind", [(128, 128, False, m.ROPE_PLAIN), (128, 64, True, m.ROPE_RAMP),
                                                (128, 48, False, m.ROPE_LINEAR), (64, 64, True, m.ROPE_PLAIN),
                                                (64, 16, False, m.ROPE_RAMP), (64, 0, False, m.ROPE_PLAIN)])
@pytest.mark.parametrize("lens,news,hq,hkv,page,layout,pads", [
    ([1], [1], 8, 8, 16, "hnd", (0, 0)),
    ([40, 3, 0, 130], [8, 1, 0, 5], 24, 3, 32, "nhd", (1, 2)),
    ([70, 5], [70, 9], 12, 1, 64, "hnd", (0, 0)),         # the second holds fewer keys than new tokens
])
def test_rope_append(dtype, dim, rot, inter, kind, lens, news, hq, hkv, page, layout, pads):
    p = ref.Problem(lens, news, hq, hkv, dim, page, dtype, layout, pads, seed=dim + rot).cuda()
    freqs, mag = m.moe_rope_freqs(rot, kind=kind, factor=4.0, original_len=64)
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(0, 1 << 24, (p.t,), generator=g, dtype=torch.int32)
    pos[0] = (1 << 24) - 1
    rope = m.Rope.from_freqs(freqs.cuda(), inter, mag)
    before_k, before_v = p.d_k.clone(), p.d_v.clone()
    qd, kd, vd = p.d_qkv[:, :hq], p.d_qkv[:, hq:hq + hkv], p.d_qkv[:, hq + hkv:]
    q_out = torch.full((p.t, hq, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    m.moe_rope_append(rope, p.cache, p.seqs, qd, kd, vd, pos.cuda(), q_out)
    torch.cuda.synchronize()

    def near(got, want, spread, eps, floor):
        bad = ~(np.abs(got - want) <= eps * np.abs(want) + floor + spread * 2.0 ** -20)
        assert not bad.any(), (got[bad][:4], want[bad][:4])

    def both(x):
        want = ref.rope(x, pos, freqs, mag, inter)
        a = np.abs(x.float().numpy()).max(axis=2, keepdims=True) * 2 * mag
        return want, np.broadcast_to(a, want.shape)

    wq, sq = both(p.qkv[:, :hq])
    live = np.zeros(p.t, bool)
    live[int(p.cu[0]):int(p.cu[-1])] = True
    got = q_out.float().cpu().numpy().astype(np.float64)
    near(got[live], wq[live], sq[live], 2.0 ** -8 * 1.001, 1e-38)
    assert np.all(got[~live] == 0)
    wk, sk = both(p.qkv[:, hq:hq + hkv])
    wv = p.qkv[:, hq + hkv:].float().numpy().astype(np.float64)
    stored = torch.zeros(p.d_k.shape[0], page, dtype=torch.bool)
    for b in range(len(lens)):
        for i in range(news[b]):
            at = lens[b] - news[b] + i
            if at < 0:
                continue
            pg, off, t = int(p.table[b, at // page]), at % page, int(p.cu[b]) + i
            stored[pg, off] = True
            for cache, want, spread, scale in ((p.d_k, wk[t], sk[t], p.k_scale), (p.d_v, wv[t], 0 * sk[t], p.v_scale)):
                x = cache[pg, :, off].float().cpu().numpy().astype(np.float64)
                if dtype == "bf16":
                    near(x, want, spread, 2.0 ** -8 * 1.001, 1e-38)
                else:
                    s = scale.numpy().astype(np.float64)[:, None]
                    near(x, np.clip(want / s, -448, 448), spread / s, 2.0 ** -4 * 1.001, 2.0 ** -10)
    # nothing else of the cache is touched
    keep = ~stored
    for a, c in ((p.d_k, before_k), (p.d_v, before_v)):
        a, c = a.permute(0, 2, 1, 3)[keep.cuda()], c.permute(0, 2, 1, 3)[keep.cuda()]
        assert torch.equal(_bytes(a), _bytes(c))
    # in place: the same q
    q2 = p.d_qkv.clone()
    m.moe_rope_append(rope, p.cache, p.seqs, q2[:, :hq], kd, vd, pos.cuda(), q2[:, :hq])
    assert torch.equal(q2[:, :hq], q_out) and torch.equal(q2[:, hq:], p.d_qkv[:, hq:])


def test_rope_drops_what_has_no_place():
    """Bad pages and places past the table are not written."""
    p = ref.Problem([40, 20], [2, 2], 8, 2, 64, 16, seed=2).cuda()
    freqs, mag = m.moe_rope_freqs(64)
    table, kv_len = p.d_table.clone(), p.d_kv_len.clone()
    table[0, 2] = p.d_k.shape[0]             # one past the end
    kv_len[1] = 10 ** 6
    seqs = m.Seqs.from_tensors(p.d_cu, kv_len, table, 2)
    before = p.d_k.clone(), p.d_v.clone()
    q_out = torch.empty(4, 8, 64, dtype=torch.bfloat16, device="cuda")
    m.moe_rope_append(m.Rope.from_freqs(freqs.cuda()), p.cache, seqs, p.d_qkv[:, :8], p.d_qkv[:, 8:10], p.d_qkv[:, 10:],
                      torch.zeros(4, dtype=torch.int32, device="cuda"), q_out)
    torch.cuda.synchronize()
    assert torch.equal(_bytes(p.d_k), _bytes(before[0])) and torch.equal(_bytes(p.d_v), _bytes(before[1]))
    assert torch.equal(q_out, p.d_qkv[:, :8])


def run_evict(p, scores, budget, recent, extra_pages=0):
    n = len(p.lens)
    to_pages = -(-budget // p.page) + extra_pages
    total = p.k.shape[0]
    shape = list(p.d_k.shape)
    shape[0] = total + n * to_pages
    def grow(x):
        raw = torch.zeros([shape[0], shape[2], shape[1], shape[3]] if x.stride(1) < x.stride(2) else shape,
                          dtype=torch.uint8 if p.dtype == "e4m3" else torch.bfloat16, device="cuda")
        raw = raw.permute(0, 2, 1, 3) if x.stride(1) < x.stride(2) else raw
        raw[:total] = x.view(torch.uint8) if p.dtype == "e4m3" else x
        return raw
    k, v = grow(p.d_k), grow(p.d_v)
    cache = m.KVCache.from_tensors(k, v, getattr(p, "d_k_scale", None), getattr(p, "d_v_scale", None))
    g = torch.Generator().manual_seed(11)
    to = (total + torch.randperm(n * to_pages, generator=g).view(n, to_pages)).int()
    kept = torch.full((n, p.hkv, budget), -9, dtype=torch.int32, device="cuda")
    so = torch.full_like(scores, -5.0)
    new_len = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    k0, v0 = k.clone(), v.clone()
    m.moe_cache_evict(cache, p.seqs, scores, budget, recent, to.cuda(), kept, so, new_len, ws)
    torch.cuda.synchronize()
    assert m.moe_get_device_error(ws) == 0
    return k, v, k0, v0, to, kept.cpu(), so.cpu(), new_len.cpu()


def bits(x):
    return x.contiguous().view(torch.int16 if x.dtype == torch.bfloat16 else torch.uint8)


@pytest.mark.parametrize("dtype,dim,layout,page", [("bf16", 128, "hnd", 64), ("e4m3", 64, "nhd", 16), ("bf16", 64, "nhd", 128),
                                                   ("e4m3", 128, "hnd", 32)])
@pytest.mark.parametrize("lens,budget,recent", [([300, 0, 100, 101], 100, 10), ([5000], 64, 64), ([5000, 1], 1, 0), ([1000], 999, 0),
                                                ([700, 65, 64], 64, 1)])
@pytest.mark.parametrize("values", ["spread", "ties", "special"])
def test_evict(dtype, dim, layout, page, lens, budget, recent, values):
    p = ref.Problem(lens, [0] * len(lens), 6, 3, dim, page, dtype, layout, seed=len(lens)).cuda()
    g = torch.Generator().manual_seed(12)
    scores = torch.rand(len(lens), 3, max(lens) + 7, generator=g).pow(-0.7)
    if values == "ties":
        scores = scores.mul(2).round().clamp(max=4)
    if values == "special":
        pick = torch.randint(0, 8, scores.shape, generator=g)
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -1e-45)):
            scores[pick == i] = x
    k, v, k0, v0, to, kept, so, new_len = run_evict(p, scores.cuda(), budget, recent, extra_pages=1)
    want = ref.evict(scores, lens, budget, recent)
    written = torch.zeros(k.shape[0], page, 3, dtype=torch.bool)
    for b, n in enumerate(lens):
        assert int(new_len[b]) == min(n, budget)
        for h in range(3):
            w = want[b][h]
            assert kept[b, h].tolist() == w + [-1] * (budget - len(w))
            assert torch.equal(so[b, h, :len(w)].view(torch.int32), scores[b, h, w].view(torch.int32))
            assert torch.all(so[b, h, len(w):] == -5.0)
            if w:
                j, r = torch.tensor(w), torch.arange(len(w))
                src, dst = p.table[b, j // page].long(), to[b, r // page].long()
                for x, x0 in ((k, k0), (v, v0)):
                    assert torch.equal(bits(x[dst.cuda(), h, (r % page).cuda()]), bits(x0[src.cuda(), h, (j % page).cuda()]))
                written[dst, r % page, h] = True
    for x, x0 in ((k, k0), (v, v0)):         # nothing else moved
        rest = (~written).cuda()
        assert torch.equal(bits(x.permute(0, 2, 1, 3)[rest]), bits(x0.permute(0, 2, 1, 3)[rest]))


def test_evict_records_bad_pages():
    p = ref.Problem([100], [0], 2, 1, 64, 16, seed=3).cuda()
    p.d_table[0, 1] = -3
    scores = torch.rand(1, 1, 100, device="cuda")
    kept = torch.zeros(1, 1, 50, dtype=torch.int32, device="cuda")
    new_len = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    to = torch.full((1, 4), 1 << 29, dtype=torch.int32, device="cuda")
    m.moe_cache_evict(p.cache, p.seqs, scores, 50, 0, to, kept, torch.empty_like(scores), new_len, ws)
    assert m.moe_get_device_error(ws) == 1


def test_attention_after_eviction():
    """The kept keys alone carry the attention afterwards."""
    p = ref.Problem([400, 250], [0, 0], 8, 2, 128, 64, seed=13).cuda()
    scores = torch.rand(2, 2, 400, generator=torch.Generator().manual_seed(1))
    k, v, _, _, to, kept, _, new_len = run_evict(p, scores.cuda(), 128, 16)
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(2)).bfloat16()
    cache = m.KVCache.from_tensors(k, v)
    seqs = m.Seqs.from_tensors(torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), new_len.cuda(), to.cuda(), 1)
    attn = m.Attn(8, 128 ** -0.5, causal=False)
    ws = torch.zeros(m.moe_attn_workspace_bytes(attn, cache), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    m.moe_paged_attention(attn, cache, seqs, q.cuda(), out, ws)
    assert m.moe_get_device_error(ws) == 0
    for b in range(2):
        for hd in range(8):
            j = kept[b, hd // 4].numpy()
            kk, vv = p.rows(p.k, None, b, hd // 4)[j], p.rows(p.v, None, b, hd // 4)[j]
            s = kk @ q[b, hd].double().numpy() * 128 ** -0.5
            e = np.exp(s - s.max())
            want, mag = e @ vv / e.sum(), e @ np.abs(vv) / e.sum()
            # the tolerance of the attention tests, with a score's error bound of 1e-4
            assert np.all(np.abs(out[b, hd].double().cpu().numpy() - want) <= mag * (2.0 ** -7 + 2e-4 + 2.0 ** -20))
    assert math.isfinite(float(out.float().sum()))
