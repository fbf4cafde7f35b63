"""Numbers that do not fit, sizes at the documented limits: recorded, refused
or answered, never left half done."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def workspace(attn, cache):
    return torch.zeros(m.moe_attn_workspace_bytes(attn, cache), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("news", [1, 6])            # few rows, and a tile of 48
@pytest.mark.parametrize("cu", ["past", "back", "first", "negative"])
def test_rows_of_a_bad_sequence_are_pad_rows(news, cu):
    """Offsets that do not fit: the sequence and those after it have no new
    tokens, and their rows are +0 and -inf as pad rows are."""
    p = ref.Problem([70, 50, 90], [news] * 3, 8, 1, 64, 16, seed=31).cuda()
    offs = {"past": [0, news, 3 * news + 1, 3 * news], "back": [0, news, news - 1, news - 1],
            "first": [3 * news + 4, 3 * news + 5, 3 * news + 6, 3 * news + 7], "negative": [-2, -1, 0, 1]}[cu]
    good = {"past": 1, "back": 1, "first": 0, "negative": 0}[cu]
    attn = m.Attn(8, p.scale, wait_timeout_us=200000)
    scores = torch.rand(3, 1, 96, generator=torch.Generator().manual_seed(1)).cuda()
    out, good_z = {}, None
    for name, c in (("good", [0, news, 2 * news, 3 * news]), ("bad", offs)):
        ws = workspace(attn, p.cache)
        o = torch.full((3 * news, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        z = torch.full((3 * news, 8), float("nan"), device="cuda")
        m.moe_paged_attention(attn, p.cache, m.Seqs.from_tensors(i32(c), p.d_kv_len, p.d_table, news), p.d_q(), o, ws, lse=z)
        assert m.moe_get_device_error(ws) == (0 if name == "good" else 1)
        sc = scores.clone()
        m.moe_key_weights(attn, p.cache, m.Seqs.from_tensors(i32(c), p.d_kv_len, p.d_table, news), p.d_q(), good_z if good_z is not None
                          else z, sc, sc, ws, decay=0.5)
        assert m.moe_get_device_error(ws) == (0 if name == "good" else 1)
        good_z = z if good_z is None else good_z
        out[name] = o, z, sc
    n = good * news
    assert torch.equal(out["bad"][0][:n], out["good"][0][:n]) and torch.equal(out["bad"][1][:n], out["good"][1][:n])
    rest = out["bad"][0][n:]
    assert torch.all(rest.view(torch.int16) == 0) and torch.all(torch.isneginf(out["bad"][1][n:]))
    assert torch.equal(out["bad"][2][:good], out["good"][2][:good])
    for b in range(good, 3):                 # no new tokens: every key's score decays
        assert torch.equal(out["bad"][2][b, :, :p.lens[b]], scores[b, :, :p.lens[b]] * 0.5)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq", [1, 4])              # few rows, and a tile
def test_window_without_limit_and_more_new_tokens_than_keys(causal, hq):
    """The largest window is none at all, also where new tokens outnumber keys."""
    p = ref.Problem([9, 20], [16, 6], hq, 1, 64, 16, seed=32).cuda()
    got = []
    for window in (0, 2 ** 31 - 1):
        attn = m.Attn(hq, p.scale, causal, window, wait_timeout_us=200000)
        ws = workspace(attn, p.cache)
        out = torch.empty((p.t, hq, 64), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((p.t, hq), device="cuda")
        m.moe_paged_attention(attn, p.cache, p.seqs, p.d_q(), out, ws, lse=lse)
        sc = torch.zeros(2, 1, 32, device="cuda")
        m.moe_key_weights(attn, p.cache, p.seqs, p.d_q(), lse, sc, sc, ws)
        assert m.moe_get_device_error(ws) == 0
        got.append((out, lse, sc))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    z = ref.attention(p, causal)[1]
    assert np.array_equal(np.isneginf(got[1][1].cpu().numpy()), np.isneginf(z))


@pytest.mark.parametrize("hq", [1, 20])             # few rows, and a tile
def test_lengths_near_2_to_31(hq):
    """The longest sequence's last keys are found; a longer length is cut to it and recorded."""
    page, dim, pages, longest, window = 128, 64, 8, 2 ** 31 - 2 ** 17, 300
    g = torch.Generator(device="cuda").manual_seed(41)
    k, v = (torch.randn(pages, 1, page, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    cache = m.KVCache.from_tensors(k, v)
    table = torch.randint(0, pages, (1, 2 ** 31 // page), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(1, hq, dim, generator=g, device="cuda").bfloat16()
    attn = m.Attn(hq, 0.125, window=window)
    places = torch.arange(longest - window, longest, device="cuda")
    rows = table[0, places // page].long()
    kk, vv = (x[rows, 0, places % page].double() for x in (k, v))
    s = q[0].double() @ kk.t() * 0.125
    want, z = torch.softmax(s, 1) @ vv, torch.logsumexp(s, 1)
    for length in (longest, 2 ** 31 - 1):
        seqs = m.Seqs.from_tensors(i32([0, 1]), i32([length]), table, hq)   # max_q picks the kernel
        ws = workspace(attn, cache)
        out = torch.empty((1, hq, dim), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((1, hq), device="cuda")
        m.moe_paged_attention(attn, cache, seqs, q, out, ws, lse=lse)
        assert m.moe_get_device_error(ws) == (0 if length == longest else 1)
        # bf16 probabilities and outputs of unit values: 2^-8 of sum p|v| and of |out|; scores' error below 2^-16
        assert bool(((out[0].double() - want).abs() <= 2.0 ** -7).all())
        assert bool(((lse[0].double() - z).abs() <= 2.0 ** -14).all())
        scores = torch.rand(1, 1, 256, device="cuda")
        got = scores.clone()
        m.moe_key_weights(attn, cache, seqs, q, lse, got, got, ws, decay=0.5)
        assert m.moe_get_device_error(ws) == (0 if length == longest else 1)
        assert torch.equal(got, scores * 0.5)


@pytest.mark.parametrize("n,h", [(4096, 16), (2100, 32), (300, 256)])
def test_evict_of_many_pairs(n, h):
    """More than 65,535 (sequence, kv head) pairs."""
    page, dim, length, budget = 16, 64, 5, 2
    g = torch.Generator(device="cuda").manual_seed(33)
    k = torch.randn(2 * n, h, page, dim, generator=g, device="cuda").bfloat16()
    v = torch.randn(2 * n, h, page, dim, generator=g, device="cuda").bfloat16()
    k0, v0 = k.clone(), v.clone()
    cache = m.KVCache.from_tensors(k, v)
    ar = torch.arange(n, dtype=torch.int32, device="cuda")
    seqs = m.Seqs.from_tensors(None, torch.full((n,), length, dtype=torch.int32, device="cuda"), ar[:, None].contiguous())
    scores = torch.rand(n, h, 8, generator=g, device="cuda")
    kept = torch.full((n, h, budget), -9, dtype=torch.int32, device="cuda")
    out, new_len = torch.zeros_like(scores), torch.zeros_like(ar)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    m.moe_cache_evict(cache, seqs, scores, budget, 1, (ar + n)[:, None].contiguous(), kept, out, new_len, ws)
    assert m.moe_get_device_error(ws) == 0
    best = scores[:, :, :length - 1].argmax(2, keepdim=True)
    want = torch.cat([best, torch.full_like(best, length - 1)], 2)
    assert torch.equal(kept.long(), want) and bool((new_len == budget).all())
    for x, x0 in ((k, k0), (v, v0)):
        rows = torch.gather(x0[:n], 2, want[..., None].expand(-1, -1, -1, dim))
        assert torch.equal(x[n:, :, :budget], rows) and torch.equal(x[:n], x0[:n]) and torch.equal(x[n:, :, budget:], x0[n:, :, budget:])


def test_evict_moves_a_bad_page_as_zeros():
    """A source page outside the cache reads as zeros; a destination outside is
    not written; both are recorded."""
    p = ref.Problem([40], [0], 2, 1, 64, 16, seed=34).cuda()
    total = p.d_k.shape[0]
    k, v = (torch.cat([x, torch.full_like(x[:3], 7.0)]) for x in (p.d_k, p.d_v))
    k0 = k.clone()
    cache = m.KVCache.from_tensors(k, v)
    table = p.d_table.clone()
    table[0, 1] = 1 << 29
    kept = torch.zeros(1, 1, 48, dtype=torch.int32, device="cuda")
    new_len = i32([0])
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    scores = torch.rand(1, 1, 48, device="cuda")
    m.moe_cache_evict(cache, m.Seqs.from_tensors(None, p.d_kv_len, table), scores, 48, 0, i32([[total, total + 1, -1]]), kept,
                      torch.empty_like(scores), new_len, ws)
    assert m.moe_get_device_error(ws) == 1
    assert int(new_len[0]) == 40 and kept[0, 0].tolist() == list(range(40)) + [-1] * 8
    for x, x0 in ((k, p.d_k), (v, p.d_v)):
        assert torch.equal(x[total], x0[int(p.table[0, 0])])
        assert bool((x[total + 1] == 0).all()) and bool((x[total + 2] == 7.0).all())
    assert torch.equal(k[:total].view(torch.int16), k0[:total].view(torch.int16))


def test_rope_with_offsets_that_run_backwards():
    """A token that two sequences claim belongs to the first; the sequences from
    the first bad offset on have none."""
    p = ref.Problem([40, 30, 50], [5, 0, 3], 8, 2, 64, 16, seed=35).cuda()
    freqs, mag = m.moe_rope_freqs(64)
    rope = m.Rope.from_freqs(freqs.cuda(), False, mag)
    got = []
    for offs in ([0, 5, 5, 5], [0, 5, 3, 8], [0, 5, 9, 8]):
        k, v = p.d_k.clone(), p.d_v.clone()
        q_out = torch.full((8, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        seqs = m.Seqs.from_tensors(i32(offs), p.d_kv_len, p.d_table, 8)
        m.moe_rope_append(rope, m.KVCache.from_tensors(k, v), seqs, p.d_qkv[:, :8], p.d_qkv[:, 8:10], p.d_qkv[:, 10:],
                          torch.arange(8, dtype=torch.int32, device="cuda"), q_out)
        got.append([x.view(torch.int16) for x in (k, v, q_out)])
    assert bool((got[0][2][5:] == 0).all())
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("wreck,code", [("none", 0), ("page", 1), ("length", 1), ("offsets", 1), ("fewer keys", 0)])
def test_rope_records_what_it_could_not_store(wreck, code):
    p = ref.Problem([40, 30], [5, 3], 8, 2, 64, 16, seed=36).cuda()
    freqs, mag = m.moe_rope_freqs(64)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    table, kv_len, cu = p.d_table.clone(), p.d_kv_len.clone(), p.d_cu.clone()
    if wreck == "page":
        table[1, 1] = p.d_k.shape[0]
    elif wreck == "length":
        kv_len[0] = 16 * table.shape[1] + 1
        table[:] = 0
    elif wreck == "offsets":
        cu[2] = 9
    elif wreck == "fewer keys":
        kv_len[1] = 2
    seqs = m.Seqs.from_tensors(cu, kv_len, table, 5)
    q_out = torch.empty(8, 8, 64, dtype=torch.bfloat16, device="cuda")
    for rope in (m.Rope.from_freqs(freqs.cuda(), False, mag, ws), m.Rope.from_freqs(freqs.cuda(), False, mag)):
        m.moe_rope_append(rope, p.cache, seqs, p.d_qkv[:, :8], p.d_qkv[:, 8:10], p.d_qkv[:, 10:],
                          torch.arange(8, dtype=torch.int32, device="cuda"), q_out)
        assert m.moe_get_device_error(ws) == code
        code = 0                             # cleared by the read, and not recorded without a word
