"""The attention-side entry points without a GPU: the rotary table, workspace
sizes, and synchronous refusals of bad arguments (no CUDA call is reached)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import moe_speculative_verify_gb300 as m

FAKE = 1 << 40                    # never dereferenced: the call is refused first
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    m.build()
    return m.load()


def cache(**kw):
    c = m.KVCache(FAKE, FAKE, None, None, 8 * 64 * 128, 64 * 128, 128, m.KV_BF16, 10, 64, 8, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def seqs(**kw):
    s = m.Seqs(FAKE, FAKE, FAKE, 2, 4, 1)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_rope_freqs_plain_is_exact_to_48_bits():
    for rot in (16, 64, 128):
        f, mag = m.moe_rope_freqs(rot, 500000.0)
        want = 500000.0 ** (-2.0 * np.arange(rot // 2) / rot) / (2 * math.pi)
        got = f.double().sum(1).numpy()
        # hi is within half a unit of 24 bits, lo within one of what it leaves
        assert np.all(np.abs(got - want) <= want * 2.0 ** -47)
        assert mag == 1.0


def test_rope_freqs_scaled():
    lin, mag = m.moe_rope_freqs(64, kind=m.ROPE_LINEAR, factor=4.0)
    plain, _ = m.moe_rope_freqs(64)
    assert torch.allclose(lin.double().sum(1) * 4, plain.double().sum(1), rtol=2 ** -40, atol=0) and mag == 1.0
    ramp, mag = m.moe_rope_freqs(64, kind=m.ROPE_RAMP, factor=4.0, original_len=4096)
    ratio = (plain.double().sum(1) / ramp.double().sum(1)).numpy()
    assert abs(mag - (0.1 * math.log(4.0) + 1)) < 1e-6
    # fast pairs as they were, slow ones divided, one way between
    turns = plain.double().sum(1).numpy() * 4096
    assert np.allclose(ratio[turns > 64], 1) and np.allclose(ratio[turns < 0.5], 4)
    assert np.all(np.diff(ratio) >= -1e-9)
    assert m.moe_rope_freqs(0)[0].shape == (0, 2)


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=8), INVALID), (dict(rot_dim=-16), INVALID), (dict(rot_dim=256), UNSUPPORTED), (dict(base=1.0), INVALID),
    (dict(base=float("nan")), INVALID), (dict(kind=3), INVALID), (dict(kind=m.ROPE_LINEAR, factor=0.0), INVALID),
    (dict(kind=m.ROPE_RAMP, factor=2.0, original_len=0), INVALID),
    (dict(kind=m.ROPE_RAMP, factor=2.0, beta_fast=0.5, beta_slow=1.0), INVALID)])
def test_rope_freqs_refusals(lib, kw, status):
    with pytest.raises(m.MoeError) as e:
        m.moe_rope_freqs(**{"rot_dim": 64, **kw})
    assert e.value.status == status


BAD_CACHE = [
    (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID), (dict(dtype=2), INVALID), (dict(n_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), INVALID), (dict(n_kv_heads=0), INVALID),
    (dict(n_kv_heads=512), UNSUPPORTED), (dict(token_stride=124), INVALID), (dict(page_stride=0), INVALID),
    (dict(head_stride=-128), INVALID), (dict(dtype=m.KV_E4M3), INVALID)]
BAD_SEQS = [
    (dict(n_seqs=-1), INVALID), (dict(n_seqs=4097), UNSUPPORTED), (dict(kv_len=None), INVALID), (dict(block_table=None), INVALID),
    (dict(kv_len=FAKE + 2), INVALID), (dict(cu_q=None), INVALID), (dict(max_q=0), INVALID), (dict(max_pages=-1), INVALID)]


def rope_call(lib, c=None, s=None, rope=None, **kw):
    a = dict(q=FAKE, qs=64 * 128, k=FAKE, ks=1024, v=FAKE, vs=1024, pos=FAKE, T=2, hq=64, out=FAKE, os=64 * 128)
    a.update(kw)
    r = rope or m.Rope(FAKE, 128, 0, 1.0)
    return lib.moe_rope_append(C.byref(r), C.byref(c or cache()), C.byref(s or seqs()), a["q"], a["qs"], a["k"], a["ks"],
                               a["v"], a["vs"], a["pos"], a["T"], a["hq"], a["out"], a["os"], None)


def attn_call(lib, at=None, c=None, s=None, **kw):
    a = dict(q=FAKE, qs=64 * 128, mask=None, T=2, out=FAKE, lse=FAKE, ws=FAKE, n=1 << 40)
    a.update(kw)
    return lib.moe_paged_attention(C.byref(at or m.Attn(64, 0.1)), C.byref(c or cache()), C.byref(s or seqs()), a["q"],
                                   a["qs"], a["mask"], a["T"], a["out"], a["lse"], a["ws"], a["n"], None)


def weights_call(lib, at=None, c=None, s=None, **kw):
    a = dict(q=FAKE, qs=64 * 128, mask=None, T=2, lse=FAKE, decay=1.0, sc=FAKE, so=FAKE, stride=64, ws=FAKE, n=1 << 40)
    a.update(kw)
    return lib.moe_key_weights(C.byref(at or m.Attn(64, 0.1)), C.byref(c or cache()), C.byref(s or seqs()), a["q"], a["qs"],
                               a["mask"], a["T"], a["lse"], a["decay"], a["sc"], a["so"], a["stride"], a["ws"], a["n"], None)


def evict_call(lib, c=None, s=None, **kw):
    a = dict(sc=FAKE, stride=64, budget=64, recent=8, to=FAKE, tp=1, kept=FAKE, so=FAKE + 4096, nl=FAKE + 64, ws=FAKE, n=256)
    a.update(kw)
    return lib.moe_cache_evict(C.byref(c or cache()), C.byref(s or seqs()), a["sc"], a["stride"], a["budget"], a["recent"],
                               a["to"], a["tp"], a["kept"], a["so"], a["nl"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches(lib, kw, status):
    for call in (rope_call, attn_call, weights_call, evict_call):
        assert call(lib, c=cache(**kw)) == status, call.__name__


@pytest.mark.parametrize("kw,status", BAD_SEQS)
def test_bad_sequences(lib, kw, status):
    for call in (rope_call, attn_call, weights_call):
        assert call(lib, s=seqs(**kw)) == status, call.__name__
    if not set(kw) & {"cu_q", "max_q"}:
        assert evict_call(lib, s=seqs(**kw)) == status


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=FAKE + 8), dict(qs=64 * 128 - 8), dict(qs=64 * 128 + 4), dict(k=None), dict(v=None),
                                dict(ks=1016), dict(pos=None), dict(pos=FAKE + 1), dict(out=None), dict(os=8), dict(hq=0), dict(T=-1)])
def test_rope_refusals(lib, kw):
    assert rope_call(lib, **kw) == INVALID
    assert rope_call(lib, T=0) == 0
    assert rope_call(lib, T=65537) == UNSUPPORTED and rope_call(lib, hq=257) == UNSUPPORTED
    for r in (m.Rope(None, 128, 0, 1.0), m.Rope(FAKE, 24, 0, 1.0), m.Rope(FAKE, 144, 0, 1.0), m.Rope(FAKE, 64, 0, float("inf"))):
        assert rope_call(lib, rope=r) == INVALID


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=FAKE + 2), dict(qs=100), dict(mask=FAKE + 4), dict(out=None), dict(out=FAKE + 8),
                                dict(lse=FAKE + 2), dict(ws=None), dict(ws=FAKE + 128), dict(T=-1), dict(s=seqs(n_seqs=0))])
def test_attention_refusals(lib, kw):
    assert attn_call(lib, **kw) == INVALID
    assert attn_call(lib, T=0) == 0
    assert attn_call(lib, T=1 << 20) == UNSUPPORTED
    assert attn_call(lib, n=1000) == WORKSPACE


@pytest.mark.parametrize("at,status", [(m.Attn(60, 0.1), INVALID), (m.Attn(0, 0.1), INVALID), (m.Attn(64, float("nan")), INVALID),
                                       (m.Attn(64, 0.1, window=-1), INVALID), (m.Attn(512, 0.1), UNSUPPORTED)])
def test_bad_attention_shapes(lib, at, status):
    assert attn_call(lib, at=at, qs=512 * 128) == status
    assert weights_call(lib, at=at, qs=512 * 128) == status
    assert m.moe_attn_workspace_bytes(at, cache()) == 0


@pytest.mark.parametrize("kw", [dict(q=None), dict(lse=None), dict(sc=None), dict(so=None), dict(stride=0), dict(decay=float("nan")),
                                dict(ws=FAKE + 8), dict(so=FAKE + 2), dict(T=-2)])
def test_weights_refusals(lib, kw):
    assert weights_call(lib, **kw) == INVALID
    assert weights_call(lib, n=255) == WORKSPACE
    assert weights_call(lib, s=seqs(n_seqs=0), T=0) == 0


@pytest.mark.parametrize("kw", [dict(sc=None), dict(so=None), dict(so=FAKE), dict(kept=None), dict(nl=None), dict(nl=FAKE), dict(to=None),
                                dict(budget=0), dict(recent=-1), dict(recent=65), dict(tp=0), dict(budget=65), dict(stride=0), dict(ws=None)])
def test_evict_refusals(lib, kw):
    assert evict_call(lib, **kw) == INVALID
    assert evict_call(lib, n=255) == WORKSPACE
    assert evict_call(lib, s=seqs(n_seqs=0)) == 0


def test_workspace_bytes(lib):
    at = m.Attn(64, 0.1)
    assert m.moe_attn_workspace_bytes(at, cache()) > m.moe_attn_workspace_bytes(at, cache(head_dim=64)) > 256
    assert m.moe_attn_workspace_bytes(at, cache(page_size=3)) == 0


def test_binding_refuses_wrong_tensors(lib):
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    c = m.KVCache.from_tensors(k, k.clone())
    nhd = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16).permute(0, 2, 1, 3)
    n = m.KVCache.from_tensors(nhd, nhd.clone())
    assert (n.page_stride, n.head_stride, n.token_stride, n.page_size, n.n_kv_heads) == (2048, 64, 128, 16, 2)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    s = m.Seqs.from_tensors(i32(3), i32(2), i32(2, 4), 1)
    for bad in (lambda: m.KVCache.from_tensors(k, nhd), lambda: m.KVCache.from_tensors(k.float(), k.float()),
                lambda: m.KVCache.from_tensors(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn)),
                lambda: m.KVCache.from_tensors(k, k[:2]),
                lambda: m.Seqs.from_tensors(i32(2), i32(2), i32(2, 4)), lambda: m.Seqs.from_tensors(i32(3), i32(2).long(), i32(2, 4)),
                lambda: m.Rope.from_freqs(torch.zeros(8, 2).double())):
        with pytest.raises(m.MoeError):
            bad()
    at, q = m.Attn(4, 0.1), torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    out, ws, lse, sc = q.clone(), torch.zeros(512, dtype=torch.uint8), torch.zeros(2, 4), torch.zeros(2, 2, 64)
    for bad in (lambda: m.moe_paged_attention(at, c, s, q.float(), out, ws), lambda: m.moe_paged_attention(at, c, s, q, out[:1], ws),
                lambda: m.moe_paged_attention(at, c, s, q, out, ws, lse=lse.double()),
                lambda: m.moe_paged_attention(at, c, s, q, out, ws, draft_mask=i32(2)),
                lambda: m.moe_key_weights(at, c, s, q, lse, sc, sc[:, :1], ws),
                lambda: m.moe_key_weights(at, c, s, q, lse[:1], sc, sc, ws),
                lambda: m.moe_cache_evict(c, s, sc, 16, 1, i32(2, 1), i32(2, 2, 8), sc.clone(), i32(2), ws),
                lambda: m.moe_rope_append(m.Rope.from_freqs(torch.zeros(8, 2)), c, s, q, q, q, i32(2), q)):
        with pytest.raises(m.MoeError) as e:
            bad()
        assert e.value.status == INVALID
