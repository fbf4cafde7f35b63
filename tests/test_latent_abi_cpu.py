"""The latent-cache entry points without a GPU: workspace sizes and synchronous
refusals of bad arguments (no CUDA call is reached)."""
import ctypes as C

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
    c = m.LatentCache(FAKE, FAKE, 64 * 576, 576, 64 * 576, 576, m.KV_BF16, 0, 10, 64, 512)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def seqs(**kw):
    s = m.Seqs(FAKE, FAKE, FAKE, 2, 4, 1)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


BAD_CACHE = [
    (dict(latent=None), INVALID), (dict(rope=FAKE + 8), INVALID), (dict(dtype=2), INVALID), (dict(n_pages=0), INVALID),
    (dict(n_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=256), UNSUPPORTED), (dict(latent_dim=0), INVALID), (dict(latent_dim=384), UNSUPPORTED),
    (dict(latent_token_stride=580), INVALID), (dict(latent_token_stride=504), INVALID), (dict(rope_token_stride=56), INVALID),
    (dict(latent_page_stride=0), INVALID), (dict(rope_page_stride=-64), INVALID),
    (dict(dtype=m.KV_E4M3, scale_log2=8), UNSUPPORTED), (dict(dtype=m.KV_E4M3, scale_log2=-65), UNSUPPORTED),
    (dict(dtype=m.KV_E4M3, latent_token_stride=520), INVALID)]
BAD_SEQS = [
    (dict(n_seqs=-1), INVALID), (dict(n_seqs=4097), UNSUPPORTED), (dict(kv_len=None), INVALID), (dict(block_table=None), INVALID),
    (dict(kv_len=FAKE + 2), INVALID), (dict(max_pages=-1), INVALID)]
BAD_QUERIES = [(dict(cu_q=None), INVALID), (dict(max_q=0), INVALID)]


def append(lib, c=None, s=None, rope=None, **kw):
    a = dict(kv=FAKE, kvs=576, gamma=FAKE, eps=1e-6, q=FAKE, qt=64 * 192, qh=192, pos=FAKE, T=2, h=64, o=FAKE, ot=64 * 576, oh=576)
    a.update(kw)
    r = rope or m.Rope(FAKE, 64, 0, 1.0)
    return lib.moe_latent_append(C.byref(r), C.byref(c or cache()), C.byref(s or seqs()), a["kv"], a["kvs"], a["gamma"], a["eps"],
                                 a["q"], a["qt"], a["qh"], a["pos"], a["T"], a["h"], a["o"], a["ot"], a["oh"], None)


def attention(lib, at=None, c=None, s=None, **kw):
    a = dict(q=FAKE, qs=64 * 576, draft=None, T=2, out=FAKE, lse=FAKE, ws=FAKE, n=1 << 40)
    a.update(kw)
    return lib.moe_latent_attention(C.byref(at or m.Attn(64, 0.1)), C.byref(c or cache()), C.byref(s or seqs()), a["q"], a["qs"],
                                    a["draft"], a["T"], a["out"], a["lse"], a["ws"], a["n"], None)


def gather(lib, c=None, s=None, **kw):
    a = dict(cu=FAKE, N=5, out=FAKE, os=576, ws=FAKE, n=256)
    a.update(kw)
    return lib.moe_latent_gather(C.byref(c or cache()), C.byref(s or seqs()), a["cu"], a["N"], a["out"], a["os"], a["ws"], a["n"], None)


def expanded(lib, at=None, s=None, **kw):
    a = dict(cu=FAKE, N=9, D=128, q=FAKE, qs=64 * 192, k=FAKE, kt=64 * 256, kh=256, r=FAKE, rs=576, v=FAKE, vt=64 * 256, vh=256, T=2,
             out=FAKE, lse=FAKE, ws=FAKE, n=1 << 40)
    a.update(kw)
    return lib.moe_expanded_attention(C.byref(at or m.Attn(64, 0.1)), C.byref(s or seqs()), a["cu"], a["N"], a["D"], a["q"], a["qs"],
                                      a["k"], a["kt"], a["kh"], a["r"], a["rs"], a["v"], a["vt"], a["vh"], a["T"], a["out"],
                                      a["lse"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_bad_caches(lib, kw, status):
    c = cache(**kw)
    assert append(lib, c) == status and attention(lib, None, c) == status and gather(lib, c) == status


@pytest.mark.parametrize("kw,status", BAD_SEQS)
def test_bad_sequences(lib, kw, status):
    s = seqs(**kw)
    assert append(lib, None, s) == status and attention(lib, None, None, s) == status and gather(lib, None, s) == status
    if "block_table" not in kw and "max_pages" not in kw:     # (the expanded form has no pages)
        assert expanded(lib, None, s) == status


@pytest.mark.parametrize("kw,status", BAD_QUERIES)
def test_bad_queries(lib, kw, status):
    s = seqs(**kw)
    assert append(lib, None, s) == status and attention(lib, None, None, s) == status and expanded(lib, None, s) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kv=None), INVALID), (dict(kvs=568), INVALID), (dict(kvs=580), INVALID), (dict(gamma=FAKE + 4), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(q=FAKE + 2), INVALID), (dict(qt=0), INVALID),
    (dict(qh=60), INVALID), (dict(qh=32), INVALID), (dict(pos=None), INVALID), (dict(T=-1), INVALID), (dict(T=65537), UNSUPPORTED),
    (dict(h=0), INVALID), (dict(h=257), UNSUPPORTED), (dict(o=None), INVALID), (dict(ot=1 << 33), INVALID), (dict(oh=-64), INVALID)])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


@pytest.mark.parametrize("rope", [m.Rope(None, 64, 0, 1.0), m.Rope(FAKE, 32, 0, 1.0), m.Rope(FAKE, 128, 0, 1.0),
                                  m.Rope(FAKE, 64, 0, float("inf")), m.Rope(FAKE, 64, 0, 1.0, FAKE + 1)])
def test_append_refuses_rotations(lib, rope):
    assert append(lib, rope=rope) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(qs=64 * 512), INVALID), (dict(qs=64 * 576 + 4), INVALID), (dict(draft=FAKE + 4), INVALID),
    (dict(T=-1), INVALID), (dict(T=65537), UNSUPPORTED), (dict(out=None), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(ws=None), INVALID), (dict(ws=FAKE + 64), INVALID), (dict(n=1000), WORKSPACE)])
def test_attention_refusals(lib, kw, status):
    assert attention(lib, **kw) == status


@pytest.mark.parametrize("at,status", [
    (m.Attn(0, 0.1), INVALID), (m.Attn(257, 0.1), UNSUPPORTED), (m.Attn(8, float("nan")), INVALID), (m.Attn(8, 0.1, True, -1), INVALID)])
def test_bad_attention_settings(lib, at, status):
    assert attention(lib, at, qs=1 << 20) == status and expanded(lib, at, qs=1 << 20) == status
    assert m.moe_latent_workspace_bytes(at, cache()) == 0 and m.moe_expanded_workspace_bytes(at, 128) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(cu=None), INVALID), (dict(N=-1), INVALID), (dict(N=(1 << 31) - 1), UNSUPPORTED), (dict(out=None), INVALID),
    (dict(os=568), INVALID), (dict(os=578), INVALID),
    (dict(ws=None), INVALID), (dict(n=255), WORKSPACE)])
def test_gather_refusals(lib, kw, status):
    assert gather(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(cu=None), INVALID), (dict(N=-1), INVALID), (dict(N=0), INVALID), (dict(D=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(qs=64 * 128), INVALID), (dict(k=FAKE + 8), INVALID), (dict(kt=0), INVALID), (dict(kh=64), INVALID),
    (dict(kh=132), INVALID), (dict(r=None), INVALID), (dict(rs=32), INVALID), (dict(v=None), INVALID), (dict(vt=-128), INVALID),
    (dict(vh=1 << 32), INVALID), (dict(T=65537), UNSUPPORTED), (dict(out=FAKE + 2), INVALID), (dict(lse=FAKE + 1), INVALID),
    (dict(ws=None), INVALID), (dict(n=100), WORKSPACE)])
def test_expanded_refusals(lib, kw, status):
    assert expanded(lib, **kw) == status


def test_nothing_to_do(lib):
    assert append(lib, T=0) == 0 and attention(lib, T=0) == 0 and gather(lib, N=0) == 0 and expanded(lib, T=0) == 0
    none = seqs(n_seqs=0)
    assert attention(lib, None, None, none) == INVALID and gather(lib, None, none) == INVALID and expanded(lib, None, none) == INVALID


def test_workspaces():
    at = m.Attn(64, 0.1)
    small, large = (m.moe_latent_workspace_bytes(at, cache(latent_dim=d)) for d in (256, 512))
    assert 0 < small < large and m.moe_latent_workspace_bytes(at, cache(latent_dim=128)) == 0
    assert 0 < m.moe_expanded_workspace_bytes(at, 64) < m.moe_expanded_workspace_bytes(at, 128)
    assert m.moe_expanded_workspace_bytes(at, 192) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    rows = torch.zeros(4, 16, 576, dtype=torch.bfloat16)
    c = m.LatentCache.from_tensors(rows[..., :512], rows[..., 512:])
    assert (c.latent_token_stride, c.rope_page_stride, c.page_size, c.latent_dim) == (576, 16 * 576, 16, 512)
    for lat, rot in ((rows[..., :512].float(), rows[..., 512:]), (rows[..., :512], rows[..., :32]), (rows[..., :512], rows[:2, :, 512:]),
                     (rows[..., :512], rows[..., 512:].float()), (rows[0, :, :512], rows[0, :, 512:]),
                     (rows.transpose(1, 2), rows[..., 512:])):
        with pytest.raises(m.MoeError):
            m.LatentCache.from_tensors(lat, rot)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    s = m.Seqs.from_tensors(i32(2), i32(1), i32(1, 3))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    r = m.Rope.from_freqs(torch.zeros(32, 2))
    at = m.Attn(4, 0.1)
    with pytest.raises(m.MoeError):           # another width of latent
        m.moe_latent_append(r, c, s, bf(2, 320), bf(2, 4, 64), i32(2), bf(2, 4, 64))
    with pytest.raises(m.MoeError):           # positions of another length
        m.moe_latent_append(r, c, s, bf(2, 576), bf(2, 4, 64), i32(3), bf(2, 4, 64))
    with pytest.raises(m.MoeError):           # queries without their rotary part
        m.moe_latent_attention(at, c, s, bf(2, 4, 512), bf(2, 4, 512), bf(8))
    with pytest.raises(m.MoeError):           # offsets of another batch
        m.moe_latent_gather(c, s, i32(3), bf(2, 576), bf(8))
    with pytest.raises(m.MoeError):           # values of another width than the keys
        m.moe_expanded_attention(at, s, i32(2), bf(2, 4, 192), bf(5, 4, 128), bf(5, 64), bf(5, 4, 64), bf(2, 4, 64), bf(8))


@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a device beside the CPU")
def test_binding_refuses_host_tensors():
    lat = torch.zeros(4, 16, 256, dtype=torch.bfloat16, device="cuda")
    rot = torch.zeros(4, 16, 64, dtype=torch.bfloat16, device="cuda")
    c = m.LatentCache.from_tensors(lat, rot)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    s = m.Seqs.from_tensors(i32(2), i32(1), i32(1, 3))
    with pytest.raises(m.MoeError):
        m.moe_latent_gather(c, s, i32(2), torch.zeros(5, 320, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8, device="cuda"))
