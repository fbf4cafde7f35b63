"""Attention where probabilities and query elements spread over many octaves:
a first key that takes most of the weight and has value zero, as trained models'
caches have it, so that the output is the average over thousands of keys of
small probability each; a query element far above the others."""
import pytest
import torch

import moe_speculative_verify_gb300 as m
from attn_one import One, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    m.build()
    m.load()
    torch.cuda.set_device(0)


def sink(keys, news, hq, hkv, dtype, dim, gap, tail, mean=0.5, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.zeros(keys, hkv, dim, device="cuda") if tail == "equal" else (randn(g, keys, hkv, dim) * 16).round() / 16
    k[:, :, 0] = 0
    k[0] = 0
    k[0, :, 0] = 16.0
    v = ((randn(g, keys, hkv, dim) + mean) * 16).round() / 16
    v[0] = 0
    q = randn(g, news, hq, dim)
    q[:, :, 0] = gap * dim ** 0.5 / 16.0                    # the first key's score; the others' are 0, or about 1 apart
    return One(k, v, q, dtype, dim ** -0.5)


# rows a kv head: 8, and 1 with a whole head a CTA (few rows); 32, 64 (repeated in the tile), 96 (one tile), 320 (two)
@pytest.mark.parametrize("news,hq,hkv,keys", [(1, 8, 1, 32768), (1, 128, 128, 8192), (4, 8, 1, 32768), (8, 8, 1, 16384),
                                              (8, 256, 32, 8192), (12, 8, 1, 32768), (40, 8, 1, 16384), (40, 8, 1, 32768)])
@pytest.mark.parametrize("tail", ["equal", "spread"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_small_probabilities_behind_a_sink(dtype, tail, news, hq, hkv, keys):
    for gap in (8.0, 10.28, 12.0, 13.0, 14.0, 15.0, 16.0):
        for dim in (64, 128):
            sink(keys, news, hq, hkv, dtype, dim, gap, tail).check()


@pytest.mark.parametrize("news", [1, 8])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_small_probabilities_of_a_million_keys(dtype, news):
    for gap in (14.0, 16.0, 18.0):
        sink(1 << 20, news, 8, 1, dtype, 128, gap, "equal").check()


@pytest.mark.parametrize("news,hq", [(8, 8), (12, 8), (40, 8)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_outlier_query_channel(dtype, dim, news, hq):
    """A query element far above the others where the keys have zero: the others
    alone make the scores."""
    for size in (1e3, 1e5, 1e6):
        g = torch.Generator(device="cuda").manual_seed(3)
        k = (randn(g, 500, 1, dim) * 16).round() / 16
        k[:, :, 5] = 0
        v = (randn(g, 500, 1, dim) * 16).round() / 16
        q = randn(g, news, hq, dim) * 3
        q[:, :, 5] = size
        One(k, v, q, dtype, dim ** -0.5).check()


@pytest.mark.parametrize("news,hq", [(1, 8), (8, 8), (40, 8)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_nan_in_the_cache(dtype, dim, news, hq):
    """A NaN value makes its column NaN and no other; a NaN key every row that sees it."""
    for code in ((0x7F, 0xFF) if dtype == "e4m3" else (0x7FC0, -0x40)):
        g = torch.Generator(device="cuda").manual_seed(4)
        k, v = ((randn(g, 400, 1, dim) * 16).round() / 16 for _ in range(2))
        p = One(k, v, randn(g, news, hq, dim), dtype, dim ** -0.5)
        clean, _ = p.run()
        bits = lambda x: x.view(torch.uint8 if dtype == "e4m3" else torch.int16)
        before = bits(p.dv)[2, 0, 7, dim - 3].clone()
        bits(p.dv)[2, 0, 7, dim - 3] = code
        out, lse = p.run()
        assert bool(torch.isnan(out[:, :, dim - 3]).all()) and not bool(torch.isnan(lse).any())
        keep = torch.arange(dim, device="cuda") != dim - 3
        assert torch.equal(out[:, :, keep], clean[:, :, keep])
        bits(p.dv)[2, 0, 7, dim - 3] = before
        bits(p.dk)[6, 0, 15, 3] = code                # key 399: the last row's own
        out, lse = p.run()
        assert bool(torch.isnan(out[-1]).all()) and bool(torch.isnan(lse[-1]).all())
        assert torch.equal(out[:-1], clean[:-1])


@pytest.mark.parametrize("dim", [64, 128])
def test_outlier_query_channel_of_a_single_token(dim):
    """As test_outlier_query_channel, in the kernel for few rows."""
    for dtype in ("bf16", "e4m3"):
        for size in (1e3, 1e5, 1e6, 1e8):
            g = torch.Generator(device="cuda").manual_seed(3)
            k = (randn(g, 500, 1, dim) * 16).round() / 16
            k[:, :, 5] = 0
            v = (randn(g, 500, 1, dim) * 16).round() / 16
            q = randn(g, 1, 8, dim) * 3
            q[:, :, 5] = size
            One(k, v, q, dtype, dim ** -0.5).check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_equal_scores_far_below_a_single_token_s_largest(dtype, dim):
    """Few keys, so that one warp's largest is the heavy key's: the others are
    21 to 27 octaves below it."""
    for gap in (14.6, 15.3, 16.3, 17.2, 18.7):
        sink(16, 1, 8, 1, dtype, dim, gap, "equal").check()


@pytest.mark.parametrize("news,hq", [(1, 16), (2, 16), (8, 16), (40, 16)])
@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_signs_of_scales(news, hq, scale):
    """Negative softmax scales and negative scales of a head's codes."""
    g = torch.Generator(device="cuda").manual_seed(6)
    ks, vs = torch.tensor([1 / 16, -1 / 16], device="cuda"), torch.tensor([-1 / 16, 1 / 16], device="cuda")
    k, v = ((randn(g, 700, 2, 64) * 16).round() / 16 for _ in range(2))
    One(k, v, randn(g, news, hq, 64), "e4m3", scale, ks, vs).check()
    One(k, v, randn(g, news, hq, 64), "bf16", scale).check()
    p = One(k, v, randn(g, news, hq, 64), "e4m3", scale)
    p.k_scale[1] = float("nan")
    out, lse = p.run()
    assert bool(torch.isnan(out[:, hq // 2:]).all()) and bool(torch.isnan(lse[:, hq // 2:]).all())
    assert bool(torch.isfinite(out[:, :hq // 2]).all())
