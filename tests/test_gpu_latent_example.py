"""The latent-cache example's layer: prompt chunks in expanded form and blocks in
absorbed form of the same text give the same rows, and its verify loop runs."""
import importlib.util
import os

import pytest
import torch

import moe_speculative_verify_gb300 as m

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    m.build()
    m.load()
    spec = importlib.util.spec_from_file_location("latent_step", os.path.join(ROOT, "examples", "latent_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_chunks_blocks_and_single_tokens_agree(ex, dtype):
    """The cached rows of both forms are the same bits.  The expanded form rounds each head's keys and values to bf16, the
    absorbed one its queries in latent space and its mixed latents: 2^-8 of each at most, with random signs over the sums
    that follow, so the attention outputs are compared in norm at 2 %, four such roundings."""
    x = torch.randn(100, ex.SHAPE.hidden, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    want = ex.Layer(cache_dtype=dtype).attend(x, True).float()
    for cuts, forms in (([60] + [8] * 5, [True] + [False] * 5), ([97, 1, 1, 1], [True] + [False] * 3), ([50, 50], [True, True]),
                        ([100], [False])):
        layer = ex.Layer(cache_dtype=dtype)
        got = torch.cat([layer.attend(part, form) for part, form in zip(x.split(cuts), forms)]).float()
        layer.check()
        assert layer.cached == 100
        assert float((got - want).norm() / want.norm()) < 0.02
    assert bool(torch.isfinite(want).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_verify_loop(ex, dtype):
    accepted, cached = ex.main(steps=6, cache_dtype=dtype, quiet=True)
    assert all(1 <= k <= 8 for k in accepted) and cached == 300 + sum(accepted)
