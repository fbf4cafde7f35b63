"""The example's layer: a chunk, a verify block and single tokens of the same
text give the same rows, and its verify loop keeps the cache to its budget."""
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
    spec = importlib.util.spec_from_file_location("verify_step", os.path.join(ROOT, "examples", "verify_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn])
def test_chunk_block_and_single_tokens_agree(ex, kv):
    """The same 100 tokens as one chunk, as 60 + 5 blocks of 8, and with the
    last ones fed one by one.  The attention outputs differ by their roundings
    (bf16 probabilities and outputs: 2^-7 of the row's scale at most), which the
    projection and the experts carry on; routing can flip only where two
    scores tie to that, so the rows are compared in norm, at a few percent."""
    x = torch.randn(100, ex.SHAPE.hidden, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    want = ex.Layer(kv_dtype=kv).forward(x)[0].float()
    for cuts in ([60] + [8] * 5, [97, 1, 1, 1]):
        layer = ex.Layer(kv_dtype=kv)
        got = torch.cat([layer.forward(part)[0] for part in x.split(cuts)]).float()
        layer.check()
        assert layer.cached == 100
        assert (got - want).norm() / want.norm() < 0.03
    assert torch.isfinite(want).all()


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn])
def test_verify_loop(ex, kv):
    accepted, lengths = ex.main(steps=6, kv_dtype=kv, quiet=True)
    assert all(1 <= k <= 8 for k in accepted)
    # 300 prompt keys are cut to 256 before the first block, then whenever a block went past it
    length = 300
    for k, n in zip(accepted, lengths):
        length = min(length, 256) + k
        assert n == length
