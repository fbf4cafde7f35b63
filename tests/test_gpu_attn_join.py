"""A long item split over 2 to all CTAs: every number of pieces is joined rightly."""
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


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news,hq,tile", [(1, 8, 64), (4, 8, 128), (12, 8, 128)])   # few rows; tiles of 32 and 96 rows
def test_every_number_of_pieces(news, hq, tile, dim, dtype):
    g = torch.Generator(device="cuda").manual_seed(5)
    for pieces in range(2, 161):               # key tiles; more than there are CTAs at the end
        k, v = ((randn(g, pieces * tile, 1, dim) * 16).round() / 16 for _ in range(2))
        One(k, v, randn(g, news, hq, dim), dtype, dim ** -0.5).check()
