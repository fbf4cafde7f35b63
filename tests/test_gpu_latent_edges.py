"""Attention through a latent cache where it can go wrong: kernels that follow one
another at once, numbers that are not finite in cached rows, every number of pieces."""
import pytest
import torch

import latent_ref as ref
import moe_speculative_verify_gb300 as m
from latent_ref import i32
from test_gpu_latent import Expanded, attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    m.build()
    m.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_kernels_that_follow_one_another(dtype):
    """Short calls of both attention kernels in turn, without a pause: a CTA's barriers lie where those of the kernel before
    lay, so an arrival of that one which came after its CTA's end would be counted here."""
    p = ref.Problem([70, 3], [2, 1], 16, 256, 32, dtype, seed=41)
    x = Expanded([40, 300], [9, 2], 2, 64, seed=42)
    attn, xa = m.Attn(16, p.scale), m.Attn(2, x.scale)
    ws = torch.zeros(m.moe_latent_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
    wx = torch.zeros(m.moe_expanded_workspace_bytes(xa, 64), dtype=torch.uint8, device="cuda")
    outs = torch.zeros(200, p.t, 16, 256, dtype=torch.bfloat16, device="cuda")
    xouts = torch.zeros(200, x.t, 2, 64, dtype=torch.bfloat16, device="cuda")
    lse, xl = torch.zeros(p.t, 16, device="cuda"), torch.zeros(x.t, 2, device="cuda")
    for k in range(200):
        m.moe_latent_attention(attn, p.cache, p.seqs, p.q, outs[k], ws, lse=lse)
        m.moe_expanded_attention(xa, x.seqs, x.d_ck, x.q, x.k, x.rope, x.v, xouts[k], wx, lse=xl)
    assert m.moe_get_device_error(ws) == 0 and m.moe_get_device_error(wx) == 0
    ref.check(outs[0], lse, *ref.latent_attention(p))
    ref.check(xouts[0], xl, *x.want())
    assert torch.equal(outs, outs[:1].expand_as(outs)) and torch.equal(xouts, xouts[:1].expand_as(xouts))
