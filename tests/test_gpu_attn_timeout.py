"""The shortest limit of device waits, one microsecond: below what a first copy
takes, though a thread that the hardware suspends in its wait may see the copy
all the same.  The call ends, right or with MOE_ERR_TIMEOUT in the error word, and
the next one on the same stream and workspace is right."""
import pytest
import torch

import moe_speculative_verify_gb300 as m
from attn_one import One, randn

pytestmark = pytest.mark.gpu
TIMEOUT = 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    m.build()
    m.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("news,hq", [(1, 16), (2, 32), (8, 16), (40, 16)])   # few rows; tiles of 32, 64 and 320 rows
def test_waits_that_run_out(news, hq, dim, dtype):
    g = torch.Generator(device="cuda").manual_seed(51)
    keys, hkv = 20000, 2
    k, v = ((randn(g, keys, hkv, dim) * 16).round() / 16 for _ in range(2))
    p = One(k, v, randn(g, news, hq, dim), dtype, dim ** -0.5)
    q = p.q.bfloat16()
    ws = torch.zeros(m.moe_attn_workspace_bytes(m.Attn(hq, p.scale), p.cache), dtype=torch.uint8, device="cuda")
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")

    def call(limit):
        attn = m.Attn(hq, p.scale, wait_timeout_us=limit)
        out = torch.zeros(news, hq, dim, dtype=torch.bfloat16, device="cuda")
        lse, scores = torch.zeros(news, hq, device="cuda"), torch.zeros(1, hkv, keys, device="cuda")
        flush.zero_()                            # the first tiles come from memory
        m.moe_paged_attention(attn, p.cache, p.seqs, q, out, ws, lse=lse)
        err = m.moe_get_device_error(ws)
        flush.zero_()
        m.moe_key_weights(attn, p.cache, p.seqs, q, want[1] if want else lse, scores, scores, ws)
        return (out, lse, scores), (err, m.moe_get_device_error(ws))

    want = None
    want, err = call(0)
    assert err == (0, 0)
    for _ in range(3):
        got, short = call(1)
        assert set(short) <= {0, TIMEOUT}
        for x, y, e in zip(got, want, (short[0], short[0], short[1])):
            assert e == TIMEOUT or torch.equal(x, y)
        got, err = call(0)
        assert err == (0, 0) and all(torch.equal(a, b) for a, b in zip(got, want))
