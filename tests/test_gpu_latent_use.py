"""The latent-cache operators as programs use them: captured graphs, streams, wait
limits, caches past 32 bits, strides and head counts at their limits."""
import threading

import pytest
import torch

import latent_ref as ref
import moe_speculative_verify_gb300 as m
from latent_ref import ROT, i32
from test_gpu_latent import Expanded, attend

pytestmark = pytest.mark.gpu
TIMEOUT = 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    m.build()
    m.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,heads", [(1, 16), (8, 16), (40, 64)])       # items of up to 64 rows, of up to 128, several
def test_waits_that_run_out(news, heads, dtype):
    """The shortest limit of device waits: the call ends, right or with MOE_ERR_TIMEOUT in the error word, and the next one on
    the same stream and workspace is right."""
    p = ref.Problem([20000], [news], heads, 512, 64, dtype, seed=51)
    ws = torch.zeros(m.moe_latent_workspace_bytes(m.Attn(heads, p.scale), p.cache), dtype=torch.uint8, device="cuda")
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")

    def call(limit):
        out, lse = torch.zeros(news, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(news, heads, device="cuda")
        flush.zero_()                            # the first tiles come from memory
        m.moe_latent_attention(m.Attn(heads, p.scale, wait_timeout_us=limit), p.cache, p.seqs, p.q, out, ws, lse=lse)
        return (out, lse), m.moe_get_device_error(ws)

    want, err = call(0)
    assert err == 0
    for _ in range(3):
        got, short = call(1)
        assert short in (0, TIMEOUT)
        assert short == TIMEOUT or all(torch.equal(a, b) for a, b in zip(got, want))
        got, err = call(0)
        assert err == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("lens,news", [([3000], [5]), ([1500], [1500])])
@pytest.mark.parametrize("dim", [64, 128])
def test_expanded_waits_that_run_out(lens, news, dim):
    p = Expanded(lens, news, 4, dim, seed=52)
    ws = torch.zeros(m.moe_expanded_workspace_bytes(m.Attn(4, p.scale), dim), dtype=torch.uint8, device="cuda")
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")

    def call(limit):
        out, lse = torch.zeros(p.t, 4, dim, dtype=torch.bfloat16, device="cuda"), torch.zeros(p.t, 4, device="cuda")
        flush.zero_()
        m.moe_expanded_attention(m.Attn(4, p.scale, wait_timeout_us=limit), p.seqs, p.d_ck, p.q, p.k, p.rope, p.v, out, ws, lse=lse)
        return (out, lse), m.moe_get_device_error(ws)

    want, err = call(0)
    assert err == 0
    for _ in range(3):
        got, short = call(1)
        assert short in (0, TIMEOUT)
        assert short == TIMEOUT or all(torch.equal(a, b) for a, b in zip(got, want))
        got, err = call(0)
        assert err == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_offsets_past_32_bits(dtype):
    """Pages whose elements lie past 2^32 of the cache, and past 2^32 bytes of the rows read back."""
    c, page, es = 512, 64, 1 if dtype == "e4m3" else 2
    n_pages = (1 << 32) // (page * c) + 40                    # 4.3e9 elements of latents
    lat = torch.empty(n_pages, page, c, dtype=torch.uint8 if es == 1 else torch.bfloat16, device="cuda")
    rot = torch.empty(n_pages, page, ROT, dtype=torch.bfloat16, device="cuda")
    last = [n_pages - 1 - 3 * k for k in range(5)]
    g = torch.Generator().manual_seed(4)
    src = torch.randn(5, page, c, generator=g)
    lat[last] = (src * 16).to(torch.float8_e4m3fn).view(torch.uint8).cuda() if es == 1 else src.bfloat16().cuda()
    rot[last] = torch.randn(5, page, ROT, generator=g).bfloat16().cuda()
    p = ref.Problem([300], [2], 16, c, page, dtype, seed=6)   # its sizes, with this cache and table
    p.latent, p.rope, p.d_table = lat, rot, i32([last])
    p.cache = m.LatentCache.from_tensors(lat, rot, p.exp)
    p.seqs = m.Seqs.from_tensors(p.d_cu, p.kv_len, p.d_table, 2)
    # appended: the last two of 300 rows
    freqs, mag = m.moe_rope_freqs(ROT)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kv = torch.randn(2, c + ROT, generator=g).bfloat16().cuda()
    q = torch.zeros(2, 16, ROT, dtype=torch.bfloat16, device="cuda")
    m.moe_latent_append(m.Rope.from_freqs(freqs.cuda(), False, mag, ws), p.cache, p.seqs, kv, q, i32([0, 0]), q)   # position 0: as they are
    rows, rk = p.rows(0)
    assert torch.equal(rk[298:], kv[:, c:].double())
    assert bool(((rows[298:] - kv[:, :c].double()).abs() <= (2.0 ** -4 * kv[:, :c].double().abs() + 2.0 ** -14 if es == 1 else 0.0)).all())
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))
    # read back to rows past 2^32 elements of their tensor
    n = 300
    wide = torch.empty((1 << 32) + (1 << 26), dtype=torch.bfloat16, device="cuda")
    step = (wide.numel() // n) // 8 * 8
    got = wide[:n * step].view(n, step)[:, :c + ROT]
    m.moe_latent_gather(p.cache, p.seqs, i32([0, n]), got, ws)
    assert m.moe_get_device_error(ws) == 0
    assert torch.equal(got.double(), torch.cat([rows, rk], 1))


def test_expanded_offsets_past_32_bits():
    """Token and head strides whose products pass 2^32 elements."""
    p = Expanded([300], [60], 3, 128, seed=7)
    wide = torch.empty((1 << 32) + (1 << 28), dtype=torch.bfloat16, device="cuda")
    step, head = (wide.numel() // 302) // 8 * 8, 1 << 20
    far = lambda at: wide.as_strided((300, 3, 128), (step, head, 1), at)
    k, v = far(0), far(head * 4)
    k.copy_(p.k), v.copy_(p.v)
    q = wide.as_strided((60, 3, 192), ((1 << 26) + 8, 192, 1), head * 9)
    q.copy_(p.q)
    want = p.want()
    p.k, p.v, p.q = k, v, q
    out, lse = p.run()
    ref.check(out, lse, *want)


def test_expanded_odd_strides():
    p = Expanded([200, 77], [130, 77], 3, 64, seed=8)
    want = p.want()

    def apart(x, *strides):                                  # NaN between the rows
        wide = torch.full((strides[0] * x.shape[0],), float("nan"), dtype=torch.bfloat16, device="cuda")
        y = wide.as_strided(x.shape, strides + (1,))
        y.copy_(x)
        return y
    p.k, p.v, p.rope, p.q = apart(p.k, 3 * 72 + 8, 72), apart(p.v, 1000, 64), apart(p.rope, 72), apart(p.q, 3 * 128 + 24, 128)
    out, lse = p.run()
    ref.check(out, lse, *want)


@pytest.mark.parametrize("scale", [0.0, -0.09])
def test_expanded_zero_and_negative_scale(scale):
    p = Expanded([400, 31], [300, 5], 2, 128, seed=9)
    p.scale = scale
    out, lse = p.run()
    ref.check(out, lse, *p.want())


def test_expanded_peaked_scores():
    p = Expanded([900], [700], 2, 64, seed=10)
    p.q *= 50
    out, lse = p.run()
    ref.check(out, lse, *p.want())


@pytest.mark.parametrize("lens,news,heads", [([200, 3], [130, 3], 256), ([0, 0], [1, 2], 2), ([1] * 300, [1] * 300, 1)])
def test_expanded_limits(lens, news, heads):
    p = Expanded(lens + [1], news + [1], heads, 64, seed=11)
    out, lse = p.run()
    ref.check(out, lse, *p.want())


@pytest.mark.parametrize("window", [1 << 20, (1 << 31) - 1])
def test_windows_past_every_length(window):
    p = ref.Problem([500, 64], [8, 1], 16, 256, 32, seed=12)
    out, lse = attend(p)
    o2, l2 = attend(p, window=window)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    x = Expanded([300], [200], 2, 64, seed=13)
    for a, b in zip(x.run(), x.run(window=window)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("max_q", [1, 7, 1 << 30])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_results_hold_for_any_max_q(max_q, dtype):
    """max_q only picks the kernel: items of 64 rows of longer blocks, and of 128 rows of single tokens."""
    p = ref.Problem([700, 90, 33], [9, 1, 33], 8, 512, 64, dtype, seed=14)
    p.seqs = m.Seqs.from_tensors(p.d_cu, p.kv_len, p.d_table, max_q)
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))


def test_sequences_that_share_pages():
    """A common prefix held once, and one page twice in a table."""
    p = ref.Problem([200, 190, 128], [1, 4, 1], 16, 512, 64, seed=15)
    p.d_table[1, :2] = p.d_table[0, :2]
    p.d_table[2, 1] = p.d_table[2, 0]
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))


def test_two_threads_and_streams_with_workspaces_of_their_own():
    def work(k, res):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            p, x = ref.Problem([3000 + 7 * k, 90], [8, 1], 16, 512, 64, seed=k), Expanded([700 + k], [600], 4, 128, seed=k)
            attn, xa = m.Attn(16, p.scale), m.Attn(4, x.scale)
            ws = torch.zeros(m.moe_latent_workspace_bytes(attn, p.cache), dtype=torch.uint8, device="cuda")
            wx = torch.zeros(m.moe_expanded_workspace_bytes(xa, 128), dtype=torch.uint8, device="cuda")
            got = []
            for _ in range(20):
                out, lse = torch.empty(9, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(9, 16, device="cuda")
                xo, xl = torch.empty(600, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(600, 4, device="cuda")
                m.moe_latent_attention(attn, p.cache, p.seqs, p.q, out, ws, lse=lse)
                m.moe_expanded_attention(xa, x.seqs, x.d_ck, x.q, x.k, x.rope, x.v, xo, wx, lse=xl)
                got.append((out, lse, xo, xl))
            s.synchronize()
            ref.check(*got[0][:2], *ref.latent_attention(p))
            ref.check(*got[0][2:], *x.want())
            res[k] = all(torch.equal(a, b) for g in got for a, b in zip(g, got[0]))
            s.synchronize()

    res = {}
    ts = [threading.Thread(target=work, args=(k, res)) for k in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert res == {0: True, 1: True}


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_graph_of_a_whole_step_follows_the_lengths(dtype):
    """Append, absorbed attention, gather and expanded attention captured as one graph; replayed with lengths, positions and
    rows that change, as often as called."""
    H, C, D, page, T, top = 4, 512, 64, 32, 6, 160
    lat = torch.zeros(16, page, C, dtype=torch.uint8 if dtype == "e4m3" else torch.bfloat16, device="cuda")
    rot = torch.zeros(16, page, ROT, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(16)
    rnd = lambda *s: torch.randn(*s, generator=g)
    old = rnd(16, page, C) * 16
    lat.copy_(old.to(torch.float8_e4m3fn).view(torch.uint8) if dtype == "e4m3" else old.bfloat16() / 16)
    rot.copy_(rnd(16, page, ROT))
    start = lat.clone(), rot.clone()
    cache = m.LatentCache.from_tensors(lat, rot, -4)
    attn = m.Attn(H, 0.07)
    ws, wx = (torch.zeros(n, dtype=torch.uint8, device="cuda")
              for n in (m.moe_latent_workspace_bytes(attn, cache), m.moe_expanded_workspace_bytes(attn, D)))
    table = torch.randperm(16, generator=g).int()[:10].view(2, 5).cuda()
    cu, kv_len, pos, ck = i32([0, 4, 6]), i32([4, 2]), i32([0] * T), i32([0, top, 2 * top])
    seqs = m.Seqs.from_tensors(cu, kv_len, table, 4)
    freqs, mag = m.moe_rope_freqs(ROT)
    rope = m.Rope.from_freqs(freqs.cuda(), True, mag, ws)
    kv, q = rnd(T, C + ROT).bfloat16().cuda(), rnd(T, H, C + ROT).bfloat16().cuda()
    wk, wv = (rnd(H * D, C).bfloat16().cuda() * C ** -0.5 for _ in range(2))
    ql, out, xo = q.clone(), torch.zeros(T, H, C, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    lse, xl = torch.zeros(T, H, device="cuda"), torch.zeros(T, H, device="cuda")
    rows = torch.zeros(2 * top, C + ROT, dtype=torch.bfloat16, device="cuda")

    def step():
        m.moe_latent_append(rope, cache, seqs, kv, q[..., C:], pos, ql[..., C:])
        m.moe_latent_attention(attn, cache, seqs, ql, out, ws, lse=lse)
        m.moe_latent_gather(cache, seqs, ck, rows, ws)
        k, v = ((rows[:, :C] @ w.t()).view(-1, H, D) for w in (wk, wv))
        m.moe_expanded_attention(attn, seqs, ck, ql[..., C - D:].contiguous(), k, rows[:, C:], v, xo, wx, lse=xl)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    res = (out, lse, rows, xo, xl, lat, rot)
    for lens in ([4, 2], [160, 2], [77, 159], [4, 33]):
        kv_len.copy_(i32(lens))
        pos.copy_(i32(list(range(lens[0] - 4, lens[0])) + list(range(lens[1] - 2, lens[1]))))
        kv.copy_(rnd(T, C + ROT))
        lat.copy_(start[0]), rot.copy_(start[1])
        step()
        want = [x.clone() for x in res]
        lat.copy_(start[0]), rot.copy_(start[1])
        for x in res[:5]:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want))
        assert bool(torch.isfinite(lse).all()) and bool(torch.isfinite(xl).all()) and float(out.float().abs().max()) > 0
    assert m.moe_get_device_error(ws) == 0 and m.moe_get_device_error(wx) == 0


@pytest.mark.parametrize("fn", ["append", "attend", "gather", "expand"])
def test_nothing_is_written_without_tokens(fn):
    """Empty calls return at once; outputs, error words and caches stay."""
    p = ref.Problem([40], [1], 4, 256, 16, seed=17)
    x = Expanded([40], [4], 2, 64, seed=17)
    ws = torch.zeros(m.moe_latent_workspace_bytes(m.Attn(4, 1.0), p.cache), dtype=torch.uint8, device="cuda")
    freqs, mag = m.moe_rope_freqs(ROT)
    before = p.latent.clone(), p.rope.clone()
    none = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    if fn == "append":
        m.moe_latent_append(m.Rope.from_freqs(freqs.cuda(), True, mag, ws), p.cache, p.seqs, none(0, 320), none(0, 4, 64), i32([]),
                            none(0, 4, 64))
    elif fn == "attend":
        m.moe_latent_attention(m.Attn(4, 1.0), p.cache, p.seqs, none(0, 4, 320), none(0, 4, 256), ws)
    elif fn == "gather":
        m.moe_latent_gather(p.cache, p.seqs, i32([0, 0]), none(0, 320), ws)
    else:
        m.moe_expanded_attention(m.Attn(2, 1.0), x.seqs, x.d_ck, none(0, 2, 128), x.k, x.rope, x.v, none(0, 2, 64), ws)
    assert m.moe_get_device_error(ws) == 0
    for a, b in zip((p.latent, p.rope), before):
        assert torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("news,heads", [([1, 1, 1], 64), ([9, 40, 2], 12)])
@pytest.mark.parametrize("scale", [0.07, -0.07])
def test_queries_with_and_without_gaps(news, heads, dtype, scale):
    """Rows one behind another, and the same with room between the tokens: the same bits; pad rows beside them hold NaN."""
    p = ref.Problem([700, 90, 64], news, heads, 512, 32, dtype, pads=(2, 3), seed=18)
    p.scale = scale
    p.q[:2] = float("nan")
    p.q[-3:] = float("nan")
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))
    wide = torch.full((p.t, heads * (p.c + ROT) + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = wide[:, :heads * (p.c + ROT)].view(p.t, heads, p.c + ROT)
    q.copy_(p.q)
    o2, l2 = attend(p, q=q)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_sequences_without_keys(dtype):
    p = ref.Problem([0, 5, 0], [1, 7, 3], 24, 256, 16, dtype, seed=19)
    out, lse = attend(p)
    ref.check(out, lse, *ref.latent_attention(p))


def test_expanded_length_past_the_rows():
    """A length past the rows there are is cut to them, and recorded."""
    p = Expanded([80], [30], 2, 64, seed=20)
    want = p.want()
    p.seqs = m.Seqs.from_tensors(i32(p.cu), i32([100]), torch.zeros(1, 0, dtype=torch.int32, device="cuda"), 30)
    out, lse = p.run(error=1)
    ref.check(out, lse, *want)
