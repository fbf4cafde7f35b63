"""A decoder layer's speculative-verify loop, its attention half and its MoE
half, through this library: a prefill chunk, then verify blocks of 8 rows over
one paged K/V cache, which is cut to a budget by accumulated attention weight.

    python examples/verify_step.py [steps]

One layer of random weights stands for the model and its output for the hidden
state that the LM head reads; the head's rows are the embedding's, one further,
so that a token mostly predicts the next number.  The drafts count up too, now
and then with a slip, which the verify rejects.  The dense projections are
plain matrix products.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_speculative_verify_gb300 as m  # noqa: E402
import synth  # noqa: E402

SHAPE = synth.LayerShape(hidden=1024, inter=512, n_experts=32, n_groups=4, topk_groups=2, topk=4, n_shared=1,
                         routed_scaling=2.5)


class Pages:
    """Free pages of one cache."""

    def __init__(self, n):
        self.free = list(range(n))

    def take(self, n):
        got, self.free = self.free[:n], self.free[n:]
        return got


class Layer:
    """Weights, cache and workspaces of one layer for one sequence."""

    def __init__(self, n_q=16, n_kv=2, dim=128, page=64, n_pages=64, capacity=2048, kv_dtype=torch.bfloat16, seed=0,
                 max_rows=512):
        dev = torch.device("cuda")
        g = torch.Generator(device=dev).manual_seed(seed)
        h = SHAPE.hidden
        rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
        self.n_q, self.n_kv, self.dim, self.page = n_q, n_kv, dim, page
        self.w_qkv = (rnd((n_q + 2 * n_kv) * dim, h) * h ** -0.5).bfloat16()
        self.w_o = (rnd(h, n_q * dim) * (n_q * dim) ** -0.5).bfloat16()
        wl = synth.Workload("example", SHAPE, rows=8)
        t = {k: v.to(dev) for k, v in synth.make_layer(wl, device="cpu").items()}
        self.router, self.bias = t["wr"], t["bias"]
        tiled = m.tile_weights(t)
        self.weights = m.Weights.from_tensors(tiled, m.LAYOUT_TILED)
        self.cfg = m.Config.from_shape(SHAPE)
        self.moe_ws = torch.zeros(m.moe_workspace_size(self.cfg, max_rows), dtype=torch.uint8, device=dev)
        # the cache and what goes with it
        shape = (n_pages, n_kv, page, dim)
        scales = {}
        if kv_dtype != torch.bfloat16:
            scales = {"k_scale": torch.full((n_kv,), 0.02, device=dev), "v_scale": torch.full((n_kv,), 0.02, device=dev)}
            k, v = (torch.zeros(shape, dtype=torch.uint8, device=dev).view(kv_dtype) for _ in range(2))
        else:
            k, v = (torch.zeros(shape, dtype=kv_dtype, device=dev) for _ in range(2))
        self.cache = m.KVCache.from_tensors(k, v, **scales)
        self.pages = Pages(n_pages)
        self.table = torch.zeros(1, capacity // page, dtype=torch.int32, device=dev)
        self.owned = []
        self.kv_len = torch.zeros(1, dtype=torch.int32, device=dev)
        self.scores = torch.zeros(1, n_kv, capacity, device=dev)
        freqs, mag = m.moe_rope_freqs(dim)
        self.attn = m.Attn(n_q, dim ** -0.5)
        self.ws = torch.zeros(m.moe_attn_workspace_bytes(self.attn, self.cache), dtype=torch.uint8, device=dev)
        self.rope = m.Rope.from_freqs(freqs.to(dev), False, mag, self.ws)
        self.cached = 0           # host's copy of kv_len
        self.position = 0         # of the next token; it runs on when keys are evicted

    def grow(self, n):
        need = -(-(self.cached + n) // self.page)
        if need > len(self.owned):
            self.owned += self.pages.take(need - len(self.owned))
            self.table[0, :need] = torch.tensor(self.owned, dtype=torch.int32)
        self.cached += n
        self.kv_len.fill_(self.cached)

    def forward(self, x):
        """Rows x [n, hidden] bf16 of new tokens: (their output, q, lse, the step's batch)."""
        n = x.shape[0]
        self.grow(n)
        cu = torch.tensor([0, n], dtype=torch.int32, device=x.device)
        seqs = m.Seqs.from_tensors(cu, self.kv_len, self.table, n)
        pos = torch.arange(self.position, self.position + n, dtype=torch.int32, device=x.device)
        self.position += n
        qkv = (x @ self.w_qkv.t()).view(n, -1, self.dim)
        q, k, v = qkv[:, :self.n_q], qkv[:, self.n_q:self.n_q + self.n_kv], qkv[:, self.n_q + self.n_kv:]
        m.moe_rope_append(self.rope, self.cache, seqs, q, k, v, pos, q)          # q in place
        a = torch.empty(n, self.n_q, self.dim, dtype=torch.bfloat16, device=x.device)
        lse = torch.empty(n, self.n_q, device=x.device)
        m.moe_paged_attention(self.attn, self.cache, seqs, q, a, self.ws, lse=lse)
        mid = x + a.view(n, -1) @ self.w_o.t()
        out = torch.empty_like(mid)
        m.moe_layer(self.cfg, mid, self.router, self.bias, self.weights, None, out, self.moe_ws)
        return mid + out, q, lse, seqs

    def settle(self, q, lse, seqs, accepted):
        """Adds the accepted rows' attention weights to the keys' scores and drops the others' keys."""
        n = q.shape[0]
        lse[accepted:] = float("inf")
        m.moe_key_weights(self.attn, self.cache, seqs, q, lse, self.scores, self.scores, self.ws)
        self.cached -= n - accepted
        self.position -= n - accepted
        self.kv_len.fill_(self.cached)

    def evict(self, budget, recent):
        """Cuts the cache to `budget` keys a kv head; its old pages go free."""
        new = self.pages.take(-(-budget // self.page))
        to = torch.zeros_like(self.table)
        to[0, :len(new)] = torch.tensor(new, dtype=torch.int32)
        kept = torch.empty(1, self.n_kv, budget, dtype=torch.int32, device=to.device)
        out, new_len = torch.zeros_like(self.scores), torch.empty_like(self.kv_len)
        seqs = m.Seqs.from_tensors(None, self.kv_len, self.table)
        m.moe_cache_evict(self.cache, seqs, self.scores, budget, recent, to, kept, out, new_len, self.ws)
        self.pages.free += self.owned
        self.owned, self.table, self.scores, self.kv_len = new, to, out, new_len
        self.cached = min(self.cached, budget)
        return kept

    def check(self):
        for ws in (self.ws, self.moe_ws):
            err = m.moe_get_device_error(ws)
            if err:
                raise RuntimeError(m.STATUS.get(err, err))


def main(steps=12, prompt=300, budget=256, recent=64, vocab=4096, seed=1, kv_dtype=torch.bfloat16, quiet=False):
    m.build()
    m.load()
    layer = Layer(kv_dtype=kv_dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    embed = torch.randn(vocab, SHAPE.hidden, generator=g, device="cuda").bfloat16()
    head = embed.roll(1, 0)
    tokens = torch.randint(0, vocab, (prompt,), generator=g, device="cuda")
    y, q, lse, seqs = layer.forward(embed[tokens])
    layer.settle(q, lse, seqs, prompt)
    committed = int((y[-1:] @ head.t()).argmax())
    am, out = (torch.empty(8, dtype=torch.int32, device="cuda") for _ in range(2))
    acc, nd = (torch.full((1,), 7, dtype=torch.int32, device="cuda") for _ in range(2))
    lengths, accepted = [], []
    for step in range(steps):
        if layer.cached > budget:
            layer.evict(budget, recent)
        slip = (5 * step) % 8                     # the draft that is wrong (0: none)
        draft = [(committed + i + (i == slip > 0)) % vocab for i in range(8)]
        draft = torch.tensor(draft, dtype=torch.int32, device="cuda")
        y, q, lse, seqs = layer.forward(embed[draft.long()])
        m.moe_greedy_verify(y @ head.t(), draft, nd, am, acc, out)
        k = int(acc)
        layer.settle(q, lse, seqs, k)
        committed = int(out[k - 1])
        accepted.append(k)
        lengths.append(layer.cached)
        if not quiet:
            print(f"step {step}: {k} tokens, {layer.cached} cached keys, position {layer.position}")
    layer.check()
    return accepted, lengths


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:2]))
