"""A decoder layer's speculative-verify loop over a latent cache, its attention half
and its MoE half, through this library: prompt chunks in expanded form, then
verify blocks of 8 rows in absorbed form, over one paged cache of a latent
vector and a shared rotary key a token.

    python examples/latent_step.py [steps]

As in verify_step.py one layer of random weights stands for the model, the head's
rows are the embedding's, one further, and the dense projections are plain matrix
products.  A rejected row needs nothing but a shorter length: the next
block writes over it.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_speculative_verify_gb300 as m  # noqa: E402
import synth  # noqa: E402

SHAPE = synth.LayerShape(hidden=1024, inter=512, n_experts=32, n_groups=4, topk_groups=2, topk=4, n_shared=1,
                         routed_scaling=2.5)
ROT = 64


class Layer:
    """Weights, cache and workspaces of one layer for one sequence."""

    def __init__(self, heads=16, dim=128, latent=512, page=64, n_pages=64, cache_dtype=torch.bfloat16, seed=0, max_rows=512):
        dev = torch.device("cuda")
        g = torch.Generator(device=dev).manual_seed(seed)
        h = SHAPE.hidden
        rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
        self.heads, self.dim, self.latent, self.page = heads, dim, latent, page
        self.w_q = (rnd(heads * (dim + ROT), h) * h ** -0.5).bfloat16()
        self.w_kv = (rnd(latent + ROT, h) * h ** -0.5).bfloat16()
        self.w_up = (rnd(heads, 2 * dim, latent) * latent ** -0.5).bfloat16()    # a head's map to keys, then to values
        self.w_o = (rnd(h, heads * dim) * (heads * dim) ** -0.5).bfloat16()
        self.gamma = torch.ones(latent, device=dev)
        wl = synth.Workload("example", SHAPE, rows=8)
        t = {k: v.to(dev) for k, v in synth.make_layer(wl, device="cpu").items()}
        self.router, self.bias = t["wr"], t["bias"]
        tiled = m.tile_weights(t)
        self.weights = m.Weights.from_tensors(tiled, m.LAYOUT_TILED)
        self.cfg = m.Config.from_shape(SHAPE)
        self.moe_ws = torch.zeros(m.moe_workspace_size(self.cfg, max_rows), dtype=torch.uint8, device=dev)
        # the cache and what goes with it; normalised latents fit e4m3 with codes of 2^-4
        rows = torch.zeros(n_pages, page, latent, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) \
            if cache_dtype == torch.float8_e4m3fn else torch.zeros(n_pages, page, latent, dtype=cache_dtype, device=dev)
        keys = torch.zeros(n_pages, page, ROT, dtype=torch.bfloat16, device=dev)
        self.cache = m.LatentCache.from_tensors(rows, keys, scale_log2=-4 if cache_dtype == torch.float8_e4m3fn else 0)
        self.table = torch.arange(n_pages, dtype=torch.int32, device=dev).view(1, -1)
        self.kv_len = torch.zeros(1, dtype=torch.int32, device=dev)
        freqs, mag = m.moe_rope_freqs(ROT)
        self.attn = m.Attn(heads, (dim + ROT) ** -0.5)
        self.ws = torch.zeros(m.moe_latent_workspace_bytes(self.attn, self.cache), dtype=torch.uint8, device=dev)
        self.ws_x = torch.zeros(m.moe_expanded_workspace_bytes(self.attn, dim), dtype=torch.uint8, device=dev)
        self.rope = m.Rope.from_freqs(freqs.to(dev), True, mag, self.ws)
        self.cached = 0           # host's copy of kv_len

    def attend(self, x, expanded):
        """Attention of new tokens x [n, hidden] bf16; expanded: over keys and values of every head's own, made from the rows
        that the cache holds; else over the rows themselves, with queries in latent space."""
        n, H, D, L = x.shape[0], self.heads, self.dim, self.latent
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=x.device)
        bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=x.device)
        pos = torch.arange(self.cached, self.cached + n, dtype=torch.int32, device=x.device)
        self.cached += n
        self.kv_len.fill_(self.cached)
        seqs = m.Seqs.from_tensors(i32([0, n]), self.kv_len, self.table, n)
        kv, q = x @ self.w_kv.t(), (x @ self.w_q.t()).view(n, H, D + ROT)
        if expanded:
            m.moe_latent_append(self.rope, self.cache, seqs, kv, q[..., D:], pos, q[..., D:], gamma=self.gamma)   # in place
            cu_k, rows = i32([0, self.cached]), bf16(self.cached, L + ROT)
            m.moe_latent_gather(self.cache, seqs, cu_k, rows, self.ws)
            up = (rows[:, :L] @ self.w_up.view(-1, L).t()).view(-1, H, 2 * D)
            out = bf16(n, H, D)
            m.moe_expanded_attention(self.attn, seqs, cu_k, q, up[..., :D], rows[:, L:], up[..., D:], out, self.ws_x)
            return out
        ql, mid = bf16(n, H, L + ROT), bf16(n, H, L)
        m.moe_latent_append(self.rope, self.cache, seqs, kv, q[..., D:], pos, ql[..., L:], gamma=self.gamma)
        ql[..., :L] = torch.bmm(q[..., :D].transpose(0, 1), self.w_up[:, :D]).transpose(0, 1)
        m.moe_latent_attention(self.attn, self.cache, seqs, ql, mid, self.ws)
        return torch.bmm(mid.transpose(0, 1), self.w_up[:, D:].transpose(1, 2)).transpose(0, 1).contiguous()

    def forward(self, x, expanded=False):
        mid = x + self.attend(x, expanded).view(x.shape[0], -1) @ self.w_o.t()
        out = torch.empty_like(mid)
        m.moe_layer(self.cfg, mid, self.router, self.bias, self.weights, None, out, self.moe_ws)
        return mid + out

    def drop(self, n):
        """Takes the last n rows back."""
        self.cached -= n
        self.kv_len.fill_(self.cached)

    def check(self):
        for ws in (self.ws, self.ws_x, self.moe_ws):
            err = m.moe_get_device_error(ws)
            if err:
                raise RuntimeError(m.STATUS.get(err, err))


def main(steps=12, prompt=300, chunk=200, vocab=4096, seed=1, cache_dtype=torch.bfloat16, quiet=False):
    m.build()
    m.load()
    layer = Layer(cache_dtype=cache_dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    embed = torch.randn(vocab, SHAPE.hidden, generator=g, device="cuda").bfloat16()
    head = embed.roll(1, 0)
    tokens = torch.randint(0, vocab, (prompt,), generator=g, device="cuda")
    for part in tokens.split(chunk):
        y = layer.forward(embed[part], expanded=True)
    committed = int((y[-1:] @ head.t()).argmax())
    am, out = (torch.empty(8, dtype=torch.int32, device="cuda") for _ in range(2))
    acc, nd = (torch.full((1,), 7, dtype=torch.int32, device="cuda") for _ in range(2))
    accepted = []
    for step in range(steps):
        slip = (5 * step) % 8                     # the draft that is wrong (0: none)
        draft = [(committed + i + (i == slip > 0)) % vocab for i in range(8)]
        draft = torch.tensor(draft, dtype=torch.int32, device="cuda")
        y = layer.forward(embed[draft.long()])
        m.moe_greedy_verify(y @ head.t(), draft, nd, am, acc, out)
        k = int(acc)
        layer.drop(8 - k)
        committed = int(out[k - 1])
        accepted.append(k)
        if not quiet:
            print(f"step {step}: {k} tokens, {layer.cached} cached rows")
    layer.check()
    return accepted, layer.cached


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:2]))
