"""The latent-cache calls refuse tensors that are not on the current device, those behind a cache, a batch or a rope table
among them: their addresses would be read by a kernel.  Without a GPU, by tensors that only say where they are."""
import pytest
import torch

import moe_speculative_verify_gb300 as m


class On(torch.Tensor):
    """A host tensor that says that it is on device `dev`."""

    @staticmethod
    def of(t, dev):
        x = t.as_subclass(On)
        x.dev = dev
        return x

    def get_device(self):
        return getattr(self, "dev", -1)


def problem(odd=None, dev=1):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    t = dict(latent=bf(3, 16, 256), rope=bf(3, 16, 64), cu=i32(2), kv_len=i32(1), table=i32(1, 3), freqs=torch.zeros(32, 2),
             err=i32(64), kv=bf(2, 320), q_rope=bf(2, 4, 64), q_out=bf(2, 4, 64), pos=i32(2), gamma=torch.zeros(256), q=bf(2, 4, 320),
             out=bf(2, 4, 256), lse=torch.zeros(2, 4), mask=torch.zeros(2, dtype=torch.int64), ws=i32(64), ck=i32(2), rows=bf(5, 320),
             qe=bf(2, 4, 128), k=bf(5, 4, 64), v=bf(5, 4, 64), k_rope=bf(5, 64), oe=bf(2, 4, 64))
    return {k: On.of(v, dev if k == odd else 0) for k, v in t.items()}


def call(fn, t):
    cache, seqs = m.LatentCache.from_tensors(t["latent"], t["rope"]), m.Seqs.from_tensors(t["cu"], t["kv_len"], t["table"], 2)
    if fn == "append":
        m.moe_latent_append(m.Rope.from_freqs(t["freqs"], ws=t["err"]), cache, seqs, t["kv"], t["q_rope"], t["pos"], t["q_out"],
                            gamma=t["gamma"])
    elif fn == "attend":
        m.moe_latent_attention(m.Attn(4, 0.1), cache, seqs, t["q"], t["out"], t["ws"], lse=t["lse"], draft_mask=t["mask"])
    elif fn == "gather":
        m.moe_latent_gather(cache, seqs, t["ck"], t["rows"], t["ws"])
    else:
        m.moe_expanded_attention(m.Attn(4, 0.1), seqs, t["ck"], t["qe"], t["k"], t["k_rope"], t["v"], t["oe"], t["ws"], lse=t["lse"])


BATCH = ["cu", "kv_len", "table"]
USES = {"append": ["latent", "rope", *BATCH, "freqs", "err", "kv", "q_rope", "q_out", "pos", "gamma"],
        "attend": ["latent", "rope", *BATCH, "q", "out", "lse", "mask", "ws"],
        "gather": ["latent", "rope", *BATCH, "ck", "rows", "ws"],
        "expand": [*BATCH, "ck", "qe", "k", "k_rope", "v", "oe", "lse", "ws"]}


@pytest.fixture
def reached(monkeypatch):
    """Calls that get past the checks end here."""
    class Reached(Exception):
        pass

    def load():
        raise Reached
    monkeypatch.setattr(m, "load", load)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return Reached


@pytest.mark.parametrize("dev", [-1, 1])
@pytest.mark.parametrize("fn,odd", [(f, x) for f, xs in USES.items() for x in xs])
def test_a_tensor_elsewhere_is_refused(reached, fn, odd, dev):
    with pytest.raises(m.MoeError):
        call(fn, problem(odd, dev))


@pytest.mark.parametrize("fn", USES)
def test_tensors_of_one_device_are_taken(reached, fn):
    with pytest.raises(reached):
        call(fn, problem())
    t = problem()
    t["table"] = On.of(torch.zeros(1, 0, dtype=torch.int32), -1)       # empty: nowhere
    with pytest.raises(reached):
        call(fn, t)


def test_structures_of_bare_pointers_have_no_device():
    assert m.LatentCache()._dev is None and m.Seqs()._dev is None and m.Rope()._dev is None
