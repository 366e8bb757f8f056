"""A small decoder served with libq4k: packed Q4_K products, paged cache, attention, pick.

Runs a random-weight model of the Qwen3 / Llama layout (RMS norms, grouped
heads, rotary positions, gated feed-forward) over several sequences at once:
prompts in chunks, then single tokens, then one sequence forked into two and
the cache compacted after the others have ended.

    python examples/serve.py [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import gguf_q4_dequant_gb300 as q4k  # noqa: E402
from gguf_q4_dequant_gb300 import synth  # noqa: E402


class Model:
    """Weights: packed Q4_K matrices (drawn row by row, scaled by 1/sqrt(K) in the norms' weights)."""

    def __init__(self, layers=2, hidden=512, heads=8, kv_heads=2, dim=64, ffn=1024, vocab=1000, seed=0, device="cuda"):
        self.layers, self.hidden, self.heads, self.kv_heads, self.dim = layers, hidden, heads, kv_heads, dim
        self.ffn, self.vocab, self.device = ffn, vocab, device
        self.shapes = {"q": (heads * dim, hidden), "k": (kv_heads * dim, hidden), "v": (kv_heads * dim, hidden),
                       "o": (hidden, heads * dim), "gate": (ffn, hidden), "up": (ffn, hidden), "down": (hidden, ffn)}
        self.host = {(l, n): synth.weight_rows(seed + 1000 * l + i, *s)
                     for l in range(layers) for i, (n, s) in enumerate(self.shapes.items())}
        self.host["head"] = synth.weight_rows(seed + 999, vocab, hidden)
        self.w = {k: t.to(device) for k, t in self.host.items()}
        g = torch.Generator().manual_seed(seed)
        self.embed = torch.randn(vocab, hidden, generator=g).to(device)
        # the drawn weights have a mean of 0.2 or so and no scale of their own: small norm weights
        # with alternating signs keep the activations near 1
        sign = torch.ones(max(hidden, ffn))
        sign[1::2] = -1
        self.norm = (0.02 * sign[:hidden]).to(device)
        self.act_scale = (0.02 * sign[:ffn]).to(device)
        self.q_norm = (torch.rand(dim, generator=g) + 0.5).to(device)
        self.k_norm = (torch.rand(dim, generator=g) + 0.5).to(device)

    def rope(self, rows):
        ang = torch.arange(rows, dtype=torch.float64)[:, None] * 1e4 ** (
            -torch.arange(self.dim // 2, dtype=torch.float64) * 2 / self.dim)
        return torch.cat([ang.cos(), ang.sin()], 1).float().to(self.device)


def rms(x, w):
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w).to(torch.bfloat16)


class Server:
    """One model, one cache, up to `slots` sequences."""

    def __init__(self, model, slots=8, max_len=256, pages=64, page_size=16):
        m = self.m = model
        self.cache = q4k.Cache.empty(m.layers, pages, m.kv_heads, page_size, m.dim, slots, max_len, m.device)
        self.workspace = self.cache.workspace()
        self.rope = m.rope(self.cache.table.shape[1] * page_size)
        self.history = {}  # tokens of each sequence

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device=self.m.device)

    def step(self, chunks):
        """chunks: {sequence: its new tokens}. Returns the logits of each sequence's last token."""
        m, cache = self.m, self.cache
        seqs, news = self.ints(list(chunks)), [len(t) for t in chunks.values()]
        ends = torch.tensor(news).cumsum(0)
        starts = self.ints([0] + ends.tolist())
        status = torch.empty(len(news), dtype=torch.int32, device=m.device)
        q4k.q4k_pages_reserve(cache, seqs, starts, status)
        if int(status.sum()):
            raise RuntimeError("no pages left")
        for s, t in chunks.items():
            self.history.setdefault(s, []).extend(t)
        T = int(ends[-1])
        x = m.embed[torch.tensor([t for c in chunks.values() for t in c], device=m.device)]
        f32 = dict(dtype=torch.float32, device=m.device)
        q = torch.empty(T, m.heads, m.dim, dtype=torch.bfloat16, device=m.device)
        att = torch.empty_like(q)
        for l in range(m.layers):
            names = ("q", "k", "v")
            ys = [torch.empty(T, m.shapes[n][0], **f32) for n in names]
            q4k.q4k_matmul_multi([m.w[l, n] for n in names], [m.shapes[n][0] for n in names], m.hidden,
                                 rms(x, m.norm), T, ys)
            q4k.q4k_cache_append(cache, l, seqs, starts, *ys, q, m.heads, self.rope, 2, m.q_norm, m.k_norm)
            q4k.q4k_cache_attention(cache, l, seqs, starts, q, att, m.heads, max(news), m.dim ** -0.5,
                                    workspace=self.workspace)
            x = x + 0.02 * q4k.matmul(m.w[l, "o"], m.hidden, m.heads * m.dim, att.view(T, -1))
            ys = [torch.empty(T, m.ffn, **f32) for _ in range(2)]
            q4k.q4k_matmul_multi([m.w[l, "gate"], m.w[l, "up"]], [m.ffn] * 2, m.hidden, rms(x, m.norm), T, ys)
            act = (torch.nn.functional.silu(ys[0]) * ys[1] * m.act_scale).to(torch.bfloat16)
            x = x + q4k.matmul(m.w[l, "down"], m.hidden, m.ffn, act)
        last = rms(x[ends.to(m.device) - 1], m.norm)
        return q4k.matmul(m.w["head"], m.vocab, m.hidden, last)

    def pick(self, seqs, logits, repeat=1.3, mask=None):
        """Greedy tokens under a repeat penalty over each sequence's tokens."""
        hist = [t for s in seqs for t in self.history[s]]
        ends = torch.tensor([len(self.history[s]) for s in seqs]).cumsum(0).tolist()
        out = torch.empty(len(seqs), dtype=torch.int64, device=self.m.device)
        penalties = torch.tensor([[repeat, 0.0, 0.0]] * len(seqs), device=self.m.device)
        q4k.q4k_logits_pick(logits, len(seqs), self.m.vocab, None, out, self.ints(hist), self.ints([0] + ends),
                            penalties, mask=mask)
        return out.tolist()

    def fork(self, parent, child):
        status = torch.empty(1, dtype=torch.int32, device=self.m.device)
        q4k.q4k_pages_fork(self.cache, self.ints([parent]), self.ints([child]), status, self.workspace)
        if int(status):
            raise RuntimeError("fork refused")
        self.history[child] = list(self.history[parent])

    def end(self, seqs):
        q4k.q4k_pages_free(self.cache, self.ints(seqs))
        for s in seqs:
            self.history.pop(s)

    def compact(self):
        q4k.q4k_pages_compact(self.cache, self.workspace)


def main(steps=8):
    q4k.q4k_init()
    srv = Server(Model())
    prompts = {0: list(range(5, 45)), 1: [7, 8, 9], 2: list(range(100, 170))}
    logits = srv.step({s: t[:32] for s, t in prompts.items()})      # chunks of up to 32 tokens
    logits = srv.step({s: t[32:] or [1] for s, t in prompts.items()})
    tokens = dict(zip(prompts, srv.pick(list(prompts), logits)))
    for _ in range(steps):
        logits = srv.step({s: [t] for s, t in tokens.items()})
        tokens = dict(zip(tokens, srv.pick(list(tokens), logits)))
    srv.end([0, 1])
    srv.fork(2, 3)
    srv.compact()
    tokens = {2: tokens[2], 3: 11}
    for _ in range(steps):
        logits = srv.step({s: [t] for s, t in tokens.items()})
        tokens = dict(zip(tokens, srv.pick(list(tokens), logits)))
    for s, t in srv.history.items():
        print(f"sequence {s}: {len(t)} tokens, last {t[-steps:]}")
    print("pages in use:", int((srv.cache.refs > 0).sum()), "highest:", int(srv.cache.refs.nonzero().max()))
    if q4k.q4k_device_error() != 0:
        raise SystemExit("device error word set")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
