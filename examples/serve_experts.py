"""The decoder of serve.py with a mixture of experts for its feed-forward part.

Every layer's norm takes what attention adds and writes the rows for the
router and the experts in bf16; the router's picks put the rows in the order
of their experts, whose packed Q4_K matrices give gate, up and down; the rows
come back to their tokens with the picks' weights, onto the residual stream.

    python examples/serve_experts.py [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "examples")):
    if path not in sys.path:
        sys.path.insert(0, path)

import gguf_q4_dequant_gb300 as q4k  # noqa: E402
import serve  # noqa: E402
from gguf_q4_dequant_gb300 import synth  # noqa: E402


class Model(serve.Model):
    """serve.Model with `experts` packed matrices each for gate, up and down, and a packed router."""

    def __init__(self, experts=16, top=4, ffn=256, seed=0, **kw):
        super().__init__(ffn=ffn, seed=seed, **kw)
        self.experts, self.top = experts, top
        for l in range(self.layers):
            self.host[l, "router"] = synth.weight_rows(seed + 1000 * l + 50, experts, self.hidden)
            for i, name in enumerate(("gate", "up", "down")):
                n, k = self.shapes[name]
                self.host[l, name] = torch.cat([synth.weight_rows(seed + 1000 * l + 100 * (i + 1) + e, n, k) for e in range(experts)])
            for name in ("router", "gate", "up", "down"):
                self.w[l, name] = self.host[l, name].to(self.device)
        self.out_scale = 0.002  # of the experts' outputs: the drawn weights have no scale of their own


class Server(serve.Server):
    def feed_forward(self, l, x, delta):
        m, (T, C) = self.m, x.shape
        P, dev = T * m.top, m.device
        def new(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=dev)
        bf16, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
        h = new(T, C, dtype=bf16)
        q4k.q4k_add_norm(x, delta, m.norm, 1e-6, sum=x, out=h)
        logits = q4k.matmul(m.w[l, "router"], m.experts, C, h)
        ids, weights, slots = new(T, m.top, dtype=i32), new(T, m.top), new(T, m.top, dtype=i32)
        order, starts = new(P, dtype=i32), new(m.experts + 1, dtype=i32)
        q4k.q4k_route(logits, m.top, q4k.ROUTE_SOFTMAX_TOP, m.out_scale, ids, weights, order, slots, starts,
                      new(q4k.q4k_route_workspace(T, m.experts), dtype=u8))
        rows, act, y = new(P, C, dtype=bf16), new(P, m.ffn, dtype=bf16), new(P, C, dtype=bf16)
        q4k.q4k_experts_gather(h, order, m.top, rows)
        q4k.q4k_experts_gated(m.w[l, "gate"], m.w[l, "up"], m.ffn, C, rows, starts, act)
        q4k.q4k_experts_matmul(m.w[l, "down"], C, m.ffn, act, starts, y)
        out = new(T, C)
        q4k.q4k_experts_combine(y, slots, weights, out, base=x)
        return out


def main(steps=8):
    q4k.q4k_init()
    srv = Server(Model())
    prompts = {0: list(range(5, 45)), 1: [7, 8, 9], 2: list(range(100, 170))}
    tokens = dict(zip(prompts, srv.pick(list(prompts), srv.step(prompts))))
    for _ in range(steps):
        tokens = dict(zip(tokens, srv.pick(list(tokens), srv.step({s: [t] for s, t in tokens.items()}))))
    for s, t in srv.history.items():
        print(f"sequence {s}: {len(t)} tokens, last {t[-steps:]}")
    if q4k.q4k_device_error() != 0:
        raise SystemExit("device error word set")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
