"""The calls together, as examples/serve.py uses them: a small decoder against
the same model in float64, and against itself after forks and compaction."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def serve(q4k):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve
    q4k.q4k_init()
    yield serve
    torch.cuda.synchronize()
    assert q4k.q4k_device_error() == 0


def dense(oracle_mod, m, tokens):
    """Logits of the last token of one sequence, everything in float64."""
    w = {k: torch.tensor(oracle_mod.dequant(t.numpy(), *(m.shapes[k[1]] if k != "head" else (m.vocab, m.hidden))),
                         dtype=torch.float64) for k, t in m.host.items()}
    norm, act_scale, qn, kn = (t.cpu().double() for t in (m.norm, m.act_scale, m.q_norm, m.k_norm))
    rms = lambda x, s: x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s  # noqa: E731
    x = m.embed.cpu().double()[tokens]
    T, h = len(tokens), m.dim // 2
    ang = torch.arange(T, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(h, dtype=torch.float64) / h)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    turn = lambda x: torch.cat([x[..., :h] * c - x[..., h:] * s, x[..., :h] * s + x[..., h:] * c], -1)  # noqa: E731
    for l in range(m.layers):
        y = rms(x, norm)
        q = turn(rms((y @ w[l, "q"].T).view(T, m.heads, m.dim), qn))
        k = turn(rms((y @ w[l, "k"].T).view(T, m.kv_heads, m.dim), kn))
        v = (y @ w[l, "v"].T).view(T, m.kv_heads, m.dim)
        g = m.heads // m.kv_heads
        k, v = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
        a = torch.einsum("ihd,jhd->hij", q, k) * m.dim ** -0.5
        a = a.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -np.inf).softmax(-1)
        x = x + 0.02 * torch.einsum("hij,jhd->ihd", a, v).reshape(T, -1) @ w[l, "o"].T
        y = rms(x, norm)
        x = x + (torch.nn.functional.silu(y @ w[l, "gate"].T) * (y @ w[l, "up"].T) * act_scale) @ w[l, "down"].T
    return rms(x[-1], norm) @ w["head"].T


def test_logits_match_the_model_in_float64(serve, oracle_mod):
    """Prompts in one chunk, in several, and token by token. About twenty
    roundings to bf16 (2^-8) lie between the tokens and the logits: 5 % of the
    logits' spread is several times what they come to."""
    m = serve.Model()
    prompts = {0: list(range(3, 40)), 1: [5], 2: list(range(200, 290))}
    ref = {s: dense(oracle_mod, m, t) for s, t in prompts.items()}
    for size in (1000, 32, 7, 1):
        srv, last = serve.Server(m), {}
        for at in range(0, 90, size):
            chunks = {s: t[at:at + size] for s, t in prompts.items() if t[at:at + size]}
            if chunks:
                last.update(zip(chunks, srv.step(chunks).cpu().double()))
        for s in prompts:
            err = float((last[s] - ref[s]).norm() / (ref[s] - ref[s].mean()).norm())
            assert err < 0.05, (size, s, err)


def test_forks_and_compaction_change_nothing(serve):
    """The same tokens give the same bits whichever pages hold the sequence."""
    m = serve.Model(seed=5)
    a, b = serve.Server(m), serve.Server(m)
    prompt = list(range(50, 123))
    a.step({0: prompt})
    b.step({4: [1] * 40, 5: [2] * 33})
    b.step({6: prompt})
    b.end([4])
    b.compact()
    b.fork(6, 1)
    b.step({6: [9, 9, 9]})
    b.end([5, 6])
    b.compact()
    for t in (3, 1, 4, 1, 5, 9):
        x, y = a.step({0: [t]}), b.step({1: [t]})
        assert torch.equal(x, y)
    assert a.pick([0], x) == b.pick([1], y)
    used = int((b.cache.refs > 0).sum())
    assert used == -(-79 // 16) and int(b.cache.refs.nonzero().max()) < used + 2


def test_example_runs(serve, capsys):
    serve.main(3)
    assert "sequence 3: " in capsys.readouterr().out
