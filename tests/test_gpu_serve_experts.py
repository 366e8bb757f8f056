"""examples/serve_experts.py runs, and gives the same bits whichever pages hold its
sequences. (Its calls together are tested step by step in test_gpu_experts.py.)"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(q4k):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_experts
    q4k.q4k_init()
    yield serve_experts
    torch.cuda.synchronize()
    assert q4k.q4k_device_error() == 0


def test_example_runs(example, capsys):
    example.main(3)
    assert "sequence 2: " in capsys.readouterr().out


def test_the_same_tokens_give_the_same_bits(example):
    m = example.Model(seed=3)
    a, b = example.Server(m), example.Server(m)
    prompt = list(range(20, 95))
    b.step({3: [4] * 30})  # other pages are taken
    x, y = a.step({0: prompt}), b.step({1: prompt})
    assert torch.equal(x, y) and bool(torch.isfinite(x).all())
    for t in (5, 6):
        x, y = a.step({0: [t]}), b.step({1: [t]})
        assert torch.equal(x, y) and bool(torch.isfinite(x).all())
