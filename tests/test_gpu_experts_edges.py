"""The expert layer's calls where numbers or sizes come to an edge, against plain
implementations in 64 bits. Tolerances count half a step for every rounding
(bf16 2^-8, fp32 2^-24, relative); they are derived at each test."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _cuda(q4k):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    torch.cuda.set_device(0)
    q4k.q4k_init()
    yield
    torch.cuda.synchronize()
    assert q4k.q4k_device_error() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def new(*shape, dtype=torch.float32, fill=0):
    return torch.full(shape, fill, dtype=dtype, device=DEV)


def route(q4k, logits, k, weighting, scale=1.0):
    """ids, weights, order, slots, starts of a call, on the device."""
    T, E = logits.shape
    i32 = torch.int32
    ids, slots, order, starts = (new(*s, dtype=i32, fill=-77) for s in ((T, k), (T, k), (T * k,), (E + 1,)))
    weights, ws = new(T, k, fill=float("nan")), new(q4k.q4k_route_workspace(T, E), dtype=torch.uint8, fill=0xEE)
    q4k.q4k_route(logits.to(DEV), k, weighting, scale, ids, weights, order, slots, starts, ws)
    return ids, weights, order, slots, starts


# ------------------------------------------------------------------- route ---

@pytest.mark.parametrize("T", [5, 900])
@pytest.mark.parametrize("spread", [1.0, 30.0, 70.0])
@pytest.mark.parametrize("top", [3.0, 0.0, -1e-3, -0.5, -10.0, -17.0, -30.0, -60.0, -63.9, -64.1, -90.0, -500.0])
def test_sigmoids_over_their_sum(q4k, T, top, spread):
    """Each weight is right relative to itself, however far below the largest it is. The exponentials are good to two
    steps each, their sums, quotients and the scale add a rounding each, five for the tree of the sum: 2^-19; the
    difference of two logits has its rounding as many times as it is large: 2^-24 |x - top|. (What is below 2^-125
    is left out: fp32 ends there.)"""
    E, k, scale = 11, 5, 1.5
    logits = top - spread * torch.rand(T, E, generator=gen(T))
    logits[:, 4] = top
    logits[:, 7] = top - spread
    got = route(q4k, logits, k, q4k.ROUTE_SIGMOID_TOP, scale)[1].cpu().double()
    x = torch.sort(logits.double(), dim=1, descending=True).values[:, :k]
    rel = torch.exp(x - top) / (1 + torch.exp(x))  # sigmoid(x) / e^top
    want = rel / rel.sum(1, keepdim=True) * scale
    tol = (2.0 ** -19 + 2.0 ** -24 * (x - top).abs()) * want
    assert bool(((got - want).abs() <= tol)[want > 2.0 ** -124].all())


def test_sigmoids_of_masks_over_their_sum(q4k):
    """A token with nothing but a type's lowest values has weights of 0; beside a score they count for nothing."""
    low = torch.tensor([-65504.0, -3.3895313892515355e38, -3.4028234663852886e38, -1e4])
    logits = low.unsqueeze(1).repeat(1, 6)
    logits = torch.cat([logits, logits])
    logits[4:, 2] = -40.0
    ids, w, _, _, _ = route(q4k, logits, 3, q4k.ROUTE_SIGMOID_TOP)
    assert bool((w[:4] == 0).all())
    assert w[4:].tolist() == [[1.0, 0.0, 0.0]] * 4 and ids[4:].tolist() == [[2, 0, 1]] * 4


# -------------------------------------------------------------------- norm ---

@pytest.mark.parametrize("C", [512, 1056, 9216, 32768])
@pytest.mark.parametrize("size", [1e18, 4e18])
def test_norm_sums_past_fp32(q4k, C, size):
    """Rows whose squares have a sum past fp32, but not a mean. The sum goes through a chain of at most 32 terms and two
    trees of 5, half of which counts after the root; the mean, the root and the products add a rounding each: 2^-19."""
    g = gen(C)
    x = torch.randn(3, C, generator=g).clamp(-4, 4) * size
    x[2] *= 2.0 ** -40  # (and one without)
    w = 0.5 + torch.rand(C, generator=g)
    out = new(3, C)
    q4k.q4k_add_norm(x.to(DEV), None, w.to(DEV), 1e-6, out=out)
    r = x.double()
    y = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    assert bool(((out.cpu().double() - y).abs() <= 2.0 ** -19 * y.abs()).all())


@pytest.mark.parametrize("C", [64, 1056, 9216])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_norm_weights_past_the_row(q4k, C, kind):
    """Weights and rows whose products leave fp32's range although the norm does not. The sum of squares goes through
    a chain of at most 32 terms and two trees of 5, half of which counts after the root; the mean, the root and the
    products add a rounding each: 2^-19."""
    g = gen(C)
    sizes = torch.tensor([1e18, 3e15, 1.0, 1e-9, 1e-15])
    x = (torch.randn(5, C, generator=g).clamp(-4, 4) * sizes.unsqueeze(1)).to(kind)
    for weight in (1e-30, 1e-20, 1e22, 1e30, 1e35):
        w = (0.5 + torch.rand(C, generator=g)) * weight
        out = new(5, C)
        q4k.q4k_add_norm(x.to(DEV), None, w.to(DEV), 0.0, out=out)
        r = x.double()
        y = r / r.square().mean(1, keepdim=True).sqrt() * w.double()
        far = y.abs() > 2.0 ** -120  # (below, fp32 has fewer bits)
        assert bool(((out.cpu().double() - y).abs() <= 2.0 ** -19 * y.abs())[far].all())


@pytest.mark.parametrize("weight", [0.25, 1.0, 4.0, -1e30])
def test_norm_of_rows_past_fp32(q4k, weight):
    """Squares past fp32: the root is infinite, the row 0, whatever the weight; codes and scales of zeros."""
    C = 96
    x = torch.full((2, C), 3e38)
    x[1, 1:] = 1.0
    out, codes, scales = new(2, C, fill=7), new(2, C, dtype=torch.uint8, fill=1), new(2, C // 32, dtype=torch.uint8, fill=1)
    q4k.q4k_add_norm(x.to(DEV), None, new(C, fill=weight), 1e-6, out=out, codes=codes, scales=scales)
    assert bool((out == 0).all()) and bool((codes & 127 == 0).all()) and bool((scales == 0).all())
