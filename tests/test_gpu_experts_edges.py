"""The expert layer's calls where numbers or sizes come to an edge, against plain
implementations in 64 bits. Tolerances count half a step for every rounding
(bf16 2^-8, fp32 2^-24, relative); they are derived at each test."""
import pytest
import torch

from captured import kernels
from gguf_q4_dequant_gb300 import synth
from test_gpu_experts import Layer

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


def check_route(q4k, logits, k, weighting):
    """Everything that a call gives, against a stable sort of 64-bit logits and of the pairs by expert."""
    T, E = logits.shape
    ids, weights, order, slots, starts = route(q4k, logits, k, weighting)
    x = logits.to(DEV).double()
    x = torch.where(x.isnan(), float("-inf"), x)
    key, want = (t[:, :k] for t in torch.sort(x, dim=1, descending=True, stable=True))
    live = key > float("-inf")
    want = torch.where(live, want, -1)
    assert torch.equal(ids.long(), want)
    flat = want.flatten()
    pairs = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    n = int(live.sum())
    assert torch.equal(order[:n].long(), pairs[:n]) and bool((order[n:] == -1).all())
    at = torch.full_like(flat, -1)
    at[pairs[:n]] = torch.arange(n, device=DEV)
    assert torch.equal(slots.flatten().long(), at)
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    assert starts.tolist() == [0, *counts.cumsum(0).tolist()]
    # exponentials to two steps, sums of at most 32 terms and a tree of 5 with a rounding each, and the quotient: 2^-18;
    # a difference's rounding as many times as it is large
    rel = torch.where(live, torch.exp(key - key[:, :1]), 0.0)
    total = (torch.exp(x - key[:, :1]) if weighting == q4k.ROUTE_SOFTMAX else rel).nan_to_num(0).sum(1, keepdim=True)
    w = torch.where(live, rel / total, 0.0)
    d = torch.where(live, key - key[:, :1], 0.0).abs()
    assert bool(((weights.double() - w).abs() <= (2.0 ** -18 + 2.0 ** -23 * d) * w + 1e-37).all())


@pytest.mark.parametrize("T", [8191, 8192, 8193, 8257, 20011])
@pytest.mark.parametrize("E,k", [(61, 4), (1000, 17), (128, 8), (1024, 32), (33, 1), (5, 5)])
def test_route_of_many_groups(q4k, T, E, k):
    """Both sides of 128 groups of 64 tokens, above which the counts are scanned by a kernel of their own."""
    g = gen(T + E)
    logits = torch.randn(T, E, generator=g) * 3
    on_device = logits.to(DEV)
    names = kernels(lambda: route(q4k, on_device, k, q4k.ROUTE_SOFTMAX))
    assert any("route_scan" in n for n in names) == (T > 8192)
    check_route(q4k, logits, k, q4k.ROUTE_SOFTMAX)
    logits = torch.round(logits)  # ties, masks, tokens without an expert, experts without a token
    logits[torch.rand(T, E, generator=g) < 0.6] = float("-inf")
    logits[torch.rand(T, E, generator=g) < 0.1] = float("nan")
    logits[::97] = float("-inf")
    logits[:, ::7] = float("-inf")
    if E > 5:
        logits[:, 3] = 1e3
    check_route(q4k, logits, k, q4k.ROUTE_SOFTMAX_TOP)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_layer_of_many_groups_captured(q4k, mode):
    """A layer whose route has all of its launches, captured twice in a row, in every launch mode."""
    layer = Layer(q4k, 8300, 6, 2, 256, 256, True, seed=5)
    old = q4k.q4k_set_pdl(mode)
    try:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(side):
            layer.run()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=side):
                layer.run()
                layer.run()
        for _ in range(2):
            layer.dx.normal_()
            layer.out.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            graph.replay()
            torch.cuda.synchronize()
            layer.check()
    finally:
        q4k.q4k_set_pdl(old)


def test_route_of_the_most_tokens(q4k):
    """2^31 - 1 tokens, every fifth without its expert: the count of the groups stays in 32 bits."""
    T, i32 = (1 << 31) - 1, torch.int32
    logits = new(T, 1)
    logits[::5] = float("-inf")
    ids, slots, order, starts = (new(n, dtype=i32, fill=-77) for n in (T, T, T, 2))
    weights, ws = new(T, fill=7), new(q4k.q4k_route_workspace(T, 1), dtype=torch.uint8)
    q4k.q4k_route(logits, 1, q4k.ROUTE_SOFTMAX, 1.0, ids, weights, order, slots, starts, ws)
    n = T - (T + 4) // 5
    assert starts.tolist() == [0, n]
    for at in range(0, T, 1 << 28):
        i = torch.arange(at, min(at + (1 << 28), T), device=DEV)
        part, live = slice(at, at + len(i)), i % 5 != 0
        assert torch.equal(ids[part], torch.where(live, 0, -1).to(i32)) and torch.equal(weights[part], live.float())
        assert torch.equal(slots[part], torch.where(live, i - i // 5 - 1, -1).to(i32))
        assert torch.equal(order[part], torch.where(i < n, i + i // 4 + 1, -1).to(i32))


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


# ---------------------------------------------------------------- products ---

def fields(w):
    """a = d sc, b = dmin m and the code q of each weight of packed rows [.., K / 256 * 144], in 64 bits: w = a q - b."""
    blocks = w.reshape(w.shape[0], -1, 144)
    d, dmin = blocks[..., :4].contiguous().view(torch.float16).double().unbind(-1)
    s, qs = blocks[..., 4:16].long(), blocks[..., 16:].long().unflatten(-1, (4, 32))
    sc = torch.cat((s[..., :4] % 64, s[..., 8:] % 16 + s[..., :4] // 64 * 16), -1)
    m = torch.cat((s[..., 4:8] % 64, s[..., 8:] // 16 + s[..., 4:8] // 64 * 16), -1)
    q = torch.stack((qs % 16, qs // 16), -2).flatten(-3, -2).double()
    a, b = d.unsqueeze(-1) * sc, dmin.unsqueeze(-1) * m
    return a.repeat_interleave(32, -1).flatten(1), b.repeat_interleave(32, -1).flatten(1), q.flatten(-2).flatten(1)


def set_heads(w, heads):
    """d and dmin of the super-blocks in turn, as fp16."""
    blocks = w.view(-1, 144)
    h = torch.tensor(heads, dtype=F64).to(torch.float16)
    blocks[:, :4] = h[torch.arange(len(blocks)) % len(h)].view(torch.uint8)


def many_bound(a, b, w):
    """How far the weights of the kernel for many rows may be off: bf16 roundings of r, of the inner FMA (|r| and 2^-8 of
    what d leaves) and of the weight; fp32 ones of a and b (2^-24), and a c on the other side of a tie, 2^-19 |a|."""
    c = torch.where(a != 0, b / a, 0.0).mul(16).round().clamp(0, 255) / 16
    return 2.0 ** -8 * (1 + 2.0 ** -6) * (w.abs() + 2 * (c * a - b).abs()) + 2.0 ** -19 * a.abs()


def product(q4k, gated, w, w2, N, K, x, starts, y):
    if gated:
        q4k.q4k_experts_gated(w, w2, N, K, x, starts, y)
    else:
        q4k.q4k_experts_matmul(w, N, K, x, starts, y)


def check_kernel(many, call):
    """Which of the two kernels the call takes."""
    name, = kernels(call)
    assert ("experts_gemm_kernel" in name) == many, name


def test_single_weights_of_many_rows(q4k):
    """Rows of x with one power of two each: the outputs are the weights that the kernel for many rows takes, exactly."""
    E, N, K = 2, 256, 512
    w = torch.stack([synth.weight_rows(40 + e, N, K) for e in range(E)])
    g = gen(4)
    w.view(-1, 144)[:, 4:] = torch.randint(0, 256, (E * N * K // 256, 140), generator=g, dtype=torch.uint8)
    d = torch.exp2(-14 * torch.rand(997, generator=g, dtype=F64))
    odd = [[0.0, 1.0], [1.0, 0.0], [0.0, 0.0], [-1.0, 2.0], [2.0, -1.0], [-1.0, -4.0], [2.0 ** -24, 2.0 ** -24],
           [2.0 ** -24, 1.0], [1.0, 2.0 ** -24], [60.0, 60.0], [6e4, 6e4], [0.830078125, 15.2265625], [0.00014150143, 0.0004968643]]
    set_heads(w, odd + torch.stack((d, d * 16 * torch.rand(997, generator=g, dtype=F64)), 1).tolist())
    # two sub-blocks whose errors are among the largest
    for row, head, sc, m, q in ((3, odd[-2], 39, 34, 14), (5, odd[-1], 21, 8, 2)):
        block = w[1].view(N, K // 256, 144)[row, 0]
        block[:4] = torch.tensor(head, dtype=torch.float16).view(torch.uint8)
        block[4], block[8], block[16] = sc, m, q
    size = torch.exp2(torch.arange(4, dtype=F64) * 3 - 6).repeat_interleave(K) * (1 - 2 * (torch.arange(4 * K) % 2))
    x = (torch.eye(K, dtype=F64).repeat(4, 1) * size.unsqueeze(1)).to(torch.bfloat16).repeat(E, 1).to(DEV)
    starts = torch.tensor([0, 4 * K, 8 * K], dtype=torch.int32, device=DEV)
    y = new(E * 4 * K, N, dtype=torch.bfloat16)
    wd = w.to(DEV)
    call = lambda: q4k.q4k_experts_matmul(wd, N, K, x, starts, y)  # noqa: E731
    check_kernel(True, call)
    for e in range(E):
        a, b, q = fields(w[e].reshape(N, -1))
        want = a * q - b
        tol = many_bound(a, b, want)
        got = y[4 * K * e:4 * K * (e + 1)].cpu().double() / size.unsqueeze(1)
        assert bool(((got.view(4, K, N) - want.T).abs() <= tol.T).all())
        # what the header says of weights around 0, and elsewhere
        inside = (a != 0) & (b / a >= 0) & (b / a <= 15.96)
        assert bool((tol <= 2.0 ** -8 * 1.03 * (want.abs() + a.abs() / 16))[inside].all())
        assert bool((tol <= 2.0 ** -8 * 3.06 * want.abs() + 2.0 ** -19 * a.abs())[~inside].all())


class Experts:
    """E packed matrices [N][K] (`distinct` different ones in turn), their products in 64 bits and how far each of the
    two kernels may be off."""

    def __init__(self, seed, E, N, K, distinct=None, change=None):
        self.E, self.N, self.K = E, N, K
        w = torch.stack([synth.weight_rows(seed + e, N, K).view(N, -1) for e in range(distinct or E)])
        if change is not None:
            change(w)
        self.fields = [[t.to(DEV) for t in fields(m)] for m in w]
        self.packed = w.repeat(E // len(w), 1, 1).to(DEV)

    def product(self, e, x, many):
        """x W_e^T, and the bound: the weights' error for many rows; for few each sum of 32 x as two bf16, 2^-16; fp32
        sums over K / 16 products of 16 and what joins them, 2^-23 each."""
        a, b, q = self.fields[e % len(self.fields)]
        w, x = a * q - b, x.double()
        tol = 2.0 ** -23 * (self.K / 16 + 64) * (x.abs() @ ((a * q).abs() + b.abs()).T)
        if many:
            tol += x.abs() @ many_bound(a, b, w).T
        else:
            tol += 2.0 ** -16 * (x.unflatten(1, (-1, 32)).sum(2).abs() @ b.abs()[:, ::32].T)
        return x @ w.T, tol


def gated_of(g, tg, u, tu):
    """silu(g) u and its bound from those of the factors: |silu'| <= 1.1, |silu(g)| <= |g|, 2^-20 for silu itself."""
    silu = g * torch.sigmoid(g)
    return silu * u, 1.1 * tg * (u.abs() + tu) + silu.abs() * tu + 2.0 ** -20 * (silu * u).abs()


def check_products(q4k, w, up, counts, x, many, lead=0):
    """The product of every expert (gated with `up`), by the kernel that is meant; rows of no expert stay."""
    starts = [lead]
    for c in counts:
        starts.append(starts[-1] + c)
    assert len(x) >= starts[-1] and len(counts) == w.E
    x[:lead], x[starts[-1]:] = float("nan"), float("nan")
    y = new(len(x), w.N, dtype=torch.bfloat16, fill=-12345)
    keep = y[0, 0].clone()
    at = torch.tensor(starts, dtype=torch.int32, device=DEV)
    check_kernel(many, lambda: product(q4k, up is not None, w.packed, None if up is None else up.packed, w.N, w.K, x, at, y))
    assert bool((y[:lead] == keep).all()) and bool((y[starts[-1]:] == keep).all())
    for e, (a, b) in enumerate(zip(starts, starts[1:])):
        if a == b:
            continue
        want, tol = w.product(e, x[a:b], many)
        if up is not None:
            want, tol = gated_of(want, tol, *up.product(e, x[a:b], many))
        err = (y[a:b].double() - want).abs()
        assert bool((err <= tol + 2.0 ** -8 * want.abs() + 1e-38).all()), (e, float((err - 2.0 ** -8 * want.abs()).div(tol).max()))


def uneven(seed, E, rows, empty):
    """E counts that add up to `rows`, a share of them 0 (the first and the last too)."""
    g = gen(seed)
    live = torch.rand(E, generator=g) >= empty
    live[0] = live[-1] = False
    cut = torch.sort(torch.randint(0, rows + 1, (int(live.sum()) - 1,), generator=g)).values.tolist()
    counts = torch.zeros(E, dtype=torch.int64)
    counts[live] = torch.tensor([0, *cut, rows]).diff()
    return counts.tolist()


def draw_x(seed, P, K, size=1.0):
    return (torch.randn(P, K, generator=gen(seed)) * size).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,K,rows,empty", [(128, 128, 256, 6000, 0.3), (40, 300, 4096, 1700, 0.2), (1024, 200, 256, 41000, 0.5),
                                              (33, 129, 512, 4000, 0.8), (3, 144, 16384, 3300, 0.0), (64, 512, 1280, 3000, 0.1)])
def test_many_rows_of_many_experts(q4k, E, N, K, rows, empty, gated):
    """More experts than lanes, most of them or none empty, and long rows, in the kernel for many rows."""
    distinct = 8 if E % 8 == 0 else E
    w = Experts(E + N, E, N, K, distinct)
    up = Experts(E + N + 5000, E, N, K, distinct) if gated else None
    check_products(q4k, w, up, uneven(E, E, rows, empty), draw_x(E + K, rows + 7, K, 0.02 if gated else 1.0), True, lead=3)


def odd_heads(w):
    """Super-blocks whose d or dmin is 0, negative, the smallest number or large."""
    set_heads(w, [[0.0, 1.0], [1.0, 0.0], [0.0, 0.0], [-1.0, 2.0], [2.0, -1.0], [-1.0, -4.0], [2.0 ** -24, 2.0 ** -24],
                  [2.0 ** -24, 1.0], [1.0, 2.0 ** -24], [60.0, 60.0]])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,many", [([3, 9], False), ([200, 90], False), ([6000, 4100], True)])
def test_odd_heads(q4k, counts, many, gated):
    w = Experts(31, 2, 40, 512, change=odd_heads)
    up = Experts(35, 2, 40, 512, change=odd_heads) if gated else None
    check_products(q4k, w, up, counts, draw_x(5, sum(counts), 512, 2.0 ** -6 if gated else 1.0), many)


@pytest.mark.parametrize("counts", [[1, 192, 0, 2400], [193, 4000, 191, 1], [385, 2303, 2305, 16]])
def test_tiles_of_many_rows(q4k, counts):
    """Rows of an expert around the borders of the tiles that they are cut into."""
    check_products(q4k, Experts(50, 4, 257, 512), None, counts, draw_x(9, sum(counts) + 1, 512), True)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,counts,many", [(1, 65536, [24], True), (2, 40000, [3, 30], False), (1, 70001, [31], True),
                                             (3, 30011, [0, 33, 20], False)])
def test_many_columns_of_few_rows(q4k, E, N, counts, many, gated):
    """Columns enough for the kernel of many rows, with fewer rows than its boxes of x have, and somewhat fewer."""
    w = Experts(E + N, E, N, 256)
    up = Experts(E + N + 5000, E, N, 256) if gated else None
    check_products(q4k, w, up, counts, draw_x(N, sum(counts), 256, 0.02 if gated else 1.0), many)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,K,counts", [(1, 64, 512, [1]), (2, 64, 512, [8, 7]), (4, 61, 2048, [8, 0, 1, 17]), (3, 36, 4352, [2, 1, 4]),
                                          (2, 300, 256, [40, 25]), (40, 64, 512, [1, 2, 3, 0] * 10), (5, 640, 768, [16, 0, 9, 3, 1])])
def test_weights_of_few_rows(q4k, E, N, K, counts, gated):
    """The kernel for few rows takes weights as they are: no bf16 rounding of them would pass."""
    w = Experts(E * N + K, E, N, K)
    up = Experts(E * N + K + 5000, E, N, K) if gated else None
    check_products(q4k, w, up, counts, draw_x(K, sum(counts), K, 0.02 if gated else 1.0), False)


def large_mins(w):
    """Mins as large as the codes' mean, so that a sum of x counts as much as all the products."""
    set_heads(w, [[1.0, 7.5], [0.25, 1.875], [0.01, 0.075]])
    blocks = w.view(-1, 144)
    blocks[:, 8:12] = blocks[:, 4:8]
    blocks[:, 12:16] = (blocks[:, 12:16] & 15) * 17  # (with the upper bits alike: every min as its scale)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,K,counts", [(1, 64, 256, [8]), (2, 64, 512, [8, 7]), (3, 61, 1024, [3, 0, 9]), (1, 640, 768, [21])])
def test_sums_of_x_of_few_rows(q4k, E, N, K, counts, gated):
    """x of one sign and large mins: the sums of x are kept to 2^-16, one bf16 each would not pass."""
    w = Experts(E * N + K, E, N, K, change=large_mins)
    up = Experts(E * N + K + 5000, E, N, K, change=large_mins) if gated else None
    x = ((0.5 + torch.rand(sum(counts), K, generator=gen(K))) * (2.0 ** -14 if gated else 1.0)).to(torch.bfloat16).to(DEV)
    check_products(q4k, w, up, counts, x, False)
