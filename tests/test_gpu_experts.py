"""The expert layer's calls on the GPU, against plain implementations in 64
bits: norm with the residual's addition, routing, gathering, the experts'
packed products, the weighted way back.

Tolerances follow from the number formats, half a step for every rounding (bf16
2^-8, fp32 2^-24, e4m3 2^-4, relative).
* norm: a sum of squares in fp32 goes through a chain of at most 32 terms and two
  trees of 5, half of which counts after the root; the residual's addition, the
  mean, the root, the division and two products add a rounding each: 2^-19.
* weights of the picks: exp and the division are good to 2 steps, sums of at most
  32 terms and a tree of 5 to 37; exp of a difference x has its rounding |x| times.
* combine: k + 1 roundings of the sums' magnitudes.
* products: the output's rounding 2^-8 |y|; where the rows are many the weights as
  bf16, w = (q - c) d + r with c the code nearest to w = 0, of two roundings: r = c d - m's,
  and the sum's, 2^-8 sum (|w| + |r|) |x| (d is kept as two bf16; c may fall to either
  side of a tie, 2^-20 |d|); where they are few the sums of x beside the mins as two bf16,
  2^-16 sum |dmin m x|; fp32 sums over K / 16 products of 16 and what is behind them,
  2^-23 (K/16 + 64) sum (|d sc q x| + |dmin m x|).
* a gated product has the errors of both factors: |silu'| <= 1.1, silu(g) <= |g|.
"""
import numpy as np
import pytest
import torch

from gguf_q4_dequant_gb300 import synth

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


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bits(t):
    return t.cpu().view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.cpu().contiguous().view(torch.uint8)


# -------------------------------------------------------------------- norm ---

def norm_ref(x, delta, w, eps):
    r = x.double() + (0 if delta is None else delta.double())
    return r, r / torch.sqrt(r.square().mean(1, keepdim=True) + eps) * w.double()


def scale_bytes(y):
    """log2(s) + 127 of the smallest power of two s >= 2^-127 with max|y| <= 448 s, per 32 columns of float32 y."""
    top = y.double().abs().view(y.shape[0], -1, 32).amax(2)
    e = torch.full(top.shape, -127.0, dtype=F64)
    while True:
        more = top > 448 * torch.exp2(e)
        if not more.any():
            return (e + 127).to(torch.uint8)
        e = torch.where(more, e + 1, e)


@pytest.mark.parametrize("T,C", [(1, 32), (3, 64), (5, 256), (2, 288), (7, 512), (4, 1024), (3, 1056), (130, 2048),
                                 (1, 4096), (2, 5120), (3, 8192), (2, 8224), (2, 16384), (2, 16416), (1, 32768)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norm(q4k, T, C, kind):
    g = gen(T * 7 + C)
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    x = (torch.randn(T, C, generator=g) * torch.exp(torch.randn(C, generator=g))).to(dt)
    delta = torch.randn(T, C, generator=g) if T != 3 else None
    w = torch.randn(C, generator=g)
    r, y = norm_ref(x, delta, w, 1e-5)
    d = None if delta is None else delta.to(DEV)
    guard = 64
    out = torch.full((T * C + guard,), float("nan"), device=DEV)
    sum_ = torch.full((T * C + guard,), 7.0, device=DEV, dtype=dt)
    codes = torch.full((T * C + guard,), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full((T * C // 32 + guard,), 0xA5, dtype=torch.uint8, device=DEV)
    q4k.q4k_add_norm(x.to(DEV), d, w.to(DEV), 1e-5, sum=sum_, out=out, codes=codes, scales=scales)
    got = out[:T * C].view(T, C).cpu()
    assert bool(((got.double() - y).abs() <= 2.0 ** -19 * y.abs()).all())
    half = 2.0 ** -24 if kind == "f32" else 2.0 ** -24 + 2.0 ** -8
    assert bool(((sum_[:T * C].view(T, C).cpu().double() - r).abs() <= half * r.abs()).all())
    # the codes are those of the fp32 rows, bit for bit
    sb = scale_bytes(got)
    assert torch.equal(scales[:T * C // 32].view(T, -1).cpu(), sb)
    v = got.double().view(T, -1, 32) * torch.exp2(127 - sb.double()).unsqueeze(2)
    want = v.float().view(T, C).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(codes[:T * C].view(T, C).cpu(), want)
    assert bool(out[T * C:].isnan().all()) and bool((sum_[T * C:] == 7).all())
    assert bool((codes[T * C:] == 0xA5).all()) and bool((scales[T * C // 32:] == 0xA5).all())
    # bf16 rows, in place
    xd, ob = x.to(DEV), torch.empty(T, C, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_add_norm(xd, d, w.to(DEV), 1e-5, sum=xd, out=ob)
    assert torch.equal(ob.cpu(), got.to(torch.bfloat16))
    assert torch.equal(bits(xd), bits(sum_[:T * C].view(T, C)))


def test_norm_special_rows(q4k):
    C = 96
    x = torch.zeros(6, C)
    x[1] = 1e-30
    x[2, 5] = float("inf")
    x[3, 40] = float("nan")
    x[4] = 448.0 * 2.0 ** torch.arange(C).div(32, rounding_mode="floor")
    x[5, 3] = 3e38
    w = torch.ones(C)
    out = torch.empty(6, C, device=DEV)
    codes = torch.empty(6, C, device=DEV, dtype=torch.float8_e4m3fn)
    scales = torch.empty(6, C // 32, device=DEV, dtype=torch.uint8)
    q4k.q4k_add_norm(x.to(DEV), None, w.to(DEV), 1e-6, out=out, codes=codes, scales=scales)
    out, s = out.cpu(), scales.cpu()
    assert bool((out[0] == 0).all()) and bool((s[0] == 0).all()) and bool((codes[0].cpu().float() == 0).all())
    assert bool(((out[1] / 1e-27 - 1).abs() < 1e-5).all())
    # an infinite residual: the infinity times 0 is NaN, the rest 0; a NaN: all NaN
    assert bool(out[2, 5].isnan()) and bool((out[2, 32:] == 0).all()) and s[2].tolist() == [255, 0, 0]
    assert bool(codes[2, :32].cpu().float().isnan().all()) and bool((codes[2, 32:].cpu().float() == 0).all())
    assert bool(out[3].isnan().all()) and s[3].tolist() == [255] * 3
    # sums of squares beyond fp32: the root is infinite and the row 0
    assert bool((out[5] == 0).all())
    assert s[4].tolist() == scale_bytes(out[4:5])[0].tolist()


# ------------------------------------------------------------------- route ---

def route_ref(logits, k, weighting, scale):
    T, E = logits.shape
    z = logits.double()
    z = torch.where(z.isnan(), float("-inf"), z)
    key, ids = torch.sort(z, dim=1, descending=True, stable=True)
    key, ids = key[:, :k], ids[:, :k]
    live = key > float("-inf")
    top = key[:, :1]
    rel = lambda x: torch.where(x == top, 1.0, torch.where(x > float("-inf"), torch.exp(x - top), 0.0))  # noqa: E731
    if weighting in (0, 1):
        w = rel(key)
        total = (rel(z) if weighting == 0 else w).sum(1, keepdim=True)
    else:
        w = torch.sigmoid(key)
        total = w.sum(1, keepdim=True) if weighting == 3 else torch.ones(T, 1, dtype=F64)
    w = torch.where(live, w / total.clamp(min=1e-300), 0.0) * scale
    ids = torch.where(live, ids, -1)
    flat = ids.reshape(-1).numpy()
    used = np.nonzero(flat >= 0)[0]
    order = np.full(T * k, -1)
    order[:len(used)] = used[np.argsort(flat[used], kind="stable")]
    slots = np.full(T * k, -1)
    slots[order[:len(used)]] = np.arange(len(used))
    starts = np.concatenate([[0], np.cumsum(np.bincount(flat[used], minlength=E))])
    return ids, w, order, slots.reshape(T, k), starts, key - top


def route(q4k, logits, k, weighting, scale=1.0, pad=5):
    T, E = logits.shape
    n = T * k
    outs = dict(ids=n, order=n, slots=n, starts=E + 1)
    b = {m: torch.full((s + pad,), -77, dtype=torch.int32, device=DEV) for m, s in outs.items()}
    w = torch.full((n + pad,), float("nan"), device=DEV)
    ws = torch.full((q4k.q4k_route_workspace(T, E) + pad,), 0xEE, dtype=torch.uint8, device=DEV)
    q4k.q4k_route(logits.to(DEV), k, weighting, scale, b["ids"], w, b["order"], b["slots"], b["starts"], ws)
    for m, s in outs.items():
        assert bool((b[m][s:] == -77).all()), m
    assert bool(w[n:].isnan().all()) and bool((ws[-pad:] == 0xEE).all())
    return (b["ids"][:n].view(T, k).cpu(), w[:n].view(T, k).cpu(), b["order"][:n].cpu(), b["slots"][:n].view(T, k).cpu(),
            b["starts"][:E + 1].cpu())


def check_route(q4k, logits, k, weighting, scale=1.0):
    got = route(q4k, logits, k, weighting, scale)
    ids, w, order, slots, starts, d = route_ref(logits, k, weighting, scale)
    assert torch.equal(got[0].long(), ids)
    assert got[2].tolist() == order.tolist() and got[3].tolist() == slots.tolist() and got[4].tolist() == starts.tolist()
    d = torch.where(torch.isfinite(d), d.abs(), 0.0)
    assert bool(((got[1].double() - w).abs() <= (2.0 ** -18 + 2.0 ** -23 * d) * w.abs() + 1e-37 * abs(scale)).all())


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (1, 128, 8), (2, 33, 3), (3, 64, 32), (48, 128, 8), (31, 61, 4),
                                   (64, 1024, 32), (65, 1024, 32), (513, 32, 4), (700, 128, 8), (1003, 61, 4),
                                   (4097, 256, 1), (2000, 512, 10), (130, 1000, 17)])
@pytest.mark.parametrize("weighting", [0, 1, 2, 3])
def test_route(q4k, T, E, k, weighting):
    g = gen(T + E + k)
    logits = torch.randn(T, E, generator=g) * 3
    check_route(q4k, logits, k, weighting, 1.0 if weighting != 2 else 2.5)
    # ties everywhere
    check_route(q4k, torch.round(logits), k, weighting)
    # experts and tokens that are masked, zeros of both signs
    m = torch.round(logits)
    m[torch.rand(T, E, generator=g) < 0.5] = float("-inf")
    m[torch.rand(T, E, generator=g) < 0.1] = float("nan")
    m[torch.rand(T, E, generator=g) < 0.2] = -0.0
    m[:, ::7] = float("-inf")
    if T > 2:
        m[1] = float("-inf")
        m[T - 1] = float("nan")
    check_route(q4k, m, k, weighting)


@pytest.mark.parametrize("T", [4, 900])
def test_route_extreme_logits(q4k, T):
    inf, big = float("inf"), 3.4e38
    rows = torch.tensor([[inf, 1, inf, -big], [big, -big, 0, 1], [-big, -big, -big, -inf], [1e-45, -1e-45, 0.0, -0.0]])
    logits = rows.repeat((T + 3) // 4, 1)[:T]
    for weighting in range(4):
        check_route(q4k, logits, 3, weighting)


@pytest.mark.parametrize("T", [4, 900])
@pytest.mark.parametrize("top", [-64.5, -87.0, -104.0, -300.0, -999.0])
def test_route_sigmoids_far_below(q4k, T, top):
    # divided by their sum they stay what they are, e^x / sum e^x, wherever fp32 ends (2^-92 off at most: 1 + e^x)
    logits = top - torch.rand(T, 9, generator=gen(T)) * 6
    logits[:, 3] = top
    _, w, _, _, _, d = route_ref(logits, 4, 1, 1.5)
    got = route(q4k, logits, 4, 3, 1.5)[1].double()
    assert bool(((got - w).abs() <= (2.0 ** -18 + 2.0 ** -23 * d.abs()) * w).all())


@pytest.mark.parametrize("T,E,k", [(5000, 2, 2), (3000, 7, 1)])
def test_route_one_expert_takes_all(q4k, T, E, k):
    logits = torch.zeros(T, E)
    logits[:, E - 1] = 1
    check_route(q4k, logits, k, 1)
    logits[:, 0] = float("-inf")
    check_route(q4k, logits, k, 1)


# ------------------------------------------------------------------ gather ---

@pytest.mark.parametrize("T,k,C,eight", [(1, 1, 8, False), (1, 8, 2048, False), (3, 2, 264, False), (37, 4, 4096, False),
                                         (300, 8, 5120, False), (2, 1, 32768, False), (1, 3, 32, True),
                                         (37, 4, 2080, True), (300, 8, 4096, True), (2, 2, 32768, True)])
def test_gather(q4k, T, k, C, eight):
    g = gen(T + C)
    x = torch.randn(T, C, generator=g).to(torch.bfloat16)
    scales = None
    order = torch.randperm(T * k, generator=g).to(torch.int32)
    order[torch.rand(T * k, generator=g) < 0.2] = -1
    if T * k > 2:
        order[0], order[1], order[2] = T * k, -(1 << 31), 0
    if eight:
        x = torch.randint(0, 256, (T, C), generator=g, dtype=torch.uint8)
        x[(x & 127) == 127] = 5
        scales = torch.randint(90, 160, (T, C // 32), generator=g, dtype=torch.uint8)
        scales[0, 0] = 255
        rows = (x.view(torch.float8_e4m3fn).double().view(T, -1, 32) * torch.exp2(scales.double() - 127).unsqueeze(2)).view(T, C)
        rows[0, :32] = float("nan")
        rows = rows.to(torch.bfloat16)
    else:
        rows = x
    out = torch.full((T * k + 2, C), 3.0, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_experts_gather(x.to(DEV), order.to(DEV), k, out, scales=None if scales is None else scales.to(DEV))
    want = torch.full((T * k + 2, C), 3.0, dtype=torch.bfloat16)
    for p, i in enumerate(order.tolist()):
        if 0 <= i < T * k:
            want[p] = rows[i // k]
    same = (out.cpu() == want) | (out.cpu().isnan() & want.isnan())
    assert bool(same.all())


def test_gather_smallest_scale(q4k):
    x = torch.full((1, 32), 0x38, dtype=torch.uint8)  # 1.0
    out = torch.empty(1, 32, dtype=torch.bfloat16, device=DEV)
    for s in (0, 1, 254):
        q4k.q4k_experts_gather(x.to(DEV), ints([0]), 1, out, scales=torch.full((1, 1), s, dtype=torch.uint8, device=DEV))
        assert bool((out.double() == 2.0 ** (s - 127)).all())


# ---------------------------------------------------------------- products ---

def parts(W, N, K):
    """d sc q and dmin m of every weight, in 64 bits, and |r|."""
    b = W.view(N, K // 256, 144).long()
    half = W.view(N, K // 256, 144)[:, :, :4].contiguous().view(torch.float16).double()
    s = b[:, :, 4:16]
    sc = torch.cat([s[..., 0:4] & 63, (s[..., 8:12] & 15) | ((s[..., 0:4] >> 6) << 4)], -1).double()
    mn = torch.cat([s[..., 4:8] & 63, (s[..., 8:12] >> 4) | ((s[..., 4:8] >> 6) << 4)], -1).double()
    q = b[:, :, 16:].view(N, K // 256, 4, 32)
    q = torch.stack([q & 15, q >> 4], 3).view(N, K // 256, 8, 32).double()
    d = (half[..., 0:1] * sc).unsqueeze(-1)
    a = d * q
    m = (half[..., 1:2] * mn).unsqueeze(-1)
    r = (m / d).nan_to_num(0, 15, 0).round().clamp(0, 15) * d - m
    flat = lambda t: t.expand_as(a).reshape(N, K)  # noqa: E731
    return flat(a), flat(m), flat(r.abs() + 2.0 ** -20 * d.abs())


class Experts:
    def __init__(self, seed, E, N, K):
        self.E, self.N, self.K = E, N, K
        self.w = torch.stack([synth.weight_rows(seed + e, N, K) for e in range(E)])
        self.dev = self.w.to(DEV)

    def product(self, e, x):
        """x W_e^T and its bound."""
        a, m, r = parts(self.w[e].reshape(self.N, -1), self.N, self.K)
        x = x.double()
        y = x @ (a - m).T
        tol = 2.0 ** -8 * (x.abs() @ ((a - m).abs() + r).T) + 2.0 ** -23 * (self.K / 16 + 64) * (x.abs() @ (a.abs() + m.abs()).T)
        return y, tol + 2.0 ** -16 * (x.abs() @ m.abs().T)


def check_experts(q4k, E, N, K, counts, gated, seed=0, lead=0, scale=1.0):
    up = Experts(seed + 5000, E, N, K) if gated else None
    w = Experts(seed, E, N, K)
    P = lead + sum(counts) + 3
    g = gen(seed + P)
    x = (torch.randn(P, K, generator=g) * (0.02 if gated else 1.0) * scale).to(torch.bfloat16)
    x[lead + sum(counts):] = float("nan")  # rows of no expert
    starts = [lead]
    for c in counts:
        starts.append(starts[-1] + c)
    sentinel = torch.tensor(-12345.0).to(torch.bfloat16)
    y = torch.full((P + 1, N), -12345.0, dtype=torch.bfloat16, device=DEV)
    if gated:
        q4k.q4k_experts_gated(w.dev, up.dev, N, K, x.to(DEV), ints(starts), y)
    else:
        q4k.q4k_experts_matmul(w.dev, N, K, x.to(DEV), ints(starts), y)
    y = y.cpu()
    assert bool((y[:lead] == sentinel).all()) and bool((y[starts[-1]:] == sentinel).all())
    worst = 0.0
    for e in range(E):
        a, b = starts[e], starts[e + 1]
        if a == b:
            continue
        want, tol = w.product(e, x[a:b])
        if gated:
            u, tu = up.product(e, x[a:b])
            silu = want * torch.sigmoid(want)
            want = silu * u
            tol = 1.1 * tol * u.abs() + silu.abs() * tu + 1.1 * tol * tu + 2.0 ** -20 * want.abs()
        tol = tol + 2.0 ** -8 * want.abs() + 1e-38
        worst = max(worst, float(((y[a:b].double() - want).abs() / tol).max()))
    assert worst <= 1.0, worst


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,K,counts", [
    (1, 32, 256, [1]), (1, 1, 256, [1]), (1, 7, 512, [3]), (2, 33, 256, [0, 8]), (2, 32, 256, [9, 0]),
    (3, 130, 768, [1, 7, 2]), (4, 64, 2048, [1, 0, 1, 1]), (4, 50, 2304, [5, 6, 7, 8]), (3, 36, 4352, [2, 1, 4]),
    (5, 16, 512, [0, 0, 3, 0, 0]), (2, 96, 1024, [16, 11]), (2, 100, 768, [17, 20]), (3, 61, 1280, [32, 1, 33]),
    (2, 128, 512, [64, 65]), (4, 129, 256, [100, 0, 1, 31])])
def test_experts_small(q4k, E, N, K, counts, gated):
    check_experts(q4k, E, N, K, counts, gated, seed=E * N + K, lead=2 if N % 2 else 0)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,K,counts", [
    (2, 128, 512, [128, 127]), (2, 257, 256, [300, 129]), (3, 192, 768, [256, 1, 512]), (2, 64, 2048, [700, 15]),
    (4, 100, 512, [0, 1000, 0, 3]), (1, 384, 1024, [513]), (1, 256, 256, [4100]), (2, 300, 256, [2000, 2501]),
    (3, 640, 512, [1537, 0, 1500]), (3, 1000, 768, [900, 193, 1700]), (5, 512, 1280, [300, 1, 0, 192, 800]),
    (1, 129, 256, [9000]), (2, 2047, 512, [400, 385])])
def test_experts_many_rows(q4k, E, N, K, counts, gated):
    check_experts(q4k, E, N, K, counts, gated, seed=E * N + K + 1, lead=3 if N % 2 else 0)


@pytest.mark.parametrize("scale", [2.0 ** -50, 2.0 ** -40, 2.0 ** 40, 2.0 ** 60])
def test_experts_scale_of_rows(q4k, scale):
    check_experts(q4k, 2, 40, 512, [3, 9], False, seed=3, scale=scale)
    check_experts(q4k, 2, 40, 512, [200, 90], False, seed=3, scale=scale)
    check_experts(q4k, 2, 256, 256, [2500, 2000], False, seed=3, scale=scale)


def test_experts_rows_with_infinity(q4k):
    """A row with an infinity or a NaN spoils no other row."""
    for counts in ([4, 5], [130, 200], [3000, 2900]):
        P, N, K = sum(counts), 256 if sum(counts) > 1000 else 64, 512
        w = Experts(9, 2, N, K)
        x = torch.randn(P, K, generator=gen(1)).to(torch.bfloat16)
        clean, dirty = (torch.empty(P, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        starts = ints([0, counts[0], P])
        q4k.q4k_experts_matmul(w.dev, N, K, x.to(DEV), starts, clean)
        x[1, 7], x[counts[0], 3] = float("inf"), float("nan")
        q4k.q4k_experts_matmul(w.dev, N, K, x.to(DEV), starts, dirty)
        keep = torch.ones(P, dtype=torch.bool)
        keep[1] = keep[counts[0]] = False
        assert torch.equal(clean.cpu()[keep], dirty.cpu()[keep])
        assert not bool(torch.isfinite(dirty[counts[0]]).any())


def test_experts_starts_out_of_range(q4k):
    """Whatever starts holds, nothing outside the rows is written."""
    N, K, P = 40, 256, 20
    w = Experts(4, 4, N, K)
    x = torch.randn(P, K, generator=gen(2)).to(torch.bfloat16).to(DEV)
    for starts in ([-5, 4, 2, 9, 1 << 30], [1 << 30] * 5, [-(1 << 31)] * 5, [20, 10, 5, 2, 0], [0, 30, 3, 30, 12]):
        y = torch.full((P + 8, N), 5.0, dtype=torch.bfloat16, device=DEV)
        q4k.q4k_experts_matmul(w.dev, N, K, x, ints(starts), y)
        assert bool((y[P:] == 5).all()) and bool(torch.isfinite(y).all())
    # values that come down are taken as the highest before them
    y = torch.full((P, N), 5.0, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_experts_matmul(w.dev, N, K, x, ints([-5, 4, 2, 9, 1 << 30]), y)
    same = torch.full((P, N), 5.0, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_experts_matmul(w.dev, N, K, x, ints([0, 4, 4, 9, 20]), same)
    assert torch.equal(y, same)


def test_experts_starts_out_of_range_many_rows(q4k):
    """The same for the kernel of many rows."""
    N, K, P = 300, 256, 2900
    w = Experts(4, 4, N, K)
    x = torch.randn(P, K, generator=gen(2)).to(torch.bfloat16).to(DEV)
    for gated in (False, True):
        def product(starts, y):
            if gated:
                q4k.q4k_experts_gated(w.dev, w.dev, N, K, x * 0.02, ints(starts), y)
            else:
                q4k.q4k_experts_matmul(w.dev, N, K, x, ints(starts), y)
            return y
        new = lambda: torch.full((P + 8, N), 5.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        # X's rows are those of Y, 8 more would be read if pairs were taken from there
        for starts in ([1 << 30] * 5, [-(1 << 31)] * 5, [P, 10, 5, 2, 0], [0, 2000, 3, 1 << 30, 12]):
            y = product(starts, new())
            assert bool((y[P:] == 5).all()) and bool(torch.isfinite(y).all())
        assert torch.equal(product([-5, 900, 2, 1900, 1 << 30], new()), product([0, 900, 900, 1900, P], new()))


@pytest.mark.parametrize("counts", [[3, 9], [200, 90], [2500, 2000]])
def test_experts_odd_heads(q4k, counts):
    """Super-blocks whose d or dmin is 0, negative, or the smallest number: the bounds hold as they are."""
    E, N, K = 2, 40, 512
    w = Experts(31, E, N, K)
    head = torch.tensor([[0.0, 1.0], [1.0, 0.0], [0.0, 0.0], [-1.0, 2.0], [2.0, -1.0], [-1.0, -4.0], [2.0 ** -24, 2.0 ** -24],
                         [2.0 ** -24, 1.0], [1.0, 2.0 ** -24], [60.0, 60.0]]).to(torch.float16)
    blocks = w.w.view(E, N, K // 256, 144)
    at = torch.arange(E * N * (K // 256)).view(E, N, K // 256) % len(head)
    blocks[..., 0:4] = head[at].view(torch.uint8)
    w.dev = w.w.to(DEV)
    P = sum(counts)
    x = torch.randn(P, K, generator=gen(5)).to(torch.bfloat16)
    y = torch.empty(P, N, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_experts_matmul(w.dev, N, K, x.to(DEV), ints([0, counts[0], P]), y)
    for e, rows in enumerate((slice(0, counts[0]), slice(counts[0], P))):
        want, tol = w.product(e, x[rows])
        assert bool(((y[rows].cpu().double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all())


def test_offsets_past_31_bits(q4k):
    """The last rows of arrays of more than 2^31 elements."""
    g, T, C = torch.Generator(device=DEV).manual_seed(1), 65700, 32768
    tail = slice(T - 3, T)
    x = torch.empty(T, C, dtype=torch.bfloat16, device=DEV)
    x[tail] = torch.randn(3, C, generator=g, device=DEV).to(torch.bfloat16)
    # rows that change places, and back, with a weight
    order = torch.arange(T, dtype=torch.int32, device=DEV)
    order[T - 1], order[0] = 0, T - 1
    x[0] = 2.0
    rows = torch.empty_like(x)
    q4k.q4k_experts_gather(x, order, 1, rows)
    assert torch.equal(rows[0], x[T - 1]) and torch.equal(rows[T - 2], x[T - 2]) and bool((rows[T - 1] == 2).all())
    out = torch.empty(T, C, device=DEV)
    q4k.q4k_experts_combine(rows, order.view(T, 1), torch.full((T, 1), 0.5, device=DEV), out)
    assert torch.equal(out[tail], 0.5 * x[tail].float()) and bool((out[0] == 1).all())
    del rows
    codes, scales = torch.empty(T, C, dtype=torch.uint8, device=DEV), torch.empty(T, C // 32, dtype=torch.uint8, device=DEV)
    w = torch.ones(C, device=DEV)
    q4k.q4k_add_norm(x, None, w, 1e-5, out=out, codes=codes, scales=scales)
    few = [torch.empty_like(t[:3]) for t in (out, codes, scales)]
    q4k.q4k_add_norm(x[tail].clone(), None, w, 1e-5, out=few[0], codes=few[1], scales=few[2])
    for t, f in zip((out, codes, scales), few):
        assert torch.equal(t[tail], f)


@pytest.mark.parametrize("E,N,K,P", [(2, 32768, 256, 65700), (1024, 8, 1 << 18, 8200)])
def test_products_past_31_bits(q4k, E, N, K, P):
    """Rows of Y (many rows an expert) and of X (few) past 2^31 elements."""
    w = synth.weight_rows(77, 8, K)
    dev = w.to(DEV).repeat(E * N // 8, 1)
    x = torch.zeros(P, K, dtype=torch.bfloat16, device=DEV)
    x[P - 3:] = torch.randn(3, K, generator=gen(6)).to(torch.bfloat16).to(DEV)
    y = torch.full((P, N), 3.0, dtype=torch.bfloat16, device=DEV)
    starts = torch.linspace(0, P, E + 1).round().int().to(DEV)
    q4k.q4k_experts_matmul(dev, N, K, x, starts, y)
    assert bool((y[:P - 3] == 0).all())
    a, m, r = parts(w.reshape(8, -1), 8, K)
    xs = x[P - 3:].cpu().double()
    want = xs @ (a - m).T
    tol = 2.0 ** -8 * (xs.abs() @ ((a - m).abs() + r).T + want.abs()) + 2.0 ** -23 * (K / 16 + 64) * (xs.abs() @ (a + m).T)
    got = y[P - 3:].cpu().double().view(3, N // 8, 8)
    assert bool(((got - want.unsqueeze(1)).abs() <= tol.unsqueeze(1)).all())


def test_experts_many_experts(q4k):
    """1024 experts, some with rows; more than a block's first pass over them."""
    E, N, K = 1024, 8, 256
    counts = [(e * 7919) % 5 if e % 3 else 0 for e in range(E)]
    w = Experts(11, 8, N, K)
    dev = w.w.repeat(E // 8, 1, 1).to(DEV)
    P = sum(counts)
    x = torch.randn(P, K, generator=gen(3)).to(torch.bfloat16)
    starts = np.concatenate([[0], np.cumsum(counts)])
    y = torch.zeros(P, N, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_experts_matmul(dev, N, K, x.to(DEV), ints(starts.tolist()), y)
    y = y.cpu().double()
    for e in range(E):
        a, b = starts[e], starts[e + 1]
        if a < b:
            want, tol = w.product(e % 8, x[a:b])
            assert bool(((y[a:b] - want).abs() <= tol + 2.0 ** -8 * want.abs()).all())


# ----------------------------------------------------------------- combine ---

@pytest.mark.parametrize("T,k,C", [(1, 1, 8), (1, 8, 2048), (3, 2, 24), (5, 32, 264), (37, 8, 4096), (64, 9, 5120),
                                   (2, 3, 32768), (1000, 4, 72)])
@pytest.mark.parametrize("base", [False, True])
def test_combine(q4k, T, k, C, base):
    g = gen(T + C)
    P = T * k
    y = torch.randn(P, C, generator=g).to(torch.bfloat16)
    slots = torch.randperm(P, generator=g).to(torch.int32).view(T, k)
    w = torch.randn(T, k, generator=g)
    gone = torch.rand(T, k, generator=g) < 0.2
    slots[gone] = -1
    if T > 1:
        slots[1] = torch.tensor([P, 1 << 30, -(1 << 31), -1] * 8)[:k]  # a token with nothing
        w[1] = float("nan")
    b = torch.randn(T, C, generator=g) if base else None
    out = torch.full((T + 1, C), 7.0, device=DEV)
    if base:
        out[:T] = b.to(DEV)
    q4k.q4k_experts_combine(y.to(DEV), slots.to(DEV), w.to(DEV), out, base=out if base else None)
    live = (slots >= 0) & (slots < P)
    terms = torch.where(live.unsqueeze(2), w.double().unsqueeze(2) * y.double()[slots.long().clamp(0, P - 1)], 0.0)
    want = terms.sum(1) + (b.double() if base else 0)
    size = terms.abs().sum(1) + (b.double().abs() if base else 0)
    got = out.cpu().double()
    assert bool(((got[:T] - want).abs() <= 2.0 ** -24 * (k + 1) * size).all())
    assert bool((got[T:] == 7).all())


# ---------------------------------------------------------------- together ---

def test_binding_refuses_another_device(q4k, monkeypatch):
    """Rows on another device than the current one, which the kernels would run on."""
    x, out = torch.zeros(4, 64, device=DEV), torch.zeros(4, 64, device=DEV)
    q4k.q4k_add_norm(x, None, torch.ones(64, device=DEV), out=out)
    monkeypatch.setattr(q4k, "_device", lambda: 1)
    i, b = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)
    for call in (lambda: q4k.q4k_add_norm(x, None, x[0], out=out),
                 lambda: q4k.q4k_route(x, 2, 0, 1.0, i, out, i, i, i, i),
                 lambda: q4k.q4k_experts_gather(b, i, 2, b),
                 lambda: q4k.q4k_experts_matmul(i, 8, 64, b, i, b),
                 lambda: q4k.q4k_experts_gated(i, i, 8, 64, b, i, b),
                 lambda: q4k.q4k_experts_combine(b, i, x, out)):
        with pytest.raises(ValueError, match="on device 0, the current one is 1"):
            call()


def test_binding_refuses_on_the_device(q4k):
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device=DEV)  # noqa: E731
    b16, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    x, w = z(4, 64), z(64)
    bad = [
        lambda: q4k.q4k_add_norm(x, z(3, 64), w, out=z(4, 64)),
        lambda: q4k.q4k_add_norm(x, None, z(63), out=z(4, 64)),
        lambda: q4k.q4k_add_norm(x, None, w, sum=z(4, 64, d=b16), out=z(4, 64)),
        lambda: q4k.q4k_add_norm(x, None, w, out=z(3, 64)),
        lambda: q4k.q4k_add_norm(x.t().contiguous().t(), None, w, out=z(4, 64)),
        lambda: q4k.q4k_add_norm(x, None, w, codes=z(4, 64, d=u8), scales=z(7, d=u8)),
        lambda: q4k.q4k_route(x, 2, 0, 1.0, z(8, d=i32), z(7), z(8, d=i32), z(8, d=i32), z(65, d=i32), z(1024, d=u8)),
        lambda: q4k.q4k_route(x, 2, 0, 1.0, z(8, d=i32), z(8), z(8, d=i32), z(8, d=i32), z(64, d=i32), z(1024, d=u8)),
        lambda: q4k.q4k_route(x, 2, 0, 1.0, z(8, d=torch.int64), z(8), z(8, d=i32), z(8, d=i32), z(65, d=i32), z(1024, d=u8)),
        lambda: q4k.q4k_experts_gather(x, z(8, d=i32), 2, z(8, 64, d=b16)),
        lambda: q4k.q4k_experts_gather(z(4, 64, d=b16), z(7, d=i32), 2, z(8, 64, d=b16)),
        lambda: q4k.q4k_experts_gather(z(4, 64, d=u8), z(8, d=i32), 2, z(8, 64, d=b16), scales=z(7, d=u8)),
        lambda: q4k.q4k_experts_matmul(z(2 * 64 * 144 - 1, d=u8), 64, 256, z(4, 256, d=b16), z(3, d=i32), z(4, 64, d=b16)),
        lambda: q4k.q4k_experts_matmul(z(2 * 64 * 144, d=u8), 64, 256, z(4, 256, d=b16), z(3, d=i32), z(255, d=b16)),
        lambda: q4k.q4k_experts_gated(z(2 * 64 * 144, d=u8), z(64 * 144, d=u8), 64, 256, z(4, 256, d=b16), z(3, d=i32), z(4, 64, d=b16)),
        lambda: q4k.q4k_experts_combine(z(8, 64, d=b16), z(4, 2, d=i32), z(7), z(4, 64)),
        lambda: q4k.q4k_experts_combine(z(8, 64, d=b16), z(4, 2, d=i32), z(8), z(3, 64)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(q4k.Q4KError) as e:
        q4k.q4k_route(x, 2, 0, 1.0, z(8, d=i32), z(8), z(8, d=i32), z(8, d=i32), z(65, d=i32), z(4 * 64 * 2 - 4, d=u8))
    assert e.value.status == q4k.Q4K_ERR_SPACE


class Layer:
    """An expert layer: norm, router, picks, gathered rows, gate and up, down, back to the tokens."""

    def __init__(self, q4k, T, E, top, hidden, ffn, eight, seed=0):
        g = gen(seed)
        self.q, self.T, self.E, self.top, self.hidden, self.ffn, self.eight = q4k, T, E, top, hidden, ffn, eight
        self.router = synth.weight_rows(seed + 77, E, hidden)
        self.gate, self.up = Experts(seed, E, ffn, hidden), Experts(seed + 1000, E, ffn, hidden)
        self.down = Experts(seed + 2000, E, hidden, ffn)
        sign = 1.0 - 2.0 * (torch.arange(hidden) % 2)
        self.weight = 0.05 * sign * (0.5 + torch.rand(hidden, generator=g))
        self.x, self.delta = torch.randn(T, hidden, generator=g), torch.randn(T, hidden, generator=g)
        d = lambda t: t.to(DEV)  # noqa: E731
        e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=DEV)  # noqa: E731
        i32, b16, u8 = torch.int32, torch.bfloat16, torch.uint8
        self.dx, self.ddelta, self.dweight, self.drouter = d(self.x), d(self.delta), d(self.weight), d(self.router)
        self.sum, self.h, self.codes, self.scales = e(T, hidden), e(T, hidden, t=b16), e(T, hidden, t=u8), e(T, hidden // 32, t=u8)
        self.logits, self.ids, self.w = e(T, E), e(T, top, t=i32), e(T, top)
        self.order, self.slots, self.starts = e(T * top, t=i32), e(T, top, t=i32), e(E + 1, t=i32)
        self.ws = e(q4k.q4k_route_workspace(T, E), t=u8)
        self.rows, self.act, self.y, self.out = (e(T * top, n, t=b16) for n in (hidden, ffn, hidden, hidden))
        self.out = e(T, hidden)

    def run(self, stream=None):
        q = self.q
        kw = dict(stream=stream)
        codes, scales = (self.codes, self.scales) if self.eight else (None, None)
        q.q4k_add_norm(self.dx, self.ddelta, self.dweight, sum=self.sum, out=self.h, codes=codes, scales=scales, **kw)
        q.matmul(self.drouter, self.E, self.hidden, self.h, self.logits, **kw)
        q.q4k_route(self.logits, self.top, q.ROUTE_SOFTMAX_TOP, 1.0, self.ids, self.w, self.order, self.slots, self.starts, self.ws, **kw)
        q.q4k_experts_gather(self.codes if self.eight else self.h, self.order, self.top, self.rows, scales=scales, **kw)
        q.q4k_experts_gated(self.gate.dev, self.up.dev, self.ffn, self.hidden, self.rows, self.starts, self.act, **kw)
        q.q4k_experts_matmul(self.down.dev, self.hidden, self.ffn, self.act, self.starts, self.y, **kw)
        q.q4k_experts_combine(self.y, self.slots, self.w, self.out, base=self.sum, **kw)
        return self.out

    def check(self):
        """Each step against 64 bits of what the step before gave, so that a pick near a border counts as it fell."""
        cpu = lambda t: t.cpu().double()  # noqa: E731
        r, h = norm_ref(self.dx.cpu(), self.ddelta.cpu(), self.weight, 1e-6)
        assert bool(((cpu(self.sum) - r).abs() <= 2.0 ** -24 * r.abs()).all())
        assert bool(((cpu(self.h) - h).abs() <= (2.0 ** -8 + 2.0 ** -18) * h.abs()).all())
        ids, w, order, slots, starts, d = route_ref(self.logits.cpu(), self.top, 1, 1.0)
        assert torch.equal(self.ids.cpu().long(), ids) and self.order.tolist() == order.tolist()
        assert bool(((cpu(self.w) - w).abs() <= (2.0 ** -18 + 2.0 ** -23 * d.abs()) * w).all())
        rows = cpu(self.h)
        if self.eight:
            rows = (self.codes.cpu().view(torch.float8_e4m3fn).double().view(self.T, -1, 32)
                    * torch.exp2(cpu(self.scales) - 127).unsqueeze(2)).view(self.T, -1)
            # half a step of 4 significant bits (or of the smallest ones, 2^-10 of the scale) from the fp32 rows
            near = 2.0 ** -4 * h.abs() * (1 + 2.0 ** -18) + 2.0 ** -10 * torch.exp2(cpu(self.scales) - 127).repeat_interleave(32, 1)
            assert bool(((rows - h).abs() <= near).all())
        assert torch.equal(cpu(self.rows), rows[order // self.top])
        for e in range(self.E):
            a, b = int(starts[e]), int(starts[e + 1])
            if a == b:
                continue
            x, act = self.rows[a:b].cpu(), self.act[a:b].cpu()
            (gt, tg), (u, tu) = self.gate.product(e, x), self.up.product(e, x)
            silu = gt * torch.sigmoid(gt)
            tol = 1.1 * tg * (u.abs() + tu) + silu.abs() * tu + (2.0 ** -8 + 2.0 ** -20) * (silu * u).abs() + 1e-38
            assert bool(((act.double() - silu * u).abs() <= tol).all())
            want, tol = self.down.product(e, act)
            assert bool(((self.y[a:b].cpu().double() - want).abs() <= tol + 2.0 ** -8 * want.abs() + 1e-38).all())
        terms = cpu(self.w).unsqueeze(2) * cpu(self.y)[torch.tensor(slots)]
        size = cpu(self.sum).abs() + terms.abs().sum(1)
        assert bool(((cpu(self.out) - cpu(self.sum) - terms.sum(1)).abs() <= 2.0 ** -24 * (self.top + 1) * size).all())


@pytest.mark.parametrize("T,E,top,hidden,ffn,eight", [(1, 8, 2, 512, 256, False), (5, 16, 4, 512, 512, True),
                                                      (33, 8, 3, 256, 768, False), (300, 6, 2, 512, 256, True),
                                                      (3000, 6, 2, 512, 512, True)])
def test_layer(q4k, T, E, top, hidden, ffn, eight):
    layer = Layer(q4k, T, E, top, hidden, ffn, eight, seed=T)
    layer.run()
    layer.check()


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("T", [3, 150, 2600])
def test_layer_captured(q4k, mode, T):
    """A captured layer replays right on new inputs, in every launch mode, back to back with itself."""
    layer = Layer(q4k, T, 6, 2, 256, 256, True, seed=3)
    old = q4k.q4k_set_pdl(mode)
    try:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(side):
            layer.run()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=side):
                layer.run()
                layer.run()
        for _ in range(3):
            layer.dx.normal_()
            layer.out.fill_(float("nan"))
            layer.act.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            graph.replay()
            torch.cuda.synchronize()
            layer.check()
    finally:
        q4k.q4k_set_pdl(old)


def test_layers_on_two_streams(q4k):
    """Two layers at once, each on a stream of its own, and the same one again: the same bits."""
    layers = [Layer(q4k, T, 8, 2, 512, 512, T == 40, seed=T) for T in (40, 2800)]
    want = []
    for layer in layers:
        layer.run()
        torch.cuda.synchronize()
        layer.check()
        want.append(layer.out.clone())
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(10):
        for layer, s in zip(layers, streams):
            layer.out.fill_(float("nan"))
        torch.cuda.synchronize()
        for layer, s in zip(layers, streams):
            layer.run(stream=s)
        torch.cuda.synchronize()
        for layer, w in zip(layers, want):
            assert torch.equal(layer.out, w)


def test_rows_do_not_depend_on_other_rows(q4k):
    """A row's product is the same bits whichever rows are beside it, while the kernel is the same."""
    N, K = 96, 1024
    w = Experts(21, 3, N, K)
    for counts in ([3, 2, 4], [90, 0, 150], [2900, 0, 4000]):
        P = sum(counts)
        x = torch.randn(P, K, generator=gen(8)).to(torch.bfloat16).to(DEV)
        a, b = (torch.empty(P, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        starts = ints(np.concatenate([[0], np.cumsum(counts)]).tolist())
        q4k.q4k_experts_matmul(w.dev, N, K, x, starts, a)
        other = x.clone()
        other[1:] = torch.randn(P - 1, K, generator=gen(9)).to(torch.bfloat16).to(DEV)
        q4k.q4k_experts_matmul(w.dev, N, K, other, starts, b)
        assert torch.equal(a[0], b[0])
