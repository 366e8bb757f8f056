"""The calls between the products on the GPU, against plain implementations in
64 bits: cache append, paged attention, page bookkeeping, logits pick.

Tolerances follow from the number formats. bf16 has 8 significant bits, so
rounding to it is off by at most 2^-8 relative. Attention rounds the output
(2^-8 |y|) and each softmax weight (2^-8 A with A the weighted mean of |v|); fp32 sums, the exponential and the scores add
(2^-13 + 2^-18 S) A at most, where S is the largest scaled sum of |q_d k_d|
(a score of 128 products in fp32 is off by at most 2^-19 S or so, and a weight
by twice that). Append rounds once to bf16: 2^-8 |y| + 2^-20 (|a| + |b|) of the
rotated pair. Logits: four fp32 roundings of values up to their sum.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _cuda(q4k):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    torch.cuda.set_device(0)
    q4k.q4k_init()
    yield
    torch.cuda.synchronize()
    assert q4k.q4k_device_error() == 0


def ints(v, dev=DEV):
    return torch.tensor(list(v), dtype=torch.int32, device=dev)


def make_cache(q4k, lens, page, kv, dim, seed=0, layers=1, fill=None, spare=3, width=None, shared=False):
    """A cache whose sequences have the given lengths, on shuffled pages; `fill`: what the
    rows that hold no position are filled with (every page of no sequence too)."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-n // page) for n in lens]
    n_pages = sum(counts) + spare
    ids = torch.randperm(n_pages, generator=g).tolist()
    width = width or max(counts + [1])
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32)
    shape = (layers, n_pages, kv, page, dim)
    if shared:  # pages of all layers, K and V side by side in one allocation
        pool = torch.randn((n_pages, layers, 2, kv, page, dim), generator=g).to(torch.bfloat16)
        k, v = pool[:, :, 0].transpose(0, 1), pool[:, :, 1].transpose(0, 1)
    else:
        k = torch.randn(shape, generator=g).to(torch.bfloat16)
        v = torch.randn(shape, generator=g).to(torch.bfloat16)
    used = torch.zeros((n_pages, page), dtype=torch.bool)
    for i, c in enumerate(counts):
        mine = [ids.pop() for _ in range(c)]
        table[i, :c] = torch.tensor(mine, dtype=torch.int32)
        for j, p in enumerate(mine):
            refs[p] = 1
            used[p, :min(page, lens[i] - j * page)] = True
    if fill is not None:
        hole = ~used[None, :, None, :, None].expand(shape)
        k[hole] = fill
        v[hole] = fill
    if shared:
        pool = pool.to(DEV)
        kd, vd = pool[:, :, 0].transpose(0, 1), pool[:, :, 1].transpose(0, 1)
    else:
        kd, vd = k.to(DEV), v.to(DEV)
    return q4k.Cache(kd, vd, refs.to(DEV), table.to(DEV), ints(lens))


def gather(cache, layer, seq):
    """K and V of a sequence's positions in float64, [kv, len, dim]."""
    page = cache.k.shape[3]
    n = int(cache.lens[seq])
    pages = cache.table[seq, :-(-n // page)].long()
    out = []
    for t in (cache.k, cache.v):
        x = t[layer][pages].cpu().double()  # [pages, kv, page, dim]
        out.append(x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :n])
    return out


def attention_ref(cache, layer, seqs, news, Q, heads, scale, window, sinks):
    """The definition, row by row over the visible keys only; and the bound."""
    Qc = Q.cpu().double()
    y = torch.zeros(Qc.shape, dtype=torch.float64)
    tol = torch.zeros(Qc.shape, dtype=torch.float64)
    t = 0
    for s, m in zip(seqs, news):
        k, v = gather(cache, layer, s) if 0 <= s < cache.lens.numel() and int(cache.lens[s]) > 0 else (None, None)
        n = k.shape[1] if k is not None else 0
        for r in range(m):
            p = n - m + r
            j = np.arange(0, p + 1)
            if window:
                j = j[(j > p - window) | (j < sinks)]
            if p < 0 or len(j) == 0:
                t += 1
                continue
            for g in range(cache.kv_heads):
                hs = slice(g * heads // cache.kv_heads, (g + 1) * heads // cache.kv_heads)
                kk, vv, q = k[g][j], v[g][j], Qc[t, hs]
                x = q @ kk.T * scale
                a = torch.softmax(x, -1)
                y[t, hs] = a @ vv
                A = a @ vv.abs()
                S = (q.abs() @ kk.abs().T * scale).max(-1, keepdim=True).values
                tol[t, hs] = 2.0 ** -8 * (y[t, hs].abs() + A) + (2.0 ** -13 + 2.0 ** -18 * S) * A
            t += 1
    return y, tol


def attend(q4k, cache, layer, seqs, news, Q, heads, scale=None, window=0, sinks=0, max_new=None, stream=None,
           ws=None, starts=None, out=None):
    starts = starts if starts is not None else ints(np.concatenate([[0], np.cumsum(news)]))
    out = out if out is not None else torch.full_like(Q, float("nan"))
    ws = ws if ws is not None else cache.workspace()
    q4k.q4k_cache_attention(cache, layer, None if seqs is None else ints(seqs), starts, Q, out, heads,
                            max(news) if max_new is None else max_new, scale or cache.head_dim ** -0.5, window,
                            sinks, ws, stream)
    torch.cuda.synchronize()
    assert int(ws[:16384].sum()) == 0, "the workspace's counters must be left at zero"
    return out


def check_attention(q4k, cache, seqs, news, heads, layer=0, window=0, sinks=0, seed=7, **kw):
    g = torch.Generator().manual_seed(seed)
    Q = (torch.randn(sum(news), heads, cache.head_dim, generator=g) * 1.5).to(torch.bfloat16).to(DEV)
    out = attend(q4k, cache, layer, seqs, news, Q, heads, window=window, sinks=sinks, **kw)
    y, tol = attention_ref(cache, layer, seqs if seqs is not None else range(len(news)), news, Q, heads,
                           cache.head_dim ** -0.5, window, sinks)
    err = (out.cpu().double() - y).abs()
    assert torch.isfinite(out).all()
    worst = float((err / (tol + 1e-30)).max())
    assert worst <= 1.0, f"error {worst:.3f} of the bound"
    return Q, out


# ------------------------------------------------------------------ attention ---

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 1), (5, 1), (8, 2), (16, 2), (6, 6), (17, 1), (40, 1)])
def test_single_tokens(q4k, dim, page, heads, kv):
    lens = [1, 2, page - 1, page, page + 1, 63, 64, 65, 127, 128, 129, 300]
    cache = make_cache(q4k, lens, page, kv, dim, fill=float("nan"))
    check_attention(q4k, cache, list(range(len(lens))), [1] * len(lens), heads)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,heads,kv,news,lens", [
    (16, 4, 1, [2], [2]),
    (16, 4, 1, [5], [133]),
    (32, 8, 2, [64, 1, 0, 33], [64, 200, 50, 257]),
    (64, 3, 1, [43, 86, 1], [300, 86, 129]),
    (128, 2, 2, [130, 257], [130, 700]),
    (16, 7, 1, [37, 18, 100], [37, 1000, 513]),
    (16, 128, 1, [3, 1], [3, 140]),
    (64, 96, 2, [9], [400]),
    (32, 1, 1, [300], [555]),
])
def test_chunks(q4k, dim, page, heads, kv, news, lens):
    cache = make_cache(q4k, lens, page, kv, dim, fill=float("inf"))
    check_attention(q4k, cache, list(range(len(lens))), news, heads)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (64, 0), (100, 130), (128, 3), (500, 4), (5000, 9)])
def test_window_and_sinks(q4k, dim, window, sinks):
    lens, news = [700, 130, 1, 300, 900], [40, 130, 1, 1, 1]
    cache = make_cache(q4k, lens, 32, 2, dim, fill=float("nan"))
    check_attention(q4k, cache, [0, 1, 2, 3, 4], news, 6, window=window, sinks=sinks)
    lens = [700, 130, 1, 513]
    cache = make_cache(q4k, lens, 16, 2, dim, fill=float("nan"), seed=3)
    check_attention(q4k, cache, [0, 1, 2, 3], [1] * 4, 8, window=window, sinks=sinks)


@pytest.mark.parametrize("heads,kv", [(4, 1), (32, 2)])
@pytest.mark.parametrize("new", [1, 60])
def test_long_sequence_split(q4k, heads, kv, new):
    """One sequence over many blocks of keys: the work is split along its length."""
    for dim, page, n in ((128, 64, 9001), (64, 16, 20000)):
        cache = make_cache(q4k, [n], page, kv, dim, fill=float("nan"))
        check_attention(q4k, cache, [0], [new], heads)


@pytest.mark.parametrize("max_new", [0, 1, 7, 100000])
def test_max_new_selects_only(q4k, max_new):
    """Whatever max_new says, the result is right."""
    lens, news = [200, 77, 1500, 40], [1, 30, 4, 40]
    cache = make_cache(q4k, lens, 16, 2, 128, fill=float("nan"))
    check_attention(q4k, cache, [0, 1, 2, 3], news, 8, max_new=max_new)


def test_sequences_by_id_layers_and_shared_allocation(q4k):
    lens = [50, 10, 333, 90]
    cache = make_cache(q4k, lens, 32, 2, 64, layers=3, fill=float("nan"), shared=True, width=20)
    for layer in range(3):
        check_attention(q4k, cache, [2, 0], [20, 1], 4, layer=layer)
        check_attention(q4k, cache, [3, 2], [1, 1], 4, layer=layer)
    check_attention(q4k, cache, None, [1, 1, 1], 4, layer=1)


def test_rows_that_see_nothing(q4k):
    """Sequence ids out of range, length zero, more new tokens than positions, and rows of no sequence."""
    cache = make_cache(q4k, [0, 5, 40], 16, 1, 128, fill=float("nan"))
    for seqs, news in (([0, 7, -1, 2], [2, 1, 3, 1]), ([1, 2], [9, 1]), ([1, 0, 2], [300, 1, 40])):
        check_attention(q4k, cache, seqs, news, 2)
    Q = torch.randn(12, 2, 128, device=DEV).to(torch.bfloat16)
    out = torch.full_like(Q, 3.0)
    attend(q4k, cache, 0, [2, 1], [4, 3], Q, 2, starts=ints([2, 6, 9]), out=out)
    assert torch.all(out[:2] == 3) and torch.all(out[9:] == 3) and torch.all(out[2:9] != 3)
    # offsets that make no sense stay inside the arrays
    for starts in ([5, 3, 40], [-7, 2, 1 << 30], [12, 12, 12], [0, 1 << 30, 5]):
        attend(q4k, cache, 0, [2, 1], [4, 3], Q, 2, starts=ints(starts))
    cache.lens.copy_(ints([-3, 1 << 30, 40]))
    attend(q4k, cache, 0, [0, 1, 2], [4, 4, 4], Q, 2)


def test_pages_out_of_range_read_as_zeros(q4k):
    cache = make_cache(q4k, [40], 16, 1, 64, seed=5)
    Q = torch.randn(1, 2, 64, device=DEV).to(torch.bfloat16)
    cache.table[0, 1] = 1 << 29
    got = attend(q4k, cache, 0, [0], [1], Q, 2)
    cache.table[0, 1] = -1
    same = attend(q4k, cache, 0, [0], [1], Q, 2)
    spare = [p for p in range(cache.k.shape[1]) if p not in cache.table[0].tolist()][0]
    cache.k[0, spare] = 0
    cache.v[0, spare] = 0
    cache.table[0, 1] = spare
    y, tol = attention_ref(cache, 0, [0], [1], Q, 2, 64 ** -0.5, 0, 0)
    assert torch.equal(got, same)
    assert bool(((got.cpu().double() - y).abs() <= tol).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("max_new", [1, 200])
def test_non_finite_values_of_unseen_tokens(q4k, bad, max_new):
    """A token whose key and value are not finite reaches the rows that see it, and no others."""
    n, m = 300, 40
    for at, window, sinks in ((280, 0, 0), (290, 0, 0), (120, 64, 4), (299, 100, 0), (3, 128, 4), (245, 64, 0)):
        cache = make_cache(q4k, [n], 16, 1, 128, seed=at)
        Q = (torch.randn(m, 4, 128, generator=torch.Generator().manual_seed(at)) * 1.5).to(torch.bfloat16).to(DEV)
        y, tol = attention_ref(cache, 0, [0], [m], Q, 4, 128 ** -0.5, window, sinks)
        page = int(cache.table[0, at // 16])
        cache.v[0, page, 0, at % 16, 5] = bad
        out = attend(q4k, cache, 0, [0], [m], Q, 4, window=window, sinks=sinks, max_new=max_new).cpu().double()
        pos = torch.arange(n - m, n)
        sees = (pos >= at) & ((pos - window < at) | (at < sinks) if window else torch.ones_like(pos, dtype=torch.bool))
        keep = torch.ones(128, dtype=torch.bool)
        keep[5] = False
        assert bool(((out[:, :, keep] - y[:, :, keep]).abs() <= tol[:, :, keep]).all())
        assert bool(((out[~sees] - y[~sees]).abs() <= tol[~sees]).all())
        hit = out[sees][:, :, 5]
        assert bool((torch.isnan(hit) if bad != bad else hit == bad).all())
        # the key too: the rows that see it are not finite or have it weigh nothing, the others are as before
        cache.k[0, page, 0, at % 16, :] = bad
        out = attend(q4k, cache, 0, [0], [m], Q, 4, window=window, sinks=sinks, max_new=max_new).cpu().double()
        assert bool(((out[~sees] - y[~sees]).abs() <= tol[~sees]).all())
        assert bool(torch.isnan(out[sees][:, :, 5]).all()) if bad != bad else True


def test_large_scores(q4k):
    """One score far above the rest, at every place among the blocks of keys, and large negative ones."""
    n = 700
    for at in (0, 1, 127, 128, 400, 699):
        cache = make_cache(q4k, [n], 64, 1, 128, seed=at)
        page = int(cache.table[0, at // 64])
        cache.k[0, page, 0, at % 64] = 12.0
        for m in (1, 20):
            Q = torch.full((m, 8, 128), 3.0, device=DEV).to(torch.bfloat16)
            Q[:, 4:] = -3.0
            out = attend(q4k, cache, 0, [0], [m], Q, 8)
            y, tol = attention_ref(cache, 0, [0], [m], Q, 8, 128 ** -0.5, 0, 0)
            assert bool(((out.cpu().double() - y).abs() <= tol).all())


def test_offsets_past_32_bits(q4k):
    """A pool of more than 2^31 elements, used at its far end."""
    kv, page, dim = 8, 128, 128
    n_pages = (1 << 31) // (kv * page * dim) + 600
    pool = torch.empty((1, n_pages, kv, page, dim), dtype=torch.bfloat16, device=DEV)
    assert pool.numel() > 1 << 31
    last = list(range(n_pages - 5, n_pages))
    pool[:, last] = torch.randn(1, 5, kv, page, dim, device=DEV).to(torch.bfloat16)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    refs[last] = 1
    cache = q4k.Cache(pool, pool, refs, ints(last).view(1, 5), ints([600]))
    check_attention(q4k, cache, [0], [1], 16)
    check_attention(q4k, cache, [0], [20], 16)
    heads = 8
    Y = [torch.randn(3, h * dim, device=DEV) for h in (heads, kv, kv)]
    q_out = torch.empty(3, heads, dim, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_cache_append(cache, 0, None, ints([0, 3]), *Y, q_out, heads)
    got = pool[0, last[4], :, 600 - 3 - 512:600 - 512].transpose(0, 1).reshape(3, -1)
    assert torch.equal(got, Y[2].to(torch.bfloat16))
    before = pool[0, last].clone()
    ws = cache.workspace()
    q4k.q4k_pages_compact(cache, ws)
    torch.cuda.synchronize()
    assert cache.table[0].tolist() == [0, 1, 2, 3, 4] and torch.equal(pool[0, :5], before)


def test_same_bits_every_time_and_on_another_stream(q4k):
    lens, news = [5000, 300, 900], [1, 1, 1]
    cache = make_cache(q4k, lens, 16, 2, 128)
    for news, heads in (([1, 1, 1], 8), ([70, 1, 300], 6)):
        Q, out = check_attention(q4k, cache, [0, 1, 2], news, heads)
        side, ws = torch.cuda.Stream(), cache.workspace()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            again = attend(q4k, cache, 0, [0, 1, 2], news, Q, heads, stream=side, ws=ws)
            assert torch.equal(out, again)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_graph_and_dependent_launch(q4k, mode):
    """A captured step (append, then attention) replays right, in every launch mode."""
    lens, news, heads, kv, dim = [400, 33], [1, 5], 4, 2, 64
    cache = make_cache(q4k, lens, 16, kv, dim, fill=float("nan"))
    Y = [torch.randn(6, h * dim, device=DEV) for h in (heads, kv, kv)]
    Q = torch.empty(6, heads, dim, dtype=torch.bfloat16, device=DEV)
    out, ws, starts, seqs = torch.empty_like(Q), cache.workspace(), ints([0, 1, 6]), ints([0, 1])

    def step():
        q4k.q4k_cache_append(cache, 0, seqs, starts, *Y, Q, heads)
        q4k.q4k_cache_attention(cache, 0, seqs, starts, Q, out, heads, 5, dim ** -0.5, 0, 0, ws)

    old = q4k.q4k_set_pdl(mode)
    try:
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=side):
                step()
        for _ in range(3):
            for y in Y:
                y.normal_()
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            y, tol = attention_ref(cache, 0, [0, 1], news, Q, heads, dim ** -0.5, 0, 0)
            assert bool(((out.cpu().double() - y).abs() <= tol).all())
    finally:
        q4k.q4k_set_pdl(old)


# --------------------------------------------------------------------- append ---

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("pairs", [0, 1, 2])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("heads,kv,page", [(1, 1, 16), (5, 1, 64), (8, 8, 32), (40, 8, 128)])
def test_append(q4k, dim, pairs, norm, heads, kv, page):
    lens, news, seqs = [1, 40, 300, 129], [1, 17, 0, 129], [0, 1, 2, 3]
    cache = make_cache(q4k, lens, page, kv, dim, layers=2, width=-(-300 // page) + 1)
    k0, v0 = cache.k.clone(), cache.v.clone()
    T = sum(news)
    g = torch.Generator().manual_seed(3)
    Yq, Yk, Yv = (torch.randn(T, h * dim, generator=g) for h in (heads, kv, kv))
    rows = cache.table.shape[1] * page
    ang = torch.arange(rows)[:, None] * 0.37 ** (torch.arange(dim // 2) / 9.0)
    rope = torch.cat([ang.cos(), ang.sin()], 1).float() if pairs else None
    qn, kn = (torch.rand(dim, generator=g) + 0.5, torch.rand(dim, generator=g) + 0.5) if norm else (None, None)
    q_out = torch.full((T, heads, dim), float("nan"), dtype=torch.bfloat16, device=DEV)
    up = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    q4k.q4k_cache_append(cache, 1, ints(seqs), ints(np.concatenate([[0], np.cumsum(news)])), Yq.to(DEV),
                         Yk.to(DEV), Yv.to(DEV), q_out, heads, up(rope), pairs, up(qn), up(kn), 1e-5)
    torch.cuda.synchronize()

    def ref(y, h, w, p):
        x = y.double().view(h, dim)
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * w.double()
        size = x.abs()
        if pairs:
            c, s = rope[p, :dim // 2].double(), rope[p, dim // 2:].double()
            ia = torch.arange(dim // 2) * 2 if pairs == 1 else torch.arange(dim // 2)
            ib = ia + 1 if pairs == 1 else ia + dim // 2
            r, both = torch.empty_like(x), x[:, ia].abs() + x[:, ib].abs()
            r[:, ia], r[:, ib] = x[:, ia] * c - x[:, ib] * s, x[:, ia] * s + x[:, ib] * c
            size = torch.empty_like(x)
            size[:, ia] = size[:, ib] = both
            x = r
        return x, 2.0 ** -8 * x.abs() + 2.0 ** -20 * size + 1e-38

    kc, vc, t = k0.cpu(), v0.cpu(), 0
    got_k, got_v = cache.k.cpu(), cache.v.cpu()
    for s, m, n in zip(seqs, news, lens):
        for r in range(m):
            p = n - m + r
            page_id, row = int(cache.table[s, p // page]), p % page
            for got, y, h, w in ((q_out[t].cpu(), Yq[t], heads, qn), (got_k[1, page_id, :, row], Yk[t], kv, kn)):
                x, tol = ref(y, h, w, p)
                assert bool(((got.double() - x).abs() <= tol).all())
            assert torch.equal(got_v[1, page_id, :, row], Yv[t].view(kv, dim).to(torch.bfloat16))
            kc[1, page_id, :, row], vc[1, page_id, :, row] = got_k[1, page_id, :, row], got_v[1, page_id, :, row]
            t += 1
    assert torch.equal(got_k, kc) and torch.equal(got_v, vc), "rows beside the new tokens' changed"


@pytest.mark.parametrize("n,most", [(7, 120), (300, 3), (1100, 1), (1100, 2), (4096, 2)])
def test_append_finds_every_token(q4k, n, most):
    """Many sequences, some without new tokens, and steps of few and many tokens: plain rounding, exact."""
    rng = np.random.default_rng(n + most)
    news = rng.integers(0, most + 1, n)
    news[rng.random(n) < 0.3] = 0
    if n == 1100 and most == 1:
        news[rng.random(n) < 0.9] = 0  # few tokens of many sequences
    lens = news + rng.integers(0, 9, n)
    page, kv, dim, heads = 16, 2, 64, 4
    cache = make_cache(q4k, lens.tolist(), page, kv, dim, width=9)
    cache.k.zero_()
    cache.v.zero_()
    T = int(news.sum())
    Y = [torch.randn(T, h * dim, device=DEV) for h in (heads, kv, kv)]
    q_out = torch.zeros(T, heads, dim, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_cache_append(cache, 0, ints(range(n)), ints(np.concatenate([[0], np.cumsum(news)])), *Y, q_out, heads)
    torch.cuda.synchronize()
    assert torch.equal(q_out, Y[0].view(T, heads, dim).to(torch.bfloat16))
    seq = np.repeat(np.arange(n), news)
    at = np.concatenate([np.arange(m - k, m) for m, k in zip(lens, news)])
    ids = cache.table.cpu().numpy()[seq, at // page]
    for got, y in ((cache.k, Y[1]), (cache.v, Y[2])):
        want = torch.zeros_like(got)
        want[0, torch.tensor(ids, device=DEV).long(), :, torch.tensor(at % page, device=DEV).long()] = \
            y.view(T, kv, dim).to(torch.bfloat16)
        assert torch.equal(got, want)


@pytest.mark.parametrize("dim,pairs,norm,heads,kv", [(128, 2, True, 40, 8), (128, 1, False, 5, 1), (64, 2, False, 32, 8),
                                                     (64, 1, True, 3, 3)])
def test_append_same_bits_in_steps_of_any_size(q4k, dim, pairs, norm, heads, kv):
    T, page = 700, 32
    cache, other = (make_cache(q4k, [T + 5], page, kv, dim) for _ in range(2))
    other.table.copy_(cache.table)
    for c in (cache, other):
        c.k.zero_()
        c.v.zero_()
    Y = [torch.randn(T, h * dim, device=DEV) for h in (heads, kv, kv)]
    rows = cache.table.shape[1] * page
    ang = torch.arange(rows, device=DEV)[:, None] * 0.37 ** (torch.arange(dim // 2, device=DEV) / 9.0)
    rope = torch.cat([ang.cos(), ang.sin()], 1).float()
    qn, kn = (torch.rand(dim, device=DEV) + 0.5, torch.rand(dim, device=DEV) + 0.5) if norm else (None, None)
    q_out = torch.zeros(T, heads, dim, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_cache_append(cache, 0, ints([0]), ints([0, T]), *Y, q_out, heads, rope, pairs, qn, kn)
    part, t = torch.zeros_like(q_out), 0
    while t < T:  # the same tokens a few at a time
        m = min(37, T - t)
        other.lens.fill_(5 + t + m)
        q4k.q4k_cache_append(other, 0, ints([0]), ints([0, m]), *(y[t:t + m] for y in Y), part[t:t + m], heads, rope,
                             pairs, qn, kn)
        t += m
    torch.cuda.synchronize()
    assert torch.equal(part, q_out) and torch.equal(cache.k, other.k) and torch.equal(cache.v, other.v)


def test_append_out_of_range(q4k):
    """Ids, positions and pages out of range store nothing; the queries are still written, unrotated."""
    cache = make_cache(q4k, [5, 20], 16, 1, 64)
    cache.table[1, 1] = -1
    k0 = cache.k.clone()
    rope = torch.randn(cache.table.shape[1] * 16, 64, device=DEV)
    Y = [torch.randn(12, h * 64, device=DEV) for h in (2, 1, 1)]
    q_out = torch.zeros(12, 2, 64, dtype=torch.bfloat16, device=DEV)
    # sequence 9 does not exist; sequence 0 has 5 positions for 7 rows; the page of sequence 1's last rows is none
    q4k.q4k_cache_append(cache, 0, ints([9, 0, 1]), ints([0, 2, 9, 11]), *Y, q_out, 2, rope, 2)
    torch.cuda.synchronize()
    plain = Y[0].view(12, 2, 64).to(torch.bfloat16)
    assert torch.equal(q_out[:4], plain[:4]) and torch.equal(q_out[11:], plain[11:])
    changed = (cache.k != k0).flatten(2).any(2)[0]
    assert changed.nonzero().flatten().tolist() == [int(cache.table[0, 0])]


# ---------------------------------------------------------------------- pages ---

class Model:
    """The bookkeeping of the page calls, written out with lists."""

    def __init__(self, cache):
        self.refs, self.table, self.lens = cache.refs.tolist(), cache.table.tolist(), cache.lens.tolist()
        self.k, self.v = cache.k.cpu().clone(), cache.v.cpu().clone()
        self.page, self.width = cache.k.shape[3], cache.table.shape[1]

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def reserve(self, seqs, news):
        status, used, free = [], 0, self.free_pages()
        for s, m in zip(seqs, news):
            if not 0 <= s < len(self.lens) or self.lens[s] + m > self.width * self.page:
                status.append(1)
                continue
            have, want = -(-self.lens[s] // self.page), -(-(self.lens[s] + m) // self.page)
            at, used = used, used + want - have
            if want > have and used > len(free):
                status.append(1)
                continue
            for i in range(want - have):
                self.table[s][have + i] = free[at + i]
                self.refs[free[at + i]] = 1
            self.lens[s] += m
            status.append(0)
        return status

    def fork(self, parents, children):
        status, free = [], self.free_pages()
        used = 0
        ok_ids = range(len(self.lens))
        start_lens = list(self.lens)
        for p, c in zip(parents, children):
            if p not in ok_ids or c not in ok_ids or start_lens[c] != 0:
                status.append(1)
                continue
            n = start_lens[p]
            full, part = n // self.page, n % self.page != 0
            used += part
            if part and used > len(free):
                status.append(1)
                continue
            row = self.table[p][:full] + [-1] * (self.width - full)
            for q in row[:full]:
                self.refs[q] += 1
            if part:
                new = free[used - 1]
                row[full] = new
                self.refs[new] = 1
                self.k[:, new], self.v[:, new] = self.k[:, self.table[p][full]], self.v[:, self.table[p][full]]
            self.table[c], self.lens[c] = row, n
            status.append(0)
        return status

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.lens):
                for p in self.table[s]:
                    if p >= 0:
                        self.refs[p] -= 1
                self.table[s], self.lens[s] = [-1] * self.width, 0

    def compact(self):
        L = sum(r > 0 for r in self.refs)
        holes = [p for p in range(L) if self.refs[p] == 0]
        movers = [p for p in range(L, len(self.refs)) if self.refs[p] > 0]
        for h, m in zip(holes, movers):
            self.refs[h], self.refs[m] = self.refs[m], 0
            self.k[:, h], self.v[:, h] = self.k[:, m], self.v[:, m]
        to = dict(zip(movers, holes))
        self.table = [[to.get(p, p) for p in row] for row in self.table]

    def check(self, cache):
        torch.cuda.synchronize()
        assert cache.refs.tolist() == self.refs
        assert cache.lens.tolist() == self.lens
        assert cache.table.tolist() == self.table
        assert torch.equal(cache.k.cpu(), self.k) and torch.equal(cache.v.cpu(), self.v)


@pytest.mark.parametrize("seed,page,kv,dim,n_pages,layers,n_seqs,shared", [
    (0, 16, 1, 64, 40, 1, 6, False), (1, 32, 2, 64, 1500, 2, 40, False), (2, 16, 3, 128, 2100, 1, 300, True),
    (3, 128, 1, 128, 25, 3, 5, True), (4, 64, 8, 64, 64, 2, 12, False)])
def test_page_calls(q4k, seed, page, kv, dim, n_pages, layers, n_seqs, shared):
    """A random life of a cache: every call leaves exactly the state that the lists have."""
    rng = np.random.default_rng(seed)
    if shared:
        pool = torch.randn(n_pages, layers, 2, kv, page, dim, device=DEV).to(torch.bfloat16)
        k, v = pool[:, :, 0].transpose(0, 1), pool[:, :, 1].transpose(0, 1)
    else:
        k = torch.randn(layers, n_pages, kv, page, dim, device=DEV).to(torch.bfloat16)
        v = torch.randn_like(k)
    width = max(3, 3 * n_pages // n_seqs)
    cache = q4k.Cache(k, v, ints([0] * n_pages), torch.full((n_seqs, width), -1, dtype=torch.int32, device=DEV),
                      ints([0] * n_seqs))
    model, ws = Model(cache), cache.workspace()
    refused = 0
    for step in range(14):
        n = int(rng.integers(1, n_seqs + 1))
        seqs = rng.permutation(n_seqs)[:n].tolist()
        if step == 3:
            seqs[0] = n_seqs  # an id that does not exist
        news = rng.integers(0, 2 * page + 3, n).tolist()
        status = ints([9] * n)
        q4k.q4k_pages_reserve(cache, ints(seqs), ints(np.concatenate([[4], 4 + np.cumsum(news)])), status)
        want = model.reserve(seqs, news)
        assert status.tolist() == want
        refused += sum(want)
        model.check(cache)
        empty = [s for s in range(n_seqs) if model.lens[s] == 0]
        used = [s for s in range(n_seqs) if model.lens[s] > 0]
        kids = empty[:max(1, len(empty) // 2)] + ([used[0], -2] if step % 4 == 1 and used else [])
        if kids and used:
            folks = [int(rng.choice(used)) for _ in kids]
            status = ints([9] * len(kids))
            q4k.q4k_pages_fork(cache, ints(folks), ints(kids), status, ws)
            assert status.tolist() == model.fork(folks, kids)
            model.check(cache)
        gone = rng.permutation(n_seqs)[:n_seqs // 2].tolist() + [n_seqs + 3]
        q4k.q4k_pages_free(cache, ints(gone), )
        model.free(gone)
        model.check(cache)
        if step % 2:
            q4k.q4k_pages_compact(cache, ws)
            model.compact()
            model.check(cache)
        assert int(ws[:16384].sum()) == 0
    assert refused > 0 or n_pages > 1000


def test_most_sequences(q4k):
    """4096 sequences in one call: reserve, fork, append, attention and free."""
    n, page, dim = 4096, 16, 64
    k = torch.randn(1, 2 * n, 1, page, dim, device=DEV).to(torch.bfloat16)
    cache = q4k.Cache(k, torch.randn_like(k), ints([0] * (2 * n)),
                      torch.full((2 * n, 4), -1, dtype=torch.int32, device=DEV), ints([0] * (2 * n)))
    model, ws = Model(cache), cache.workspace()
    news = [1 + i % 20 for i in range(n)]
    starts, status = ints(np.concatenate([[0], np.cumsum(news)])), ints([9] * n)
    q4k.q4k_pages_reserve(cache, None, starts, status)
    assert status.tolist() == model.reserve(range(n), news) and sum(status.tolist()) == 0
    kids = list(range(n, 2 * n))
    q4k.q4k_pages_fork(cache, ints(range(n)), ints(kids), status, ws)
    want = model.fork(list(range(n)), kids)
    assert status.tolist() == want and 0 < sum(want) < n
    model.check(cache)
    T = sum(news)
    Y = [torch.randn(T, dim, device=DEV) for _ in range(3)]
    q = torch.empty(T, 1, dim, dtype=torch.bfloat16, device=DEV)
    q4k.q4k_cache_append(cache, 0, None, starts, *Y, q, 1)
    out = attend(q4k, cache, 0, None, news, q, 1, ws=ws)
    picks = [0, 17, 2000, 4095]
    rows = [r for s in picks for r in range(sum(news[:s]), sum(news[:s + 1]))]
    y, tol = attention_ref(cache, 0, picks, [news[s] for s in picks], q[rows], 1, dim ** -0.5, 0, 0)
    assert bool(((out[rows].cpu().double() - y).abs() <= tol).all())
    q4k.q4k_pages_free(cache, ints(range(2 * n)))
    assert int(cache.refs.abs().sum()) == 0 and int(cache.lens.sum()) == 0


def test_pages_copy(q4k):
    cache = make_cache(q4k, [100], 16, 3, 64, layers=4, spare=20)
    k0, v0 = cache.k.clone(), cache.v.clone()
    q4k.q4k_pages_copy(cache, ints([0, 3, -1, 5, 1 << 29]), ints([9, 11, 12, 1 << 29, 13]))
    torch.cuda.synchronize()
    for t, t0 in ((cache.k, k0), (cache.v, v0)):
        t0[:, 9], t0[:, 11] = t0[:, 0].clone(), t0[:, 3].clone()
        assert torch.equal(t, t0)


# --------------------------------------------------------------------- logits ---

def pick_ref(x, hist, pen, bias, allowed):
    """float64, from the definition; also each element's size for the rounding bound."""
    x = x.astype(np.float64).copy()
    size = np.abs(x)
    for m in range(x.shape[0]):
        if hist is not None:
            ids, counts = np.unique([v for v in hist[m] if 0 <= v < x.shape[1]], return_counts=True)
            ids = ids.astype(int)
            rep, pres, freq = (float(p) for p in pen[m])
            y = np.where(x[m, ids] > 0, x[m, ids] / rep, x[m, ids] * rep)
            size[m, ids] = np.abs(y) + np.abs(counts * freq) + abs(pres)
            x[m, ids] = y - counts * freq - pres
        if bias is not None:
            for v, b in {v: b for v, b in bias[m] if 0 <= v < x.shape[1]}.items():
                x[m, v] += b
                size[m, v] += abs(b)
    best = np.empty(x.shape[0], dtype=np.int64)
    for m in range(x.shape[0]):
        ok = np.ones(x.shape[1], bool) if allowed is None else allowed[m]
        x[m, ~ok] = -np.inf
        y = np.where(np.isnan(x[m]), -np.inf, x[m])
        number = ok & ~np.isnan(x[m])
        pool = number if number.any() else ok
        best[m] = np.flatnonzero(pool)[np.argmax(y[pool])] if pool.any() else -1
    return x, best, size


def pick_run(q4k, x, hist=None, pen=None, bias=None, allowed=None, keep=True, pick=True, alias=False):
    R, V = x.shape
    logits = torch.tensor(x, device=DEV)
    out = logits if alias else torch.full_like(logits, 7.0) if keep else None
    picks = torch.full((R,), -9, dtype=torch.int64, device=DEV) if pick else None
    flat = lambda rows: np.concatenate([[0], np.cumsum([len(r) for r in rows])])  # noqa: E731
    a = {}
    if hist is not None:
        a.update(history=ints([v for r in hist for v in r]), hist_starts=ints(flat(hist)),
                 penalties=torch.tensor(np.asarray(pen, np.float32), device=DEV))
    if bias is not None:
        a.update(bias_ids=ints([v for r in bias for v, _ in r]),
                 bias=torch.tensor([b for r in bias for _, b in r], dtype=torch.float32, device=DEV),
                 bias_starts=ints(flat(bias)))
    if allowed is not None:
        bits = np.zeros((R, -(-V // 32) * 32), np.uint8)
        bits[:, :V] = allowed
        words = np.packbits(bits, axis=1, bitorder="little").view(np.uint32)
        a["mask"] = torch.tensor(words.astype(np.int64) - (words.astype(np.int64) >> 31 << 32), device=DEV).to(torch.int32)
    q4k.q4k_logits_pick(logits, R, V, out, picks, **a)
    torch.cuda.synchronize()
    return None if out is None else out.cpu().numpy(), None if picks is None else picks.cpu().numpy()


@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (5, 31), (2, 33), (4, 4095), (7, 4097), (1, 8191), (3, 20001),
                                 (2, 50257), (1, 128256), (65, 9001), (500, 130)])
def test_pick_exact_values(q4k, R, V):
    """Values on a coarse grid, where fp32 is exact: outputs and picks (with their many ties) equal the definition's."""
    rng = np.random.default_rng(R * 1000 + V)
    x = (rng.integers(-40, 41, (R, V)) / 8).astype(np.float32)
    x[x == 0] = np.where(rng.random((x == 0).sum()) < 0.5, 0.0, -0.0)
    hist = [rng.integers(-2, V + 2, rng.integers(0, 60)).tolist() for _ in range(R)]
    hist[0] = hist[0] + [V // 2] * 70
    pen = [[rng.choice([0.5, 1, 2, 4]), rng.integers(0, 9) / 8, rng.integers(0, 5) / 8] for _ in range(R)]
    bias = [[(int(v), float(rng.integers(-16, 17)) / 4) for v in rng.integers(-1, V + 1, rng.integers(0, 9))] for _ in range(R)]
    allowed = rng.random((R, V)) < 0.5
    if R > 1:
        allowed[1] = False
        allowed[R - 1, :-1] = False
    for h, b, ok in ((hist, bias, allowed), (hist, None, None), (None, bias, None), (None, None, allowed),
                     (None, None, None), (hist, bias, None)):
        y, best, _ = pick_ref(x, h, pen, b, ok)
        out, got = pick_run(q4k, x, h, pen, b, ok)
        assert np.array_equal(got, best)
        assert np.array_equal(out, y.astype(np.float32))
    out, got = pick_run(q4k, x, hist, pen, bias, allowed, alias=True)
    y, best, _ = pick_ref(x, hist, pen, bias, allowed)
    assert np.array_equal(got, best) and np.array_equal(out, y.astype(np.float32))
    assert np.array_equal(pick_run(q4k, x, hist, pen, bias, allowed, keep=False)[1], best)
    assert np.array_equal(pick_run(q4k, x, hist, pen, bias, allowed, pick=False)[0], y.astype(np.float32))


@pytest.mark.parametrize("R,V,H", [(1, 128256, 5000), (33, 151936, 3000), (4, 77777, 100000)])
def test_pick_real_values(q4k, R, V, H):
    rng = np.random.default_rng(V)
    x = rng.normal(0, 3, (R, V)).astype(np.float32)
    hist = [rng.choice(np.r_[np.argsort(-x[m])[:40], rng.integers(0, V, 40)], H).tolist() for m in range(R)]
    pen = np.stack([rng.uniform(1, 1.4, R), rng.uniform(0, 1, R), rng.uniform(0, 1e-2, R)], 1).astype(np.float32)
    bias = [[(int(v), float(np.float32(rng.normal()))) for v in rng.choice(V, 20, replace=False)] for _ in range(R)]
    y, best, size = pick_ref(x, hist, pen, bias, None)
    out, got = pick_run(q4k, x, hist, pen, bias, None)
    assert np.all(np.abs(out - y) <= 4 * 2.0 ** -24 * size)
    # the pick is the output's own largest, and the definition's up to the rounding
    assert np.array_equal(got, out.argmax(1))
    rows = np.arange(R)
    assert np.all(y[rows, got] >= y[rows, best] - 8 * 2.0 ** -24 * size[rows, best])


def test_pick_special_values(q4k):
    inf, nan = float("inf"), float("nan")
    V = 300
    x = np.full((8, V), -1.0, np.float32)
    x[0, 5], x[0, 7] = nan, 2.0          # NaN below every number
    x[1, :] = nan                         # nothing but NaN: the lowest index
    x[2, :] = -inf                        # nothing but -inf: the lowest index
    x[3, :] = -inf
    x[3, :9] = nan                        # -inf above NaN
    x[4, 100], x[4, 200] = inf, inf
    x[5, :] = nan
    x[6, 10], x[6, 20] = inf, 3.0         # forbidden infinity
    x[7, :] = -inf                        # allowed -inf beside forbidden numbers
    x[7, :150] = 8.0
    allowed = np.ones((8, V), bool)
    allowed[5, :40] = False
    allowed[6, 10] = False
    allowed[7, :150] = False
    for keep in (True, False):
        _, got = pick_run(q4k, x, allowed=allowed, keep=keep)
        assert got.tolist() == [7, 0, 0, 9, 100, 40, 20, 150]
    # adjusted to -inf and NaN: a ban by bias, infinities that meet, in rows that have nothing else
    x = np.full((4, V), -inf, np.float32)
    x[0, :] = 1.0
    x[1, 3:6] = 2.0
    x[2, :] = nan
    x[2, 77] = inf
    x[3, 9] = inf
    allowed = np.zeros((4, V), bool)
    allowed[0, [20, 30]] = True    # both banned
    allowed[1, 3:6] = True         # one of them not
    allowed[2, 70:80] = True       # inf - inf is NaN like the others
    allowed[3, [9, 12]] = True     # inf - inf is NaN, -inf beside it
    bias = [[(20, -inf), (30, -inf)], [(3, -inf), (4, -inf), (5, -1.0)], [(77, -inf)], [(9, -inf)]]
    hist = [[20, 20, 30], [], [], [12]]
    pen = [[1.0, 0.5, 0.5]] * 4
    for keep in (True, False):
        out, got = pick_run(q4k, x, hist, pen, bias, allowed, keep=keep)
        assert got.tolist() == [20, 5, 70, 12]


@pytest.mark.parametrize("R,V", [(1, 300000), (2, 151937), (600, 70001)])
def test_pick_long_rows_and_histories(q4k, R, V):
    """More logits than one set of tables covers, and a token that occurs more often than 16 bits count."""
    rng = np.random.default_rng(V)
    x = (rng.integers(-40, 41, (R, V)) / 8).astype(np.float32)
    long_one = 70000 if R < 10 else 50
    hist = [[int(rng.integers(0, V))] * long_one + rng.integers(0, V, 90).tolist() for _ in range(R)]
    pen = [[2.0, 0.5, 1.0 / 1024]] * R
    bias = [[(int(v), float(rng.integers(-16, 17)) / 4) for v in rng.integers(0, V, 5)] for _ in range(R)]
    y, best, _ = pick_ref(x, hist, pen, bias, None)
    out, got = pick_run(q4k, x, hist, pen, bias)
    assert np.array_equal(got, best) and np.array_equal(out, y.astype(np.float32))


@pytest.mark.parametrize("total", [32766, 32767, 32768, 32769, 65535, 65536])
def test_pick_counts_of_neighbours(q4k, total):
    """Histories about as long as a 15-bit and a 16-bit count, of two tokens side by side, with and without biases."""
    V = 23
    x = (np.random.default_rng(total).integers(-40, 41, (4, V)) / 8).astype(np.float32)
    split = [total, 0, total // 2, total - 1]
    hist = [[8] * k + [9] * (total - k) for k in split]
    pen = [[2.0, 0.5, 1.0 / 4096]] * 4
    bias = [[(8, 2.0), (9, -1.0), (8, 40.0)], [(9, 40.0)], [], [(8, 16.0)]]
    for b in (bias, None):
        y, best, _ = pick_ref(x, hist, pen, b, None)
        out, got = pick_run(q4k, x, hist, pen, b)
        assert np.array_equal(got, best) and np.array_equal(out, y.astype(np.float32))


@pytest.mark.parametrize("n", [1, 31, 32, 33, 700])
def test_pick_last_bias_counts(q4k, n):
    """Biases of few tokens over and over, more than one at a time is looked at."""
    rng = np.random.default_rng(n)
    V = 37
    x = (rng.integers(-40, 41, (5, V)) / 8).astype(np.float32)
    bias = [[(int(v), float(rng.integers(-64, 65)) / 4) for v in rng.integers(-2, V + 2, n)] for _ in range(5)]
    hist = [rng.integers(0, V, 12).tolist() for _ in range(5)]
    pen = [[2.0, 0.25, 0.125]] * 5
    for h in (hist, None):
        y, best, _ = pick_ref(x, h, pen, bias, None)
        out, got = pick_run(q4k, x, h, pen, bias)
        assert np.array_equal(got, best) and np.array_equal(out, y.astype(np.float32))


@pytest.mark.parametrize("V,seen,biased", [(5000, 3000, 0), (5003, 900, 1500), (4097, 4097, 4097), (40001, 0, 30000)])
def test_pick_many_adjusted_tokens(q4k, V, seen, biased):
    """More penalised and biased tokens than wait for the end of the row on their own."""
    rng = np.random.default_rng(V)
    R = 2
    x = (rng.integers(-40, 41, (R, V)) / 8).astype(np.float32)
    hist = [np.r_[rng.choice(V, seen, replace=False), rng.integers(0, V, seen // 3)].tolist() for _ in range(R)]
    pen = [[2.0, 0.25, 0.125]] * R
    bias = [[(int(v), float(rng.integers(-64, 65)) / 4) for v in np.r_[rng.choice(V, biased, replace=False), rng.integers(0, V, 9)]]
            for _ in range(R)]
    allowed = rng.random((R, V)) < 0.7
    for ok in (None, allowed):
        y, best, _ = pick_ref(x, hist, pen, bias, ok)
        for alias in (False, True):
            out, got = pick_run(q4k, x, hist, pen, bias, ok, alias=alias)
            assert np.array_equal(got, best) and np.array_equal(out, y.astype(np.float32))


@pytest.mark.parametrize("V", [1, 2, 3, 5, 6, 7, 8, 23, 41, 42, 4097, 9003])
def test_pick_of_a_sole_allowed_token_at_the_ends_of_a_row(q4k, V):
    """One allowed token among the row's first or last four (in a group of four that the row fills in part, for most V
    and rows), in the history, biased or both, adjusted to -infinity or NaN: it is the pick, as no other is allowed."""
    inf = float("inf")
    # (the logit, in the history, presence penalty, bias): -inf, -inf, NaN, NaN, NaN, -inf, and a number
    forms = [(1.0, False, 0.0, -inf), (1.0, True, inf, None), (inf, False, 0.0, -inf), (inf, True, inf, None),
             (-inf, True, 0.0, inf), (-inf, True, 0.5, 2.0), (1.0, True, 0.5, 3.0)]
    ends = sorted({v for v in (*range(4), *range(V - 4, V)) if 0 <= v < V})
    rows = [(v, *f) for f in forms for v in ends]
    rows = [r for r in rows for _ in range(2)]  # (an even number of each, so that V = 2 has both offsets)
    x = np.random.default_rng(V).integers(-40, 41, (len(rows), V)).astype(np.float32)
    allowed = np.zeros(x.shape, bool)
    hist, pen, bias = [], [], []
    for m, (v, logit, listed, presence, b) in enumerate(rows):
        x[m, v] = logit
        allowed[m, v] = True
        hist.append([v] if listed else [])
        pen.append([1.0, presence, 0.0])
        bias.append([] if b is None else [(v, b)])
    sole = [r[0] for r in rows]
    for keep, alias in ((True, False), (False, False), (True, True)):
        out, got = pick_run(q4k, x, hist, pen, bias, allowed, keep=keep, alias=alias)
        assert got.tolist() == sole
        if out is not None:
            with np.errstate(invalid="ignore"):
                y, _, _ = pick_ref(x, hist, pen, bias, allowed)
            assert np.array_equal(out, y.astype(np.float32), equal_nan=True)
    none = np.zeros(x.shape, bool)
    assert set(pick_run(q4k, x, hist, pen, bias, none)[1].tolist()) == {-1}


@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 4, (1 << 31) - 40])
@pytest.mark.parametrize("max_new", [8, 100])
def test_largest_windows_with_more_new_tokens_than_positions(q4k, window, max_new):
    """Positions below 0 less a window near 2^31 lie below -2^31."""
    lens, news = [5, 40, 1, 129], [8, 3, 8, 60]
    cache = make_cache(q4k, lens, 16, 2, 128, fill=float("nan"))
    check_attention(q4k, cache, [0, 1, 2, 3], news, 4, window=window, max_new=max_new)
    check_attention(q4k, cache, [0, 1, 2, 3], news, 4, window=window, sinks=2, max_new=max_new)


@pytest.mark.parametrize("T", [1, 37, 700])
@pytest.mark.parametrize("dim,kv,pairs,norm", [(64, 8, 0, False), (64, 1, 2, True), (64, 16, 1, False), (128, 4, 0, True),
                                               (128, 8, 2, False), (128, 3, 1, True)])
def test_append_to_a_cache_of_one_tensor(q4k, T, dim, kv, pairs, norm):
    """K and V the same tensor, in steps of few and of many tokens: the values remain, in every row."""
    page, heads = 32, 2 * kv
    c = make_cache(q4k, [T + 5], page, kv, dim)
    cache = q4k.Cache(c.k, c.k, c.refs, c.table, c.lens)
    Y = [torch.randn(T, h * dim, device=DEV) for h in (heads, kv, kv)]
    rope = torch.rand(c.table.shape[1] * page, dim, device=DEV)
    w = torch.rand(dim, device=DEV) + 0.5 if norm else None
    q_out = torch.empty(T, heads, dim, dtype=torch.bfloat16, device=DEV)
    at = torch.arange(5, T + 5, device=DEV)
    want = c.k.clone()
    want[0, c.table[0, at // page].long(), :, at % page] = Y[2].view(T, kv, dim).to(torch.bfloat16)
    for _ in range(3):
        cache.k.fill_(7.0)
        q4k.q4k_cache_append(cache, 0, None, ints([0, T]), *Y, q_out, heads, rope, pairs, w, w)
        torch.cuda.synchronize()
        rows = c.table[0, at // page].long(), at % page
        assert torch.equal(cache.k[0][rows[0], :, rows[1]], want[0][rows[0], :, rows[1]])
        assert int((cache.k != 7.0).flatten(2).any(2).sum()) <= c.table.shape[1]


def test_raw_addresses(q4k):
    """Device addresses in the tensors' place, where no count is taken from the tensor: the same results."""
    T, heads, kv, dim, page = 40, 4, 2, 64, 16
    Y = [torch.randn(T, h * dim, device=DEV) for h in (heads, kv, kv)]
    starts, seqs, w = ints([0, 40]), ints([0]), torch.rand(dim, device=DEV)
    results = []
    for raw in (False, True):
        to = (lambda t: t.data_ptr()) if raw else (lambda t: t)
        cache = make_cache(q4k, [100, 0], page, kv, dim, spare=5)
        cache.k.nan_to_num_(0.0)
        ws, status = cache.workspace(), ints([9])
        rope = torch.arange(cache.table.shape[1] * page * dim, device=DEV).view(-1, dim).float().cos()
        Q = torch.zeros(T, heads, dim, dtype=torch.bfloat16, device=DEV)
        out = torch.zeros_like(Q)
        q4k.q4k_cache_append(cache, 0, to(seqs), starts, Y[0], to(Y[1]), to(Y[2]), to(Q), heads, to(rope), 2, to(w), to(w))
        q4k.q4k_cache_attention(cache, 0, to(seqs), starts, Q, to(out), heads, T, dim ** -0.5, workspace=to(ws))
        q4k.q4k_pages_fork(cache, ints([0]), to(ints([1])), to(status), to(ws))
        q4k.q4k_pages_free(cache, ints([0]))
        q4k.q4k_pages_compact(cache, to(ws))
        torch.cuda.synchronize()
        assert int(status) == 0
        results.append([t.clone() for t in (Q, out, cache.k, cache.v, cache.table, cache.lens, cache.refs)])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_strides_of_single_layers_pages_and_heads_do_not_matter(q4k):
    """A dimension of one entry may have any stride, and another one in V than in K."""
    def odd(shape, strides, seed):
        base = torch.empty(1 << 16, dtype=torch.bfloat16, device=DEV)
        base.copy_(torch.randn(1 << 16, generator=torch.Generator().manual_seed(seed)))
        return base.as_strided(shape, strides)

    for shape, page_stride, a, b in (((1, 4, 2, 16, 64), 4096, (99, 4096, 1024), (4096 * 7, 4096, 1024)),
                                     ((1, 4, 1, 16, 64), 2048, (8, 2048, 5), (1, 2048, 1)),
                                     ((3, 1, 2, 16, 64), 0, (4096, 17, 1024), (4096, 4096, 1024))):
        k, v = odd(shape, (*a, 64, 1), 1), odd(shape, (*b, 64, 1), 2)
        n_pages, kv = shape[1:3]
        lens = [16 * n_pages - 5]
        refs, table = ints([1] * n_pages), torch.arange(n_pages, dtype=torch.int32, device=DEV)[None]
        cache = q4k.Cache(k, v, refs, table, ints(lens))
        for layer in range(shape[0]):
            check_attention(q4k, cache, [0], [1], 2 * kv, layer=layer)
            check_attention(q4k, cache, [0], [11], 2 * kv, layer=layer)
    k = odd((2, 4, 2, 16, 64), (8192, 2048, 1024, 64, 1), 1)
    v = odd((2, 4, 2, 16, 64), (10240, 2048, 1024, 64, 1), 1)
    with pytest.raises(ValueError, match="same shape and strides"):
        q4k.Cache(k, v, ints([0] * 4), ints([0]).view(1, 1), ints([0]))
    v = odd((2, 4, 2, 16, 64), (8192, 2048, 1024, 32, 1), 1)
    with pytest.raises(ValueError, match="contiguous"):
        q4k.Cache(k, v, ints([0] * 4), ints([0]).view(1, 1), ints([0]))


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_a_whole_step_in_every_launch_mode(q4k, mode):
    """Reserve, append, attention, fork, free, compaction and pick, each on what the call before it wrote, captured
    and replayed: the state and results of the same calls made one at a time."""
    heads, kv, dim, page, n_pages, V = 8, 2, 64, 16, 700, 1001
    table = torch.full((12, 60), -1, dtype=torch.int32, device=DEV)
    k, v = (torch.randn(3, n_pages, kv, page, dim, device=DEV).to(torch.bfloat16) for _ in range(2))
    cache = q4k.Cache(k, v, ints([0] * n_pages), table, ints([0] * 12))
    ws, status = cache.workspace(), ints([9] * 6)
    seqs, news = ints(range(6)), [300, 1, 77, 16, 31, 200]
    starts, T = ints(np.concatenate([[0], np.cumsum(news)])), sum(news)
    Y = [torch.randn(T, h * dim, device=DEV) for h in (heads, kv, kv)]
    Q = torch.zeros(T, heads, dim, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros_like(Q)
    one, ones = ints(range(7)), [torch.randn(6, h * dim, device=DEV) for h in (heads, kv, kv)]
    Q1 = torch.zeros(6, heads, dim, dtype=torch.bfloat16, device=DEV)
    out1 = torch.zeros_like(Q1)
    logits, pick = torch.randn(6, V, device=DEV), torch.zeros(6, dtype=torch.int64, device=DEV)
    adjusted, pen = torch.zeros_like(logits), torch.rand(6, 3, device=DEV) + 0.5
    scale = dim ** -0.5
    state = (cache.k, cache.v, cache.refs, cache.table, cache.lens)
    results = (Q, out, Q1, out1, status, adjusted, pick)
    begin = [t.clone() for t in state]
    calls = [
        lambda: q4k.q4k_pages_reserve(cache, seqs, starts, status),
        lambda: q4k.q4k_cache_append(cache, 1, seqs, starts, *Y, Q, heads),
        lambda: q4k.q4k_cache_attention(cache, 1, seqs, starts, Q, out, heads, 300, scale, workspace=ws),
        lambda: q4k.q4k_pages_fork(cache, seqs, ints_b, status, ws),
        lambda: q4k.q4k_pages_free(cache, odd),
        lambda: q4k.q4k_pages_compact(cache, ws),
        lambda: q4k.q4k_pages_copy(cache, src, dst),
        lambda: q4k.q4k_pages_reserve(cache, ints_b, one, status),
        lambda: q4k.q4k_cache_append(cache, 1, ints_b, one, *ones, Q1, heads),
        lambda: q4k.q4k_cache_attention(cache, 1, ints_b, one, Q1, out1, heads, 1, scale, workspace=ws),
        lambda: q4k.q4k_logits_pick(logits, 6, V, adjusted, pick, status, one, pen),
        lambda: q4k.q4k_pages_compact(cache, ws),
    ]
    ints_b, odd = ints(range(6, 12)), ints([0, 2, 4])
    src, dst = ints([0, 3]), ints([n_pages - 1, n_pages - 2])
    old = q4k.q4k_set_pdl(0)
    try:
        for call in calls:
            call()
            torch.cuda.synchronize()
        want = [t.clone() for t in (*state, *results)]
        assert int(status.sum()) == 0 and int((cache.refs > 0).sum()) > 40
        q4k.q4k_set_pdl(mode)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            for call in calls:
                call()
        for _ in range(20):
            for t, b in zip(state, begin):
                t.copy_(b)
            for t in results:
                t.fill_(5)
            graph.replay()
            torch.cuda.synchronize()
            for t, w in zip((*state, *results), want):
                assert torch.equal(t, w)
    finally:
        q4k.q4k_set_pdl(old)


def attention_rows(cache, ids, news, Q, heads, window=0, sinks=0, p_bits=None):
    """The definition on the GPU in float64, a sequence at a time, and the bound (each weight rounded to bf16: p_bits
    None, or to the sum of two, 15 bits of it: p_bits 15). Ids out of range give zeros."""
    page, dim = cache.k.shape[3], cache.head_dim
    scale = dim ** -0.5
    y = torch.zeros(Q.shape, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(y)
    lens, at = cache.lens.tolist(), 0
    for b, m in zip(ids, news):
        rows = slice(at, at + m)
        at += m
        n = lens[b] if 0 <= b < len(lens) else 0
        if m == 0 or n == 0:
            continue
        pages = cache.table[b, :-(-n // page)].long()
        k, v = (t[0][pages].transpose(0, 1).reshape(cache.kv_heads, -1, dim)[:, :n].double() for t in (cache.k, cache.v))
        q = Q[rows].double().view(m, cache.kv_heads, -1, dim)
        x = torch.einsum("mghd,gjd->mghj", q, k) * scale
        size = torch.einsum("mghd,gjd->mghj", q.abs(), k.abs()).amax(-1, keepdim=True) * scale
        p, j = torch.arange(n - m, n, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
        sees = (j <= p) & ((j > p - window) | (j < sinks) if window else j >= 0)
        x = x.masked_fill(~sees[:, None, None], -float("inf"))
        a = torch.exp(x - x.amax(-1, keepdim=True).nan_to_num(neginf=0.0))
        total = a.sum(-1, keepdim=True)
        a = torch.where(total > 0, a / total, 0.0)
        want, mean = (torch.einsum("mghj,gjd->mghd", a, t) for t in (v, v.abs()))
        bound = 2.0 ** -8 * want.abs() + (2.0 ** -(p_bits or 8) + 2.0 ** -13 + 2.0 ** -18 * size) * mean
        y[rows], tol[rows] = want.reshape(m, heads, dim), bound.reshape(m, heads, dim)
    return y, tol


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,group,most", [(33, 1, 1), (33, 16, 1), (64, 5, 1), (64, 8, 1), (64, 12, 1), (300, 4, 4), (300, 2, 3),
                                          (4096, 4, 1), (4096, 9, 1), (40, 4, 30), (200, 2, 70)])
def test_many_sequences(q4k, dim, n, group, most):
    """Steps of more than 32 sequences, single tokens and chunks, every row: lengths from 0 on (some shared out over
    several blocks), sequences without new tokens, more new tokens than positions, ids out of range."""
    rng = np.random.default_rng(n + group + dim)
    kv, page = 2, 32
    lens = np.where(rng.random(n) < 0.1, rng.integers(0, 3, n), rng.integers(1, 900 if n < 1000 else 80, n))
    lens[n // 3] = 30000 if n < 1000 else 9000  # one that is shared out
    lens[n // 2] = 5000
    news = rng.integers(0, most + 1, n) if most > 1 else (rng.random(n) < 0.9).astype(int)
    news[n // 3] = most
    ids = np.arange(n)
    ids[[5, n - 2]] = [n + 3, -1]
    counts = -(-lens // page)
    cache = make_cache(q4k, [0], page, kv, dim, spare=int(counts.sum()) + 2)  # (the pool; its table is made here)
    order = torch.randperm(cache.k.shape[1], generator=torch.Generator().manual_seed(n)).tolist()
    table = np.full((n, int(counts.max())), -1, dtype=np.int32)
    for i, c in enumerate(counts):
        table[i, :c] = [order.pop() for _ in range(c)]
    k, v = cache.k.clone(), cache.v.clone()
    for i, length in enumerate(lens):  # what lies past a sequence's end must not matter
        if length % page:
            k[0, table[i, length // page], :, length % page:] = float("nan")
            v[0, table[i, length // page], :, length % page:] = float("nan")
    cache = q4k.Cache(k, v, cache.refs, torch.tensor(table, device=DEV), ints(lens))
    heads = kv * group
    Q = (torch.randn(int(news.sum()), heads, dim, generator=torch.Generator().manual_seed(3)) * 1.5).to(torch.bfloat16).to(DEV)
    for window, sinks in ((0, 0), (300, 3))[:2 if n < 1000 else 1]:
        out = attend(q4k, cache, 0, ids, news, Q, heads, window=window, sinks=sinks, max_new=most)
        y, tol = attention_rows(cache, ids, news.tolist(), Q, heads, window, sinks, 15 if most * group <= 16 else None)
        worst = float(((out.double() - y).abs() / (tol + 1e-30)).max())
        assert worst <= 1.0, f"error {worst:.3f} of the bound"


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 8, 16])
def test_weights_of_single_tokens_have_more_bits_than_one_bf16(q4k, dim, group):
    """Values that are unit vectors give the weights themselves: within the output's own rounding, 2^-8, and 2^-15
    for the sum of two bf16 (the upper cut off, at most 2^-7 away, the lower rounded to 8 bits)."""
    n, kv = dim, 2
    cache = make_cache(q4k, [n], 64, kv, dim)
    cache.k.mul_(0.5)  # (scores, and so the fp32 part of the bound, small)
    for j in range(n):
        cache.v[0, cache.table[0, j // 64].long(), :, j % 64] = 0.0
        cache.v[0, cache.table[0, j // 64].long(), :, j % 64, j] = 1.0
    Q = torch.randn(1, kv * group, dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    out = attend(q4k, cache, 0, [0], [1], Q, kv * group).double()
    y, tol = attention_rows(cache, [0], [1], Q, kv * group, p_bits=15)
    assert bool(((out - y).abs() <= tol).all())
    # the bound tells the two apart: weights rounded to one bf16 pass it
    once = y.float().to(torch.bfloat16).double()
    low = (y / y.amax(-1, keepdim=True)).float().to(torch.bfloat16).double()  # as the kernel has them, 1 at the largest
    low = (low * y.amax(-1, keepdim=True)).float().to(torch.bfloat16).double()
    assert bool(((once - y).abs() <= tol).all()) and not bool(((low - y).abs() <= tol).all())
