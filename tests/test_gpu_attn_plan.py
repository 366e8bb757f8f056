"""How the attention kernels share out a step: blocks' ranges against the same
rule with Python's integers, past 2^32 units of work too, where running the
step itself would take most of a minute."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

KEYS = 128          # positions of a key tile
CHUNK = (3, 1, 4)   # item, snap, q_min of the chunk kernel
SINGLE = (2, 3, 4)  # of the single-token kernel
HEAD, ITEM = 8, 10


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from gguf_q4_dequant_gb300 import build
    import os
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "attn_plan_walk.cu")
    lib = str(tmp_path_factory.mktemp("plan") / "plan_walk.so")
    subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, f"-I{build.CSRC}", "-shared", src, "-o", lib],
                   check=True, capture_output=True)
    L = ctypes.CDLL(lib)
    ci, vp = ctypes.c_int, ctypes.c_void_p
    L.plan_walk.argtypes = [vp, vp] + [ci] * 14 + [vp]
    L.plan_walk.restype = ci

    def run(lens, news, kv, group, tt, cost, window=0, sinks=0, grid=152, most=1, wide=2):
        n = len(lens)
        dev = lambda v: torch.tensor(np.asarray(v, dtype=np.int32), device="cuda:0")  # noqa: E731
        starts = np.concatenate([[0], np.cumsum(news)])
        out = torch.full((grid, HEAD + most * ITEM), -99, dtype=torch.int64, device="cuda:0")
        lens_d, starts_d = dev(lens), dev(starts)
        assert starts[-1] * kv * group < 1 << 31
        run.count_bytes = L.plan_walk(lens_d.data_ptr(), starts_d.data_ptr(), n, int(starts[-1]),
                                      max(1, -(-max(lens) // 128)), kv, group, tt, *cost, window, sinks, grid, most,
                                      wide, out.data_ptr())
        assert run.count_bytes != 0
        return out.cpu().numpy()

    return run


class Rule:
    """Units of every row tile: what the header of the shared part says, in 64 bits."""

    def __init__(self, lens, news, kv, tt, cost, window, sinks, grid):
        self.item, self.snap, q_min = cost
        self.kv, self.tt = kv, tt
        self.tiles = []
        for n, m in zip(lens, news):
            t = np.arange(-(-m // tt), dtype=np.int64)
            p0 = n - m + t * tt
            p1 = p0 + np.minimum(tt, m - t * tt) - 1
            end = p1 // KEYS + 1
            w0 = np.maximum(p0 - window + 1, 0) // KEYS if window else np.zeros_like(t)
            st = np.minimum((np.minimum(sinks, p1 + 1) + KEYS - 1) // KEYS, w0) if window else np.zeros_like(t)
            self.tiles.append(np.where(p1 < 0, 1, st + end - w0) + self.item)
        self.before = [np.concatenate([[0], np.cumsum(t)]) for t in self.tiles]
        self.per_head = [int(b[-1]) for b in self.before]
        at = [0]
        for u in self.per_head:
            at.append(at[-1] + u * kv)
        self.at, self.total = at, at[-1]
        self.q = max(-(-self.total // grid), q_min)

    def cut(self, u):
        """(the boundary moved, sequence, head, row tile, units inside it)"""
        if u >= self.total:
            return self.total, 0, 0, 0, 0
        b = int(np.searchsorted(np.array(self.at[1:], dtype=np.int64), u, side="right"))
        h, rest = divmod(u - self.at[b], self.per_head[b])
        t = int(np.searchsorted(self.before[b][1:], rest, side="right"))
        off, n = rest - int(self.before[b][t]), int(self.tiles[b][t])
        if off <= self.item + self.snap:
            return u - off, b, h, t, 0
        if n - off <= self.snap:
            return u + n - off, b, h, t + 1, 0
        return u, b, h, t, off


def check(walk, lens, news, kv, group, tt, cost, window=0, sinks=0, grid=152, most=1, wide=2):
    rule = Rule(lens, news, kv, tt, cost, window, sinks, grid)
    got = walk(lens, news, kv, group, tt, cost, window, sinks, grid, most, wide)
    for c in range(grid):
        begin, end = rule.cut(c * rule.q), rule.cut((c + 1) * rule.q)
        assert got[c, 2] == rule.q
        if c * rule.q < rule.total:
            assert tuple(got[c, [0, 3, 4, 5, 6]]) == begin and got[c, 1] == end[0], c
        else:
            assert got[c, 0] == got[c, 1]
    return rule, got


@pytest.mark.parametrize("lens,news,kv,group,tt,cost", [
    ([2_200_000], [2_200_000], 8, 8, 32, CHUNK),                           # one prompt, a row tile after the other
    ([2_200_000, 7, 2_000_000], [2_100_000, 7, 1], 8, 8, 32, CHUNK),
    ([400_000 + i for i in range(40)], [400_000] * 40, 8, 8, 32, CHUNK),   # more than 32 sequences: by all warps
    ([1 << 30] * 4096, [1] * 4096, 8, 4, 2, SINGLE),                       # single tokens over the longest sequences
    ([1 << 30] * 32, [1] * 32, 1024, 1, 8, SINGLE),
])
def test_more_than_32_bits_of_units(walk, lens, news, kv, group, tt, cost):
    rule, got = check(walk, lens, news, kv, group, tt, cost)
    assert rule.total > 1 << 32 and walk.count_bytes == 8
    assert got[0, 0] == 0 and got[-1, 1] == rule.total and (got[1:, 0] == got[:-1, 1]).all()
    for c, row in enumerate(got):  # the range's first item begins at the boundary
        t_first, tokens, p0, h, _, n, i0, i1, first, last = row[HEAD:HEAD + ITEM]
        b, tile, off = row[3], row[5], row[6]
        if tile == len(rule.tiles[b]):
            continue
        assert h == row[4] and t_first == sum(news[:b]) + tile * tt and p0 == lens[b] - news[b] + tile * tt
        assert n == rule.tiles[b][tile] - rule.item and i0 == max(off - rule.item, 0)
        assert first <= c <= last and (first < c) == (off > 0)


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("wide", [0, 1])
def test_every_key_tile_once(walk, seed, wide):
    """The items of all blocks are each key tile of each row tile once, and say which blocks share it."""
    rng = np.random.default_rng(seed)
    n = int(rng.choice([1, 2, 5, 32, 33, 70]))
    kv, group = int(rng.integers(1, 4)), int(rng.integers(1, 6))
    single = seed % 2 == 0
    tt, cost = (8 // group, SINGLE) if single else (2 * (128 // group), CHUNK)
    news = rng.integers(0, 9 if single else 700, n)
    lens = np.maximum(news + rng.integers(-3, 4000, n), 0)
    window, sinks = [(0, 0), (900, 4), (64, 130)][seed % 3]
    rule, got = check(walk, lens.tolist(), news.tolist(), kv, group, tt, cost, window, sinks, most=3000, wide=wide)
    starts = np.concatenate([[0], np.cumsum(news)])
    seen = {}
    for c, row in enumerate(got):
        assert row[7] < 3000
        for x in row[HEAD:HEAD + row[7] * ITEM].reshape(-1, ITEM):
            t_first, tokens, p0, h, _, keys, i0, i1, first, last = (int(v) for v in x)
            seen.setdefault((t_first, h), []).append((c, i0, i1, keys, first, last, tokens, p0))
    want = {(int(starts[b]) + t * tt, h) for b in range(n) for t in range(len(rule.tiles[b])) for h in range(kv)}
    assert set(seen) == want
    for (t_first, h), parts in seen.items():
        b = int(np.searchsorted(starts[1:], t_first, side="right"))
        t = (t_first - int(starts[b])) // tt
        assert parts[0][1] == 0 and parts[-1][2] == parts[0][3] == rule.tiles[b][t] - rule.item
        assert all(p[2] == q[1] and p[0] < q[0] for p, q in zip(parts, parts[1:]))
        assert all(p[4] == parts[0][0] and p[5] == parts[-1][0] for p in parts)
        assert [p[0] for p in parts] == list(range(parts[0][0], parts[-1][0] + 1))
        assert all(p[6] == min(tt, news[b] - t * tt) and p[7] == lens[b] - news[b] + t * tt for p in parts)


@pytest.mark.parametrize("n,news,heads,kv,lens", [(2, 300, 128, 2, [700, 450]), (16, 1, 16, 16, [130 * i + 1 for i in range(16)])])
def test_attention_with_a_table_for_the_longest_sequences(q4k, n, news, heads, kv, lens):
    """The calls themselves where the table has room for 2^30 positions, so that units are counted in 64 bits."""
    from test_gpu_serve import check_attention, make_cache
    small = make_cache(q4k, lens, 16, kv, 64, fill=float("nan"))
    table = torch.full((n, 1 << 26), -1, dtype=torch.int32, device="cuda:0")
    table[:, :small.table.shape[1]] = small.table
    cache = q4k.Cache(small.k, small.v, small.refs, table, small.lens)
    tt = 8 if heads == kv else 2 * (128 // (heads // kv))
    assert n * (n * news // tt + 1) * kv * (1 << 23) > 4.2e9
    check_attention(q4k, cache, list(range(n)), [news] * n, heads)
    check_attention(q4k, cache, list(range(n)), [news] * n, heads, window=200, sinks=3)
