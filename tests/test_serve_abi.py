"""The calls between the products without a GPU: what they refuse, on the host,
before any CUDA call."""
import ctypes

import pytest

A = 1 << 20  # an aligned fake address, never followed


def cache(q4k, **kw):
    c = dict(k=A, v=A, layer_stride=10 * 2 * 16 * 64, page_stride=2 * 16 * 64, refs=A, table=A, lens=A, n_pages=10,
             layers=3, kv_heads=2, page_size=16, head_dim=64, n_seqs=4, width=8)
    c.update(kw)
    return ctypes.byref(q4k._CacheStruct(*[c[n] for n, _ in q4k._CacheStruct._fields_]))


def append(q4k, c, layer=0, n=1, starts=A, tokens=4, Yq=A, Yk=A, Yv=A, q_out=A, heads=4, rope=A, rows=128, pairs=1,
           qn=None, kn=None, eps=1e-6, seqs=A):
    return q4k.lib().q4k_cache_append(c, layer, seqs, n, starts, tokens, Yq, Yk, Yv, q_out, heads, rope, rows, pairs,
                                      qn, kn, eps, None)


def attend(q4k, c, layer=0, n=1, starts=A, tokens=4, Q=A, out=A, heads=4, max_new=1, scale=0.1, window=0, sinks=0,
           ws=A, ws_bytes=1 << 40, seqs=A):
    return q4k.lib().q4k_cache_attention(c, layer, seqs, n, starts, tokens, Q, out, heads, max_new, scale, window,
                                         sinks, ws, ws_bytes, None)


def every_call(q4k, c):
    L = q4k.lib()
    return [append(q4k, c), attend(q4k, c), L.q4k_pages_reserve(c, A, 1, A, A, None),
            L.q4k_pages_fork(c, A, A, 1, A, A, 1 << 40, None), L.q4k_pages_free(c, A, 1, None),
            L.q4k_pages_copy(c, A, A, 1, None), L.q4k_pages_compact(c, A, 1 << 40, None),
            L.q4k_cache_workspace(c)]


@pytest.mark.parametrize("field", ["k", "v", "refs", "table", "lens"])
def test_cache_pointers(q4k, field):
    assert set(every_call(q4k, cache(q4k, **{field: None}))) == {q4k.Q4K_ERR_NULL}
    off = 8 if field in "kv" else 2
    assert set(every_call(q4k, cache(q4k, **{field: A + off}))) == {q4k.Q4K_ERR_ALIGN}
    assert set(every_call(q4k, None)) == {q4k.Q4K_ERR_NULL}


@pytest.mark.parametrize("kw", [
    dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(page_size=0), dict(head_dim=96),
    dict(head_dim=0), dict(head_dim=256), dict(n_pages=0), dict(n_pages=(1 << 30) + 1), dict(layers=0),
    dict(layers=65536), dict(kv_heads=0), dict(kv_heads=1025), dict(n_seqs=0), dict(n_seqs=(1 << 24) + 1),
    dict(width=0), dict(width=(1 << 26) + 1), dict(page_stride=2 * 16 * 64 - 8), dict(page_stride=2 * 16 * 64 + 4),
    dict(layer_stride=10 * 2 * 16 * 64 - 8), dict(layer_stride=0), dict(layer_stride=-(1 << 20)),
    dict(page_stride=1 << 39), dict(layer_stride=2 * 16 * 64 + 8)])
def test_cache_dimensions(q4k, kw):
    assert set(every_call(q4k, cache(q4k, **kw))) == {q4k.Q4K_ERR_BAD_DIM}


@pytest.mark.parametrize("kw,status", [
    (dict(layer=-1), -2), (dict(layer=3), -2), (dict(n=0), -2), (dict(n=4097), -2), (dict(tokens=0), -2),
    (dict(heads=3), -2), (dict(heads=0), -2), (dict(heads=1), -2), (dict(tokens=(1 << 31) // 4), -2),
    (dict(starts=None), -1), (dict(starts=A + 2), -4), (dict(seqs=A + 1), -4), (dict(seqs=None, n=5), -2)])
def test_step_arguments(q4k, kw, status):
    c = cache(q4k)
    assert append(q4k, c, **kw) == status
    assert attend(q4k, c, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(Yq=None), -1), (dict(Yk=None), -1), (dict(Yv=None), -1), (dict(q_out=None), -1), (dict(rope=None), -1),
    (dict(rows=127), -2), (dict(pairs=3), -2), (dict(pairs=-1), -2), (dict(Yq=A + 4), -4), (dict(Yk=A + 8), -4),
    (dict(Yv=A + 8), -4), (dict(q_out=A + 8), -4), (dict(rope=A + 4), -4), (dict(qn=A + 4), -4), (dict(kn=A + 4), -4),
    (dict(qn=A, eps=-1.0), -2), (dict(kn=A, eps=float("nan")), -2), (dict(kn=A, eps=float("inf")), -2)])
def test_append_arguments(q4k, kw, status):
    assert append(q4k, cache(q4k), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(heads=258), -2), (dict(max_new=-1), -2),
    (dict(window=-1), -2), (dict(sinks=-1), -2), (dict(scale=0.0), -2), (dict(scale=-0.1), -2),
    (dict(scale=float("inf")), -2), (dict(scale=float("nan")), -2), (dict(Q=A + 8), -4), (dict(out=A + 8), -4),
    (dict(ws=A + 128), -4)])
def test_attention_arguments(q4k, kw, status):
    assert attend(q4k, cache(q4k), **kw) == status


def test_page_arguments(q4k):
    L, c = q4k.lib(), cache(q4k)
    assert L.q4k_pages_reserve(c, A, 1, None, A, None) == -1
    assert L.q4k_pages_reserve(c, A, 1, A, None, None) == -1
    assert L.q4k_pages_reserve(c, A, 0, A, A, None) == -2
    assert L.q4k_pages_reserve(c, A, 4097, A, A, None) == -2
    assert L.q4k_pages_reserve(c, None, 5, A, A, None) == -2
    assert L.q4k_pages_reserve(c, A, 1, A, A + 2, None) == -4
    for i in (0, 1, 3):
        args = [A, A, 1, A]
        args[i] = None
        assert L.q4k_pages_fork(c, *args, A, 1 << 40, None) == -1
    assert L.q4k_pages_fork(c, A, A, 1, A, None, 1 << 40, None) == -1
    assert L.q4k_pages_fork(c, A, A, 0, A, A, 1 << 40, None) == -2
    assert L.q4k_pages_fork(c, A, A, 4097, A, A, 1 << 40, None) == -2
    assert L.q4k_pages_fork(c, A, A, 1, A, A + 4, 1 << 40, None) == -4
    assert L.q4k_pages_free(c, None, 1, None) == -1
    assert L.q4k_pages_free(c, A, 0, None) == -2
    assert L.q4k_pages_free(c, A + 1, 1, None) == -4
    assert L.q4k_pages_copy(c, None, A, 1, None) == -1
    assert L.q4k_pages_copy(c, A, None, 1, None) == -1
    assert L.q4k_pages_copy(c, A, A, 0, None) == -2
    assert L.q4k_pages_copy(c, A, A, 1 << 31, None) == -2
    assert L.q4k_pages_copy(c, A, A + 2, 1, None) == -4
    assert L.q4k_pages_compact(c, None, 1 << 40, None) == -1
    assert L.q4k_pages_compact(c, A + 64, 1 << 40, None) == -4


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), -1), (dict(out=None, pick=None), -1), (dict(hist_starts=None), -1), (dict(penalties=None), -1),
    (dict(bias=None), -1), (dict(bias_starts=None), -1), (dict(M=0), -2), (dict(M=65536), -2), (dict(V=0), -2),
    (dict(V=1 << 31), -2), (dict(logits=A + 4), -4), (dict(out=A + 8), -4), (dict(pick=A + 4), -4),
    (dict(history=A + 2), -4), (dict(mask=A + 2), -4), (dict(bias_ids=A + 1), -4)])
def test_pick_arguments(q4k, kw, status):
    a = dict(logits=A, M=2, V=100, out=A, pick=A, history=A, hist_starts=A, penalties=A, bias_ids=A, bias=A,
             bias_starts=A, mask=A)
    a.update(kw)
    assert q4k.lib().q4k_logits_pick(*a.values(), None) == status


def test_space_status(q4k):
    assert q4k.status_string(q4k.Q4K_ERR_SPACE).startswith("Q4K_ERR_SPACE")


def test_binding_refusals(q4k):
    """The binding refuses wrong types, shapes and sizes before the C call."""
    torch = pytest.importorskip("torch")
    k = torch.zeros(1, 2, 1, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 3, dtype=torch.int32)
    for bad in (dict(k=k.float()), dict(v=k[..., :32]), dict(k=k[0]), dict(refs=i.long()), dict(table=i), dict(lens=t)):
        with pytest.raises(ValueError):
            q4k.Cache(**{**dict(k=k, v=k, refs=i, table=t, lens=i), **bad})
    with pytest.raises(ValueError, match="CUDA device memory"):
        q4k.Cache(k, k, i, t, i)
    x = torch.zeros(2, 10)
    with pytest.raises(ValueError, match="the call needs"):
        q4k.q4k_logits_pick(x, 3, 10, x)
    with pytest.raises(ValueError, match="must be torch.float32"):
        q4k.q4k_logits_pick(x.double(), 2, 10, x)


class Tensor:
    """Stands for a CUDA tensor: what the binding looks at."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.is_cuda = dtype, shape, True

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A


@pytest.mark.parametrize("ids,values,refused", [(5, 4, True), (5, 0, True), (1, 0, True), (5, 5, None), (5, 6, None)])
def test_pick_refuses_fewer_biases_than_ids(q4k, ids, values, refused):
    """Every id's value is read, so there must be one for each."""
    torch = pytest.importorskip("torch")
    i32, f32 = torch.int32, torch.float32
    call = lambda: q4k.q4k_logits_pick(  # noqa: E731
        A, 0, 10, A, A, bias_ids=Tensor(i32, ids), bias=Tensor(f32, values), bias_starts=A, stream=0)
    if refused:
        with pytest.raises(ValueError, match="bias holds"):
            call()
    else:
        with pytest.raises(q4k.Q4KError, match="Q4K_ERR_BAD_DIM"):  # (M = 0: nothing is launched)
            call()


def test_counts_come_from_tensors(q4k):
    """An address says nothing of how many entries there are: refused where the call has no other argument for it."""
    for call in (lambda: q4k.q4k_pages_fork(None, A, A, A, A), lambda: q4k.q4k_pages_free(None, A),
                 lambda: q4k.q4k_pages_copy(None, A, A), lambda: q4k.q4k_pages_reserve(None, A, A, A)):
        with pytest.raises(ValueError, match="must be a tensor"):
            call()
