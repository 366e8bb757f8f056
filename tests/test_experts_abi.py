"""The expert layer's calls without a GPU: what they refuse, on the host, before
any CUDA call, and what the binding refuses before the call."""
import pytest

A = 1 << 20  # an aligned fake address, never followed


def norm(q4k, **kw):
    a = dict(x=A, x_type=0, delta=A, weight=A, eps=1e-6, T=3, C=64, sum=A, out=A, out_type=1, codes=A, scales=A)
    a.update(kw)
    return q4k.lib().q4k_add_norm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(weight=None), -1), (dict(out=None, codes=None, scales=None), -1), (dict(codes=None), -1),
    (dict(scales=None), -1), (dict(x_type=2), -2), (dict(x_type=-1), -2), (dict(out_type=2), -2), (dict(T=0), -2),
    (dict(T=1 << 31), -2), (dict(C=0), -2), (dict(C=16), -2), (dict(C=48), -2), (dict(C=32800), -2), (dict(eps=-1e-6), -2),
    (dict(eps=float("nan")), -2), (dict(eps=float("inf")), -2), (dict(x=A + 8), -4), (dict(delta=A + 4), -4),
    (dict(weight=A + 4), -4), (dict(sum=A + 8), -4), (dict(out=A + 8), -4), (dict(codes=A + 4), -4)])
def test_norm_arguments(q4k, kw, status):
    assert norm(q4k, **kw) == status


def route(q4k, **kw):
    a = dict(logits=A, T=9, E=8, k=2, weighting=1, scale=1.0, ids=A, weights=A, order=A, slots=A, starts=A, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    return q4k.lib().q4k_route(*a.values(), None)


@pytest.mark.parametrize("kw,status", [(dict([(n, None)]), -1) for n in
                                       ("logits", "ids", "weights", "order", "slots", "starts", "ws")] + [
    (dict(T=0), -2), (dict(T=1 << 30), -2), (dict(E=0), -2), (dict(E=1025), -2), (dict(k=0), -2), (dict(k=9), -2),
    (dict(k=33, E=64), -2), (dict(weighting=-1), -2), (dict(weighting=4), -2), (dict(scale=float("nan")), -2),
    (dict(scale=float("inf")), -2), (dict(logits=A + 2), -4), (dict(ids=A + 1), -4), (dict(weights=A + 2), -4),
    (dict(order=A + 2), -4), (dict(slots=A + 2), -4), (dict(starts=A + 2), -4), (dict(ws=A + 1), -4),
    (dict(ws_bytes=4 * 8 * 2 - 1), -7), (dict(T=65, ws_bytes=4 * 8 * 3 - 1), -7)])
def test_route_arguments(q4k, kw, status):
    assert route(q4k, **kw) == status


def test_route_workspace(q4k):
    for T, E in ((1, 1), (64, 128), (65, 128), (8192, 60), ((1 << 31) - 1, 1024)):
        assert q4k.q4k_route_workspace(T, E) == 4 * E * (-(-T // 64) + 1)
    for T, E in ((0, 8), (1 << 31, 8), (8, 0), (8, 1025)):
        with pytest.raises(q4k.Q4KError):
            q4k.q4k_route_workspace(T, E)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), -1), (dict(order=None), -1), (dict(out=None), -1), (dict(T=0), -2), (dict(k=0), -2), (dict(k=33), -2),
    (dict(T=1 << 30, k=2), -2), (dict(C=0), -2), (dict(C=12), -2), (dict(C=40, scales=A), -2), (dict(C=32776), -2),
    (dict(X=A + 8), -4), (dict(X=A + 4, scales=A), -4), (dict(order=A + 2), -4), (dict(out=A + 8), -4)])
def test_gather_arguments(q4k, kw, status):
    a = dict(X=A, scales=None, order=A, T=4, k=2, C=64, out=A)
    a.update(kw)
    assert q4k.lib().q4k_experts_gather(*a.values(), None) == status


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(W=None), -1), (dict(X=None), -1), (dict(starts=None), -1), (dict(Y=None), -1), (dict(E=0), -2), (dict(E=1025), -2),
    (dict(N=0), -2), (dict(N=1 << 31), -2), (dict(E=1024, N=1 << 21), -2), (dict(K=0), -2), (dict(K=128), -2),
    (dict(K=300), -2), (dict(K=(1 << 24) + 256), -2), (dict(pairs=0), -2), (dict(pairs=1 << 31), -2), (dict(W=A + 8), -4),
    (dict(X=A + 8), -4), (dict(Y=A + 8), -4), (dict(starts=A + 2), -4)])
def test_product_arguments(q4k, kw, status, gated):
    a = dict(W=A, E=4, N=64, K=256, X=A, starts=A, pairs=10, Y=A)
    a.update(kw)
    L = q4k.lib()
    if gated:
        assert L.q4k_experts_gated(a["W"], A, *list(a.values())[1:], None) == status
        if "W" in kw:
            assert L.q4k_experts_gated(A, a["W"], *list(a.values())[1:], None) == status
    else:
        assert L.q4k_experts_matmul(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(Y=None), -1), (dict(slots=None), -1), (dict(weights=None), -1), (dict(out=None), -1), (dict(pairs=0), -2),
    (dict(pairs=1 << 31), -2), (dict(T=0), -2), (dict(T=1 << 30), -2), (dict(k=0), -2), (dict(k=33), -2), (dict(C=0), -2),
    (dict(C=12), -2), (dict(C=32776), -2), (dict(Y=A + 8), -4), (dict(base=A + 8), -4), (dict(out=A + 8), -4),
    (dict(slots=A + 2), -4), (dict(weights=A + 1), -4)])
def test_combine_arguments(q4k, kw, status):
    a = dict(Y=A, pairs=8, slots=A, weights=A, base=A, T=4, k=2, C=64, out=A)
    a.update(kw)
    assert q4k.lib().q4k_experts_combine(*a.values(), None) == status


def test_binding_refuses(q4k):
    """Tensors that are too small, of another type or shape, not contiguous or not on the device."""
    torch = pytest.importorskip("torch")
    f, b, i, u = (lambda *s, d=d: torch.zeros(*s, dtype=d) for d in
                  (torch.float32, torch.bfloat16, torch.int32, torch.uint8))
    with pytest.raises(ValueError):
        q4k.q4k_add_norm(f(2, 64), None, f(64), out=b(2, 64))      # host memory
    with pytest.raises(ValueError):
        q4k.q4k_add_norm(f(64), None, f(64), out=b(64))            # one dimension
    with pytest.raises(ValueError):
        q4k.q4k_add_norm(i(2, 64), None, f(64), out=b(2, 64))      # type of x
    with pytest.raises(ValueError):
        q4k.q4k_add_norm(f(2, 64), None, f(64), out=A)             # an address has no type
    with pytest.raises(ValueError):
        q4k.q4k_route(f(8), 2, 0, 1.0, i(2), f(2), i(2), i(2), i(9), u(1000))
    with pytest.raises(ValueError):
        q4k.q4k_experts_gather(b(4), i(4), 1, b(4, 64))
    with pytest.raises(ValueError):
        q4k.q4k_experts_matmul(u(10), 64, 256, b(4, 512), i(5), b(4, 64))   # columns of X
    with pytest.raises(ValueError):
        q4k.q4k_experts_matmul(u(10), 64, 256, b(4, 256), A, b(4, 64))      # starts are counted
    with pytest.raises(ValueError):
        q4k.q4k_experts_combine(b(8, 64), i(8), f(8), f(4, 64))
