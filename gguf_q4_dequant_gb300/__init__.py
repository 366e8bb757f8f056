"""Python binding of libq4k, the GB300 packed Q4_K dequant-matmul library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/q4k.h``. The functions mirror
the C names and take torch tensors (device memory, caller-owned) or raw device
pointers (ints; an array that a count is taken from, as the step's ``starts`` or
sequences to free, has to be a tensor). There is no fallback: if ``libq4k.so``
has not been built, or a call fails, a ``Q4KError`` is raised.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libq4k.so")

Q4K_OK = 0
Q4K_ERR_NULL = -1
Q4K_ERR_BAD_DIM = -2
Q4K_ERR_CUDA = -3
Q4K_ERR_ALIGN = -4
Q4K_ERR_ARCH = -5
Q4K_ERR_TIMEOUT = -6
Q4K_ERR_SPACE = -7

#: every symbol include/q4k.h declares
EXPORTS = ("q4k_status_string", "q4k_init", "q4k_dequant", "q4k_matmul", "q4k_matmul_bf16",
           "q4k_matmul_multi", "q4k_matmul_multi_bf16", "q4k_matmul_argmax",
           "q4k_matmul_argmax_bf16", "q4k_set_pdl", "q4k_device_error", "q4k_selftest_timeout",
           "q4k_cache_workspace", "q4k_cache_append", "q4k_cache_attention", "q4k_pages_reserve",
           "q4k_pages_fork", "q4k_pages_free", "q4k_pages_copy", "q4k_pages_compact", "q4k_logits_pick",
           "q4k_add_norm", "q4k_route_workspace", "q4k_route", "q4k_experts_gather", "q4k_experts_matmul",
           "q4k_experts_gated", "q4k_experts_combine")
MAX_GROUP = 8

#: weightings of q4k_route
ROUTE_SOFTMAX, ROUTE_SOFTMAX_TOP, ROUTE_SIGMOID, ROUTE_SIGMOID_TOP = range(4)


_STATUS_NAMES = {Q4K_OK: "Q4K_OK", Q4K_ERR_NULL: "Q4K_ERR_NULL", Q4K_ERR_BAD_DIM: "Q4K_ERR_BAD_DIM",
                 Q4K_ERR_CUDA: "Q4K_ERR_CUDA", Q4K_ERR_ALIGN: "Q4K_ERR_ALIGN",
                 Q4K_ERR_ARCH: "Q4K_ERR_ARCH", Q4K_ERR_TIMEOUT: "Q4K_ERR_TIMEOUT",
                 Q4K_ERR_SPACE: "Q4K_ERR_SPACE"}


class Q4KError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS_NAMES.get(status, 'unknown status')} ({status})")


class _CacheStruct(ctypes.Structure):
    """struct q4k_cache of include/q4k.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("refs", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("layers", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_seqs", ctypes.c_int32), ("width", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libq4k.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise Q4KError(Q4K_ERR_CUDA, f"libq4k.so not built at {LIB_PATH} "
                               "(run gguf_q4_dequant_gb300.build.build())")
            L = ctypes.CDLL(LIB_PATH)
            vp, i64 = ctypes.c_void_p, ctypes.c_int64
            L.q4k_status_string.argtypes = [ctypes.c_int]
            L.q4k_status_string.restype = ctypes.c_char_p
            L.q4k_init.argtypes = []
            L.q4k_init.restype = ctypes.c_int
            L.q4k_dequant.argtypes = [vp, i64, i64, vp, vp]
            L.q4k_dequant.restype = ctypes.c_int
            L.q4k_matmul.argtypes = [vp, i64, i64, vp, i64, vp, vp]
            L.q4k_matmul.restype = ctypes.c_int
            L.q4k_matmul_bf16.argtypes = [vp, i64, i64, vp, i64, vp, vp]
            L.q4k_matmul_bf16.restype = ctypes.c_int
            vpp = ctypes.POINTER(ctypes.c_void_p)
            i64p = ctypes.POINTER(ctypes.c_int64)
            L.q4k_matmul_multi.argtypes = [ctypes.c_int, vpp, i64p, i64, vp, i64, vpp, vp]
            L.q4k_matmul_multi.restype = ctypes.c_int
            L.q4k_matmul_multi_bf16.argtypes = [ctypes.c_int, vpp, i64p, i64, vp, i64, vpp, vp]
            L.q4k_matmul_multi_bf16.restype = ctypes.c_int
            L.q4k_matmul_argmax.argtypes = [vp, i64, i64, vp, i64, vp, vp]
            L.q4k_matmul_argmax.restype = ctypes.c_int
            L.q4k_matmul_argmax_bf16.argtypes = [vp, i64, i64, vp, i64, vp, vp]
            L.q4k_matmul_argmax_bf16.restype = ctypes.c_int
            L.q4k_set_pdl.argtypes = [ctypes.c_int]
            L.q4k_set_pdl.restype = ctypes.c_int
            L.q4k_device_error.argtypes = [ctypes.c_int]
            L.q4k_device_error.restype = ctypes.c_int
            L.q4k_selftest_timeout.argtypes = [i64, vp]
            L.q4k_selftest_timeout.restype = ctypes.c_int
            ci, cf, cp = ctypes.c_int, ctypes.c_float, ctypes.POINTER(_CacheStruct)
            L.q4k_route_workspace.argtypes = [i64, i64]
            L.q4k_route_workspace.restype = i64
            L.q4k_cache_workspace.argtypes = [cp]
            L.q4k_cache_workspace.restype = i64
            for name, args in (
                    ("q4k_cache_append", [cp, ci, vp, ci, vp, i64, vp, vp, vp, vp, ci, vp, i64, ci, vp, vp, cf, vp]),
                    ("q4k_cache_attention", [cp, ci, vp, ci, vp, i64, vp, vp, ci, ci, cf, ci, ci, vp, i64, vp]),
                    ("q4k_pages_reserve", [cp, vp, ci, vp, vp, vp]),
                    ("q4k_pages_fork", [cp, vp, vp, ci, vp, vp, i64, vp]),
                    ("q4k_pages_free", [cp, vp, ci, vp]),
                    ("q4k_pages_copy", [cp, vp, vp, i64, vp]),
                    ("q4k_pages_compact", [cp, vp, i64, vp]),
                    ("q4k_logits_pick", [vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
                    ("q4k_add_norm", [vp, ci, vp, vp, cf, i64, i64, vp, vp, ci, vp, vp, vp]),
                    ("q4k_route", [vp, i64, i64, ci, ci, cf, vp, vp, vp, vp, vp, vp, i64, vp]),
                    ("q4k_experts_gather", [vp, vp, vp, i64, ci, i64, vp, vp]),
                    ("q4k_experts_matmul", [vp, i64, i64, i64, vp, vp, i64, vp, vp]),
                    ("q4k_experts_gated", [vp, vp, i64, i64, i64, vp, vp, i64, vp, vp]),
                    ("q4k_experts_combine", [vp, i64, vp, vp, vp, i64, ci, i64, vp, vp])):
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = ci
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().q4k_status_string(int(status)).decode()


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor must live in CUDA device memory")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


_current_stream = None  # a function that gives the address of the current stream


def _find_current_stream():
    global _current_stream
    import torch
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
    if raw is not None:  # the same address without building a Stream object (2.9 us of a call's host time)
        _current_stream = lambda: raw(device())  # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731


def _stream(stream) -> int:
    if stream is None:
        if _current_stream is None:
            _find_current_stream()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != Q4K_OK:
        raise Q4KError(rc, where)


def _check_dtype(t, dtype, name):
    if not isinstance(t, int) and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _dims_valid(N, K, M=1):
    return N >= 1 and M >= 1 and K >= 256 and K % 256 == 0


def _check_size(t, need: int, name: str):
    """A tensor (not a raw pointer) must hold at least `need` elements, so that
    no kernel reads or writes past it."""
    if t is not None and not isinstance(t, int) and t.numel() < need:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs {need}")


def _w_bytes(N, K):
    return N * (K // 256) * 144


def _check_matmul_sizes(W, N, K, X, M, Y):
    if not _dims_valid(N, K, M):
        return  # the C ABI rejects the dimensions themselves
    _check_size(W, _w_bytes(N, K), "W")
    _check_size(X, M * K, "X")
    _check_size(Y, M * N, "Y")


def q4k_init():
    _check(lib().q4k_init(), "q4k_init")


def q4k_dequant(W, N: int, K: int, out, stream=None):
    """out[n*K + k] = w(n, k): packed uint8 W -> fp32 out (both on the device)."""
    import torch
    _check_dtype(W, torch.uint8, "W")
    _check_dtype(out, torch.float32, "out")
    if _dims_valid(N, K):
        _check_size(W, _w_bytes(N, K), "W")
        _check_size(out, N * K, "out")
    _check(lib().q4k_dequant(_ptr(W), N, K, _ptr(out), _stream(stream)), "q4k_dequant")


def q4k_matmul(W, N: int, K: int, X, M: int, Y, stream=None):
    """Y[M, N] = X[M, K] (fp32) * W^T."""
    import torch
    _check_dtype(W, torch.uint8, "W")
    _check_dtype(X, torch.float32, "X")
    _check_dtype(Y, torch.float32, "Y")
    _check_matmul_sizes(W, N, K, X, M, Y)
    _check(lib().q4k_matmul(_ptr(W), N, K, _ptr(X), M, _ptr(Y), _stream(stream)), "q4k_matmul")


def q4k_matmul_bf16(W, N: int, K: int, X, M: int, Y, stream=None):
    """Y[M, N] = X[M, K] (bf16) * W^T."""
    import torch
    _check_dtype(W, torch.uint8, "W")
    _check_dtype(X, torch.bfloat16, "X")
    _check_dtype(Y, torch.float32, "Y")
    _check_matmul_sizes(W, N, K, X, M, Y)
    _check(lib().q4k_matmul_bf16(_ptr(W), N, K, _ptr(X), M, _ptr(Y), _stream(stream)),
           "q4k_matmul_bf16")


def q4k_matmul_multi(Ws, Ns, K: int, X, M: int, Ys, stream=None):
    """Y_i[M, N_i] = X[M, K] * W_i^T for matrices sharing K and X (fp32 or bf16 X)."""
    import torch
    count = len(Ws)
    if not (len(Ns) == len(Ys) == count):
        raise ValueError("Ws, Ns and Ys must have the same length")
    for W, Y in zip(Ws, Ys):
        _check_dtype(W, torch.uint8, "W")
        _check_dtype(Y, torch.float32, "Y")
    bf16 = not isinstance(X, int) and X.dtype == torch.bfloat16
    if not bf16:
        _check_dtype(X, torch.float32, "X")
    for W, N, Y in zip(Ws, Ns, Ys):
        _check_matmul_sizes(W, int(N), K, X, M, Y)
    w_arr = (ctypes.c_void_p * count)(*[_ptr(W) for W in Ws])
    n_arr = (ctypes.c_int64 * count)(*[int(n) for n in Ns])
    y_arr = (ctypes.c_void_p * count)(*[_ptr(Y) for Y in Ys])
    fn = lib().q4k_matmul_multi_bf16 if bf16 else lib().q4k_matmul_multi
    _check(fn(count, w_arr, n_arr, K, _ptr(X), M, y_arr, _stream(stream)), "q4k_matmul_multi")


def q4k_matmul_argmax(W, N: int, K: int, X, M: int, out, stream=None):
    """out[m] = argmax_n (X[M, K] * W^T)[m, n] (int64, lowest n on ties), fp32 or bf16 X, M <= 16."""
    import torch
    _check_dtype(W, torch.uint8, "W")
    _check_dtype(out, torch.int64, "out")
    bf16 = not isinstance(X, int) and X.dtype == torch.bfloat16
    if not bf16:
        _check_dtype(X, torch.float32, "X")
    _check_matmul_sizes(W, N, K, X, M, None)
    if M >= 1:
        _check_size(out, M, "out")
    fn = lib().q4k_matmul_argmax_bf16 if bf16 else lib().q4k_matmul_argmax
    _check(fn(_ptr(W), N, K, _ptr(X), M, _ptr(out), _stream(stream)), "q4k_matmul_argmax")


def argmax(W, N: int, K: int, X, out=None, stream=None):
    """Convenience: the fused argmax, allocating out with torch if not given."""
    import torch
    M = X.shape[0]
    if out is None:
        out = torch.empty(M, dtype=torch.int64, device=X.device)
    q4k_matmul_argmax(W, N, K, X, M, out, stream)
    return out


def q4k_selftest_timeout(limit_ns: int, stream=None):
    """Runs the one-thread kernel whose bounded wait runs out after limit_ns
    (the library's timeout path, without a fault); q4k_device_error() then
    reports Q4K_ERR_TIMEOUT."""
    _check(lib().q4k_selftest_timeout(int(limit_ns), _stream(stream)), "q4k_selftest_timeout")


def q4k_set_pdl(mode: int) -> int:
    """Programmatic-dependent-launch mode for later calls (0, 1 or 2); returns the old mode."""
    rc = lib().q4k_set_pdl(int(mode))
    if rc < 0:
        raise Q4KError(rc, "q4k_set_pdl")
    return rc


def q4k_device_error(clear: bool = True) -> int:
    """Status of the device error word (synchronous)."""
    return lib().q4k_device_error(1 if clear else 0)


def matmul(W, N: int, K: int, X, Y=None, stream=None):
    """Convenience: dispatch on X's dtype, allocating Y with torch if not given."""
    import torch
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    if X.dtype == torch.bfloat16:
        q4k_matmul_bf16(W, N, K, X, M, Y, stream)
    else:
        q4k_matmul(W, N, K, X, M, Y, stream)
    return Y


# ------------------------------------------------- between the products ---

class Cache:
    """The paged cache of a model: caller-owned tensors and the struct q4k_cache that names them.

    k, v   bf16 [layers, n_pages, kv_heads, page_size, head_dim]; the layer and page strides are
           free (k and v may be views into one allocation), a page of a layer is contiguous
    refs   int32 [n_pages], sequences that hold each page
    table  int32 [n_seqs, width], pages of each sequence (-1: none)
    lens   int32 [n_seqs], positions of each sequence

    The object keeps the tensors alive; it holds no state of its own.
    """

    def __init__(self, k, v, refs, table, lens):
        import torch
        for t, name in ((k, "k"), (v, "v")):
            _check_dtype(t, torch.bfloat16, name)
            if t.dim() != 5:
                raise ValueError(f"{name} must be [layers, n_pages, kv_heads, page_size, head_dim]")
        for t, dims, name in ((refs, 1, "refs"), (table, 2, "table"), (lens, 1, "lens")):
            _check_dtype(t, torch.int32, name)
            if t.dim() != dims:
                raise ValueError(f"{name} must have {dims} dimension{'s' if dims > 1 else ''}")
            _ptr(t)
        layers, n_pages, kv_heads, page_size, head_dim = k.shape
        # a stride of a single layer, page or head is never used: any one will do
        used = [i for i in range(5) if k.shape[i] > 1]
        if v.shape != k.shape or any(v.stride(i) != k.stride(i) for i in used if i < 2):
            raise ValueError("k and v must have the same shape and strides")
        for t, name in ((k, "k"), (v, "v")):
            if any(t.stride(i) != (page_size * head_dim, head_dim, 1)[i - 2] for i in used if i >= 2):
                raise ValueError(f"a page of a layer of {name} must be contiguous")
            if not t.is_cuda:
                raise ValueError("tensor must live in CUDA device memory")
        if refs.numel() != n_pages or table.shape[0] != lens.numel():
            raise ValueError("refs must have n_pages entries, and table a row for each entry of lens")
        if len({t.device for t in (k, v, refs, table, lens)}) != 1:
            raise ValueError("the tensors of a cache must be on one device")
        self.k, self.v, self.refs, self.table, self.lens = k, v, refs, table, lens
        self.layers, self.kv_heads, self.head_dim = layers, kv_heads, head_dim
        page = kv_heads * page_size * head_dim
        page_stride = k.stride(1) if n_pages > 1 else page
        layer_stride = k.stride(0) if layers > 1 else page_stride * n_pages
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), layer_stride, page_stride, refs.data_ptr(),
                                    table.data_ptr(), lens.data_ptr(), n_pages, layers, kv_heads, page_size,
                                    head_dim, lens.numel(), table.shape[1])
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def empty(cls, layers, n_pages, kv_heads, page_size, head_dim, n_seqs, max_len, device="cuda"):
        """A cache with all pages free, allocated with torch."""
        import torch
        shape = (layers, n_pages, kv_heads, page_size, head_dim)
        return cls(torch.empty(shape, dtype=torch.bfloat16, device=device),
                   torch.empty(shape, dtype=torch.bfloat16, device=device),
                   torch.zeros(n_pages, dtype=torch.int32, device=device),
                   torch.full((n_seqs, -(-max_len // page_size)), -1, dtype=torch.int32, device=device),
                   torch.zeros(n_seqs, dtype=torch.int32, device=device))

    def workspace(self):
        """A workspace for the calls that take one (a zeroed uint8 tensor)."""
        import torch
        return torch.zeros(q4k_cache_workspace(self), dtype=torch.uint8, device=self.k.device)


def q4k_cache_workspace(cache: Cache) -> int:
    """Bytes of the workspace of a cache's calls."""
    n = lib().q4k_cache_workspace(cache._ref)
    if n < 0:
        raise Q4KError(n, "q4k_cache_workspace")
    return n


def _tensor(t, dtype, need, name):
    """Device address of a contiguous tensor of at least `need` elements (an int is passed through)."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype is dtype and t.numel() >= need and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:  # (what is wrong with it)
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < need:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs {need}")
    return _ptr(t)


def _step(seqs, starts):
    """(seqs address, n, starts address) of a step's batch."""
    import torch
    if isinstance(starts, int) or starts.dim() != 1 or starts.numel() < 2:
        raise ValueError("starts must be a tensor of n + 1 offsets")
    n = starts.numel() - 1
    return _tensor(seqs, torch.int32, n, "seqs"), n, _tensor(starts, torch.int32, n + 1, "starts")


def _count(t, name):
    if isinstance(t, int):
        raise ValueError(f"{name} must be a tensor, its entries are counted")
    return t.numel()


def _workspace(cache, ws, uint8):
    """(address, bytes) of a workspace; an address is taken to have the bytes that the calls need."""
    if ws is None or isinstance(ws, int):
        return ws, q4k_cache_workspace(cache) if ws else 0
    return _tensor(ws, uint8, 0, "workspace"), ws.numel()


def q4k_cache_append(cache: Cache, layer: int, seqs, starts, Yq, Yk, Yv, q_out, heads: int, rope=None,
                     pairs: int = 0, q_norm=None, k_norm=None, eps: float = 1e-6, stream=None):
    """A step's keys and values into the pages of a layer, its queries to q_out [tokens, heads, head_dim]
    (bf16), from the fp32 products Yq, Yk, Yv; optional per-head norm and rotation (see include/q4k.h)."""
    import torch
    f32, D, G = torch.float32, cache.head_dim, cache.kv_heads
    s, n, st = _step(seqs, starts)
    if isinstance(Yq, int) or Yq.dim() < 2:
        raise ValueError("Yq must be a tensor of a row per token")
    tokens = Yq.shape[0]
    rows = 0
    if isinstance(rope, int):  # taken to have a row for every position
        rows = cache.table.shape[1] * cache.k.shape[3]
    elif rope is not None:
        rows = rope.shape[0]
        if rope.numel() != rows * D:
            raise ValueError("rope must be [rows, head_dim]")
    _check(lib().q4k_cache_append(
        cache._ref, layer, s, n, st, tokens, _tensor(Yq, f32, tokens * heads * D, "Yq"),
        _tensor(Yk, f32, tokens * G * D, "Yk"), _tensor(Yv, f32, tokens * G * D, "Yv"),
        _tensor(q_out, torch.bfloat16, tokens * heads * D, "q_out"), heads, _tensor(rope, f32, 0, "rope"), rows,
        pairs, _tensor(q_norm, f32, D, "q_norm"), _tensor(k_norm, f32, D, "k_norm"), eps, _stream(stream)),
        "q4k_cache_append")


def q4k_cache_attention(cache: Cache, layer: int, seqs, starts, Q, out, heads: int, max_new: int, scale: float,
                        window: int = 0, sinks: int = 0, workspace=None, stream=None):
    """out[tokens, heads, head_dim] = attention of the step's new tokens Q over their sequences' pages."""
    import torch
    s, n, st = _step(seqs, starts)
    if isinstance(Q, int) or Q.dim() < 2:
        raise ValueError("Q must be a tensor of a row per token")
    tokens = Q.shape[0]
    need = tokens * heads * cache.head_dim
    _check(lib().q4k_cache_attention(
        cache._ref, layer, s, n, st, tokens, _tensor(Q, torch.bfloat16, need, "Q"),
        _tensor(out, torch.bfloat16, need, "out"), heads, max_new, scale, window, sinks,
        *_workspace(cache, workspace, torch.uint8), _stream(stream)), "q4k_cache_attention")


def q4k_pages_reserve(cache: Cache, seqs, starts, status, stream=None):
    """Room for the step's new tokens: lengths and pages of the sequences grow; status int32 [n], 0 or 1."""
    import torch
    s, n, st = _step(seqs, starts)
    _check(lib().q4k_pages_reserve(cache._ref, s, n, st, _tensor(status, torch.int32, n, "status"),
                                   _stream(stream)), "q4k_pages_reserve")


def q4k_pages_fork(cache: Cache, parents, children, status, workspace=None, stream=None):
    """Sequence children[i] becomes a copy of parents[i] (shared pages; the last partial page copied)."""
    import torch
    n = _count(parents, "parents")
    i32 = torch.int32
    _check(lib().q4k_pages_fork(
        cache._ref, _tensor(parents, i32, n, "parents"), _tensor(children, i32, n, "children"), n,
        _tensor(status, i32, n, "status"), *_workspace(cache, workspace, torch.uint8), _stream(stream)), "q4k_pages_fork")


def q4k_pages_free(cache: Cache, seqs, stream=None):
    """Ends the sequences: their pages lose a reference."""
    import torch
    n = _count(seqs, "seqs")
    _check(lib().q4k_pages_free(cache._ref, _tensor(seqs, torch.int32, n, "seqs"), n, _stream(stream)),
           "q4k_pages_free")


def q4k_pages_copy(cache: Cache, src, dst, stream=None):
    """Copies page src[i] to page dst[i] in every layer."""
    import torch
    n = _count(src, "src")
    _check(lib().q4k_pages_copy(cache._ref, _tensor(src, torch.int32, n, "src"),
                                _tensor(dst, torch.int32, n, "dst"), n, _stream(stream)), "q4k_pages_copy")


def q4k_pages_compact(cache: Cache, workspace=None, stream=None):
    """Moves the pages in use to the lowest ids, in every layer; refs and table follow."""
    import torch
    _check(lib().q4k_pages_compact(cache._ref, *_workspace(cache, workspace, torch.uint8), _stream(stream)),
           "q4k_pages_compact")


def q4k_logits_pick(logits, M: int, V: int, out=None, pick=None, history=None, hist_starts=None, penalties=None,
                    bias_ids=None, bias=None, bias_starts=None, mask=None, stream=None):
    """Penalties, biases and grammar mask on fp32 logits [M, V] (to out, if given) and the greedy pick
    (int64 [M], -1 where nothing is allowed); see include/q4k.h."""
    import torch
    f32, i32 = torch.float32, torch.int32
    if not isinstance(mask, (int, type(None))) and mask.dtype == torch.uint32:
        mask = mask.view(i32)
    biases = 0 if isinstance(bias_ids, (int, type(None))) else bias_ids.numel()  # a value is read for each
    _check(lib().q4k_logits_pick(
        _tensor(logits, f32, M * V, "logits"), M, V, _tensor(out, f32, M * V, "out"),
        _tensor(pick, torch.int64, M, "pick"), _tensor(history, i32, 0, "history") or None,
        _tensor(hist_starts, i32, M + 1, "hist_starts"), _tensor(penalties, f32, 3 * M, "penalties"),
        _tensor(bias_ids, i32, 0, "bias_ids") or None, _tensor(bias, f32, biases, "bias"),
        _tensor(bias_starts, i32, M + 1, "bias_starts"), _tensor(mask, i32, M * ((V + 31) // 32), "mask"),
        _stream(stream)), "q4k_logits_pick")


# ------------------------------------------------------- the expert layer ---

_dtypes = None  # torch's float32, bfloat16, int32, uint8, float8_e4m3fn


def _types():
    global _dtypes
    if _dtypes is None:
        import torch
        _dtypes = (torch.float32, torch.bfloat16, torch.int32, torch.uint8, torch.float8_e4m3fn)
    return _dtypes


_device = None  # a function that gives the current device


def _rows(t, name):
    """(rows, columns) of a tensor of a row per token or pair, which is on the device that the call goes to."""
    global _device
    if isinstance(t, int) or t.dim() != 2:
        raise ValueError(f"{name} must be a tensor of two dimensions")
    device = t.get_device()
    if device < 0:
        raise ValueError("tensor must live in CUDA device memory")
    if _device is None:
        import torch
        _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    if device != _device():
        raise ValueError(f"{name} is on device {device}, the current one is {_device()}")
    return t.shape


def _bytes(t, need, name):
    """Address of a tensor of 8-bit codes (uint8, or torch's e4m3)."""
    _, _, _, u8, e4m3 = _types()
    return _tensor(t, e4m3 if not isinstance(t, (int, type(None))) and t.dtype is e4m3 else u8, need, name)


def q4k_add_norm(x, delta, weight, eps: float = 1e-6, sum=None, out=None, codes=None, scales=None, stream=None):
    """sum = x + delta [T, C] (x and sum fp32 or bf16; delta fp32 or None), and its RMS norm times weight as out
    (fp32 or bf16) and as e4m3 codes with scales [T, C/32] (uint8 exponents); each output may be None."""
    f32, bf16, _, u8, _ = _types()
    T, C = _rows(x, "x")
    n, kind = T * C, x.dtype
    if kind is not f32 and kind is not bf16:
        raise ValueError(f"x must be {f32} or {bf16}, got {kind}")
    if isinstance(out, int):
        raise ValueError("out must be a tensor, its type is taken from it")
    out_kind = bf16 if out is None else out.dtype
    if out_kind is not f32 and out_kind is not bf16:
        raise ValueError(f"out must be {f32} or {bf16}, got {out_kind}")
    _check(lib().q4k_add_norm(
        _tensor(x, kind, n, "x"), kind is bf16, _tensor(delta, f32, n, "delta"), _tensor(weight, f32, C, "weight"), eps, T, C,
        _tensor(sum, kind, n, "sum"), _tensor(out, out_kind, n, "out"), out_kind is bf16, _bytes(codes, n, "codes"),
        _tensor(scales, u8, T * (C // 32), "scales"), _stream(stream)), "q4k_add_norm")


def q4k_route_workspace(T: int, E: int) -> int:
    """Bytes of the workspace of q4k_route."""
    n = lib().q4k_route_workspace(T, E)
    if n < 0:
        raise Q4KError(n, "q4k_route_workspace")
    return n


def q4k_route(logits, k: int, weighting: int, scale: float, ids, weights, order, slots, starts, workspace, stream=None):
    """The k largest of the router's logits [T, E] of each token: ids, weights, slots [T, k], and the pairs by expert:
    order [T*k], starts [E + 1] (see include/q4k.h)."""
    f32, _, i32, u8, _ = _types()
    T, E = _rows(logits, "logits")
    n = T * k
    if isinstance(workspace, int):
        ws_bytes = q4k_route_workspace(T, E)  # an address is taken to have the bytes that the call needs
    else:
        ws_bytes = 0 if workspace is None else workspace.numel()
    _check(lib().q4k_route(
        _tensor(logits, f32, T * E, "logits"), T, E, k, weighting, scale, _tensor(ids, i32, n, "ids"),
        _tensor(weights, f32, n, "weights"), _tensor(order, i32, n, "order"), _tensor(slots, i32, n, "slots"),
        _tensor(starts, i32, E + 1, "starts"), _tensor(workspace, u8, 0, "workspace"), ws_bytes, _stream(stream)), "q4k_route")


def q4k_experts_gather(X, order, k: int, out, scales=None, stream=None):
    """out[p] = X[order[p] // k] (bf16 [T*k, C]) from rows X [T, C] in bf16, or in e4m3 codes with their scales."""
    _, bf16, i32, u8, _ = _types()
    T, C = _rows(X, "X")
    x = _tensor(X, bf16, T * C, "X") if scales is None else _bytes(X, T * C, "X")
    _check(lib().q4k_experts_gather(
        x, _tensor(scales, u8, T * (C // 32), "scales"), _tensor(order, i32, T * k, "order"), T, k, C,
        _tensor(out, bf16, T * k * C, "out"), _stream(stream)), "q4k_experts_gather")


def _experts(N, K, X, starts, Y):
    """(E, bytes of E packed matrices, X, starts, pairs, Y) of an experts' product, checked."""
    _, bf16, i32, _, _ = _types()
    pairs, cols = _rows(X, "X")
    if cols != K:
        raise ValueError(f"X has {cols} columns, K is {K}")
    E = _count(starts, "starts") - 1
    return (E, E * _w_bytes(N, K) if _dims_valid(N, K) else 0, _tensor(X, bf16, pairs * K, "X"),
            _tensor(starts, i32, E + 1, "starts"), pairs, _tensor(Y, bf16, pairs * max(N, 0), "Y"))


def q4k_experts_matmul(W, N: int, K: int, X, starts, Y, stream=None):
    """Y[p] = X[p] W_e^T (bf16) for the rows p of each expert e: starts [E + 1], W the E packed matrices [N, K]."""
    E, need, x, st, pairs, y = _experts(N, K, X, starts, Y)
    _check(lib().q4k_experts_matmul(_tensor(W, _types()[3], need, "W"), E, N, K, x, st, pairs, y, _stream(stream)),
           "q4k_experts_matmul")


def q4k_experts_gated(gate, up, N: int, K: int, X, starts, Y, stream=None):
    """Y[p] = silu(X[p] gate_e^T) * (X[p] up_e^T) (bf16) for the rows p of each expert e."""
    E, need, x, st, pairs, y = _experts(N, K, X, starts, Y)
    u8 = _types()[3]
    _check(lib().q4k_experts_gated(_tensor(gate, u8, need, "gate"), _tensor(up, u8, need, "up"), E, N, K, x, st, pairs, y,
                                   _stream(stream)), "q4k_experts_gated")


def q4k_experts_combine(Y, slots, weights, out, base=None, stream=None):
    """out[t] = base[t] + sum_j weights[t, j] * Y[slots[t, j]] (fp32 [T, C]); slots below 0 add nothing."""
    f32, bf16, i32, _, _ = _types()
    pairs, C = _rows(Y, "Y")
    T, k = _rows(slots, "slots")
    _check(lib().q4k_experts_combine(
        _tensor(Y, bf16, pairs * C, "Y"), pairs, _tensor(slots, i32, T * k, "slots"), _tensor(weights, f32, T * k, "weights"),
        _tensor(base, f32, T * C, "base"), T, k, C, _tensor(out, f32, T * C, "out"), _stream(stream)), "q4k_experts_combine")
