"""The names of the kernels that a call launches, from a graph that captures it."""
import ctypes

import torch


class _KernelNode(ctypes.Structure):
    """CUDA_KERNEL_NODE_PARAMS of the driver API, version 2."""
    _fields_ = [("func", ctypes.c_void_p), ("grid_block_smem", ctypes.c_uint * 7), ("params", ctypes.c_void_p),
                ("extra", ctypes.c_void_p), ("kernel", ctypes.c_void_p), ("context", ctypes.c_void_p)]


def kernels(call):
    """The (mangled) names of the kernels of call(), in no order. The call runs once before; captured, it does not run."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cuda, n = ctypes.CDLL("libcuda.so.1"), ctypes.c_size_t()
    raw = ctypes.c_void_p(graph.raw_cuda_graph())
    assert cuda.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes, names = (ctypes.c_void_p * n.value)(), []
    assert cuda.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    for node in nodes:
        kind, p, name = ctypes.c_int(), _KernelNode(), ctypes.c_char_p()
        assert cuda.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value != 0:  # no kernel
            continue
        assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        assert cuda.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)) == 0
        names.append(name.value.decode())
    return names
