"""What a call launches: its kernels' names, grids, blocks and shared memory (of the launch, and the
most that the kernel may be launched with at that moment), read from a captured graph (driver API, read
only).  Template arguments stand in the mangled name: Li4E is the int 4."""
import ctypes
from collections import namedtuple

import torch

Launch = namedtuple("Launch", "name grid block smem most_smem")

_MOST_DYNAMIC_SMEM = 8  # CU_FUNC_ATTRIBUTE_MAX_DYNAMIC_SHARED_SIZE_BYTES


class _Params(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("dims", ctypes.c_uint * 6), ("smem", ctypes.c_uint),
                ("args", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launches_of(call):
    """The kernels that call() launches on the current stream, without running them."""
    cu = ctypes.CDLL("libcuda.so.1")

    def do(fn, *args):
        assert getattr(cu, fn)(*args) == 0, fn

    graph = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    do("cuGraphGetNodes", raw, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    do("cuGraphGetNodes", raw, nodes, ctypes.byref(n))
    found = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        do("cuGraphNodeGetType", ctypes.c_void_p(node), ctypes.byref(kind))
        if kind.value != 0:  # CU_GRAPH_NODE_TYPE_KERNEL
            continue
        p, name, most = _Params(), ctypes.c_char_p(), ctypes.c_int(-1)
        do("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node), ctypes.byref(p))
        if p.func:
            do("cuFuncGetName", ctypes.byref(name), ctypes.c_void_p(p.func))
            do("cuFuncGetAttribute", ctypes.byref(most), _MOST_DYNAMIC_SMEM, ctypes.c_void_p(p.func))
        else:
            do("cuKernelGetName", ctypes.byref(name), ctypes.c_void_p(p.kern))
            do("cuKernelGetAttribute", ctypes.byref(most), _MOST_DYNAMIC_SMEM, ctypes.c_void_p(p.kern),
               torch.cuda.current_device())
        found.append(Launch(name.value.decode(), tuple(p.dims[:3]), tuple(p.dims[3:]), p.smem, most.value))
    return found
