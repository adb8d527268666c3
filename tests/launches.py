"""Which kernels a call launches, so that a test can say that it reaches the one it is about: the call is captured into a graph,
which is not run, and the names of the graph's kernels are read."""
from __future__ import annotations

import ctypes

import torch


class _KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _ok(status):
    assert status == 0, f"driver call failed: {status}"


def kernels(call):
    """Mangled names of the kernels that call(stream) launches, in order; template arguments read as in k_fewILi128ELi2EE."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    raw, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    _ok(cu.cuStreamBeginCapture_v2(raw, 1))  # thread-local
    try:
        call(stream)
    finally:
        ended = cu.cuStreamEndCapture(raw, ctypes.byref(graph))
    _ok(ended)
    n = ctypes.c_size_t()
    _ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
    nodes = (ctypes.c_void_p * max(n.value, 1))()
    _ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
    names = []
    for node in nodes[:n.value]:
        kind, p, name = ctypes.c_int(), _KernelNode(), ctypes.c_char_p()
        _ok(cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)))
        if kind.value != 0:  # CU_GRAPH_NODE_TYPE_KERNEL
            continue
        _ok(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)))
        if p.func:
            _ok(cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)))
        else:
            _ok(cu.cuKernelGetName(ctypes.byref(name), ctypes.c_void_p(p.kern)))
        names.append(name.value.decode())
    _ok(cu.cuGraphDestroy(graph))
    return names
