"""The nodes that a call puts into a captured graph, through the driver API."""
from __future__ import annotations

import ctypes

import torch

KINDS = {0: "kernel", 1: "memcpy", 2: "memset"}


def captured_nodes(call):
    """(kinds of the nodes that `call` captures, number of nodes without a predecessor).

    `call` runs once before the capture, and allocates nothing.  The graph is
    never launched."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
        stream.synchronize()
        raw, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
        assert cu.cuStreamBeginCapture_v2(raw, 2) == 0                      # relaxed
        try:
            call()
        finally:
            end = cu.cuStreamEndCapture(raw, ctypes.byref(graph))
    assert end == 0
    count, roots = ctypes.c_size_t(), ctypes.c_size_t()
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(count)) == 0
    assert cu.cuGraphGetRootNodes(graph, None, ctypes.byref(roots)) == 0
    kinds = []
    for node in nodes:
        kind = ctypes.c_int()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        kinds.append(KINDS.get(kind.value, kind.value))
    assert cu.cuGraphDestroy(graph) == 0
    return kinds, roots.value
