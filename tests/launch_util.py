"""Which kernel a call launches, without running it: the call is captured into a
graph and the graph's kernel nodes are read through the HIP runtime.

The kernel of 256x256 tiles has 768 threads a workgroup, the one of few rows 256
or 512, so the sizes that a test means for one of them can be held to it."""
import ctypes

import mxfp4_microscaled_precision_amd as mx

TILE_THREADS = 768
_KERNEL_NODE = 0        # hipGraphNodeTypeKernel


class _Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint32), ("y", ctypes.c_uint32), ("z", ctypes.c_uint32)]


class _KernelNodeParams(ctypes.Structure):
    """hipKernelNodeParams"""
    _fields_ = [("blockDim", _Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p),
                ("gridDim", _Dim3), ("kernelParams", ctypes.c_void_p),
                ("sharedMemBytes", ctypes.c_uint32)]


def block_threads(call):
    """Threads of a workgroup of each kernel that call() launches, in order of
    capture. Nothing is run."""
    import torch
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    hip = ctypes.CDLL(mx._hip_runtimes_mapped()[0])
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert hip.hipGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * max(1, n.value))()
    assert hip.hipGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    threads = []
    for node in nodes[:n.value]:
        kind, params = ctypes.c_int(-1), _KernelNodeParams()
        assert hip.hipGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == _KERNEL_NODE:
            assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(params)) == 0
            threads.append(params.blockDim.x)
    return threads


def only_tiles(call):
    """Whether the call launches one kernel and it is the one of 256x256 tiles."""
    return block_threads(call) == [TILE_THREADS]
