"""The layer's weight-streaming launches have no more blocks than the GPU holds at once.

A block's shared memory grows with the lists of chosen experts, so that with many experts and pairs an SM holds one block
instead of two; a grid of two an SM would then run as two waves, one after the other.  The grids are read from a captured
graph, the blocks an SM holds from the driver's occupancy calculation.
"""
import ctypes

import pytest
import torch

from test_gpu_layer import check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


class KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "smem")] + [
        (n, ctypes.c_void_p) for n in ("params", "extra", "kern", "ctx")]


def launches(graph):
    """[(name, blocks, blocks an SM holds)] of a captured graph's kernels."""
    cu = ctypes.CDLL("libcuda.so.1")

    def call(name, *args):
        rc = getattr(cu, name)(*args)
        assert rc == 0, (name, rc)
    g, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    call("cuGraphGetNodes", g, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    call("cuGraphGetNodes", g, nodes, ctypes.byref(n))
    found = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        call("cuGraphNodeGetType", ctypes.c_void_p(node), ctypes.byref(kind))
        if kind.value != 0:
            continue
        p, name, held = KernelNode(), ctypes.c_char_p(), ctypes.c_int(0)
        call("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node), ctypes.byref(p))
        func = ctypes.c_void_p(p.func)
        if not func:
            call("cuKernelGetFunction", ctypes.byref(func), ctypes.c_void_p(p.kern))
        call("cuFuncGetName", ctypes.byref(name), func)
        call("cuOccupancyMaxActiveBlocksPerMultiprocessor", ctypes.byref(held), func, ctypes.c_int(p.bx * p.by * p.bz),
             ctypes.c_size_t(p.smem))
        found.append((name.value.decode(), p.gx * p.gy * p.gz, held.value))
    return found


@pytest.mark.parametrize("N,E,K,H,I", [(1, 128, 8, 2048, 768), (8, 128, 8, 2048, 768), (61, 64, 6, 1024, 128), (64, 384, 8, 512, 64),
                                       (32, 512, 10, 512, 64), (8, 512, 8, 2048, 64), (8, 1024, 32, 1024, 32), (5, 600, 24, 5128, 16),
                                       (64, 1024, 32, 128, 16)])
def test_grids(m, N, E, K, H, I):  # noqa: E741
    a = inputs(N, E, H, I)
    m.layer(K=K, **a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        m.layer(K=K, **a)
    streaming = [x for x in launches(graph) if "layer_rows" in x[0] or "layer_down" in x[0]]
    assert len(streaming) == 2
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for name, blocks, held in streaming:
        assert held in (1, 2) and blocks <= held * sms, (name, blocks, held)


@pytest.mark.parametrize("N,E,K,H,I,bits", [(64, 384, 8, 512, 72, 16), (32, 512, 10, 256, 200, 8), (8, 512, 8, 2056, 72, 16),
                                            (6, 1024, 32, 5136, 40, 8), (1, 1024, 32, 264, 1032, 16)])
def test_many_experts(m, N, E, K, H, I, bits):  # noqa: E741
    check(m, inputs(N, E, H, I, bits=bits), K)
