"""The grid of a call depends on the call alone, not on what was called before."""
import ctypes

import pytest
import torch

import bit_quantized_all_gb300 as qr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_quantized_all_gb300 import build
    build.build()
    qr.lib()


class _KernelNode(ctypes.Structure):
    """CUDA_KERNEL_NODE_PARAMS_v2."""
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _launch(call):
    """(CTAs, threads of one) of a call that is a single launch, from a captured graph."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cu = ctypes.CDLL("libcuda.so.1")
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0 and n.value == 1
    node, params = ctypes.c_void_p(), _KernelNode()
    assert cu.cuGraphGetNodes(raw, ctypes.byref(node), ctypes.byref(n)) == 0
    assert cu.cuGraphKernelNodeGetParams_v2(node, ctypes.byref(params)) == 0
    return params.grid[0] * params.grid[1] * params.grid[2], params.block[0]


@pytest.mark.parametrize("eight", [False, True])
def test_a_row_per_cta(eight):
    """One kernel serves rows of 2048 to 16384 values with 64 to 512 threads: its waves differ."""
    call = qr.qr_rms_norm_q8 if eight else qr.qr_rms_norm
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    widths = (16384, 8192, 2048)
    x = [torch.zeros((20 * sms, cols), dtype=torch.bfloat16, device="cuda") for cols in widths]
    w = [torch.ones(cols, dtype=torch.bfloat16, device="cuda") for cols in widths]

    def shape(i):
        return _launch(lambda: call(x[i], w[i]))

    seen = [shape(i) for i in range(3)]
    assert [t for _, t in seen] == [512, 256, 64]
    assert all(grid % sms == 0 for grid, _ in seen)
    assert seen[0][0] < seen[1][0] < seen[2][0]
    assert [shape(i) for i in reversed(range(3))] == seen[::-1]
