"""The amax that a norm or an epilogue hands out, given to a quantizer in the very next launch (the raw calls, with nothing
between them): x's writer is then the kernel in front of the quantizer, which may not start reading x before that kernel is
through.  Without a given amax the quantizer overlaps its own amax pass's tail."""
import ctypes

import pytest
import torch

import operator_refs as R
from test_gpu_host_threads import kernels_of
from test_gpu_layernorm import activations, randn

pytestmark = pytest.mark.gpu
M, K, N = 300, 2048, 1024


def quantizers(lib, x, amax, given, q):
    """{name: raw call of a quantizer of x into q}."""
    rows, k = x.shape
    a = (x, rows, k, k)
    out = (q.codes, q.sf, lib.SF_TCGEN05, q.g, amax, given)
    return {
        "quantize": lambda: lib.nvfp4_quantize(*a, *out),
        "stochastic": lambda: lib.nvfp4_quantize_stochastic(*a, *out, 3, 4),
        "hadamard": lambda: lib.nvfp4_quantize_hadamard(*a, 64, *out),
        "hadamard_stochastic": lambda: lib.nvfp4_quantize_hadamard_stochastic(*a, 128, *out, 3, 4),
    }


QUANTIZERS = ["quantize", "stochastic", "hadamard", "hadamard_stochastic"]


def writers(lib, y, amax):
    """{name: raw call that writes y [M, N] bf16 and its amax, nothing launched behind the kernel that writes y}."""
    x = activations(1, M, N).bfloat16().cuda()
    a, b = lib.quantize(activations(2, M, K).bfloat16().cuda()), lib.quantize(randn(3, N, K, scale=K ** -0.5).bfloat16().cuda())
    dd, pre = randn(4, M, N).bfloat16().cuda(), randn(5, M, N).bfloat16().cuda()
    torch.cuda.synchronize()
    return {
        "layernorm": lambda: lib.nvfp4_layernorm(x, 0, M, N, N, None, None, 0, 1e-5, y, 0, N, None, None, amax),
        "gemm_epilogue": lambda: lib.nvfp4_gemm_epilogue(a.codes, a.sf, a.g, b.codes, b.sf, b.g, M, N, K, None, 0, lib.ACT_GELU,
                                                         None, 0, y, N, lib.OUT_BF16, None, 0, amax),
        "epilogue_backward": lambda: lib.nvfp4_epilogue_backward(dd, N, pre, N, 0, lib.ACT_SILU, M, N, y, N, None, amax, None, 0),
    }


WRITERS = ["layernorm", "gemm_epilogue", "epilogue_backward"]


class EdgeData(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte), ("reserved", ctypes.c_ubyte * 5)]


def programmatic_edges(graph):
    """Edges of a captured graph that let a kernel start before the one in front of it is through."""
    cuda, raw = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(graph.raw_cuda_graph())
    count = ctypes.c_size_t()
    assert cuda.cuGraphGetEdges_v2(raw, None, None, None, ctypes.byref(count)) == 0
    at, to, data = (ctypes.c_void_p * count.value)(), (ctypes.c_void_p * count.value)(), (EdgeData * count.value)()
    assert cuda.cuGraphGetEdges_v2(raw, at, to, data, ctypes.byref(count)) == 0
    return sum(d.type == 1 for d in data)                    # CU_GRAPH_DEPENDENCY_TYPE_PROGRAMMATIC


@pytest.mark.parametrize("writer", WRITERS)
@pytest.mark.parametrize("quantizer", QUANTIZERS)
def test_quantizer_waits_for_the_writer(lib, writer, quantizer):
    y, amax = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")
    q = lib.empty_quantized(M, N)
    write = writers(lib, y, amax)[writer]
    for given, overlapping in ((1, 0), (0, 1)):
        graph = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(graph):
            write()
            quantizers(lib, y, amax, given, q)[quantizer]()
        assert len(kernels_of(graph)) == 3 - given
        assert programmatic_edges(graph) == overlapping


@pytest.mark.parametrize("writer", WRITERS)
@pytest.mark.parametrize("quantizer", ["quantize", "stochastic"])
@pytest.mark.parametrize("graphed", [False, True], ids=["calls", "graph"])
def test_hand_over(lib, writer, quantizer, graphed):
    """Equal to a quantizer that finds the amax itself, once all is written; y holds other rows before every run."""
    y, amax, own = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    q, want = lib.empty_quantized(M, N), lib.empty_quantized(M, N)
    write, quantize = writers(lib, y, amax)[writer], quantizers(lib, y, amax, 1, q)[quantizer]
    write()                                                  # (first calls load their kernels)
    quantize()
    graph = torch.cuda.CUDAGraph()
    if graphed:
        with torch.cuda.graph(graph):
            write()
            quantize()
    for _ in range(20):
        y.fill_(100.0)
        q.codes.fill_(0xFF)
        torch.cuda.synchronize()
        if graphed:
            graph.replay()
        else:
            write()
            quantize()
        torch.cuda.synchronize()
        quantizers(lib, y, own, 0, want)[quantizer]()
        assert float(own) == float(amax) == float(y.float().abs().max())
        assert torch.equal(q.codes, want.codes) and torch.equal(q.sf, want.sf) and torch.equal(q.g, want.g)
    assert lib.nvfp4_check_device_status() == lib.OK
