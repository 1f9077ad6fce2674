"""Calls from two host threads at once, each on its own stream with its own buffers: a kernel's shared-memory limit belongs
to the function, so a call that lowers it to its own size would make the other thread's launch fail."""
import ctypes
import threading

import pytest
import torch

from test_gpu_layernorm import activations, placed, randn

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ROUNDS = 500


def forward(lib, rows, k, dtype, pad):
    x, _ = placed(activations(k, rows, k), dtype, pad)
    y, _ = placed(torch.zeros(rows, k), dtype, pad)
    out = torch.empty(2 * rows + 1, device="cuda")

    def call(stream):
        lib.nvfp4_layernorm(x, lib._dtype_of(x), rows, k, k + pad, None, None, 0, 1e-5, y, lib._dtype_of(y), k + pad, out[:rows],
                            out[rows:2 * rows], out[2 * rows:], stream)

    return call, (y, out)


def backward(lib, rows, k, dtype, pad, sums=True):
    x, _ = placed(activations(k, rows, k), dtype, pad)
    dy, _ = placed(randn(rows, rows, k), dtype, pad)
    dx, _ = placed(torch.zeros(rows, k), dtype, pad)
    n = lib.layernorm(x)
    mean, rstd = n.mean, n.rstd
    out = torch.zeros(2 * k + 1, device="cuda")
    ws = torch.empty(lib.nvfp4_workspace_bytes(lib.OP_LAYERNORM_BACKWARD, rows, k, 0), dtype=torch.uint8, device="cuda")
    dg, db = (out[:k], out[k:2 * k]) if sums else (None, None)

    def call(stream):
        t = lib._dtype_of(x)
        lib.nvfp4_layernorm_backward(dy, t, k + pad, x, t, k + pad, mean, rstd, None, 0, None, 0, rows, k, dx, k + pad, dg, db,
                                     out[2 * k:], ws, ws.numel(), stream)

    return call, (dx, out if sums else out[2 * k:])


# each pair takes the same kernel with much and with little shared memory
PAIRS = {
    "forward, bf16 rows that start anywhere": [lambda lib: forward(lib, 4, 8001, BF16, 0), lambda lib: forward(lib, 4, 301, BF16, 0)],
    "backward, ring": [lambda lib: backward(lib, 4, 8192, BF16, 0), lambda lib: backward(lib, 1, 72, BF16, 0)],
    "backward, ring over a cluster": [lambda lib: backward(lib, 4, 16384, F32, 0), lambda lib: backward(lib, 4, 13600, F32, 0)],
    "backward, rows straight from memory": [lambda lib: backward(lib, 4, 8001, F32, 0),
                                            lambda lib: backward(lib, 4, 8001, F32, 0, sums=False)],
}


class KernelNode(ctypes.Structure):
    """CUDA_KERNEL_NODE_PARAMS_v2 of the driver's API."""
    _fields_ = ([("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "shared")] +
                [(n, ctypes.c_void_p) for n in ("params", "extra", "kern", "ctx")])


def kernels_of(graph):
    """[(function, dynamic shared memory)] of a captured graph's kernel nodes."""
    cuda, raw = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(graph.raw_cuda_graph())
    count = ctypes.c_size_t()
    assert cuda.cuGraphGetNodes(raw, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert cuda.cuGraphGetNodes(raw, nodes, ctypes.byref(count)) == 0
    found = []
    for node in nodes:
        kind, params = ctypes.c_int(), KernelNode()
        assert cuda.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value != 0:                                  # CU_GRAPH_NODE_TYPE_KERNEL
            continue
        assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(params)) == 0
        func = ctypes.c_void_p(params.func)
        if not func:
            assert cuda.cuKernelGetFunction(ctypes.byref(func), ctypes.c_void_p(params.kern)) == 0
        found.append((func.value, params.shared))
    return found


def limit_of(func):
    value = ctypes.c_int()                                   # CU_FUNC_ATTRIBUTE_MAX_DYNAMIC_SHARED_SIZE_BYTES
    assert ctypes.CDLL("libcuda.so.1").cuFuncGetAttribute(ctypes.byref(value), 8, ctypes.c_void_p(func)) == 0
    return value.value


@pytest.mark.parametrize("pair", list(PAIRS))
def test_a_smaller_call_leaves_the_limit(lib, pair):
    """The larger call's launch stays possible whatever another thread calls between its preparation and its launch."""
    (large, _), (small, _) = [make(lib) for make in PAIRS[pair]]
    torch.cuda.synchronize()
    used = []
    for call in (large, small):
        graph = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(graph):
            call(None)
        used.append((graph, max(kernels_of(graph), key=lambda f: f[1])))
    (func, most), (_, (_, least)) = used[0][1], used[1]
    assert most > 48 * 1024 and most > least and func in [f for f, _ in kernels_of(used[1][0])], "the same kernel"
    assert limit_of(func) >= most


@pytest.mark.parametrize("pair", list(PAIRS))
def test_two_host_threads(lib, pair):
    made = [make(lib) for make in PAIRS[pair]]
    want = []
    for call, outputs in made:
        call(None)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outputs])
        for t in outputs:
            t.fill_(3.0)
    torch.cuda.synchronize()
    start, errors = threading.Barrier(2), []

    def work(call, stream):
        start.wait()
        try:
            for _ in range(ROUNDS):
                call(stream)
        except Exception as e:                               # noqa: BLE001 (reported by the test's thread)
            errors.append(e)

    streams = [torch.cuda.Stream() for _ in made]
    threads = [threading.Thread(target=work, args=(call, s.cuda_stream)) for (call, _), s in zip(made, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for (_, outputs), w in zip(made, want):
        for a, b in zip(outputs, w):
            assert torch.equal(a, b)
