"""Helpers on a stream that is not the current one, with their outputs and workspaces left to them, while the current
stream allocates and writes at once what the helpers may have dropped."""
import pytest
import torch

import operator_refs as R
from test_gpu_block import params_of, weights
from test_gpu_layernorm import activations, randn

pytestmark = pytest.mark.gpu
M, N, K = 24, 1000, 1024


@pytest.fixture(scope="module")
def operands(lib):
    x = activations(3, M, K).bfloat16().cuda()
    g, b = params_of(K, 7)
    n = lib.layernorm(x, g, b)
    w, _ = weights(lib, N, K, 40)
    dd, pre = randn(1, M, N).bfloat16().cuda(), randn(2, M, N).bfloat16().cuda()
    torch.cuda.synchronize()
    return dict(x=x, g=g, b=b, n=n, w=w, a=lib.quantize(x), dd=dd, pre=pre, bias=randn(8, N).cuda())


def calls(lib, o, **kw):
    n = o["n"]
    few = o["x"][:9]
    return {
        "layernorm": lambda: vars(lib.layernorm(o["x"], o["g"], o["b"], **kw)).values(),
        "layernorm_backward": lambda: lib.layernorm_backward(o["x"], o["x"], n.mean, n.rstd, o["g"], **kw),
        "gemm_epilogue": lambda: lib.gemm_epilogue(o["a"], o["w"], o["bias"], "gelu", pre=True, **kw),
        "gemv_batched_epilogue": lambda: [lib.gemv_batched_epilogue(few, o["w"], o["bias"], "silu", **kw)],
        "gemv_batched": lambda: [lib.gemv_batched(few, o["w"], **kw)],
        "epilogue_backward": lambda: lib.epilogue_backward(o["dd"], o["pre"], "silu", **kw),
        "gemm_quant_a": lambda: [lib.gemm_quant_a(o["x"], o["w"], **kw)],
        "quantize": lambda: (lambda q: [q.codes, q.sf, q.g, q.amax])(lib.quantize(n.y, amax=n.amax, **kw)),
    }


HELPERS = ["layernorm", "layernorm_backward", "gemm_epilogue", "gemv_batched_epilogue", "gemv_batched", "epilogue_backward",
           "gemm_quant_a", "quantize"]


@pytest.mark.parametrize("helper", HELPERS)
@pytest.mark.parametrize("given", ["stream", "handle"])
def test_call_on_another_stream(lib, operands, helper, given, monkeypatch):
    want = [t.clone() for t in calls(lib, operands)[helper]()]
    side = torch.cuda.Stream()
    handed_out = []                                          # what the helper allocates: (address, bytes)
    empty = torch.empty
    torch.cuda.synchronize()
    with monkeypatch.context() as mp:
        def recorded(*args, **kw):
            t = empty(*args, **kw)
            handed_out.append((t.data_ptr(), t.numel() * t.element_size()))
            return t
        mp.setattr(torch, "empty", recorded)
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                    # the call's kernels run well after what follows is enqueued
        got = list(calls(lib, operands, stream=side if given == "stream" else side.cuda_stream)[helper]())
    assert handed_out
    behind = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _, size in handed_out for _ in range(2)]
    for t in behind:
        for at, size in handed_out:
            assert t.data_ptr() + t.numel() <= at or at + size <= t.data_ptr(), "memory of the call handed out on another stream"
    side.synchronize()
    assert lib.nvfp4_check_device_status() == lib.OK
    for i, (a, v) in enumerate(zip(got, want)):
        assert torch.equal(a, v), i


def test_default_stream_by_its_handle(lib, operands):
    """0 is the legacy default stream, which is torch's default one."""
    o = operands
    y = lib.layernorm(o["x"], o["g"], o["b"], stream=0)
    assert torch.equal(y.y, o["n"].y) and torch.cuda.current_stream() == torch.cuda.default_stream()


@pytest.mark.parametrize("given", ["stream", "handle"])
def test_captured_with_the_stream_named(lib, operands, given):
    """Helpers given the very stream that a graph is captured on: what they allocate is the graph's, replays take new
    contents."""
    o = operands
    x = o["x"].clone()
    side = torch.cuda.Stream()

    def step(**kw):
        n = lib.layernorm(x, o["g"], o["b"], **kw)
        q = lib.quantize(n.y, amax=n.amax, **kw)
        d, pre = lib.gemm_epilogue(q, o["w"], o["bias"], "gelu", pre=True, **kw)
        few = lib.gemv_batched_epilogue(x[:9], o["w"], o["bias"], "silu", **kw)
        back = lib.epilogue_backward(o["dd"], pre, "gelu", **kw)
        return [d, pre, few, *back, *lib.layernorm_backward(o["x"], x, n.mean, n.rstd, o["g"], **kw)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step(stream=side if given == "stream" else side.cuda_stream)
    for seed in (5, 6):
        x.copy_(activations(seed, M, K))
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, v) in enumerate(zip(got, step())):
            assert torch.equal(a, v), i
    assert lib.nvfp4_check_device_status() == lib.OK
