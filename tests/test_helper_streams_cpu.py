"""The torch helpers' own work for a call on a given stream (outputs, workspaces, small copies) belongs to that stream: what
the allocator hands out on another one may still be in use there, and is handed out again there while the kernels run.  The
library's calls and torch's streams are stood in for, so no GPU is needed."""
import contextlib

import pytest
import torch

SIDE = 64                                                   # the handle of the stream that the calls are given


@pytest.fixture
def nv(monkeypatch):
    from nvfp4_block_scaled_15_b200 import build
    build.build()
    from nvfp4_block_scaled_15_b200 import nvfp4

    class Stream:
        def __init__(self, handle, *_):
            self.cuda_stream = handle

    current = [None]                                        # handle of torch's current stream
    log = []                                                # ("empty" | "copy_" | the library's call, handle it happens on)

    @contextlib.contextmanager
    def switch(s):
        before, current[0] = current[0], s.cuda_stream
        yield
        current[0] = before

    def logged(module, name):
        real = getattr(module, name)

        def call(*args, **kw):
            log.append((name, current[0]))
            return real(*args, **kw)
        monkeypatch.setattr(module, name, call)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", switch)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: Stream(current[0]))
    for module, name in ((torch, "empty"), (torch.Tensor, "copy_")):
        logged(module, name)
    for name in nvfp4._SIGS:
        if not name.endswith(("_bytes", "_string")):
            monkeypatch.setattr(nvfp4, name, lambda *args, _n=name, **kw: log.append((_n, args[-1])))
    monkeypatch.setattr(nvfp4, "_test_log", log, raising=False)
    return nvfp4


def calls(nv, stream):
    """One call per helper that allocates or copies, on `stream`."""
    m, n, k = 9, 128, 64
    x, wide = torch.zeros(m, k, dtype=torch.bfloat16), torch.zeros(m, n, dtype=torch.bfloat16)
    one, stat = torch.ones(1), torch.zeros(m)
    a, w = nv.empty_quantized(m, k, device="cpu"), nv.empty_quantized(n, k, device="cpu")
    codes = lambda rows: nv.MXQuantized(torch.zeros(rows, k, dtype=torch.uint8), torch.zeros(4096, dtype=torch.uint8), rows, 2 * k,
                                        nv.SF_TCGEN05)
    return {
        "quantize": lambda: nv.quantize(x, amax=one, stream=stream),
        "quantize_stochastic": lambda: nv.quantize_stochastic(x, 1, 2, amax=one, stream=stream),
        "quantize_hadamard": lambda: nv.quantize_hadamard(x, 16, amax=one, stream=stream),
        "quantize_hadamard_stochastic": lambda: nv.quantize_hadamard_stochastic(x, 16, 1, 2, amax=one, stream=stream),
        "gemm": lambda: nv.gemm(a, w, stream=stream),
        "gemm_by_position": lambda: nv.gemm(a, w, torch.bfloat16, None, stream),
        "gemm_requant": lambda: nv.gemm_requant(a, w, one, stream=stream),
        "gemm_fp8_out": lambda: nv.gemm_fp8_out(a, w, one, stream=stream),
        "gemv_batched": lambda: nv.gemv_batched(x, w, stream=stream),
        "gemm_quant_a": lambda: nv.gemm_quant_a(x, w, stream=stream),
        "mxfp4_quantize": lambda: nv.mxfp4_quantize(torch.zeros(m, 128, dtype=torch.bfloat16), stream=stream),
        "mxfp4_gemm": lambda: nv.mxfp4_gemm(codes(m), codes(n), stream=stream),
        "layernorm": lambda: nv.layernorm(x, stream=stream),
        "layernorm_backward": lambda: nv.layernorm_backward(x, x, stat, stat, stream=stream),
        "gemm_epilogue": lambda: nv.gemm_epilogue(a, w, pre=True, stream=stream),
        "gemv_batched_epilogue": lambda: nv.gemv_batched_epilogue(x, w, stream=stream),
        "epilogue_backward": lambda: nv.epilogue_backward(wide, None, stream=stream),
    }


HELPERS = ["quantize", "quantize_stochastic", "quantize_hadamard", "quantize_hadamard_stochastic", "gemm", "gemm_by_position",
           "gemm_requant", "gemm_fp8_out", "gemv_batched", "gemm_quant_a", "mxfp4_quantize", "mxfp4_gemm", "layernorm",
           "layernorm_backward", "gemm_epilogue", "gemv_batched_epilogue", "epilogue_backward"]


@pytest.mark.parametrize("helper", HELPERS)
@pytest.mark.parametrize("given", ["stream", "handle"])
def test_work_of_a_call_is_on_its_stream(nv, helper, given):
    call = calls(nv, SIDE if given == "handle" else torch.cuda.Stream(SIDE))[helper]
    nv._test_log.clear()
    call()
    own = [(what, where) for what, where in nv._test_log if not what.startswith("nvfp4_")]
    assert own and all(where == SIDE for _, where in own), nv._test_log
    assert any(what.startswith("nvfp4_") for what, _ in nv._test_log)


@pytest.mark.parametrize("helper", HELPERS)
def test_no_stream_is_the_current_one(nv, helper):
    call = calls(nv, None)[helper]
    nv._test_log.clear()
    call()
    own = [(what, where) for what, where in nv._test_log if not what.startswith("nvfp4_")]
    assert own and all(where is None for _, where in own), nv._test_log
