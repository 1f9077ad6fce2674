"""The operators as a transformer block's MLP uses them: norm, quantize, up projection with bias and GELU, quantize, down
projection onto the residual stream; the same for single tokens through the GEMV; and the backward pass of the norm and the
up projection's epilogue.  Each call's inputs are the outputs of the one before, taken as they are by the reference."""
import pytest
import torch

import operator_refs as R
from oracle import nvfp4_oracle as O
from nvfp4_block_scaled_15_b200 import inputs
from parity import dev_bf16, host_bf16_bits
from test_gpu_layernorm import activations, randn

pytestmark = pytest.mark.gpu


def weights(lib, n, k, seed):
    bits = inputs.gaussian_bf16((n, k), seed=seed, std=1.0 / k ** 0.5)
    return lib.quantize(dev_bf16(bits)), O.quantize(bits)[:3]


def product_ref(a, w):
    return O.gemm_ref(*O.quantize(host_bf16_bits(a))[:3], *w)


@pytest.mark.parametrize("m,hidden,inner", [(300, 256, 1024), (40, 320, 640)], ids=str)
def test_block_forward_and_backward(lib, m, hidden, inner):
    x = activations(m, m, hidden).bfloat16().cuda()
    g, b = (1 + 0.1 * randn(1, hidden)).bfloat16().cuda(), (0.1 * randn(2, hidden)).bfloat16().cuda()
    w1, w1_ref = weights(lib, inner, hidden, 11)
    w2, w2_ref = weights(lib, hidden, inner, 12)
    b1, b2 = randn(3, inner).cuda(), randn(4, hidden).cuda()
    n = lib.layernorm(x, g, b)
    yq = lib.quantize(n.y, amax=n.amax)
    amax_h = torch.zeros(1, device="cuda")
    h, pre = lib.gemm_epilogue(yq, w1, b1, "gelu_tanh", pre=True, amax=amax_h)
    out = lib.gemm_epilogue(lib.quantize(h, amax=amax_h), w2, b2, residual=x)
    assert lib.nvfp4_check_device_status() == lib.OK
    R.check(n.y, *R.layernorm(x, g, b, 1e-5)["y"], "norm")
    ref = R.epilogue(*product_ref(n.y, w1_ref), b1, "gelu_tanh", None)
    R.check(h, *ref["d"], "up")
    R.check(pre, *ref["pre"], "before the activation")
    R.check(out, *R.epilogue(*product_ref(h, w2_ref), b2, "none", x)["d"], "down")

    # backward from a gradient of h and of the stream
    dh, dstream = randn(5, m, inner, scale=0.05).bfloat16().cuda(), randn(6, m, hidden, scale=0.05).bfloat16().cuda()
    dpre, db1, amax_dpre = lib.epilogue_backward(dh, pre, "gelu_tanh")
    ref = R.epilogue_backward(dh, pre, "gelu_tanh")
    R.check(dpre, *ref["dpre"], "dpre")
    R.check(db1, *ref["dbias"], "db1")
    wt, wt_ref = weights(lib, hidden, inner, 13)                     # stands for W1^T, quantized along its own K
    dy = lib.gemm(lib.quantize(dpre, amax=amax_dpre), wt)
    dx, dg, db, amax_dx = lib.layernorm_backward(dy, x, n.mean, n.rstd, g, dstream)
    ref = R.layernorm_backward(dy, x, n.mean, n.rstd, g, dstream)
    R.check(dx, *ref["dx"], "dx")
    R.check(dg, *ref["dgamma"], "dgamma")
    R.check(db, *ref["dbeta"], "dbeta")
    assert float(amax_dx) == float(dx.float().abs().max())


@pytest.mark.parametrize("m", [1, 12])
def test_block_decode_in_a_graph(lib, m):
    """Single tokens: norm, GEMV with bias and SiLU, GEMV back onto the stream in place, captured once and replayed."""
    hidden, inner = 512, 1536
    w1, w1_ref = weights(lib, inner, hidden, 21)
    w2, w2_ref = weights(lib, hidden, inner, 22)
    b1, b2 = randn(3, inner).bfloat16().cuda(), randn(4, hidden).bfloat16().cuda()
    g, b = (1 + 0.1 * randn(1, hidden)).cuda(), (0.1 * randn(2, hidden)).cuda()
    x = torch.zeros(m, hidden, dtype=torch.bfloat16, device="cuda")
    y, h = torch.empty_like(x), torch.empty(m, inner, dtype=torch.bfloat16, device="cuda")
    ws1 = torch.empty(lib.nvfp4_workspace_bytes(lib.OP_GEMV_BATCHED, m, inner, hidden), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(lib.nvfp4_workspace_bytes(lib.OP_GEMV_BATCHED, m, hidden, inner), dtype=torch.uint8, device="cuda")

    def step():
        lib.layernorm(x, g, b, out=y)
        lib.gemv_batched_epilogue(y, w1, b1, "silu", out=h, workspace=ws1)
        lib.gemv_batched_epilogue(h, w2, b2, residual=x, out=x, workspace=ws2)

    x.copy_(activations(1, m, hidden))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (31, 32):
        x.copy_(activations(seed, m, hidden))
        before = x.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert lib.nvfp4_check_device_status() == lib.OK
        R.check(y, *R.layernorm(before, g, b, 1e-5)["y"], "norm")
        R.check(h, *R.epilogue(*product_ref(y, w1_ref), b1, "silu", None)["d"], "up")
        R.check(x, *R.epilogue(*product_ref(h, w2_ref), b2, "none", before)["d"], "down")
