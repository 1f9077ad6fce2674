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


def calls(lib, seed):
    """One call of each operator on tensors of its own, as (function, outputs); every output is the call's alone."""
    m, n, k = 300, 1000, 1024
    w, _ = weights(lib, n, k, 40)
    x = activations(seed, m, k).bfloat16().cuda()
    g, b, bias = params_of(k, 7) + (randn(8, n).bfloat16().cuda(),)
    a = lib.quantize(x)
    f32 = dict(device="cuda", dtype=torch.float32)
    y, mean, rstd, top = torch.empty_like(x), torch.empty(m, **f32), torch.empty(m, **f32), torch.empty(1, **f32)
    d, pre, res = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    res.copy_(randn(seed + 1, m, n))
    top_d, top_p, dbias, dpre = torch.empty(1, **f32), torch.empty(1, **f32), torch.empty(n, **f32), torch.empty_like(d)
    dx, dg, db, top_x = torch.empty_like(x), torch.empty(k, **f32), torch.empty(k, **f32), torch.empty(1, **f32)
    few = torch.empty(9, n, dtype=torch.bfloat16, device="cuda")
    ws = [torch.empty(lib.nvfp4_workspace_bytes(op, *dims), dtype=torch.uint8, device="cuda")
          for op, dims in ((lib.OP_LAYERNORM_BACKWARD, (m, k, 0)), (lib.OP_EPILOGUE_BACKWARD, (m, n, 0)),
                           (lib.OP_GEMV_BATCHED, (9, n, k)))]

    def run(s):
        lib.nvfp4_layernorm(x, 0, m, k, k, g, b, lib._dtype_of(g), 1e-5, y, 0, k, mean, rstd, top, s)
        lib.nvfp4_gemm_epilogue(a.codes, a.sf, a.g, w.codes, w.sf, w.g, m, n, k, bias, 0, lib.ACTIVATIONS["gelu"], res, n, d, n, 0,
                                pre, n, top_d, s)
        lib.nvfp4_gemv_batched_epilogue(x, 9, k, w.codes, w.sf, w.g, n, k, bias, 0, lib.ACTIVATIONS["silu"], res, n, few, n,
                                        ws[2], ws[2].numel(), s)
        lib.nvfp4_epilogue_backward(res, n, pre, n, 0, lib.ACTIVATIONS["gelu"], m, n, dpre, n, dbias, top_p, ws[1], ws[1].numel(), s)
        lib.nvfp4_layernorm_backward(y, 0, k, x, 0, k, mean, rstd, g, lib._dtype_of(g), x, k, m, k, dx, k, dg, db, top_x,
                                     ws[0], ws[0].numel(), s)

    return run, x, (y, mean, rstd, top, d, pre, top_d, few, dpre, dbias, top_p, dx, dg, db, top_x), (a, w, g, b, bias, res, ws)


def params_of(k, seed):
    return (1 + 0.1 * randn(seed, k)).cuda(), (0.1 * randn(seed + 1, k)).cuda()


def test_two_streams_at_once(lib):
    """Each operator from two streams at the same time, workspaces apart: the bits of a call on its own."""
    sets = [calls(lib, 60), calls(lib, 70)]
    alone = []
    for run, _, outs, _ in sets:
        run(None)
        torch.cuda.synchronize()
        alone.append([o.clone() for o in outs])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _, _, outs, _ in sets:
        for o in outs: o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        for (run, *_), s in zip(sets, streams): run(s)
    torch.cuda.synchronize()
    assert lib.nvfp4_check_device_status() == lib.OK
    for (_, _, outs, _), want in zip(sets, alone):
        for i, (o, v) in enumerate(zip(outs, want)): assert torch.equal(o, v), i


def test_every_operator_captured(lib):
    """One graph of all five, replayed on other inputs: each replay gives the bits of the calls on those inputs, amax and
    column sums included, which must not hold what an earlier replay left."""
    run, x, outs, _ = calls(lib, 80)
    run(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(None)
    for scale in (30.0, 1.0):                                 # the larger maxima first
        x.copy_(activations(int(scale), *x.shape) * scale)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for o in outs: o.fill_(float("nan"))
        run(None)
        torch.cuda.synchronize()
        assert lib.nvfp4_check_device_status() == lib.OK
        for i, (o, v) in enumerate(zip(outs, got)): assert torch.equal(o, v), i
