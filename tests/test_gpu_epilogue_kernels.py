"""The GEMM epilogue where the tiles are more than the SMs, so that the larger tiles' kernels run: the CTA-pair kernel and,
for M <= 128, the one of 128 x 256 tiles, each with its outputs by TMA boxes or by rows, bf16 and fp32, several tiles per
block, ragged in M and N."""
import pytest
import torch

import operator_refs as R
from test_gpu_epilogue import product, run_gemm
from test_gpu_layernorm import BF16, F32, placed, randn, untouched

pytestmark = pytest.mark.gpu
# 128 x 128 tiles: 630, 195, 150, 152 (148 SMs)
SHAPES = [(2304, 4361, 64), (513, 4872, 192), (128, 19200, 128), (65, 19337, 320)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("out,bd,act,res,pre,pad,off", [
    (BF16, BF16, "gelu_tanh", True, True, 0, 0), (F32, F32, "silu", True, True, 0, 0), (F32, BF16, "relu", False, False, 4, 0),
    (BF16, None, "none", True, False, 3, 1), (F32, None, "gelu", True, True, 1, 1)],
    ids=["bf16_all", "f32_all", "f32_pitch", "bf16_odd", "f32_odd"])
def test_outputs(lib, shape, out, bd, act, res, pre, pad, off):
    m, n, k = shape
    a, w, _, (d_ref, s_ref, alpha) = product(lib, *shape)
    bias = randn(n, n).to(bd).cuda() if bd is not None else None
    r = placed(randn(m, m, n), out, pad, off)[0] if res else None
    d, d_flat = placed(torch.full((m, n), 7.0), out, pad, off)
    p, p_flat = placed(torch.full((m, n), 7.0), out, pad, off) if pre else (None, None)
    amax = torch.full((1,), float("nan"), device="cuda")
    run_gemm(lib, a, w, bias, act, r, d, p, amax)
    assert lib.nvfp4_check_device_status() == lib.OK
    ref = R.epilogue(d_ref, s_ref, alpha, bias, act, r)
    R.check(d, *ref["d"], "d")
    untouched(d_flat, d)
    assert float(amax) == float(d.float().abs().max())
    if pre:
        R.check(p, *ref["pre"], "pre")
        untouched(p_flat, p)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("out", [BF16, F32], ids=["bf16", "f32"])
def test_residual_in_place_and_repeats(lib, shape, out):
    m, n, k = shape
    a, w, _, (d_ref, s_ref, alpha) = product(lib, *shape)
    bias, r = randn(1, n).cuda(), randn(2, m, n).to(out).cuda()
    ref = R.epilogue(d_ref, s_ref, alpha, bias, "silu", r)
    apart = lib.gemm_epilogue(a, w, bias, "silu", residual=r, out_dtype=out)
    lib.gemm_epilogue(a, w, bias, "silu", residual=r, out=r)
    R.check(r, *ref["d"], "d")
    assert torch.equal(r, apart)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_nothing_asked_for_is_the_gemm(lib, shape):
    a, w, _, _ = product(lib, *shape)
    for t in (BF16, F32):
        assert torch.equal(lib.gemm_epilogue(a, w, out_dtype=t), lib.gemm(a, w, t))
