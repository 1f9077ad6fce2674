"""The gradients' maximum where no column sums are asked for: no kernel behind joins the blocks' maxima then, so each kernel
clears and raises it itself.  A larger maximum comes first, so that one left from it would show."""
import pytest
import torch

import operator_refs as R
from test_gpu_layernorm import BF16, F32, backward_inputs, placed, randn, untouched

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,k,xd,pad,off", [
    (70, 64, BF16, 0, 0), (3000, 33, F32, 1, 0),             # short rows
    (50, 1155, F32, 0, 0), (50, 301, BF16, 0, 1),            # rows that start anywhere, straight from memory
    (50, 2048, BF16, 0, 0), (700, 72, F32, 0, 0),            # the ring
    (4003, 1155, BF16, 0, 0),                                # the ring, rows that start anywhere
    (40, 16384, BF16, 0, 0), (20, 9001, F32, 0, 0),          # rows cut between the blocks of a cluster
    (9, 70001, BF16, 0, 0), (9, 70008, F32, 0, 0)], ids=str)  # rows of any length
def test_layernorm_backward(lib, rows, k, xd, pad, off):
    amax = torch.full((1,), float("nan"), device="cuda")
    largest = []
    for scale in (8.0, 1.0):
        dy, *others = backward_inputs(rows, k, xd, xd, F32, True, pad, off)
        dy.mul_(scale)
        others[-1].mul_(scale)
        x, mean, rstd, g, res = others
        dx, flat = placed(torch.full((rows, k), 7.0), xd, pad, off)
        lib.nvfp4_layernorm_backward(dy, lib._dtype_of(dy), dy.stride(0), x, lib._dtype_of(x), x.stride(0), mean, rstd, g,
                                     lib.DTYPE_F32, res, res.stride(0), rows, k, dx, dx.stride(0), None, None, amax, None, 0)
        R.check(dx, *R.layernorm_backward(dy, x, mean, rstd, g, res)["dx"], "dx")
        untouched(flat, dx)
        largest.append(float(amax))
        assert largest[-1] == float(dx.float().abs().max())
    assert largest[0] > largest[1]


@pytest.mark.parametrize("n", [264, 1001])
@pytest.mark.parametrize("t", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("stored", [True, False], ids=["dpre", "amax_alone"])
def test_epilogue_backward(lib, n, t, stored):
    m = 700
    amax = torch.full((1,), float("nan"), device="cuda")
    largest = []
    for scale in (8.0, 1.0):
        dd, pre = (scale * randn(1, m, n)).to(t).cuda(), randn(2, m, n).to(t).cuda()
        dpre = torch.full_like(dd, float("nan"))
        lib.nvfp4_epilogue_backward(dd, n, pre, n, lib._dtype_of(dd), lib.ACT_SILU, m, n, dpre if stored else None,
                                    n if stored else 0, None, amax, None, 0)
        ref, tol = R.epilogue_backward(dd, pre, "silu")["dpre"]
        if stored:
            R.check(dpre, ref, tol, "dpre")
            assert float(amax) == float(dpre.float().abs().max())
        at = int(ref.abs().argmax())                         # the maximum lies within the largest element's tolerance
        R.check(amax.to(t), ref.abs().max().reshape(1), tol.reshape(-1)[at].reshape(1) + tol.max(), "amax")
        largest.append(float(amax))
    assert largest[0] > largest[1]
