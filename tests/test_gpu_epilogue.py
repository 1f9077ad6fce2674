"""The GEMM and the decode GEMV with bias, activation and residual, and the epilogue's gradient, against the oracle's
product and the 64-bit definition of the rest."""
import pytest
import torch

import operator_refs as R
from oracle import nvfp4_oracle as O
from nvfp4_block_scaled_15_b200 import inputs
from parity import dev_bf16
from test_gpu_layernorm import placed, randn, untouched

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
_products = {}


def product(lib, m, n, k):
    """(A on the device, W on the device, x in bf16, (D, S, alpha) of the oracle): made once per shape."""
    if (m, n, k) not in _products:
        x = inputs.gaussian_bf16((m, k), seed=m + 7 * n)
        w = inputs.gaussian_bf16((n, k), seed=n + 3 * k, std=0.7 / k ** 0.5)
        px, sx, gx, _ = O.quantize(x)
        pw, sw, gw, _ = O.quantize(w)
        xd = dev_bf16(x)
        _products[(m, n, k)] = (lib.quantize(xd), lib.quantize(dev_bf16(w)), xd, O.gemm_ref(px, sx, gx, pw, sw, gw))
    return _products[(m, n, k)]


def run_gemm(lib, a, w, bias, act, res, d, pre, amax):
    lib.nvfp4_gemm_epilogue(a.codes, a.sf, a.g, w.codes, w.sf, w.g, a.rows, w.rows, a.k, bias, lib._dtype_of(bias),
                            lib.ACTIVATIONS[act], res, 0 if res is None else res.stride(0), d, d.stride(0), lib._dtype_of(d),
                            pre, 0 if pre is None else pre.stride(0), amax)


# narrow, short and paired tiles; one element; one K step; whole and ragged tiles in both directions
GEMM_SHAPES = [(1, 1, 64), (128, 128, 256), (130, 100, 320), (5, 300, 192), (100, 1000, 448), (129, 257, 64), (256, 512, 512),
               (300, 520, 1088), (513, 264, 640)]


@pytest.mark.parametrize("m,n,k", GEMM_SHAPES, ids=str)
@pytest.mark.parametrize("out,bd,act,res,pre,pad,off", [
    (BF16, BF16, "gelu_tanh", True, True, 0, 0), (F32, F32, "silu", True, True, 0, 0), (BF16, F32, "gelu", False, True, 8, 0),
    (F32, BF16, "relu", False, False, 4, 0), (BF16, None, "none", True, False, 3, 1), (F32, None, "gelu", True, True, 1, 1)],
    ids=["bf16_all", "f32_all", "bf16_pre_pitch", "f32_pitch", "bf16_odd", "f32_odd"])
def test_gemm_epilogue(lib, m, n, k, out, bd, act, res, pre, pad, off):
    a, w, _, (d_ref, s_ref, alpha) = product(lib, m, n, k)
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


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(70, 90, 128), (60, 300, 128), (300, 300, 128)], ids=str)
def test_gemm_every_activation_with_far_values(lib, m, n, k, act):
    """A bias that takes the value before the activation to +-40."""
    a, w, _, (d_ref, s_ref, alpha) = product(lib, m, n, k)
    bias = torch.linspace(-40, 40, n).cuda()
    d = lib.gemm_epilogue(a, w, bias, act, out_dtype=F32)
    R.check(d, *R.epilogue(d_ref, s_ref, alpha, bias, act, None)["d"], "d")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("m,n,k", [(100, 90, 128), (60, 300, 128), (300, 520, 1088)], ids=str)
def test_gemm_residual_in_place(lib, m, n, k, out):
    a, w, _, (d_ref, s_ref, alpha) = product(lib, m, n, k)
    bias = randn(1, n).cuda()
    r = randn(2, m, n).to(out).cuda()
    ref = R.epilogue(d_ref, s_ref, alpha, bias, "silu", r)
    lib.gemm_epilogue(a, w, bias, "silu", residual=r, out=r)
    R.check(r, *ref["d"], "d")


def test_gemm_without_an_epilogue_is_the_gemm(lib):
    for m, n, k in [(130, 100, 320), (100, 1000, 448), (300, 520, 1088)]:
        a, w, _, _ = product(lib, m, n, k)
        for t in (BF16, F32):
            assert torch.equal(lib.gemm_epilogue(a, w, out_dtype=t), lib.gemm(a, w, t))


def test_gemm_many_tiles_per_block(lib):
    """More tiles than CTA pairs: the accumulators and the output staging take turns."""
    m, n, k = 2304, 4360, 128
    a, w, _, (d_ref, s_ref, alpha) = product(lib, m, n, k)
    bias, r = randn(1, n).bfloat16().cuda(), randn(2, m, n).bfloat16().cuda()
    d, pre = lib.gemm_epilogue(a, w, bias, "gelu_tanh", r, pre=True)
    assert lib.nvfp4_check_device_status() == lib.OK
    ref = R.epilogue(d_ref, s_ref, alpha, bias, "gelu_tanh", r)
    R.check(d, *ref["d"], "d")
    R.check(pre, *ref["pre"], "pre")


@pytest.mark.parametrize("n,k,res,pre", [(4352, 64, False, False), (4352, 1024, True, False), (4352, 64, True, False), (4352, 64, True, True),
                                         (4354, 64, True, False)], ids=str)
def test_gemm_epilogue_slower_than_the_product(lib, n, k, res, pre):
    """Short K and several tiles per CTA pair: the products run ahead of the epilogue warps, which then differ in how far
    they are (the warps of one half release the shared columns and go on, those of the other may be a tile behind)."""
    m = 2304
    a, w, _, (d_ref, s_ref, alpha) = product(lib, m, n, k)
    bias = randn(1, n).bfloat16().cuda()
    r = randn(2, m, n).bfloat16().cuda() if res else None
    p = torch.empty(m, n, dtype=BF16, device="cuda") if pre else None
    for _ in range(3):
        d = lib.gemm_epilogue(a, w, bias, "gelu", r, pre=p if pre else False)
    assert lib.nvfp4_check_device_status() == lib.OK
    ref = R.epilogue(d_ref, s_ref, alpha, bias, "gelu", r)
    R.check(d, *ref["d"], "d")
    if pre:
        R.check(p, *ref["pre"], "pre")


@pytest.mark.parametrize("n", [264, 296, 328, 376, 392, 424, 456, 488, 504, 904])
@pytest.mark.parametrize("res,pre", [(True, True), (True, False), (False, True)], ids=["res_pre", "res", "pre"])
def test_gemm_ends_inside_a_tile(lib, n, res, pre):
    """N ends in each of a tile's eight boxes of 32 columns (the boxes shared between the accumulators are taken first, so
    the first ones may lie past N and the later ones before it), with enough rows for tiles in both accumulators."""
    m, k = 18944 + 300, 64
    _, w, x, ref = product(lib, 300, n, k)
    bias = randn(1, n).bfloat16().cuda()
    # the rows of one small product over and over: enough tiles that every CTA pair takes several
    rows = torch.arange(m, device="cuda") % 300
    big = lib.quantize(x[rows])
    d_ref, s_ref, alpha = ref
    r = randn(2, m, n).bfloat16().cuda() if res else None
    p = torch.empty(m, n, dtype=BF16, device="cuda") if pre else None
    for _ in range(2):
        d = lib.gemm_epilogue(big, w, bias, "relu", r, pre=p if pre else False)
    assert lib.nvfp4_check_device_status() == lib.OK
    idx = rows.cpu().numpy()
    ref = R.epilogue(d_ref[idx], s_ref[idx], alpha, bias, "relu", r)
    R.check(d, *ref["d"], "d")
    if pre:
        R.check(p, *ref["pre"], "pre")


def test_gemm_nonfinite_bias_and_residual(lib):
    a, w, _, _ = product(lib, 300, 520, 1088)
    bias = torch.zeros(520, device="cuda")
    bias[100] = float("nan")
    r = torch.zeros(300, 520, dtype=BF16, device="cuda")
    r[7, 9] = float("inf")
    amax = torch.zeros(1, device="cuda")
    d = lib.gemm_epilogue(a, w, bias, "relu", r, amax=amax)
    assert bool(torch.isnan(d[:, 100]).all()) and float(d[7, 9]) == float("inf")
    mask = torch.ones_like(d, dtype=torch.bool)
    mask[:, 100] = False
    mask[7, 9] = False
    assert bool(torch.isfinite(d[mask]).all()) and not bool(torch.isfinite(amax))


# both GEMV kernels (M <= 8 and K <= 8192, or not), whole and split tiles, ragged N and K
@pytest.mark.parametrize("m", [1, 3, 8, 9, 16, 32])
@pytest.mark.parametrize("n,k", [(1, 64), (1000, 1024), (384, 4096), (640, 2880), (160 * 128, 1024), (100, 8192), (9000, 2112)], ids=str)
def test_gemv_epilogue(lib, m, n, k):
    _, w, x, (d_ref, s_ref, alpha) = product(lib, m, n, k)
    for bd, act, res, pad, off in [(BF16, "gelu_tanh", True, 0, 0), (F32, "gelu", False, 3, 1), (None, "none", True, 1, 0),
                                   (F32, "silu", True, 8, 0), (BF16, "relu", False, 0, 0)]:
        bias = randn(n, n).to(bd).cuda() if bd is not None else None
        r = placed(randn(m, m, n), BF16, pad, off)[0] if res else None
        y, flat = placed(torch.full((m, n), 7.0), BF16, pad, off)
        ws = torch.randint(0, 256, (lib.nvfp4_workspace_bytes(lib.OP_GEMV_BATCHED, m, n, k),), dtype=torch.uint8, device="cuda")
        lib.nvfp4_gemv_batched_epilogue(x, m, x.stride(0), w.codes, w.sf, w.g, n, k, bias, lib._dtype_of(bias),
                                        lib.ACTIVATIONS[act], r, 0 if r is None else r.stride(0), y, y.stride(0), ws, ws.numel())
        assert lib.nvfp4_check_device_status() == lib.OK
        R.check(y, *R.epilogue(d_ref, s_ref, alpha, bias, act, r)["d"], act)
        untouched(flat, y)


@pytest.mark.parametrize("m,k", [(2, 1024), (12, 1024), (2, 8256)], ids=str)
def test_gemv_residual_in_place_and_plain(lib, m, k):
    n = 1000
    _, w, x, (d_ref, s_ref, alpha) = product(lib, m, n, k)
    R.check(lib.gemv_batched_epilogue(x, w), *R.epilogue(d_ref, s_ref, alpha, None, "none", None)["d"], "plain")
    r = randn(2, m, n).bfloat16().cuda()
    ref = R.epilogue(d_ref, s_ref, alpha, None, "none", r)
    lib.gemv_batched_epilogue(x, w, residual=r, out=r)
    R.check(r, *ref["d"], "y")


# ---------------------------------------------------------------------------
# the epilogue's gradient
# ---------------------------------------------------------------------------
def run_backward(lib, dd, pre, act, dpre, want_bias=True, amax=True):
    m, n = dd.shape
    out = torch.full((n + 1,), float("nan"), device="cuda")
    nbytes = lib.nvfp4_workspace_bytes(lib.OP_EPILOGUE_BACKWARD, m, n, 0)
    ws = torch.full((nbytes + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    lib.nvfp4_epilogue_backward(dd, dd.stride(0), pre, 0 if pre is None else pre.stride(0), lib._dtype_of(dd),
                                lib.ACTIVATIONS[act], m, n, dpre, 0 if dpre is None else dpre.stride(0),
                                out[:n] if want_bias else None, out[n:] if amax else None, ws, nbytes)
    assert bool((ws[nbytes:] == 0xFF).all()), "written past the workspace"
    return out[:n], out[n:]


@pytest.mark.parametrize("m,n", [(1, 1), (3, 5), (1, 4096), (64, 256), (65, 264), (1000, 1001), (7, 2056), (5000, 72), (130, 8192)],
                         ids=str)
@pytest.mark.parametrize("t,act,pad,off", [(BF16, "gelu_tanh", 0, 0), (F32, "silu", 0, 0), (BF16, "gelu", 8, 0), (F32, "gelu", 1, 1),
                                           (BF16, "relu", 3, 1), (F32, "none", 0, 0)], ids=str)
def test_epilogue_backward(lib, m, n, t, act, pad, off):
    dd, _ = placed(randn(m, m, n, scale=0.05), t, pad, off)
    pre, _ = placed(randn(n, m, n, scale=2.0), t, pad, off)
    dpre, flat = placed(torch.full((m, n), 7.0), t, pad, off)
    dbias, amax = run_backward(lib, dd, None if act == "none" else pre, act, dpre)
    ref = R.epilogue_backward(dd, pre, act)
    R.check(dpre, *ref["dpre"], "dpre")
    R.check(dbias, *ref["dbias"], "dbias")
    assert float(amax) == float(dpre.float().abs().max())
    untouched(flat, dpre)


@pytest.mark.parametrize("act", ACTS)
def test_epilogue_backward_far_values_and_limits(lib, act):
    v = torch.cat([torch.linspace(-60, 60, 4001), torch.tensor([0.0, -0.0, 1e4, -1e4, 1e30, -1e30])])
    pre = v.repeat(4, 1).cuda()
    dd = torch.ones_like(pre)
    dpre = torch.empty_like(pre)
    run_backward(lib, dd, pre, act, dpre)
    R.check(dpre, *R.epilogue_backward(dd, pre.clamp(-1e5, 1e5), act)["dpre"], "slope")
    if act != "none":
        pre = torch.tensor([[float("inf"), float("-inf"), float("nan")]], device="cuda")
        run_backward(lib, torch.ones_like(pre), pre, act, dpre[:1, :3])
        assert dpre[0, :2].tolist() == [1.0, 0.0] and bool(torch.isnan(dpre[0, 2]))


@pytest.mark.parametrize("n", [264, 1001])
def test_epilogue_backward_in_place_parts_and_repeats(lib, n):
    m = 700
    dd, pre = randn(1, m, n).bfloat16().cuda(), randn(2, m, n).bfloat16().cuda()
    ref = R.epilogue_backward(dd, pre, "silu")
    dbias, amax = run_backward(lib, dd, pre, "silu", None)
    R.check(dbias, *ref["dbias"], "dbias alone")
    again, _ = run_backward(lib, dd, pre, "silu", None, amax=False)
    assert torch.equal(again, dbias)
    none, _ = run_backward(lib, dd, pre, "silu", dd.clone(), want_bias=False)
    assert bool(torch.isnan(none).all())
    inplace, amax2 = run_backward(lib, dd, pre, "silu", dd)
    R.check(dd, *ref["dpre"], "dpre in place")
    assert torch.equal(inplace, dbias) and torch.equal(amax, amax2)


def test_epilogue_backward_no_rows(lib):
    out = torch.full((9,), 5.0, device="cuda")
    lib.nvfp4_epilogue_backward(None, 8, None, 8, 0, 1, 0, 8, None, 8, out[:8], out[8:], None, 0)
    assert bool((out == 0).all())


@pytest.mark.parametrize("act", ACTS[1:])
def test_epilogue_backward_against_differences(lib, act):
    """Central differences of the 64-bit activation, h = 1e-5 (error h^2 / 6 times a third derivative below 4, and
    2^-52 / h of the value), away from relu's corner."""
    pre = randn(3, 40, 50, scale=2.0)
    pre = torch.where(pre.abs() < 1e-3, torch.ones_like(pre), pre).cuda()
    dd = randn(4, 40, 50).cuda()
    dpre, _, _ = lib.epilogue_backward(dd, pre, act)
    v, h = pre.double().cpu(), 1e-5
    slope = (R.act(v + h, act)[0] - R.act(v - h, act)[0]) / (2 * h)
    R.check(dpre, dd.double().cpu() * slope, R.epilogue_backward(dd, pre, act)["dpre"][1] + dd.double().cpu().abs() * 1e-9, "dpre")
