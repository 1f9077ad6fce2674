"""Layer norm forward and backward against the 64-bit definition: every output, at sizes, types, pitches and
alignments around each kernel's limits."""
import pytest
import torch

import operator_refs as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def randn(seed, *shape, scale=1.0):
    return scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def placed(t, dtype, pad=0, offset=0, fill=7.0):
    """t on the device in `dtype` with `pad` more elements per row, `offset` elements past an aligned address;
    (view, the whole buffer)."""
    rows, k = t.shape
    flat = torch.full((offset + (rows + 1) * (k + pad) + 8,), fill, dtype=dtype, device="cuda")
    v = flat[offset:].as_strided((rows, k), (k + pad, 1))
    v.copy_(t)
    return v, flat


def untouched(flat, view):
    """Everything of the buffer outside the view still holds the fill."""
    inside = torch.zeros_like(flat, dtype=torch.bool)
    inside[view.storage_offset() - flat.storage_offset():].as_strided(view.shape, view.stride()).fill_(True)
    assert bool((flat[~inside] == 7.0).all()), "written outside the rows"


def activations(seed, rows, k):
    x = randn(seed, rows, k)
    x[:, ::97] *= 40.0
    return x + 0.3 * randn(seed + 1, k)


def params(seed, k, dtype, which="gb"):
    g = (1 + 0.2 * randn(seed, k)).to(dtype).cuda() if "g" in which else None
    b = (0.3 * randn(seed + 1, k)).to(dtype).cuda() if "b" in which else None
    return g, b


def run_forward(lib, x, g, b, y, eps=EPS, stream=None):
    """The raw call, outputs pre-filled with NaN so that a missing store shows."""
    rows, k = x.shape
    stats = torch.full((2 * rows + 1,), float("nan"), device="cuda")
    pd = lib._dtype_of(g if g is not None else b)
    lib.nvfp4_layernorm(x, lib._dtype_of(x), rows, k, x.stride(0), g, b, pd, eps, y, lib._dtype_of(y), y.stride(0),
                        stats[:rows], stats[rows:2 * rows], stats[2 * rows:], stream)
    return stats[:rows], stats[rows:2 * rows], stats[2 * rows:]


def check_forward(lib, x, g, b, y, stats, eps=EPS):
    ref = R.layernorm(x, g, b, eps)
    R.check(y, *ref["y"], "y")
    R.check(stats[0], *ref["mean"], "mean")
    R.check(stats[1], *ref["rstd"], "rstd")
    assert float(stats[2]) == float(y.float().abs().max()), "amax of the stored y"


# (rows, k): one element, one warp's and one block's limits on both sides, a whole vector less or more, lengths past
# what registers hold, more rows than a grid
SHAPES = [(1, 1), (1, 8192), (8, 8192), (3, 7), (5, 33), (130, 1000), (64, 1155), (33, 1024), (33, 1032), (9, 2048),
          (300, 2056), (5, 4096), (3, 8200), (2, 16384), (3, 28672), (2, 32768), (2, 32776), (2, 40001), (2, 70001), (2500, 64), (400, 8191), (170, 20001), (700, 63), (90, 65), (1300, 256), (50, 257)]


@pytest.mark.parametrize("rows,k", SHAPES, ids=str)
@pytest.mark.parametrize("xd,yd,pd,pad,off", [(BF16, BF16, BF16, 0, 0), (F32, BF16, F32, 8, 0), (BF16, F32, F32, 1, 1),
                                              (F32, F32, BF16, 0, 3)], ids=["bf16", "f32_bf16_pitch", "bf16_f32_odd", "f32_offset"])
def test_forward(lib, rows, k, xd, yd, pd, pad, off):
    x, _ = placed(activations(rows * 31 + k, rows, k), xd, pad, off)
    y, flat = placed(torch.full((rows, k), 7.0), yd, pad, off)
    g, b = params(k, k, pd)
    stats = run_forward(lib, x, g, b, y)
    check_forward(lib, x, g, b, y, stats)
    untouched(flat, y)


@pytest.mark.parametrize("which", ["", "g", "b"], ids=["none", "gamma", "beta"])
@pytest.mark.parametrize("k", [96, 1155, 40000])
def test_forward_without_parameters(lib, which, k):
    x, _ = placed(activations(3, 6, k), BF16)
    y, _ = placed(torch.zeros(6, k), BF16)
    g, b = params(k, k, F32, which)
    check_forward(lib, x, g, b, y, run_forward(lib, x, g, b, y))


@pytest.mark.parametrize("xd", [BF16, F32])
@pytest.mark.parametrize("k", [100, 4096, 33000])
def test_forward_far_mean_and_constant_rows(lib, xd, k):
    """Rows far from zero (their spread is a thousandth of their mean), constant rows and rows of zeros."""
    x = 1000.0 + randn(5, 6, k)
    x[2] = 3.0
    x[4] = 0.0
    x, _ = placed(x, xd)
    y, _ = placed(torch.zeros(6, k), F32)
    g, b = params(9, k, F32)
    check_forward(lib, x, g, b, y, run_forward(lib, x, g, b, y))


@pytest.mark.parametrize("k", [40, 4096, 33000])
def test_forward_nonfinite_rows_stay_apart(lib, k):
    x = activations(4, 7, k)
    x[1, k // 2] = float("inf")
    x[5, 3] = float("nan")
    x, _ = placed(x, BF16)
    y, _ = placed(torch.zeros(7, k), BF16)
    g, b = params(9, k, BF16)
    stats = run_forward(lib, x, g, b, y)
    assert bool(torch.isnan(y[[1, 5]]).all())
    keep = [0, 2, 3, 4, 6]
    ref = R.layernorm(x[keep], g, b, EPS)
    R.check(y[keep], *ref["y"], "y")
    assert not bool(torch.isfinite(stats[2]))


def test_forward_no_rows_and_no_outputs(lib):
    stats = torch.full((1,), 5.0, device="cuda")
    lib.nvfp4_layernorm(None, 0, 0, 64, 64, None, None, 0, EPS, None, 0, 64, None, None, stats)
    assert float(stats) == 0.0
    x, _ = placed(activations(1, 5, 300), BF16)
    y, _ = placed(torch.zeros(5, 300), BF16)
    lib.nvfp4_layernorm(x, 0, 5, 300, 300, None, None, 0, EPS, y, 0, 300)
    R.check(y, *R.layernorm(x, None, None, EPS)["y"], "y")


def test_forward_offsets_past_32_bits(lib):
    """Two rows 2^31 + 64 elements apart."""
    ld, k = (1 << 31) + 64, 1000
    buf = torch.empty(ld + k, dtype=BF16, device="cuda")
    x = buf.as_strided((2, k), (ld, 1))
    x.copy_(activations(8, 2, k))
    g, b = params(1, k, F32)
    y, _ = placed(torch.zeros(2, k), F32)
    check_forward(lib, x, g, b, y, run_forward(lib, x, g, b, y))


def test_amax_makes_the_quantizer_one_pass(lib):
    x, _ = placed(activations(21, 200, 1024), BF16)
    g, b = params(2, 1024, F32)
    n = lib.layernorm(x, g, b)
    one, two = lib.quantize(n.y, amax=n.amax), lib.quantize(n.y)
    assert torch.equal(one.codes, two.codes) and torch.equal(one.sf, two.sf) and torch.equal(one.g, two.g)


def run_backward(lib, dy, x, mean, rstd, g, res, dx, want=(True, True), amax=True):
    rows, k = x.shape
    out = torch.full((2 * k + 1,), float("nan"), device="cuda")
    nbytes = lib.nvfp4_workspace_bytes(lib.OP_LAYERNORM_BACKWARD, rows, k, 0)
    ws = torch.full((nbytes + 64,), 0xFF, dtype=torch.uint8, device="cuda")       # NaN patterns; a guard behind
    lib.nvfp4_layernorm_backward(dy, lib._dtype_of(dy), dy.stride(0), x, lib._dtype_of(x), x.stride(0), mean, rstd, g,
                                 lib._dtype_of(g), res, 0 if res is None else res.stride(0), rows, k, dx, dx.stride(0),
                                 out[:k] if want[0] else None, out[k:2 * k] if want[1] else None,
                                 out[2 * k:] if amax else None, ws, nbytes)
    assert bool((ws[nbytes:] == 0xFF).all()), "written past the workspace"
    return out[:k], out[k:2 * k], out[2 * k:]


def backward_inputs(rows, k, xd, dyd, pd, res, pad=0, off=0):
    x, _ = placed(activations(rows * 13 + k, rows, k), xd, pad, off)
    dy, _ = placed(randn(k + 5, rows, k, scale=0.05), dyd, pad, off)
    ref = R.layernorm(x, None, None, EPS)
    mean, rstd = ref["mean"][0].float().cuda(), ref["rstd"][0].float().cuda()
    g = params(k, k, pd)[0] if pd is not None else None
    r = placed(randn(k + 9, rows, k, scale=0.05), xd, pad, off)[0] if res else None
    return dy, x, mean, rstd, g, r


def check_backward(inputs, dx, grads):
    ref = R.layernorm_backward(*inputs)
    R.check(dx, *ref["dx"], "dx")
    R.check(grads[0], *ref["dgamma"], "dgamma")
    R.check(grads[1], *ref["dbeta"], "dbeta")
    assert float(grads[2]) == float(dx.float().abs().max()), "amax of the stored dx"


@pytest.mark.parametrize("rows,k", SHAPES, ids=str)
@pytest.mark.parametrize("xd,dyd,pd,res,pad,off", [(BF16, BF16, BF16, True, 0, 0), (F32, BF16, F32, False, 8, 0),
                                                   (BF16, F32, None, True, 1, 1), (F32, F32, BF16, True, 0, 3)],
                         ids=["bf16", "f32_bf16_pitch", "bf16_f32_odd", "f32_offset"])
def test_backward(lib, rows, k, xd, dyd, pd, res, pad, off):
    inputs = backward_inputs(rows, k, xd, dyd, pd, res, pad, off)
    dx, flat = placed(torch.full((rows, k), 7.0), xd, pad, off)
    grads = run_backward(lib, *inputs, dx)
    check_backward(inputs, dx, grads)
    untouched(flat, dx)


@pytest.mark.parametrize("rows,k", [(20000, 66), (9001, 301), (4003, 1155), (1200, 4095), (700, 8191)], ids=str)
@pytest.mark.parametrize("xd,dyd", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)], ids=["f32", "f32_bf16", "bf16_f32", "bf16"])
def test_backward_many_rows_that_start_anywhere(lib, rows, k, xd, dyd):
    """Several rounds of rows per group, on both sides of the choice between the ring and rows straight from memory."""
    inputs = backward_inputs(rows, k, xd, dyd, BF16, True, 1, 1)
    dx, flat = placed(torch.full((rows, k), 7.0), xd, 1, 1)
    check_backward(inputs, dx, run_backward(lib, *inputs, dx))
    untouched(flat, dx)


@pytest.mark.parametrize("k", [72, 1155, 8192, 33000])
def test_backward_in_place_on_the_residual_gradient(lib, k):
    inputs = backward_inputs(20, k, BF16, BF16, F32, True)
    kept = inputs[:5] + (inputs[5].clone(),)
    grads = run_backward(lib, *inputs, inputs[5])
    check_backward(kept, inputs[5], grads)


@pytest.mark.parametrize("want", [(True, False), (False, True), (False, False)], ids=str)
@pytest.mark.parametrize("k", [64, 2048, 33000])
def test_backward_outputs_left_out(lib, want, k):
    inputs = backward_inputs(50, k, BF16, BF16, BF16, False)
    dx, _ = placed(torch.zeros(50, k), BF16)
    grads = run_backward(lib, *inputs, dx, want, amax=False)
    ref = R.layernorm_backward(*inputs)
    R.check(dx, *ref["dx"], "dx")
    for on, got, name in zip(want, grads, ("dgamma", "dbeta")):
        if on:
            R.check(got, *ref[name], name)
        else:
            assert bool(torch.isnan(got).all()), "an output that was not asked for"


def test_backward_no_rows(lib):
    out = torch.full((2 * 48 + 1,), 5.0, device="cuda")
    lib.nvfp4_layernorm_backward(None, 0, 48, None, 0, 48, None, None, None, 0, None, 0, 0, 48, None, 48, out[:48], out[48:96],
                                 out[96:], None, 0)
    assert bool((out == 0).all())


@pytest.mark.parametrize("rows,k", [(4000, 96), (700, 1155), (513, 8192)], ids=str)
def test_backward_same_bits_every_time(lib, rows, k):
    inputs = backward_inputs(rows, k, BF16, BF16, BF16, True)
    dx, _ = placed(torch.zeros(rows, k), BF16)
    first = [t.clone() for t in run_backward(lib, *inputs, dx)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run_backward(lib, *inputs, dx)))


@pytest.mark.parametrize("k", [48, 1155])
def test_backward_against_differences(lib, k):
    """Central differences of the 64-bit forward pass in random directions of x, gamma and beta.  The difference
    quotient's own error is h^2 / 6 of a third derivative (h = 1e-4, values of order one: below 1e-6 of the sum of
    magnitudes) and is allowed beside the elementwise tolerances."""
    rows = 6
    x, _ = placed(randn(2, rows, k), F32)
    g, b = params(3, k, F32)
    w, _ = placed(randn(4, rows, k), F32)
    n = lib.layernorm(x, g, b, EPS, F32)
    dx, dg, db, _ = lib.layernorm_backward(w, x, n.mean, n.rstd, g)
    ref = R.layernorm_backward(w, x, n.mean, n.rstd, g, None)
    x64, g64, b64, w64 = (t.double().cpu() for t in (x, g, b, w))

    def loss(x, g, b):
        return (R.layernorm(x, g, b, EPS)["y"][0] * w64).sum()

    h = 1e-4
    for grad, name, at in ((dx, "dx", 0), (dg, "dgamma", 1), (db, "dbeta", 2)):
        for seed in range(3):
            v = randn(100 + seed, *grad.shape).double()
            args = [x64, g64, b64]
            hi, lo = list(args), list(args)
            hi[at], lo[at] = args[at] + h * v, args[at] - h * v
            want = float((loss(*hi) - loss(*lo)) / (2 * h))
            got = float((grad.double().cpu() * v).sum())
            scale = float((grad.double().cpu() * v).abs().sum())
            # the statistics handed to the backward pass are the fp32 ones: their tolerance moves dx by as much again
            stats = R.layernorm(x, g, b, EPS)
            rel = float((stats["rstd"][1] / stats["rstd"][0]).max() + (stats["mean"][1] * stats["rstd"][0]).max())
            tol = float((ref[name][1] * v.abs()).sum()) + scale * (1e-6 + 4 * rel + 2.0 ** -24)
            assert abs(got - want) <= tol, (name, got, want, tol)


def test_streams_and_graph(lib):
    """Calls on a side stream, captured into a graph with the quantizer behind, replayed on new contents."""
    rows, k = 70, 2048
    x, _ = placed(activations(1, rows, k), BF16)
    g, b = params(5, k, BF16)
    y, _ = placed(torch.zeros(rows, k), BF16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        stats = run_forward(lib, x, g, b, y)
    s.synchronize()
    check_forward(lib, x, g, b, y, stats)
    inputs = backward_inputs(rows, k, BF16, BF16, BF16, True)
    dx, _ = placed(torch.zeros(rows, k), BF16)
    out = torch.empty(2 * k + 1, device="cuda")
    ws = torch.empty(lib.nvfp4_workspace_bytes(lib.OP_LAYERNORM_BACKWARD, rows, k, 0), dtype=torch.uint8, device="cuda")
    dy, x2, mean, rstd, g2, res = inputs
    rs = torch.empty(2 * rows + 1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.nvfp4_layernorm(x, 0, rows, k, k, g, b, 0, EPS, y, 0, k, rs[:rows], rs[rows:2 * rows], rs[2 * rows:])
        lib.nvfp4_layernorm_backward(dy, 0, k, x2, 0, k, mean, rstd, g2, 0, res, k, rows, k, dx, k, out[:k], out[k:2 * k],
                                     out[2 * k:], ws, ws.numel())
    for seed in (50, 51):
        x.copy_(activations(seed, rows, k))
        dy.copy_(randn(seed, rows, k, scale=0.05))
        graph.replay()
        torch.cuda.synchronize()
        check_forward(lib, x, g, b, y, (rs[:rows], rs[rows:2 * rows], rs[2 * rows:]))
        check_backward(inputs, dx, (out[:k], out[k:2 * k], out[2 * k:]))


def test_helpers_refuse(lib):
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    with pytest.raises(AssertionError):
        lib.layernorm(x.t())
    with pytest.raises(AssertionError):
        lib.layernorm(x.half())
    with pytest.raises(AssertionError):
        lib.layernorm(x, torch.ones(63, device="cuda"))
    with pytest.raises(AssertionError):
        lib.layernorm(x, torch.ones(64, device="cuda"), torch.ones(64, device="cuda", dtype=BF16))
    with pytest.raises(lib.NVFP4Error):
        lib.layernorm(x, eps=-1.0)
