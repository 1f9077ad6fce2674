"""Argument checks of the layer norm and product epilogue entry points (no GPU needed): refusals come before any
device work, valid arguments stop only at the device check."""
import pytest
import torch

FAKE = 1 << 20                      # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def nv():
    from nvfp4_block_scaled_15_b200 import build
    build.build()
    from nvfp4_block_scaled_15_b200 import nvfp4
    return nvfp4


def call(nv, name, base, **change):
    args = dict(base)
    assert set(change) <= set(args), change
    args.update(change)
    return nv.raw_status(name, *args.values())


def passes(nv, status):
    return status in ((nv.ERR_CUDA, nv.ERR_ARCH) if not torch.cuda.is_available() else (nv.OK,))


LN = dict(x=FAKE, x_dtype=0, rows=4, k=33, ldx=33, gamma=FAKE, beta=FAKE, p_dtype=1, eps=1e-5, y=FAKE, y_dtype=0, ldy=33,
          mean=FAKE, rstd=FAKE, amax=FAKE, stream=None)
LNB = dict(dy=FAKE, dy_dtype=0, lddy=33, x=FAKE, x_dtype=0, ldx=33, mean=FAKE, rstd=FAKE, gamma=FAKE, p_dtype=0, res=None,
           ldr=0, rows=4, k=33, dx=FAKE, lddx=33, dgamma=FAKE, dbeta=FAKE, amax=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)
GEMM = dict(a=FAKE, a_sf=FAKE, g_a=FAKE, b=FAKE, b_sf=FAKE, g_b=FAKE, m=8, n=10, k=64, bias=FAKE, b_dtype=0, act=2,
            res=None, ldr=0, d=FAKE, ldd=10, out=0, pre=None, ldp=0, amax=FAKE, stream=None)
GEMV = dict(x=FAKE, m=4, ldx=64, w=FAKE, w_sf=FAKE, g_w=FAKE, n=10, k=64, bias=FAKE, b_dtype=0, act=2, res=None, ldr=0,
            y=FAKE, ldy=10, ws=FAKE, ws_bytes=1 << 30, stream=None)
EB = dict(dd=FAKE, ldd=10, pre=FAKE, ldp=10, dtype=0, act=2, m=8, n=10, dpre=FAKE + (1 << 16), lddp=10, dbias=FAKE,
          amax=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), "INVALID_ARG"), (dict(k=0, ldx=0, ldy=0), "INVALID_ARG"), (dict(ldx=32), "INVALID_ARG"),
    (dict(ldy=32), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"),
    (dict(x_dtype=2), "INVALID_ARG"), (dict(y_dtype=-1), "INVALID_ARG"), (dict(p_dtype=7), "INVALID_ARG"),
    (dict(eps=-1e-5), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"),
    (dict(rows=1 << 31), "UNSUPPORTED_SHAPE"), (dict(k=1 << 31, ldx=1 << 31, ldy=1 << 31), "UNSUPPORTED_SHAPE"),
    (dict(k=(1 << 28) + 1, ldx=1 << 30, ldy=1 << 30), "UNSUPPORTED_SHAPE"),
    (dict(x=FAKE + 1), "MISALIGNED"), (dict(x=FAKE + 2, x_dtype=1), "MISALIGNED"), (dict(y=FAKE + 1), "MISALIGNED"),
    (dict(gamma=FAKE + 2), "MISALIGNED"), (dict(beta=FAKE + 1, p_dtype=0), "MISALIGNED"), (dict(mean=FAKE + 2), "MISALIGNED"),
    (dict(amax=FAKE + 1), "MISALIGNED")], ids=str)
def test_layernorm_refuses(nv, change, status):
    assert call(nv, "nvfp4_layernorm", LN, **change) == getattr(nv, "ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"), (dict(dy=None), "INVALID_ARG"),
    (dict(mean=None), "INVALID_ARG"), (dict(rstd=None), "INVALID_ARG"), (dict(dx=None), "INVALID_ARG"),
    (dict(lddy=32), "INVALID_ARG"), (dict(lddx=32), "INVALID_ARG"), (dict(res=FAKE + 64, ldr=32), "INVALID_ARG"),
    (dict(res=FAKE, ldr=40), "INVALID_ARG"), (dict(dy_dtype=3), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"),
    (dict(ws_bytes=64), "WORKSPACE"), (dict(ws=FAKE + 8), "MISALIGNED"), (dict(dgamma=FAKE + 2), "MISALIGNED"),
    (dict(res=FAKE + 1, ldr=33), "MISALIGNED"), (dict(rows=1 << 31), "UNSUPPORTED_SHAPE"),
    (dict(k=(1 << 28) + 1, ldx=1 << 30, lddy=1 << 30, lddx=1 << 30), "UNSUPPORTED_SHAPE")], ids=str)
def test_layernorm_backward_refuses(nv, change, status):
    assert call(nv, "nvfp4_layernorm_backward", LNB, **change) == getattr(nv, "ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(m=0), "INVALID_ARG"), (dict(k=96), "UNSUPPORTED_SHAPE"), (dict(act=5), "INVALID_ARG"), (dict(act=-1), "INVALID_ARG"),
    (dict(b_dtype=2), "INVALID_ARG"), (dict(out=2), "INVALID_ARG"), (dict(ldd=9), "INVALID_ARG"), (dict(d=None), "INVALID_ARG"),
    (dict(res=FAKE + 64, ldr=9), "INVALID_ARG"), (dict(res=FAKE, ldr=12), "INVALID_ARG"), (dict(pre=FAKE, ldp=10), "INVALID_ARG"),
    (dict(pre=FAKE + 64, ldp=9), "INVALID_ARG"), (dict(pre=FAKE + 64, ldp=10, res=FAKE + 64, ldr=10), "INVALID_ARG"),
    (dict(d=FAKE + 1), "MISALIGNED"), (dict(pre=FAKE + 65, ldp=10), "MISALIGNED"), (dict(bias=FAKE + 1), "MISALIGNED"),
    (dict(bias=FAKE + 2, b_dtype=1), "MISALIGNED"), (dict(a=FAKE + 8), "MISALIGNED"), (dict(amax=FAKE + 2), "MISALIGNED"),
    (dict(res=FAKE + 66, ldr=10, out=1), "MISALIGNED")], ids=str)
def test_gemm_epilogue_refuses(nv, change, status):
    assert call(nv, "nvfp4_gemm_epilogue", GEMM, **change) == getattr(nv, "ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(m=33), "UNSUPPORTED_SHAPE"), (dict(m=0), "INVALID_ARG"), (dict(act=9), "INVALID_ARG"), (dict(b_dtype=2), "INVALID_ARG"),
    (dict(res=FAKE, ldr=12), "INVALID_ARG"), (dict(res=FAKE + 64, ldr=9), "INVALID_ARG"), (dict(res=FAKE + 1, ldr=10), "MISALIGNED"),
    (dict(bias=FAKE + 1), "MISALIGNED"), (dict(ws_bytes=64), "WORKSPACE"), (dict(ws=None), "INVALID_ARG"),
    (dict(ldy=9), "INVALID_ARG")], ids=str)
def test_gemv_epilogue_refuses(nv, change, status):
    assert call(nv, "nvfp4_gemv_batched_epilogue", GEMV, **change) == getattr(nv, "ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), "INVALID_ARG"), (dict(n=0), "INVALID_ARG"), (dict(pre=None), "INVALID_ARG"), (dict(dd=None), "INVALID_ARG"),
    (dict(act=6), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"), (dict(ldd=9), "INVALID_ARG"), (dict(lddp=9), "INVALID_ARG"),
    (dict(dpre=FAKE, lddp=12), "INVALID_ARG"), (dict(pre=FAKE + (1 << 16)), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"),
    (dict(ws_bytes=16), "WORKSPACE"), (dict(ws=FAKE + 4), "MISALIGNED"), (dict(dd=FAKE + 1), "MISALIGNED"),
    (dict(dbias=FAKE + 1), "MISALIGNED"), (dict(m=1 << 31), "UNSUPPORTED_SHAPE"),
    (dict(n=(1 << 28) + 1, ldd=1 << 30, ldp=1 << 30, lddp=1 << 30), "UNSUPPORTED_SHAPE")], ids=str)
def test_epilogue_backward_refuses(nv, change, status):
    assert call(nv, "nvfp4_epilogue_backward", EB, **change) == getattr(nv, "ERR_" + status)


def test_valid_arguments_stop_at_the_device_check(nv):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for name, base, changes in [
            ("nvfp4_layernorm", LN, [{}, dict(gamma=None, beta=None, mean=None, rstd=None, amax=None), dict(rows=0, x=None, y=None)]),
            ("nvfp4_layernorm_backward", LNB, [{}, dict(dgamma=None, dbeta=None, ws=None, ws_bytes=0), dict(res=FAKE, ldr=33),
                                               dict(rows=0, ws=None)]),
            ("nvfp4_gemm_epilogue", GEMM, [{}, dict(bias=None, act=0, amax=None), dict(res=FAKE, ldr=10)]),
            ("nvfp4_gemv_batched_epilogue", GEMV, [{}, dict(bias=None, act=0), dict(res=FAKE, ldr=10)]),
            ("nvfp4_epilogue_backward", EB, [{}, dict(pre=None, act=0), dict(dpre=None), dict(dbias=None, ws=None), dict(m=0)])]:
        for change in changes:
            assert passes(nv, call(nv, name, base, **change)), (name, change)


def test_workspace_sizes(nv):
    for op in (nv.OP_LAYERNORM_BACKWARD, nv.OP_EPILOGUE_BACKWARD):
        assert nv.nvfp4_workspace_bytes(op, 4, 33, 0) > 0
        assert nv.nvfp4_workspace_bytes(op, 0, 33, 0) > 0
        assert nv.nvfp4_workspace_bytes(op, -1, 33, 0) == 0
        assert nv.nvfp4_workspace_bytes(op, 4, 0, 0) == 0
        assert nv.nvfp4_workspace_bytes(op, 1 << 31, 33, 0) == 0
        assert nv.nvfp4_workspace_bytes(op, 4, (1 << 28) + 1, 0) == 0


# ---------------------------------------------------------------------------
# the torch helpers
# ---------------------------------------------------------------------------
def quantized(nv, rows, k):
    return nv.empty_quantized(rows, k, device="cpu")


def overlapping(rows, k, dtype):
    """A broadcast vector (pitch 0) and windows that overlap (pitch 10): rows that share memory."""
    return [torch.zeros(k, dtype=dtype).expand(rows, k), torch.zeros(10 * rows + k, dtype=dtype).as_strided((rows, k), (10, 1))]


def helper_calls(nv, rows=300, k=64, n=128):
    """{operand: call of its helper with that operand replaced}; no call gets as far as the device."""
    t = torch.zeros(rows, k, dtype=torch.bfloat16)
    few, wide = torch.zeros(9, k, dtype=torch.bfloat16), torch.zeros(rows, n, dtype=torch.bfloat16)
    stat = torch.zeros(rows)
    a, w = quantized(nv, rows, k), quantized(nv, n, k)
    back = lambda **c: nv.layernorm_backward(c.get("dy", t), c.get("x", t), stat, stat, d_residual=c.get("res"), out=c.get("out"))
    return {
        "layernorm x": (rows, k, lambda v: nv.layernorm(v)),
        "layernorm out": (rows, k, lambda v: nv.layernorm(t, out=v)),
        "layernorm_backward dy": (rows, k, lambda v: back(dy=v)),
        "layernorm_backward x": (rows, k, lambda v: back(x=v)),
        "layernorm_backward d_residual": (rows, k, lambda v: back(res=v)),
        "layernorm_backward out": (rows, k, lambda v: back(out=v)),
        "gemm_epilogue residual": (rows, n, lambda v: nv.gemm_epilogue(a, w, residual=v)),
        "gemm_epilogue out": (rows, n, lambda v: nv.gemm_epilogue(a, w, out=v)),
        "gemm_epilogue pre": (rows, n, lambda v: nv.gemm_epilogue(a, w, pre=v)),
        "gemv_batched_epilogue x": (9, k, lambda v: nv.gemv_batched_epilogue(v, w)),
        "gemv_batched_epilogue residual": (9, n, lambda v: nv.gemv_batched_epilogue(few, w, residual=v)),
        "gemv_batched_epilogue out": (9, n, lambda v: nv.gemv_batched_epilogue(few, w, out=v)),
        "epilogue_backward dd": (rows, n, lambda v: nv.epilogue_backward(v, None)),
        "epilogue_backward pre": (rows, n, lambda v: nv.epilogue_backward(wide, v, "relu")),
        "epilogue_backward out": (rows, n, lambda v: nv.epilogue_backward(wide, None, out=v)),
    }


@pytest.mark.parametrize("operand", [
    "layernorm x", "layernorm out", "layernorm_backward dy", "layernorm_backward x", "layernorm_backward d_residual",
    "layernorm_backward out", "gemm_epilogue residual", "gemm_epilogue out", "gemm_epilogue pre", "gemv_batched_epilogue x",
    "gemv_batched_epilogue residual", "gemv_batched_epilogue out", "epilogue_backward dd", "epilogue_backward pre",
    "epilogue_backward out"])
def test_helpers_refuse_rows_that_overlap(nv, operand):
    """Their buffer holds fewer elements than rows times columns: taken as dense rows they would be read, or written,
    past its end."""
    rows, cols, call = helper_calls(nv)[operand]
    for v in overlapping(rows, cols, torch.bfloat16):
        with pytest.raises(AssertionError, match="overlap"):
            call(v)


def test_pitch_of_a_single_row(nv):
    """The stride of a matrix of one row (or none) says nothing; of more rows it is the pitch."""
    flat = torch.zeros(1000)
    assert nv._rows_of(flat.as_strided((1, 64), (0, 1))) == 64
    assert nv._rows_of(flat.as_strided((1, 64), (999, 1))) == 64
    assert nv._rows_of(flat.as_strided((0, 64), (0, 1))) == 64
    assert nv._rows_of(flat.as_strided((2, 64), (70, 1))) == 70
    assert nv._rows_of(flat.as_strided((5, 1), (3, 9))) == 3
    with pytest.raises(AssertionError, match="overlap"):
        nv._rows_of(flat.as_strided((5, 1), (0, 1)))


def test_helpers_refuse_an_output_on_an_input(nv):
    """Kernels read rows again, or other blocks read them, after outputs are written: only a residual (or its gradient, or
    the gradient that an epilogue is given) may be written in place."""
    t, dy, square = (torch.zeros(9, 64, dtype=torch.bfloat16) for _ in range(3))
    stat, w = torch.zeros(9), quantized(nv, 64, 64)
    for call in (lambda: nv.layernorm(t, out=t), lambda: nv.layernorm_backward(dy, t, stat, stat, out=t),
                 lambda: nv.layernorm_backward(dy, t, stat, stat, out=dy),
                 lambda: nv.gemv_batched_epilogue(square, w, out=square),
                 lambda: nv.gemv_batched_epilogue(square, w, residual=square, out=square)):
        with pytest.raises(AssertionError, match="in place"):
            call()


def test_helpers_take_rows_side_by_side(nv, monkeypatch):
    """An input and an output may be columns of one buffer; the in-place forms that the library has stay."""
    for name in ("nvfp4_layernorm", "nvfp4_layernorm_backward", "nvfp4_gemv_batched_epilogue", "nvfp4_epilogue_backward"):
        monkeypatch.setattr(nv, name, lambda *a, **kw: None)
    both, stat, w = torch.zeros(9, 128, dtype=torch.bfloat16), torch.zeros(9), quantized(nv, 64, 64)
    x, y, r = both[:, :64], both[:, 64:], torch.zeros(9, 64, dtype=torch.bfloat16)
    nv.layernorm(x, out=y)
    nv.layernorm_backward(x, x, stat, stat, d_residual=r, out=r)
    nv.gemv_batched_epilogue(x, w, residual=r, out=r)
    nv.gemv_batched_epilogue(x, w, out=y)
    nv.epilogue_backward(r, x, "relu", out=r)
