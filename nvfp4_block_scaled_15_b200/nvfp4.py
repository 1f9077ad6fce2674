"""Thin Python binding of libnvfp4 (include/nvfp4.h).

Argument marshalling only: every function passes raw pointers, sizes and the
current CUDA stream to the C ABI and raises NVFP4Error on a non-zero status.
PyTorch provides device memory and streams; no computation happens here.
The library must be built (``python -m nvfp4_block_scaled_15_b200.build``);
importing this module fails loudly otherwise.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with `python -m nvfp4_block_scaled_15_b200.build`")
_lib = ctypes.CDLL(_LIB_PATH)

# status codes (nvfp4_status)
OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED_SHAPE = 2
ERR_MISALIGNED = 3
ERR_ARCH = 4
ERR_CUDA = 5
ERR_TIMEOUT = 6
ERR_RANGE = 7
ERR_WORKSPACE = 8
# nvfp4_sf_layout
SF_ROWMAJOR = 0
SF_TCGEN05 = 1
# nvfp4_out_dtype
OUT_BF16 = 0
OUT_F32 = 1
# nvfp4_op
OP_GEMV_BATCHED = 1
OP_GEMM_QUANT_A = 2
OP_LAYERNORM_BACKWARD = 3
OP_EPILOGUE_BACKWARD = 4
# nvfp4_dtype
DTYPE_BF16 = 0
DTYPE_F32 = 1
# nvfp4_act
ACT_NONE = 0
ACT_RELU = 1
ACT_GELU = 2
ACT_GELU_TANH = 3
ACT_SILU = 4

_vp, _i64, _sz, _i32, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint64
_f32 = ctypes.c_float
_SIGS = {
    "nvfp4_abi_version": ([], _i32),
    "nvfp4_status_string": ([_i32], ctypes.c_char_p),
    "nvfp4_sf_bytes": ([_i64, _i64, _i32], _sz),
    "nvfp4_amax": ([_vp, _i64, _i64, _i64, _vp, _vp], _i32),
    "nvfp4_quantize": ([_vp, _i64, _i64, _i64, _vp, _vp, _i32, _vp, _vp, _i32, _vp], _i32),
    "nvfp4_quantize_stochastic": ([_vp, _i64, _i64, _i64, _vp, _vp, _i32, _vp, _vp, _i32, _u64, _u64, _vp],
                                  _i32),
    "nvfp4_quantize_hadamard_stochastic": ([_vp, _i64, _i64, _i64, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _u64, _u64,
                                            _vp], _i32),
    "nvfp4_quantize_hadamard": ([_vp, _i64, _i64, _i64, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp], _i32),
    "nvfp4_swizzle_sf": ([_vp, _i64, _i64, _vp, _vp], _i32),
    "nvfp4_gemm": ([_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _i32, _vp], _i32),
    "nvfp4_gemm_fp8_out": ([_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp], _i32),
    "nvfp4_gemm_requant": ([_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _vp, _vp],
                           _i32),
    "nvfp4_workspace_bytes": ([_i32, _i64, _i64, _i64], _sz),
    "nvfp4_gemv_batched": ([_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _sz, _vp], _i32),
    "nvfp4_gemm_quant_a": ([_vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _i32, _vp, _sz, _vp], _i32),
    "nvfp4_gemm_quant_a_prepare": ([_vp, _i64, _i64, _i64, _i64, _vp, _sz, _vp], _i32),
    "nvfp4_gemm_quant_a_run": ([_vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _i32, _vp, _sz, _vp], _i32),
    "nvfp4_gemm_quant_a_amax": ([_vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _i32, _vp, _sz, _vp],
                                _i32),
    "nvfp4_gemv_batched_noalloc": ([_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _i64, _vp], _i32),
    "nvfp4_mxfp4_sf_bytes": ([_i64, _i64, _i32], _sz),
    "nvfp4_mxfp4_quantize": ([_vp, _i64, _i64, _i64, _vp, _vp, _i32, _vp], _i32),
    "nvfp4_mxfp4_gemm": ([_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _i32, _vp], _i32),
    "nvfp4_layernorm": ([_vp, _i32, _i64, _i64, _i64, _vp, _vp, _i32, _f32, _vp, _i32, _i64, _vp, _vp, _vp, _vp], _i32),
    "nvfp4_layernorm_backward": ([_vp, _i32, _i64, _vp, _i32, _i64, _vp, _vp, _vp, _i32, _vp, _i64, _i64, _i64, _vp,
                                  _i64, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "nvfp4_gemm_epilogue": ([_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _i32, _vp, _i64, _vp, _i64,
                             _i32, _vp, _i64, _vp, _vp], _i32),
    "nvfp4_gemv_batched_epilogue": ([_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _i32, _i32, _vp, _i64, _vp, _i64,
                                     _vp, _sz, _vp], _i32),
    "nvfp4_epilogue_backward": ([_vp, _i64, _vp, _i64, _i32, _i32, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp],
                                _i32),
    "nvfp4_check_device_status": ([_vp], _i32),
    "nvfp4_set_wait_limit_ns": ([_u64], None),
    "nvfp4_selftest_wait_timeout": ([_u64, _vp], _i32),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def nvfp4_status_string(status: int) -> str:
    return _lib.nvfp4_status_string(int(status)).decode()


status_string = nvfp4_status_string


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _s(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str) -> None:
    if status != OK:
        raise NVFP4Error(status, where)


# ---------------------------------------------------------------------------
# one wrapper per C entry point
# ---------------------------------------------------------------------------
def nvfp4_abi_version() -> int:
    return _lib.nvfp4_abi_version()


def nvfp4_sf_bytes(rows: int, k: int, layout: int) -> int:
    return _lib.nvfp4_sf_bytes(rows, k, layout)


def nvfp4_workspace_bytes(op: int, m: int, n: int, k: int) -> int:
    return _lib.nvfp4_workspace_bytes(op, m, n, k)


def nvfp4_amax(x, rows, k, ldx, amax_dev, stream=None) -> None:
    _check(_lib.nvfp4_amax(_p(x), rows, k, ldx, _p(amax_dev), _s(stream)), "nvfp4_amax")


def nvfp4_quantize(x, rows, k, ldx, codes, sf, layout, g_dev, amax_dev, amax_given=0, stream=None) -> None:
    _check(_lib.nvfp4_quantize(_p(x), rows, k, ldx, _p(codes), _p(sf), layout, _p(g_dev), _p(amax_dev),
                               int(amax_given), _s(stream)), "nvfp4_quantize")


def nvfp4_quantize_stochastic(x, rows, k, ldx, codes, sf, layout, g_dev, amax_dev, amax_given, seed, offset,
                              stream=None) -> None:
    _check(_lib.nvfp4_quantize_stochastic(_p(x), rows, k, ldx, _p(codes), _p(sf), layout, _p(g_dev), _p(amax_dev),
                                          int(amax_given), int(seed), int(offset), _s(stream)),
           "nvfp4_quantize_stochastic")


def nvfp4_quantize_hadamard(x, rows, k, ldx, order, codes, sf, layout, g_dev, amax_dev, amax_given=0,
                            stream=None) -> None:
    _check(_lib.nvfp4_quantize_hadamard(_p(x), rows, k, ldx, int(order), _p(codes), _p(sf), layout, _p(g_dev),
                                        _p(amax_dev), int(amax_given), _s(stream)), "nvfp4_quantize_hadamard")


def nvfp4_quantize_hadamard_stochastic(x, rows, k, ldx, order, codes, sf, layout, g_dev, amax_dev, amax_given,
                                       seed, offset, stream=None) -> None:
    _check(_lib.nvfp4_quantize_hadamard_stochastic(_p(x), rows, k, ldx, int(order), _p(codes), _p(sf), layout,
                                                   _p(g_dev), _p(amax_dev), int(amax_given), int(seed), int(offset),
                                                   _s(stream)), "nvfp4_quantize_hadamard_stochastic")


def nvfp4_swizzle_sf(sf_rowmajor, rows, k, sf_tc, stream=None) -> None:
    _check(_lib.nvfp4_swizzle_sf(_p(sf_rowmajor), rows, k, _p(sf_tc), _s(stream)), "nvfp4_swizzle_sf")


def nvfp4_gemm(a_codes, a_sf, g_a, b_codes, b_sf, g_b, m, n, k, d, ldd, out_dtype=OUT_BF16, stream=None) -> None:
    _check(_lib.nvfp4_gemm(_p(a_codes), _p(a_sf), _p(g_a), _p(b_codes), _p(b_sf), _p(g_b), m, n, k, _p(d), ldd,
                           out_dtype, _s(stream)), "nvfp4_gemm")


def nvfp4_gemm_fp8_out(a_codes, a_sf, g_a, b_codes, b_sf, g_b, m, n, k, g_d, d, ldd, amax_d=None,
                       stream=None) -> None:
    _check(_lib.nvfp4_gemm_fp8_out(_p(a_codes), _p(a_sf), _p(g_a), _p(b_codes), _p(b_sf), _p(g_b), m, n, k,
                                   _p(g_d), _p(d), ldd, _p(amax_d), _s(stream)), "nvfp4_gemm_fp8_out")


def nvfp4_gemm_requant(a_codes, a_sf, g_a, b_codes, b_sf, g_b, m, n, k, g_d, d_codes, ldd_bytes, d_sf, layout,
                       amax_d=None, stream=None) -> None:
    _check(_lib.nvfp4_gemm_requant(_p(a_codes), _p(a_sf), _p(g_a), _p(b_codes), _p(b_sf), _p(g_b), m, n, k,
                                   _p(g_d), _p(d_codes), ldd_bytes, _p(d_sf), layout, _p(amax_d), _s(stream)),
           "nvfp4_gemm_requant")


def nvfp4_gemv_batched(x, m, ldx, w_codes, w_sf, g_w, n, k, y, ldy, workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_gemv_batched(_p(x), m, ldx, _p(w_codes), _p(w_sf), _p(g_w), n, k, _p(y), ldy,
                                   _p(workspace), ws_bytes, _s(stream)), "nvfp4_gemv_batched")


def nvfp4_gemv_batched_noalloc(x, m, ldx, w_codes, w_sf, g_w, n, k, y, ldy, stream=None) -> None:
    """nvfp4_gemv_batched on the library's fixed scratch (no workspace argument)."""
    _check(_lib.nvfp4_gemv_batched_noalloc(_p(x), m, ldx, _p(w_codes), _p(w_sf), _p(g_w), n, k, _p(y), ldy,
                                           _s(stream)), "nvfp4_gemv_batched_noalloc")


def nvfp4_gemm_quant_a(a, lda, b_codes, b_sf, g_b, m, n, k, d, ldd, out_dtype, workspace, ws_bytes,
                       stream=None) -> None:
    _check(_lib.nvfp4_gemm_quant_a(_p(a), lda, _p(b_codes), _p(b_sf), _p(g_b), m, n, k, _p(d), ldd, out_dtype,
                                   _p(workspace), ws_bytes, _s(stream)), "nvfp4_gemm_quant_a")


def nvfp4_gemm_quant_a_prepare(a, lda, m, n, k, workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_gemm_quant_a_prepare(_p(a), lda, m, n, k, _p(workspace), ws_bytes, _s(stream)),
           "nvfp4_gemm_quant_a_prepare")


def nvfp4_gemm_quant_a_run(a, lda, b_codes, b_sf, g_b, m, n, k, d, ldd, out_dtype, workspace, ws_bytes,
                           stream=None) -> None:
    _check(_lib.nvfp4_gemm_quant_a_run(_p(a), lda, _p(b_codes), _p(b_sf), _p(g_b), m, n, k, _p(d), ldd, out_dtype,
                                       _p(workspace), ws_bytes, _s(stream)), "nvfp4_gemm_quant_a_run")


def nvfp4_gemm_quant_a_amax(a, lda, amax, b_codes, b_sf, g_b, m, n, k, d, ldd, out_dtype, workspace, ws_bytes,
                            stream=None) -> None:
    _check(_lib.nvfp4_gemm_quant_a_amax(_p(a), lda, _p(amax), _p(b_codes), _p(b_sf), _p(g_b), m, n, k, _p(d), ldd,
                                        out_dtype, _p(workspace), ws_bytes, _s(stream)), "nvfp4_gemm_quant_a_amax")


def nvfp4_mxfp4_sf_bytes(rows: int, k: int, layout: int) -> int:
    return _lib.nvfp4_mxfp4_sf_bytes(rows, k, layout)


def nvfp4_mxfp4_quantize(x, rows, k, ldx, codes, sf, layout, stream=None) -> None:
    _check(_lib.nvfp4_mxfp4_quantize(_p(x), rows, k, ldx, _p(codes), _p(sf), layout, _s(stream)),
           "nvfp4_mxfp4_quantize")


def nvfp4_mxfp4_gemm(a_codes, a_sf, b_codes, b_sf, m, n, k, d, ldd, out_dtype=OUT_BF16, stream=None) -> None:
    _check(_lib.nvfp4_mxfp4_gemm(_p(a_codes), _p(a_sf), _p(b_codes), _p(b_sf), m, n, k, _p(d), ldd, out_dtype,
                                 _s(stream)), "nvfp4_mxfp4_gemm")


def nvfp4_layernorm(x, x_dtype, rows, k, ldx, gamma, beta, param_dtype, eps, y, y_dtype, ldy, mean=None, rstd=None,
                    amax_dev=None, stream=None) -> None:
    _check(_lib.nvfp4_layernorm(_p(x), x_dtype, rows, k, ldx, _p(gamma), _p(beta), param_dtype, eps, _p(y), y_dtype,
                                ldy, _p(mean), _p(rstd), _p(amax_dev), _s(stream)), "nvfp4_layernorm")


def nvfp4_layernorm_backward(dy, dy_dtype, lddy, x, x_dtype, ldx, mean, rstd, gamma, param_dtype, d_residual, ldr,
                             rows, k, dx, lddx, dgamma, dbeta, amax_dx, workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_layernorm_backward(_p(dy), dy_dtype, lddy, _p(x), x_dtype, ldx, _p(mean), _p(rstd), _p(gamma),
                                         param_dtype, _p(d_residual), ldr, rows, k, _p(dx), lddx, _p(dgamma),
                                         _p(dbeta), _p(amax_dx), _p(workspace), ws_bytes, _s(stream)),
           "nvfp4_layernorm_backward")


def nvfp4_gemm_epilogue(a_codes, a_sf, g_a, b_codes, b_sf, g_b, m, n, k, bias, bias_dtype, act, residual, ldr, d, ldd,
                        out_dtype=OUT_BF16, pre=None, ldp=0, amax_d=None, stream=None) -> None:
    _check(_lib.nvfp4_gemm_epilogue(_p(a_codes), _p(a_sf), _p(g_a), _p(b_codes), _p(b_sf), _p(g_b), m, n, k, _p(bias),
                                    bias_dtype, act, _p(residual), ldr, _p(d), ldd, out_dtype, _p(pre), ldp,
                                    _p(amax_d), _s(stream)), "nvfp4_gemm_epilogue")


def nvfp4_gemv_batched_epilogue(x, m, ldx, w_codes, w_sf, g_w, n, k, bias, bias_dtype, act, residual, ldr, y, ldy,
                                workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_gemv_batched_epilogue(_p(x), m, ldx, _p(w_codes), _p(w_sf), _p(g_w), n, k, _p(bias), bias_dtype,
                                            act, _p(residual), ldr, _p(y), ldy, _p(workspace), ws_bytes, _s(stream)),
           "nvfp4_gemv_batched_epilogue")


def nvfp4_epilogue_backward(dd, ldd, pre, ldp, dtype, act, m, n, dpre, lddp, dbias, amax_dpre, workspace, ws_bytes,
                            stream=None) -> None:
    _check(_lib.nvfp4_epilogue_backward(_p(dd), ldd, _p(pre), ldp, dtype, act, m, n, _p(dpre), lddp, _p(dbias),
                                        _p(amax_dpre), _p(workspace), ws_bytes, _s(stream)), "nvfp4_epilogue_backward")


def nvfp4_check_device_status(stream=None) -> int:
    """Synchronises the stream; returns (and clears) the device status code."""
    return _lib.nvfp4_check_device_status(_s(stream))


def nvfp4_set_wait_limit_ns(limit_ns: int) -> None:
    _lib.nvfp4_set_wait_limit_ns(int(limit_ns))


def nvfp4_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    _check(_lib.nvfp4_selftest_wait_timeout(int(limit_ns), _s(stream)), "nvfp4_selftest_wait_timeout")


def raw_status(name: str, *args) -> int:
    """Call a C entry point with raw arguments and return its status (for tests of argument checks)."""
    return getattr(_lib, name)(*args)


# ---------------------------------------------------------------------------
# allocation helpers (torch owns the memory; the work runs in the library)
# ---------------------------------------------------------------------------
def _on_its_stream(helper):
    """A helper called with ``stream=`` runs with that stream current, so that what it allocates (outputs, workspace) and
    copies belongs to that stream: torch's allocator hands memory out, and again once it is dropped, in the order of
    the stream that it was allocated on.  Outputs are the given stream's then; the inputs have to be ready on it."""
    at = list(inspect.signature(helper).parameters).index("stream")

    @functools.wraps(helper)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return helper(*args, **kw)
        with torch.cuda.stream(_stream_of(stream)):
            return helper(*args, **kw)

    return call


def _stream_of(stream):
    """torch's stream of a stream or a cudaStream_t handle (0 and 1 name the default stream)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream)) if int(stream) > 1 else torch.cuda.default_stream()


class Quantized:
    """NVFP4 tensor: codes [rows, k/2] uint8, sf (layout bytes), g and amax (one fp32 each, on device)."""

    def __init__(self, codes, sf, g, amax, rows, k, layout):
        self.codes, self.sf, self.g, self.amax = codes, sf, g, amax
        self.rows, self.k, self.layout = rows, k, layout


def empty_quantized(rows: int, k: int, layout: int = SF_TCGEN05, device="cuda") -> Quantized:
    codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=device)
    sf = torch.empty(max(1, nvfp4_sf_bytes(rows, k, layout)), dtype=torch.uint8, device=device)
    scal = torch.empty(8, dtype=torch.float32, device=device)
    return Quantized(codes, sf, scal[0:1], scal[4:5], rows, k, layout)


@_on_its_stream
def quantize(x: torch.Tensor, layout: int = SF_TCGEN05, out: Quantized | None = None, amax=None,
             stream=None) -> Quantized:
    """bf16 [rows, k] (row pitch x.stride(0)) -> NVFP4.  ``amax`` (device fp32) skips the amax pass."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    q = out if out is not None else empty_quantized(rows, k, layout, x.device)
    if amax is not None:
        q.amax.copy_(amax)
    nvfp4_quantize(x, rows, k, x.stride(0), q.codes, q.sf, layout, q.g, q.amax, 1 if amax is not None else 0,
                   stream)
    return q


@_on_its_stream
def quantize_stochastic(x: torch.Tensor, seed: int, offset: int, layout: int = SF_TCGEN05,
                        out: Quantized | None = None, amax=None, stream=None) -> Quantized:
    """bf16 [rows, k] -> NVFP4 with stochastically rounded codes (Philox4x32-10 bits from seed, offset)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    q = out if out is not None else empty_quantized(rows, k, layout, x.device)
    if amax is not None:
        q.amax.copy_(amax)
    nvfp4_quantize_stochastic(x, rows, k, x.stride(0), q.codes, q.sf, layout, q.g, q.amax,
                              1 if amax is not None else 0, seed, offset, stream)
    return q


@_on_its_stream
def quantize_hadamard(x: torch.Tensor, order: int, layout: int = SF_TCGEN05, out: Quantized | None = None,
                      amax=None, stream=None) -> Quantized:
    """bf16 [rows, k] -> NVFP4 of y = x H (block-diagonal Walsh-Hadamard of the given order over
    sqrt(order)).  ``amax`` (device fp32, max |y|) skips the amax pass."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    q = out if out is not None else empty_quantized(rows, k, layout, x.device)
    if amax is not None:
        q.amax.copy_(amax)
    nvfp4_quantize_hadamard(x, rows, k, x.stride(0), order, q.codes, q.sf, layout, q.g, q.amax,
                            1 if amax is not None else 0, stream)
    return q


@_on_its_stream
def quantize_hadamard_stochastic(x: torch.Tensor, order: int, seed: int, offset: int, layout: int = SF_TCGEN05,
                                 out: Quantized | None = None, amax=None, stream=None) -> Quantized:
    """bf16 [rows, k] -> NVFP4 of y = x H with stochastically rounded codes."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    q = out if out is not None else empty_quantized(rows, k, layout, x.device)
    if amax is not None:
        q.amax.copy_(amax)
    nvfp4_quantize_hadamard_stochastic(x, rows, k, x.stride(0), order, q.codes, q.sf, layout, q.g, q.amax,
                                       1 if amax is not None else 0, seed, offset, stream)
    return q


@_on_its_stream
def gemm(a: Quantized, b: Quantized, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """D [M, N] = alpha (s_a A)(s_b B)^T for two TCGEN05-layout NVFP4 operands."""
    assert a.layout == SF_TCGEN05 and b.layout == SF_TCGEN05 and a.k == b.k
    od = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    d = out if out is not None else torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    nvfp4_gemm(a.codes, a.sf, a.g, b.codes, b.sf, b.g, a.rows, b.rows, a.k, d, d.stride(0), od, stream)
    return d


@_on_its_stream
def gemm_requant(a: Quantized, b: Quantized, g_d: torch.Tensor, layout: int = SF_TCGEN05,
                 out: Quantized | None = None, stream=None) -> Quantized:
    """D = alpha (s_a A)(s_b B)^T quantized to NVFP4 under the given encode
    scale g_d (one fp32 on the device); out.amax receives max |D|."""
    assert a.layout == SF_TCGEN05 and b.layout == SF_TCGEN05 and a.k == b.k
    q = out if out is not None else empty_quantized(a.rows, b.rows, layout, a.codes.device)
    q.g.copy_(g_d.reshape(1))
    nvfp4_gemm_requant(a.codes, a.sf, a.g, b.codes, b.sf, b.g, a.rows, b.rows, a.k, q.g, q.codes,
                       q.codes.stride(0), q.sf, q.layout, q.amax, stream)
    return q


@_on_its_stream
def gemm_fp8_out(a: Quantized, b: Quantized, g_d: torch.Tensor, out: torch.Tensor | None = None,
                 amax_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """FP8 (float8_e4m3fn) e4m3(v * g_d) for v = alpha (s_a A)(s_b B)^T; amax_out receives max |v|."""
    assert a.layout == SF_TCGEN05 and b.layout == SF_TCGEN05 and a.k == b.k
    d = out if out is not None else torch.empty((a.rows, b.rows), dtype=torch.float8_e4m3fn, device=a.codes.device)
    nvfp4_gemm_fp8_out(a.codes, a.sf, a.g, b.codes, b.sf, b.g, a.rows, b.rows, a.k, g_d, d, d.stride(0), amax_out,
                       stream)
    return d


@_on_its_stream
def gemv_batched(x: torch.Tensor, w: Quantized, out: torch.Tensor | None = None, workspace=None,
                 stream=None) -> torch.Tensor:
    """y [M, N] for bf16 activations x [M, K] (M <= 32) and NVFP4 weights w [N, K]."""
    m, k = x.shape
    n = w.rows
    ws_bytes = nvfp4_workspace_bytes(OP_GEMV_BATCHED, m, n, k)
    ws = workspace if workspace is not None else torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    nvfp4_gemv_batched(x, m, x.stride(0), w.codes, w.sf, w.g, n, k, y, y.stride(0), ws, ws.numel(), stream)
    return y


@_on_its_stream
def gemm_quant_a(a: torch.Tensor, b: Quantized, out_dtype=torch.bfloat16, out=None, workspace=None,
                 stream=None, amax: torch.Tensor | None = None) -> torch.Tensor:
    """D = A_q @ B_q^T with a bf16 A quantized inside the call; amax: A's tensor
    amax already on the device (1-element fp32), which skips the amax pass."""
    m, k = a.shape
    n = b.rows
    ws_bytes = nvfp4_workspace_bytes(OP_GEMM_QUANT_A, m, n, k)
    ws = workspace if workspace is not None else torch.empty(ws_bytes, dtype=torch.uint8, device=a.device)
    od = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    d = out if out is not None else torch.empty((m, n), dtype=out_dtype, device=a.device)
    if amax is None:
        nvfp4_gemm_quant_a(a, a.stride(0), b.codes, b.sf, b.g, m, n, k, d, d.stride(0), od, ws, ws.numel(), stream)
    else:
        nvfp4_gemm_quant_a_amax(a, a.stride(0), amax, b.codes, b.sf, b.g, m, n, k, d, d.stride(0), od, ws,
                                ws.numel(), stream)
    return d


def quant_a_workspace_views(ws: torch.Tensor, m: int, k: int):
    """A's codes [m, k/2], its tensor-core scales and g_a (1-element fp32) inside a
    gemm_quant_a workspace (the layout include/nvfp4.h states)."""
    codes_bytes = m * (k // 2)
    sf_off = (codes_bytes + 255) // 256 * 256
    sf_bytes = nvfp4_sf_bytes(m, k, SF_TCGEN05)
    g_off = sf_off + (sf_bytes + 255) // 256 * 256
    return (ws[:codes_bytes].view(m, k // 2), ws[sf_off:sf_off + sf_bytes],
            ws[g_off:g_off + 4].view(torch.float32))


class MXQuantized:
    """MXFP4 tensor: codes [rows, k/2] uint8 and E8M0 scales (layout bytes); no global scale."""

    def __init__(self, codes, sf, rows, k, layout):
        self.codes, self.sf = codes, sf
        self.rows, self.k, self.layout = rows, k, layout


@_on_its_stream
def mxfp4_quantize(x: torch.Tensor, layout: int = SF_TCGEN05, out: MXQuantized | None = None,
                   stream=None) -> MXQuantized:
    """bf16 [rows, k] (row pitch x.stride(0)) -> MXFP4 (one pass)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, k = x.shape
    if out is None:
        codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=x.device)
        sf = torch.empty(max(1, nvfp4_mxfp4_sf_bytes(rows, k, layout)), dtype=torch.uint8, device=x.device)
        out = MXQuantized(codes, sf, rows, k, layout)
    nvfp4_mxfp4_quantize(x, rows, k, x.stride(0), out.codes, out.sf, layout, stream)
    return out


@_on_its_stream
def mxfp4_gemm(a: MXQuantized, b: MXQuantized, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """D [M, N] = (s_a A)(s_b B)^T for two TCGEN05-layout MXFP4 operands."""
    assert a.layout == SF_TCGEN05 and b.layout == SF_TCGEN05 and a.k == b.k
    od = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    d = out if out is not None else torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    nvfp4_mxfp4_gemm(a.codes, a.sf, b.codes, b.sf, a.rows, b.rows, a.k, d, d.stride(0), od, stream)
    return d


# ---------------------------------------------------------------------------
# layer norm and the product epilogues
# ---------------------------------------------------------------------------
ACTIVATIONS = {None: ACT_NONE, "none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH,
               "silu": ACT_SILU}


def _dtype_of(t) -> int:
    """nvfp4_dtype of a tensor (bf16 for None, where the library reads nothing)."""
    if t is None:
        return DTYPE_BF16
    assert t.dtype in (torch.bfloat16, torch.float32), t.dtype
    return DTYPE_F32 if t.dtype == torch.float32 else DTYPE_BF16


def _rows_of(t, shape=None):
    """Row pitch of a row-major matrix.  Rows may not overlap (a broadcast's pitch is 0): the library takes rows times
    pitch elements of memory.  The stride of a single row says nothing."""
    assert t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1), "a row-major matrix"
    assert shape is None or tuple(t.shape) == tuple(shape), (tuple(t.shape), tuple(shape))
    if t.shape[0] <= 1:
        return t.shape[1]
    assert t.stride(0) >= t.shape[1], f"rows that overlap: a pitch of {t.stride(0)} for {t.shape[1]} columns"
    return t.stride(0)


def _apart(out, *inputs):
    """Outputs that would be written while the kernels still read these inputs (columns of one buffer are apart)."""
    assert all(out.data_ptr() != t.data_ptr() or out.numel() == 0 for t in inputs), "not in place: out is an input that is still read"


class Normalized:
    """Result of layernorm: y [rows, k], mean and rstd [rows] fp32, amax (max |y|, one fp32) for quantize(y, amax=)."""

    def __init__(self, y, mean, rstd, amax):
        self.y, self.mean, self.rstd, self.amax = y, mean, rstd, amax


@_on_its_stream
def layernorm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
              eps: float = 1e-5, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
              stream=None) -> Normalized:
    """Layer norm of x [rows, k] (bf16 or fp32), not in place; weight and bias [k] of one dtype.  The amax makes the
    quantizer behind it a single pass: ``quantize(n.y, amax=n.amax)``."""
    rows, k = x.shape
    ldx = _rows_of(x)
    for t in (weight, bias):
        assert t is None or (t.shape == (k,) and t.is_contiguous()), "contiguous [k] weight and bias"
    assert weight is None or bias is None or weight.dtype == bias.dtype, "weight and bias of one dtype"
    y = out if out is not None else torch.empty((rows, k), dtype=out_dtype, device=x.device)
    _apart(y, x)
    stats = torch.empty(2 * rows + 1, dtype=torch.float32, device=x.device)
    mean, rstd, amax = stats[:rows], stats[rows:2 * rows], stats[2 * rows:]
    nvfp4_layernorm(x, _dtype_of(x), rows, k, ldx, weight, bias, _dtype_of(weight if weight is not None else bias), eps,
                    y, _dtype_of(y), _rows_of(y, (rows, k)), mean, rstd, amax, stream)
    return Normalized(y, mean, rstd, amax)


@_on_its_stream
def layernorm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                       weight: torch.Tensor | None = None, d_residual: torch.Tensor | None = None,
                       out: torch.Tensor | None = None, workspace=None, stream=None):
    """(dx, dweight, dbias, amax of dx): dx in x's dtype with d_residual added (out may be d_residual), dweight and dbias
    fp32."""
    rows, k = x.shape
    for t in (mean, rstd):
        assert t.shape == (rows,) and t.dtype == torch.float32 and t.is_contiguous(), "mean and rstd of the forward call"
    assert weight is None or (weight.shape == (k,) and weight.is_contiguous()), "contiguous [k] weight"
    assert d_residual is None or d_residual.dtype == x.dtype, "d_residual in x's dtype"
    dx = out if out is not None else torch.empty((rows, k), dtype=x.dtype, device=x.device)
    assert dx.dtype == x.dtype, "dx in x's dtype"
    _apart(dx, dy, x)
    grads = torch.empty(2 * k + 1, dtype=torch.float32, device=x.device)
    ws_bytes = nvfp4_workspace_bytes(OP_LAYERNORM_BACKWARD, rows, k, 0)
    ws = workspace if workspace is not None else torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    nvfp4_layernorm_backward(dy, _dtype_of(dy), _rows_of(dy, (rows, k)), x, _dtype_of(x), _rows_of(x), mean, rstd, weight,
                             _dtype_of(weight), d_residual, 0 if d_residual is None else _rows_of(d_residual, (rows, k)),
                             rows, k, dx, _rows_of(dx, (rows, k)), grads[:k], grads[k:2 * k], grads[2 * k:], ws,
                             ws.numel(), stream)
    return dx, grads[:k], grads[k:2 * k], grads[2 * k:]


def _check_epilogue(m, n, bias, residual, dtype) -> int:
    assert bias is None or (bias.shape == (n,) and bias.is_contiguous()), "contiguous [n] bias"
    assert residual is None or residual.dtype == dtype, "residual in the output's dtype"
    return 0 if residual is None else _rows_of(residual, (m, n))


@_on_its_stream
def gemm_epilogue(a: Quantized, b: Quantized, bias: torch.Tensor | None = None, act: str | None = None,
                  residual: torch.Tensor | None = None, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                  pre: torch.Tensor | bool = False, amax: torch.Tensor | None = None, stream=None):
    """D = act(alpha (s_a A)(s_b B)^T + bias) + residual.  pre: a tensor (or True: a new one, returned as
    (D, pre)) for the value before act; amax: one fp32 on the device that receives max |D|."""
    assert a.layout == SF_TCGEN05 and b.layout == SF_TCGEN05 and a.k == b.k
    m, n = a.rows, b.rows
    d = out if out is not None else torch.empty((m, n), dtype=out_dtype, device=a.codes.device)
    p = torch.empty((m, n), dtype=d.dtype, device=d.device) if pre is True else (None if pre is False else pre)
    assert p is None or p.dtype == d.dtype, "pre in the output's dtype"
    ldr = _check_epilogue(m, n, bias, residual, d.dtype)
    nvfp4_gemm_epilogue(a.codes, a.sf, a.g, b.codes, b.sf, b.g, m, n, a.k, bias, _dtype_of(bias), ACTIVATIONS[act],
                        residual, ldr, d, _rows_of(d, (m, n)), _dtype_of(d), p, 0 if p is None else _rows_of(p, (m, n)),
                        amax, stream)
    return (d, p) if pre is True else d


@_on_its_stream
def gemv_batched_epilogue(x: torch.Tensor, w: Quantized, bias: torch.Tensor | None = None, act: str | None = None,
                          residual: torch.Tensor | None = None, out: torch.Tensor | None = None, workspace=None,
                          stream=None) -> torch.Tensor:
    """y [M, N] = act(x w^T + bias) + residual for bf16 activations x [M, K] (M <= 32) and NVFP4 weights w; out may be
    residual, not x."""
    assert x.dtype == torch.bfloat16 and x.shape[1] == w.k and w.layout == SF_TCGEN05
    m, k = x.shape
    n = w.rows
    ws_bytes = nvfp4_workspace_bytes(OP_GEMV_BATCHED, m, n, k)
    ws = workspace if workspace is not None else torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    assert y.dtype == torch.bfloat16
    _apart(y, x)
    ldr = _check_epilogue(m, n, bias, residual, y.dtype)
    nvfp4_gemv_batched_epilogue(x, m, _rows_of(x), w.codes, w.sf, w.g, n, k, bias, _dtype_of(bias), ACTIVATIONS[act],
                                residual, ldr, y, _rows_of(y, (m, n)), ws, ws.numel(), stream)
    return y


@_on_its_stream
def epilogue_backward(dd: torch.Tensor, pre: torch.Tensor | None, act: str | None = None,
                      out: torch.Tensor | None = None, workspace=None, stream=None):
    """(dpre, dbias, amax of dpre) of D = act(pre) [+ residual], pre = product + bias; dbias fp32."""
    m, n = dd.shape
    assert pre is None or pre.dtype == dd.dtype, "pre in dd's dtype"
    dpre = out if out is not None else torch.empty((m, n), dtype=dd.dtype, device=dd.device)
    assert dpre.dtype == dd.dtype, "dpre in dd's dtype"
    grads = torch.empty(n + 1, dtype=torch.float32, device=dd.device)
    ws_bytes = nvfp4_workspace_bytes(OP_EPILOGUE_BACKWARD, m, n, 0)
    ws = workspace if workspace is not None else torch.empty(ws_bytes, dtype=torch.uint8, device=dd.device)
    nvfp4_epilogue_backward(dd, _rows_of(dd), pre, 0 if pre is None else _rows_of(pre, (m, n)), _dtype_of(dd),
                            ACTIVATIONS[act], m, n, dpre, _rows_of(dpre, (m, n)), grads[:n], grads[n:], ws, ws.numel(),
                            stream)
    return dpre, grads[:n], grads[n:]
