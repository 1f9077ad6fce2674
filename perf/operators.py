"""Layer norm, the GEMM and GEMV with bias, activation and residual in their epilogue, and the
gradients of both, as they run in a transformer block around the NVFP4 products:

    y = layernorm(x)                       -> quantize(y, amax of y)
    h = act(y_q W1^T + b1)                 -> quantize(h, amax of h)     (the value before act kept for training)
    x = (h_q W2^T + b2) + x                (the residual stream)
    backward: d(pre) = d(h) act'(pre), d(b1) = column sums; layernorm backward + the residual stream's gradient

`run` computes a case in plain torch (own == False) or through the library's entry points
(own == True); `exact` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
LN, LN_BWD, GEMM, GEMV, ACT_BWD = "layernorm", "layernorm_backward", "gemm_epilogue", "gemv_epilogue", "epilogue_backward"
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a small batch: 8 tokens of an 8192-wide model; latency is all
        dict(name="ln_decode", op=LN, rows=8, k=8192, x="bf16", y="bf16", p="bf16", pad=0),
        # prefill or training: the residual stream of 16384 tokens, as the quantizer's own workload
        dict(name="ln_tokens", op=LN, rows=16384, k=8192, x="bf16", y="bf16", p="bf16", pad=0),
        # an fp32 residual stream of odd width and odd pitch (no 16-byte alignment anywhere)
        dict(name="ln_odd", op=LN, rows=3001, k=1155, x="f32", y="bf16", p="f32", pad=2),
        # training: backward of the block's norm, with the gradient that arrives along the residual stream
        dict(name="ln_bwd_tokens", op=LN_BWD, rows=16384, k=8192, dy="bf16", x="bf16", p="bf16", res=True, pad=0),
        # the same at an odd width, fp32 stream, bf16 gradient from the product behind
        dict(name="ln_bwd_odd", op=LN_BWD, rows=1537, k=1155, dy="bf16", x="f32", p="f32", res=True, pad=2),
        # MLP up projection in training: bias + GELU, the value before GELU kept, amax for the quantizer behind
        dict(name="gemm_up", op=GEMM, m=4096, n=28672, k=8192, act="gelu_tanh", bias="bf16", res=False, pre=True,
             out="bf16", pad=0),
        # MLP down projection (the long-K workload): bias and residual stream
        dict(name="gemm_down", op=GEMM, m=4096, n=8192, k=28672, act="none", bias="bf16", res=True, pre=False,
             out="bf16", pad=0),
        # a short ragged batch, fp32 out, everything at once
        dict(name="gemm_ragged", op=GEMM, m=301, n=1001, k=2112, act="silu", bias="f32", res=True, pre=True,
             out="f32", pad=3),
        # decoding one token: up projection
        dict(name="gemv_up", op=GEMV, m=1, n=28672, k=8192, act="gelu", bias="bf16", res=False),
        # decoding 16 tokens: square projection back onto the residual stream
        dict(name="gemv_res", op=GEMV, m=16, n=8192, k=8192, act="none", bias="f32", res=True),
        # training: gradient through the up projection's bias and GELU
        dict(name="act_bwd_up", op=ACT_BWD, m=4096, n=28672, act="gelu_tanh", t="bf16", pad=0),
        # a ragged batch of an odd width in fp32
        dict(name="act_bwd_odd", op=ACT_BWD, m=777, n=1001, act="silu", t="f32", pad=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice([LN, LN_BWD, GEMM, GEMV, ACT_BWD])
    act = rng.choice(list(ACTS))
    if op in (LN, LN_BWD):
        k = _log(rng, 16, 28672)
        if rng.random() < 0.6:
            k = max(16, k // 16 * 16)
        rows = _log(rng, 1, min(32768, 16384 * 8192 // k))
        c = dict(op=op, rows=rows, k=k, x=rng.choice(["bf16", "bf16", "f32"]), p=rng.choice(["bf16", "f32"]),
                 pad=rng.choice([0, 0, 8, 1]))
        if c["x"] == "f32" and rows * k > 8192 * 8192:
            c["x"] = "bf16"
        if op == LN:
            return dict(c, y=rng.choice(["bf16", "bf16", "f32"]))
        return dict(c, dy=rng.choice(["bf16", c["x"]]), res=rng.random() < 0.5)
    if op == GEMM:
        n, k = _log(rng, 16, 28672), 64 * _log(rng, 1, 448)
        m = _log(rng, 1, max(1, min(8192, 4096 * 28672 * 8192 // (n * k), 4096 * 28672 // n)))
        out = "f32" if m * n <= 2048 * 28672 and rng.random() < 0.3 else "bf16"
        return dict(op=op, m=m, n=n, k=k, act=act, bias=rng.choice(["bf16", "f32"]), res=rng.random() < 0.5,
                    pre=rng.random() < 0.4, out=out, pad=rng.choice([0, 0, 8, 1]))
    if op == GEMV:
        return dict(op=op, m=_log(rng, 1, 32), n=_log(rng, 64, 28672), k=64 * _log(rng, 4, 256), act=act,
                    bias=rng.choice(["bf16", "f32"]), res=rng.random() < 0.5)
    n = _log(rng, 1, 28672)
    m = _log(rng, 1, min(32768, 4096 * 28672 // n))
    t = "f32" if m * n <= 2048 * 28672 and rng.random() < 0.4 else "bf16"
    return dict(op=op, m=m, n=n, act=act, t=t, pad=rng.choice([0, 0, 8, 1]))


def work(case):
    size = {"bf16": 2, "f32": 4}
    op = case["op"]
    if op == LN:
        n = case["rows"] * case["k"]
        return {"bytes": n * (size[case["x"]] + size[case["y"]]) + 2 * case["k"] * size[case["p"]] + 8 * case["rows"] + 4,
                "flops": 8 * n}
    if op == LN_BWD:
        n = case["rows"] * case["k"]
        b = n * (size[case["dy"]] + size[case["x"]] * (3 if case["res"] else 2))
        return {"bytes": b + case["k"] * (size[case["p"]] + 8) + 8 * case["rows"] + 4, "flops": 14 * n}
    if op in (GEMM, GEMV):
        m, n, k = case["m"], case["n"], case["k"]
        o = size[case["out"]] if op == GEMM else 2
        tensors = 1 + bool(case["res"]) + bool(case.get("pre"))
        a = m * k * 9 // 16 if op == GEMM else m * k * 2
        return {"bytes": a + n * k * 9 // 16 + m * n * o * tensors + n * size[case["bias"]] + 12,
                "flops": 2 * m * n * k + 10 * m * n}
    n = case["m"] * case["n"]
    return {"bytes": 3 * n * size[case["t"]] + 4 * case["n"] + 4, "flops": 15 * n}


# ---------------------------------------------------------------------------
# what a user's program holds before the call
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, k):
    """N(0, 1) with a few outlier channels, each channel about a mean of its own."""
    x = _randn(g, rows, k)
    out = torch.rand(k, generator=g, device="cuda") < 0.01
    x *= torch.where(out, 30.0, 1.0)
    x += 0.3 * _randn(g, k)
    return x


def _pitched(t, dtype, pad):
    """t in `dtype` inside rows of k + pad elements."""
    buf = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def _one(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def _encode(x):
    """The quantizer's rule on bf16 x [rows, k], every fp32 step rounded once: the global scale g, the
    block scales as E4M3, and the code number (0..7, sign apart) of each element."""
    rows, k = x.shape
    x = x.float().reshape(rows, k // 16, 16)
    g = _one(2688.0) / x.abs().amax()
    s = ((x.abs().amax(2) * g) / _one(6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float().unsqueeze(2)
    u = torch.where(d > 0, (x * g) / d, _one(0.0))
    a = u.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code += 8 * torch.signbit(u).to(torch.uint8)
    return code.reshape(rows, k), s, g


def _quantized(x):
    """(codes [rows, k/2], scales in the tensor core's layout, g) of bf16 x: what a program keeps of its weights."""
    code, s, g = _encode(x)
    rows, k = x.shape
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    rp, kb = (rows + 127) // 128 * 128, k // 16
    full = torch.zeros((rp, kb), dtype=torch.uint8, device="cuda")
    full[:rows] = s.view(torch.uint8)
    sf = full.reshape(rp // 128, 4, 32, kb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)
    return codes.contiguous(), sf, g.reshape(1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case, op=op)
    if op in (LN, LN_BWD):
        rows, k, p = case["rows"], case["k"], DTYPES[case["p"]]
        x = _pitched(_activations(g, rows, k), DTYPES[case["x"]], case["pad"])
        s.update(x=x, gamma=(1.0 + 0.1 * _randn(g, k)).to(p), beta=(0.1 * _randn(g, k)).to(p))
        if op == LN_BWD:
            x64 = x.double()
            mean = x64.mean(1)
            rstd = ((x64 - mean[:, None]).square().mean(1) + EPS).rsqrt()
            s.update(mean=mean.float(), rstd=rstd.float(),
                     dy=_pitched(0.02 * _randn(g, rows, k), DTYPES[case["dy"]], case["pad"]),
                     res=_pitched(0.02 * _randn(g, rows, k), DTYPES[case["x"]], case["pad"]) if case["res"] else None)
        return s
    if op == ACT_BWD:
        m, n, t = case["m"], case["n"], DTYPES[case["t"]]
        s.update(pre=_pitched(1.5 * _randn(g, m, n), t, case["pad"]), dd=_pitched(0.02 * _randn(g, m, n), t, case["pad"]))
        return s
    m, n, k = case["m"], case["n"], case["k"]
    x = _activations(g, m, k).bfloat16()
    w = (0.02 * math.sqrt(8192 / k) * _randn(g, n, k)).bfloat16()
    s.update(w=_quantized(w), bias=(0.5 * _randn(g, n)).to(DTYPES[case["bias"]]))
    if op == GEMV:
        s.update(x=x, res=_randn(g, m, n).bfloat16() if case["res"] else None)
    else:
        s.update(a=_quantized(x), res=_pitched(_randn(g, m, n), DTYPES[case["out"]], case["pad"]) if case["res"] else None)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _act_grad(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * v * v)
    if act == "silu":
        e = 1.0 / (1.0 + torch.exp(-v))
        return e * (1.0 + v * (1.0 - e))
    return torch.ones_like(v)


_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _decoded(q):
    """s * code of (codes, scales, g) in fp32, [rows, k]; the product is exact."""
    codes, sf, _ = q
    rows, k = codes.shape[0], codes.shape[1] * 2
    table = torch.tensor(_VALUES + [-v for v in _VALUES], dtype=torch.float32, device="cuda")
    v = table[torch.stack((codes & 15, codes >> 4), 2).reshape(rows, k).int()]
    scales = sf.reshape(-1, k // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, k // 16)[:rows]
    return (v.reshape(rows, k // 16, 16) * scales.view(torch.float8_e4m3fn).float().unsqueeze(2)).reshape(rows, k)


def _amax(t):
    return t.float().abs().amax().reshape(1)


def _plain(s):
    c, op = s["case"], s["op"]
    if op == LN:
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1.0 / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)
        y = (d * rstd * s["gamma"].float() + s["beta"].float()).to(DTYPES[c["y"]])
        return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0], "amax": _amax(y)}
    if op == LN_BWD:
        rstd = s["rstd"][:, None]
        xh = (s["x"].float() - s["mean"][:, None]) * rstd
        dy = s["dy"].float()
        a = dy * s["gamma"].float()
        dx = rstd * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
        if s["res"] is not None:
            dx = dx + s["res"].float()
        dx = dx.to(DTYPES[c["x"]])
        return {"dx": dx, "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0), "amax": _amax(dx)}
    if op == ACT_BWD:
        d = s["dd"].float() * _act_grad(s["pre"].float(), c["act"])
        dpre = d.to(DTYPES[c["t"]])
        return {"dpre": dpre, "dbias": d.sum(0), "amax": _amax(dpre)}
    if op == GEMV:
        code, sc, g_a = _encode(s["x"])
        table = torch.tensor(_VALUES + [-v for v in _VALUES], dtype=torch.float32, device="cuda")
        a = (table[code.int()].reshape(*sc.shape, 16) * sc.float().unsqueeze(2)).reshape(code.shape)
        out = torch.bfloat16
    else:
        a, g_a, out = _decoded(s["a"]), s["a"][2], DTYPES[c["out"]]
    alpha = _one(1.0) / (g_a * s["w"][2])
    v = torch.matmul(a, _decoded(s["w"]).t()) * alpha + s["bias"].float()
    d = _act(v, c["act"])
    if s["res"] is not None:
        d = d + s["res"].float()
    d = d.to(out)
    if op == GEMV:
        return {"d": d}
    return {"d": d, "pre": v.to(out) if c["pre"] else None, "amax": _amax(d)}


def _dtype(t):
    return 1 if t.dtype == torch.float32 else 0


def _empty_like_pitched(rows, k, dtype, pad):
    return torch.empty((rows, k + pad), dtype=dtype, device="cuda")[:, :k]


def _buffers(s, nv):
    """Outputs and workspace that a program allocates once and keeps."""
    c, op = s["case"], s["op"]
    f32 = dict(dtype=torch.float32, device="cuda")
    if op == LN:
        return dict(y=_empty_like_pitched(c["rows"], c["k"], DTYPES[c["y"]], c["pad"]), mean=torch.empty(c["rows"], **f32),
                    rstd=torch.empty(c["rows"], **f32), amax=torch.empty(1, **f32))
    if op == LN_BWD:
        ws = nv.nvfp4_workspace_bytes(nv.OP_LAYERNORM_BACKWARD, c["rows"], c["k"], 0)
        return dict(dx=_empty_like_pitched(c["rows"], c["k"], DTYPES[c["x"]], c["pad"]), dgamma=torch.empty(c["k"], **f32),
                    dbeta=torch.empty(c["k"], **f32), amax=torch.empty(1, **f32),
                    ws=torch.empty(ws, dtype=torch.uint8, device="cuda"))
    if op == ACT_BWD:
        ws = nv.nvfp4_workspace_bytes(nv.OP_EPILOGUE_BACKWARD, c["m"], c["n"], 0)
        return dict(dpre=_empty_like_pitched(c["m"], c["n"], DTYPES[c["t"]], c["pad"]), dbias=torch.empty(c["n"], **f32),
                    amax=torch.empty(1, **f32), ws=torch.empty(ws, dtype=torch.uint8, device="cuda"))
    if op == GEMV:
        ws = nv.nvfp4_workspace_bytes(nv.OP_GEMV_BATCHED, c["m"], c["n"], c["k"])
        return dict(d=torch.empty((c["m"], c["n"]), dtype=torch.bfloat16, device="cuda"),
                    ws=torch.empty(ws, dtype=torch.uint8, device="cuda"))
    t = DTYPES[c["out"]]
    return dict(d=_empty_like_pitched(c["m"], c["n"], t, c["pad"]),
                pre=_empty_like_pitched(c["m"], c["n"], t, c["pad"]) if c["pre"] else None, amax=torch.empty(1, **f32))


def _pitch(t):
    return t.stride(0) if t is not None else 0


def _own(s):
    from nvfp4_block_scaled_15_b200 import nvfp4 as nv
    if "buffers" not in s:
        s["buffers"] = _buffers(s, nv)
    c, op, b = s["case"], s["op"], s["buffers"]
    if op == LN:
        x, y, gamma = s["x"], b["y"], s["gamma"]
        nv.nvfp4_layernorm(x, _dtype(x), c["rows"], c["k"], x.stride(0), gamma, s["beta"], _dtype(gamma), EPS, y, _dtype(y),
                           y.stride(0), b["mean"], b["rstd"], b["amax"])
        return {"y": y, "mean": b["mean"], "rstd": b["rstd"], "amax": b["amax"]}
    if op == LN_BWD:
        dy, x, dx, res, gamma = s["dy"], s["x"], b["dx"], s["res"], s["gamma"]
        nv.nvfp4_layernorm_backward(dy, _dtype(dy), dy.stride(0), x, _dtype(x), x.stride(0), s["mean"], s["rstd"], gamma,
                                    _dtype(gamma), res, _pitch(res), c["rows"], c["k"], dx, dx.stride(0), b["dgamma"],
                                    b["dbeta"], b["amax"], b["ws"], b["ws"].numel())
        return {"dx": dx, "dgamma": b["dgamma"], "dbeta": b["dbeta"], "amax": b["amax"]}
    if op == ACT_BWD:
        dd, pre, dpre = s["dd"], s["pre"], b["dpre"]
        nv.nvfp4_epilogue_backward(dd, dd.stride(0), pre, pre.stride(0), _dtype(pre), ACTS[c["act"]], c["m"], c["n"], dpre,
                                   dpre.stride(0), b["dbias"], b["amax"], b["ws"], b["ws"].numel())
        return {"dpre": dpre, "dbias": b["dbias"], "amax": b["amax"]}
    w, g_w, w_sf = s["w"][0], s["w"][2], s["w"][1]
    bias, res, d = s["bias"], s["res"], b["d"]
    if op == GEMV:
        nv.nvfp4_gemv_batched_epilogue(s["x"], c["m"], c["k"], w, w_sf, g_w, c["n"], c["k"], bias, _dtype(bias),
                                       ACTS[c["act"]], res, _pitch(res), d, d.stride(0), b["ws"], b["ws"].numel())
        return {"d": d}
    a, a_sf, g_a = s["a"]
    nv.nvfp4_gemm_epilogue(a, a_sf, g_a, w, w_sf, g_w, c["m"], c["n"], c["k"], bias, _dtype(bias), ACTS[c["act"]], res,
                           _pitch(res), d, d.stride(0), _dtype(d), b["pre"], _pitch(b["pre"]), b["amax"])
    return {"d": d, "pre": b["pre"], "amax": b["amax"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _grid(v, mantissa, least, top):
    """v >= 0 rounded to nearest even onto a small float's values (mantissa bits, least normal exponent, largest value)."""
    e = torch.frexp(v.clamp(min=2.0 ** least))[1].double() - 1.0
    q = torch.exp2(e - mantissa)
    return (torch.round(v / q) * q).clamp(max=top)


def _values64(codes, sf, cols=None):
    """scale * value of the codes from their bits, [rows, k] in 64 bits."""
    rows, kb = codes.shape[0], codes.shape[1] // 8
    r = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(kb, device="cuda")[None, :]
    at = 512 * ((r // 128) * (kb // 4) + b // 4) + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    byte = sf[at].int()
    e, f = (byte >> 3) & 15, (byte & 7).double()
    scale = torch.where(e > 0, (8.0 + f) * torch.exp2(e.double() - 10.0), f * 2.0 ** -9)
    nib = torch.stack((codes & 15, codes >> 4), 2).reshape(rows, kb, 16).int()
    e, f = (nib >> 1) & 3, (nib & 1).double()
    v = torch.where(e > 0, (2.0 + f) * torch.exp2(e.double() - 2.0), 0.5 * f)
    return (torch.where(nib >= 8, -v, v) * scale[:, :, None]).reshape(rows, kb * 16)


def _quantized64(x):
    """The quantizer's definition: its fp32 roundings are part of it (a 64-bit quotient of fp32 values rounds to fp32 as
    the fp32 quotient does), the E4M3 and E2M1 roundings are on their grids."""
    rows, k = x.shape
    x = x.double().reshape(rows, k // 16, 16)
    g = (2688.0 / x.abs().amax()).float().double()
    t = (x.abs().amax(2) * g).float().double()
    scale = _grid((t / 6.0).float().double(), 3, -6, 448.0)[:, :, None]
    t = (x * g).float().double()
    u = torch.where(scale > 0, (t / scale).float().double(), 0.0)
    return (torch.sign(u) * _grid(u.abs(), 1, 0, 6.0) * scale).reshape(rows, k), g


def _act64(v, act):
    if act == "gelu":
        return v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v.clamp(min=0.0) if act == "relu" else v


def _act_grad64(v, act):
    if act == "gelu":
        return 0.5 * torch.special.erfc(-v / math.sqrt(2.0)) + v * torch.exp(-v * v / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        u = 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
        p = torch.sigmoid(u)
        return p + v * p * torch.sigmoid(-u) * 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * v * v)
    if act == "silu":
        p = torch.sigmoid(v)
        return p + v * p * torch.sigmoid(-v)
    return (v > 0).double() if act == "relu" else torch.ones_like(v)


def _stored_amax(t, dtype):
    return t.to(dtype).double().abs().max().reshape(1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in (LN, LN_BWD):
        k = case["k"]
        x, gamma = s["x"].double(), s["gamma"].double()
        if op == LN:
            mean = x.sum(1) / k
            x -= mean[:, None]
            rstd = (torch.einsum("rk,rk->r", x, x) / k + EPS) ** -0.5
            y = torch.addcmul(s["beta"].double(), x * rstd[:, None], gamma)
            return {"y": y, "mean": mean, "rstd": rstd, "amax": _stored_amax(y, DTYPES[case["y"]])}
        rstd = s["rstd"].double()
        xh = (x - s["mean"].double()[:, None]) * rstd[:, None]
        dy = s["dy"].double()
        c1 = torch.mv(dy, gamma) / k
        c2 = torch.mv(dy * xh, gamma) / k
        dx = (dy * gamma - c1[:, None] - xh * c2[:, None]) * rstd[:, None]
        if s["res"] is not None:
            dx += s["res"].double()
        return {"dx": dx, "dgamma": torch.einsum("rk,rk->k", dy, xh), "dbeta": torch.einsum("rk->k", dy),
                "amax": _stored_amax(dx, DTYPES[case["x"]])}
    if op == ACT_BWD:
        d = s["dd"].double() * _act_grad64(s["pre"].double(), case["act"])
        return {"dpre": d, "dbias": torch.einsum("mn->n", d), "amax": _stored_amax(d, DTYPES[case["t"]])}
    if op == GEMV:
        a, g_a = _quantized64(s["x"])
        out = torch.bfloat16
    else:
        a, g_a = _values64(s["a"][0], s["a"][1]), s["a"][2].double()
        out = DTYPES[case["out"]]
    codes, sf, g_w = s["w"]
    alpha = 1.0 / (g_a * g_w.double())
    kb = codes.shape[1] // 8
    step = 128 * max(1, (1 << 26) // (128 * case["k"]))            # whole scale groups of weight rows at a time
    v = torch.cat([a @ _values64(codes[i:i + step], sf[i * kb:]).t() for i in range(0, case["n"], step)], 1)
    v = v * alpha + s["bias"].double()
    d = _act64(v, case["act"])
    if s["res"] is not None:
        d = d + s["res"].double()
    if op == GEMV:
        return {"d": d}
    return {"d": d, "pre": v if case["pre"] else None, "amax": _stored_amax(d, out)}
