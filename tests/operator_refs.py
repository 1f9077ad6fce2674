"""64-bit references of the layer norm, the product epilogue and their gradients, each with an elementwise
bound on a kernel that computes in fp32 and rounds its output once.

Notation: u = 2^-24 (half a step of fp32); a sum whose longest chain of additions is c is off by at most
c u sum |terms| (to first order); a rounding to type t is off by finfo(t).eps / 2 relative to the value, or half
of its smallest subnormal.  No sum of the kernels has a longer chain than CHAIN + n / 256 additions for rows of
n elements (a thread's share, 5 shuffle steps, one step per warp), nor than CHAIN + rows / 64 for column sums.
"""
import math

import torch

U = 2.0 ** -24
CHAIN = 80


def rounding(ref, dtype):
    if dtype == torch.float64:
        return torch.zeros_like(ref)
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def check(got, ref, tol, what):
    """|got - ref| <= tol + the rounding of a value that is off by tol; NaNs and infinities in the same places."""
    assert tuple(got.shape) == tuple(ref.shape), (what, got.shape, ref.shape)
    g, ref = got.detach().double().cpu(), ref.cpu()
    tol = tol.cpu() if torch.is_tensor(tol) else torch.full_like(ref, tol)
    finite = torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{what}: NaNs in other places"
    assert torch.equal(g[~finite & ~torch.isnan(ref)], ref[~finite & ~torch.isnan(ref)]), f"{what}: infinities"
    lim = tol + rounding(ref.abs() + tol, got.dtype)
    err = (g - ref).abs()
    bad = finite & ~(err <= lim)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, err / lim, torch.zeros_like(err))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {ref.numel()} off, worst {float(g.reshape(-1)[i])!r} for "
                             f"{float(ref.reshape(-1)[i])!r}, allowed {float(lim.reshape(-1)[i])!r}")


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def layernorm(x, gamma, beta, eps):
    """{name: (reference, tolerance before the output's rounding)} for y, mean, rstd."""
    x = x.double().cpu()
    k = x.shape[1]
    g = gamma.double().cpu() if gamma is not None else torch.ones(k, dtype=torch.float64)
    b = beta.double().cpu() if beta is not None else torch.zeros(k, dtype=torch.float64)
    mean = x.mean(1)
    d = x - mean[:, None]
    var = d.square().mean(1)
    rstd = 1.0 / torch.sqrt(var + eps)
    c = (CHAIN + k / 256) * U
    # mean: the sum, times 1/k (rounded), rounded
    e_mean = (c + 2 * U) * x.abs().mean(1) + U * mean.abs()
    # sum (x - m')^2 = k (var + (m - m')^2) exactly; each difference is rounded (2u on its square), then the
    # square, the sum, the factor 1/k, eps added
    e_var = e_mean.square() + (c + 5 * U) * (var + e_mean.square()) + U * eps
    rel = torch.where(var + eps > 0, 0.5 * e_var / (var + eps), torch.zeros_like(var)) * 1.01 + 2 * U
    xh = d * rstd[:, None]
    # (x - m') rstd' g + b: the difference, two products, one sum
    e_y = g.abs() * (rstd[:, None] * (1 + rel[:, None]) * (e_mean[:, None] + U * d.abs()) + xh.abs() * (rel[:, None] + 3 * U))
    y = xh * g + b
    return {"y": (y, e_y + U * (y.abs() + b.abs())), "mean": (mean, e_mean), "rstd": (rstd, rel * rstd)}


def layernorm_backward(dy, x, mean, rstd, gamma, res):
    """The same for dx, dgamma, dbeta; mean and rstd are inputs."""
    dy, x, mean, rstd = (t.double().cpu() for t in (dy, x, mean, rstd))
    rows, k = x.shape
    g = gamma.double().cpu() if gamma is not None else torch.ones(k, dtype=torch.float64)
    xh = (x - mean[:, None]) * rstd[:, None]
    a = dy * g
    c1, c2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    c = (CHAIN + k / 256) * U
    # xh carries 2 roundings, a one; sums, then the factor 1/k
    e1 = (c + 4 * U) * a.abs().mean(1, keepdim=True)
    e2 = (c + 7 * U) * (a * xh).abs().mean(1, keepdim=True)
    core = rstd[:, None] * (a - c1 - xh * c2)
    e = rstd[:, None].abs() * (e1 + xh.abs() * e2 + 6 * U * (a.abs() + c1.abs() + (xh * c2).abs())) + 2 * U * core.abs()
    dx = core
    if res is not None:
        dx = core + res.double().cpu()
        e = e + U * dx.abs()
    cr = (CHAIN + rows / 64) * U
    return {"dx": (dx, e), "dgamma": ((dy * xh).sum(0), (cr + 4 * U) * (dy * xh).abs().sum(0)),
            "dbeta": (dy.sum(0), cr * dy.abs().sum(0))}


# ---------------------------------------------------------------------------
# activations: the fp32 forms use the 2-ulp exponential (error 2 + 1.2 |x| ulps of 2^-23 for e^x), erfc (4 ulps) and
# a 2-ulp division; a rounding of the argument w of e^w or erfc changes the value by |w| 2 u (e^w, three roundings)
# or (v^2 + 1) u (erfc(v / sqrt 2)).  With X the size of that argument: relative error (8 + 2 X) 2^-23.  That holds
# for normal numbers: an exponential, erfc or quotient below 2^-126 has no relative accuracy (fp32 values there are
# 2^-149 apart, and the fast forms may give 0), so it is off by up to 2^-126 itself, the value v p by |v| 2^-126, and
# the slope p + v w'(v) p (1 - p) by (1 + |v w'|) 2^-126, |v w'| <= 1.6 |v| + 0.22 |v|^3, which is below
# (1 + |v|^3) 2^-125.
# ---------------------------------------------------------------------------
TINY = 2.0 ** -125


def _u2(v):
    return 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)


def act(v, name):
    """(act(v), bound on the evaluation's error, bound on |act'|)."""
    if name == "relu":
        return v.clamp(min=0.0), torch.zeros_like(v), 1.0
    if name == "gelu":
        f, x = 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0)), v.square()
    elif name == "gelu_tanh":
        f, x = v * torch.sigmoid(_u2(v)), _u2(v).abs()
    elif name == "silu":
        f, x = v * torch.sigmoid(v), v.abs()
    else:
        return v, torch.zeros_like(v), 1.0
    return f, f.abs() * (8 + 2 * x) * 2.0 ** -23 + TINY * (1 + v.abs()), 1.14


def act_slope(v, name):
    """(act'(v), bound on the evaluation's error)."""
    if name == "relu":
        return (v > 0).double(), torch.zeros_like(v)
    if name == "gelu":
        p, t, x = 0.5 * torch.special.erfc(-v / math.sqrt(2.0)), v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi), v.square()
    elif name == "gelu_tanh":
        p = torch.sigmoid(_u2(v))
        t = v * p * torch.sigmoid(-_u2(v)) * 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * v * v)
        x = _u2(v).abs()
    elif name == "silu":
        p = torch.sigmoid(v)
        t, x = v * p * torch.sigmoid(-v), v.abs()
    else:
        return torch.ones_like(v), torch.zeros_like(v)
    return p + t, (p + t.abs()) * (8 + 2 * x) * 2.0 ** -23 + 2 * U * (p + t).abs() + TINY * (1 + v.abs() ** 3)


def epilogue(d_ref, s_ref, alpha, bias, name, res):
    """{d, pre} of alpha acc + bias; the product's own bound is 2^-20 alpha sum |a b|."""
    v = torch.as_tensor(d_ref)
    e = torch.as_tensor(s_ref) * (2.0 ** -20 * float(alpha))
    if bias is not None:
        v = v + bias.double().cpu()
    e = e + U * v.abs()
    f, e_f, slope = act(v, name)
    e_d = e_f + slope * e
    if res is not None:
        f = f + res.double().cpu()
        e_d = e_d + U * f.abs()
    return {"d": (f, e_d), "pre": (v, e)}


def epilogue_backward(dd, pre, name):
    dd, pre = dd.double().cpu(), pre.double().cpu()
    s, e_s = act_slope(pre, name)
    d = dd * s
    e = dd.abs() * e_s + U * d.abs()
    c = (CHAIN + dd.shape[0] / 64) * U
    return {"dpre": (d, e), "dbias": (d.sum(0), e.sum(0) + c * d.abs().sum(0))}
