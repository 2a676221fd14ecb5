"""Plain references, in 64 bits, of the operators around the MXFP4 products
(include/nvfp4_layer.h), with bounds of how far fp32 arithmetic may be off:
written from the definitions in torch, sharing nothing with the library."""
import math

import torch

U = 2.0 ** -24   # half a step of fp32, relative


def act(name, z):
    """The activation of float64 z."""
    if name in (None, "none"):
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def act_bound(name, z, dz):
    """How far the activation of a z that is off by dz may be: the slope, at
    most 1.13 (gelu at sqrt 2, silu 1.1), times dz, and the evaluation's own
    error.  silu: the exponent -1.4427 z is rounded (|z| u of the exponential)
    and the power of two, sum, reciprocal and product add at most 8 u: (|z| + 8)
    u relative, doubled.  gelu_tanh: the same for an exponent of up to four
    roundings.  gelu: erf to 8 u (and its argument's roundings) beside 1: |z|
    16 u."""
    own = {"silu": (z.abs() + 8) * 2 * U * act("silu", z).abs(),
           "gelu": z.abs() * 16 * U,
           "gelu_tanh": (1.6 * z.abs() * (1 + 0.05 * z * z) + 8) * 8 * U * act("gelu_tanh", z).abs()}.get(name, 0.0)
    return 1.13 * dz + own


def product(a, b, alpha=1.0):
    """(alpha a b^T, bound) of float64 values: every matrix instruction (64
    elements deep at least) and each of at most 17 partial sums adds with at
    most two units in the last place (2^-22 of the magnitudes); alpha rounds."""
    z = alpha * (a @ b.T)
    mag = abs(alpha) * (a.abs() @ b.abs().T)
    return z, (a.shape[1] / 64 + 17) * 4 * U * mag + 2 * U * z.abs()


def epilogue(z, dz, activation=None, bias=None, gate=None, gate_bias=None, residual=None):
    """(result, bound before the output is rounded); z and gate: (values, bound)
    of products."""
    if bias is not None:
        z = z + bias
        dz = dz + 2 * U * z.abs()
    if gate is None:
        out, d = act(activation, z), act_bound(activation, z, dz)
    else:
        v, dv = gate
        if gate_bias is not None:
            v = v + gate_bias
            dv = dv + 2 * U * v.abs()
        g, dg = act(activation, v), act_bound(activation, v, dv)
        out, d = g * z, dg * z.abs() + (g.abs() + dg) * dz + 2 * U * (g * z).abs()
    if residual is not None:
        out = out + residual
        d = d + 2 * U * (out.abs() + d)
    return out, d


def check(got, want, bound, what=""):
    """got (rounded to its type) is within bound and half a step of want; NaN
    where want is."""
    eps = torch.finfo(got.dtype).eps
    g, w = got.double(), want.double()
    assert torch.equal(g.isnan(), w.isnan()), f"{what}: NaN in other places"
    fine = w.isfinite()
    assert torch.equal(g[~fine & ~w.isnan()], w[~fine & ~w.isnan()]), f"{what}: infinities"
    off = ((g - w).abs() - (bound + eps / 2 * (w.abs() + bound) + 1e-37))[fine]
    assert not off.numel() or off.max() <= 0, f"{what}: {int((off > 0).sum())} elements off, by up to {off.max():.3g} over the bound"


# ---- norms: everything in float64, (value, bound before rounding) ---------------
# A mean of squares adds at most 60 times on its way (pieces of a lane, lanes,
# waves): off by 62 u with the mean and eps, its root's inverse by half of that
# and the instruction's error, 40 u in all.

def inverse_rms(x, eps):
    return (x.square().mean(-1, keepdim=True) + eps).rsqrt()


def norm_h(y, residual=None, post=False, post_weight=None, gate=None, scale=1.0, residual_scale=1.0, eps=1e-6):
    u = y * inverse_rms(y, eps) if post else y
    if post_weight is not None:
        u = u * post_weight
    b = scale * u if gate is None else scale * gate * u
    r = 0.0 if residual is None else residual_scale * residual
    return b + r, 48 * U * b.abs() + 4 * U * (b.abs() + abs(r))


def norm_n(h, pre_weight=None, eps=1e-6):
    n = h * inverse_rms(h, eps) * (1.0 if pre_weight is None else pre_weight)
    return n, 48 * U * n.abs()


def _norm_back(d, dd, x, w, eps):
    """Gradients of x / rms(x) * w for d, which is off by dd: ((dx, bound), (dw, bound) by rows)."""
    r = inverse_rms(x, eps)
    v, dv = d * w, dd * abs(w) + 2 * U * (d * w).abs()
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    along = mean(v * x)
    dx = r * v - x * r ** 3 * along
    bound = r * (dv + 50 * U * v.abs()) + x.abs() * r ** 3 * (mean(dv * x.abs()) + 70 * U * mean((v * x).abs())
                                                              + 130 * U * along.abs()) + 4 * U * dx.abs()
    dw = d * x * r
    return (dx, bound), (dw, (dd + 46 * U * d.abs()) * (x * r).abs())


def norm_grads(dh, dn, y, h, post=False, post_weight=None, gate=None, pre_weight=None, scale=1.0, residual_scale=1.0,
               eps=1e-6, channel=False):
    """{name: (value, bound)}; sums over rows add at most as often as there are rows, plus 40."""
    rows = (dh if dh is not None else dn).shape[0]
    total = lambda t, b: (t.sum(0), b.sum(0) + (rows + 40) * U * t.abs().sum(0))  # noqa: E731
    out = {}
    d = torch.zeros_like(dn) if dh is None else dh
    b = torch.zeros_like(d)
    if dn is not None:
        w = torch.ones_like(dn[0]) if pre_weight is None else pre_weight
        (dx, bx), dw = _norm_back(dn, torch.zeros_like(dn), h, w, eps)
        b = bx + 2 * U * (d.abs() + dx.abs())
        d = d + dx
        out["pre_weight"] = total(*dw)
    out["residual"] = residual_scale * d, abs(residual_scale) * b + 2 * U * (residual_scale * d).abs()
    d, b = scale * d, abs(scale) * b + U * (scale * d).abs()
    if gate is not None:
        u = y
        if post:
            u = y * inverse_rms(y, eps) * (1.0 if post_weight is None else post_weight)
        g, bg = d * u, b * u.abs() + 46 * U * (d * u).abs()
        out["gate"] = total(g, bg) if channel else (g, bg)
        d, b = d * gate, b * abs(gate) + U * (d * gate).abs()
    if post:
        w = torch.ones_like(y[0]) if post_weight is None else post_weight
        (d, b), dw = _norm_back(d, b, y, w, eps)
        out["post_weight"] = total(*dw)
    out["y"] = d, b
    return out


# ---- a layer of experts ------------------------------------------------------------

def moe_hidden(x, ids, w, act_name, gate=None, bias=None, gate_bias=None):
    """{(t, e): (h, bound)} before its rounding; x, w, gate: float64 values that MXFP4 holds."""
    out = {}
    for e in sorted(set(ids.flatten().tolist())):
        if 0 <= e < w.shape[0]:
            t = sorted(set(torch.nonzero(ids == e)[:, 0].tolist()))
            more = {}
            if bias is not None:
                more["bias"] = bias[e]
            if gate is not None:
                more["gate"] = product(x[t], gate[e])
                if gate_bias is not None:
                    more["gate_bias"] = gate_bias[e]
            h, d = epilogue(*product(x[t], w[e]), activation=act_name, **more)
            for i, token in enumerate(t):
                out[token, e] = h[i], d[i]
    return out
