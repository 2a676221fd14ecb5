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
