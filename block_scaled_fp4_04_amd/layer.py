"""Python binding of the operators around the MXFP4 products of a transformer
layer (``include/nvfp4_layer.h``): argument marshalling only, like the rest of
the package.

``MxEpilogue`` names what a product adds in its epilogue; ``mx_gemm``,
``mx_gemm_quantized``, ``mx_linear`` and ``mx_grouped_gemm`` take one as
``epilogue``:

    gated = MxEpilogue(activation="silu", gate=w_gate)
    h = mx_linear(x, w_up, epilogue=gated)
    x = mx_linear(h, w_down, epilogue=MxEpilogue(bias=b, residual=x))

The products have no backward form, with an epilogue as without: results carry
no autograd history.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

from . import _i64, _vp, lib
from .mx import _GEMM, _GEMM_Q, _GROUPED, _KINDS, _kind

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}   # NVFP4_ACT_*

LAYER_EXPORTS = ["nvfp4_mx_gemm_fused", "nvfp4_mx_gemm_quantized_fused", "nvfp4_mx_grouped_gemm_fused",
                 "nvfp4_sequence_add_mx_gemm_fused", "nvfp4_sequence_add_mx_gemm_quantized_fused",
                 "nvfp4_sequence_add_mx_grouped_gemm_fused"]

_int, _f32 = ctypes.c_int, ctypes.c_float
_bound = None


class _EpilogueT(ctypes.Structure):
    _fields_ = [("activation", _int), ("gate_packed", _vp), ("gate_scales", _vp), ("bias", _vp), ("gate_bias", _vp),
                ("bias_type", _int), ("residual", _vp), ("ld_residual", _i64)]


_epi = ctypes.POINTER(_EpilogueT)


def _with_epilogue(types: list) -> list:
    """The argument types of a product with an epilogue behind alpha."""
    at = types.index(_f32) + 1
    return types[:at] + [_epi] + types[at:]


def layer_lib() -> ctypes.CDLL:
    """The library with the argument types of its layer functions set."""
    global _bound
    L = lib()
    if _bound is not L:
        for name, types in (("mx_gemm_fused", _with_epilogue(_GEMM)),
                            ("mx_gemm_quantized_fused", _with_epilogue(_GEMM_Q)),
                            ("mx_grouped_gemm_fused", _with_epilogue(_GROUPED))):
            f, g = getattr(L, "nvfp4_" + name), getattr(L, "nvfp4_sequence_add_" + name)
            f.restype = g.restype = _int
            f.argtypes, g.argtypes = types + [_vp], [_vp] + types
        _bound = L
    return L


def _activation(name) -> int:
    kind = ACTIVATIONS.get(name or "none")
    if kind is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, not {name!r}")
    return kind


def _bias(name: str, b, shape: tuple):
    """Checks a bias and returns (address, type code); (None, None) for none."""
    if b is None:
        return None, None
    kind = _KINDS.get(b.dtype)
    if kind is None or tuple(b.shape) != shape or not b.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 or bfloat16 tensor of shape {shape}")
    return b.data_ptr(), kind


@dataclass
class MxEpilogue:
    """What a product of activations A with a weight B (``mx_gemm`` and the
    others) adds before its result is rounded, in fp32: act(alpha A B^T +
    ``bias``) + ``residual``, or with a ``gate`` weight, of B's class and sizes,
    act(alpha A gate^T + ``gate_bias``) * (alpha A B^T + ``bias``) + ``residual``.

    ``activation``: "none", "relu", "silu", "gelu" or "gelu_tanh".  Biases are
    [N] (grouped: [groups, N]), float32 or bfloat16, both of one type.  The
    ``residual`` has the shape and type of the result, rows may be strided; it
    may be the ``out`` tensor itself, but must not overlap it otherwise."""
    activation: "str | None" = None
    bias: "object" = None
    gate: "object" = None
    gate_bias: "object" = None
    residual: "object" = None

    def _marshal(self, b, out, args: tuple):
        """(C arguments, tensors) for a product of B = b into out whose
        arguments without an epilogue are `args`."""
        shape = (b.rows,) if not hasattr(b, "groups") else (b.groups, b.rows)
        bias, kind = _bias("bias", self.bias, shape)
        gate_bias, gate_kind = _bias("gate_bias", self.gate_bias, shape)
        g, r = self.gate, self.residual
        if g is None:
            if gate_bias is not None:
                raise ValueError("gate_bias needs a gate")
        else:
            _kind(g, "gate", type(b))
            if (g.rows, g.K) != (b.rows, b.K) or getattr(g, "groups", 0) != getattr(b, "groups", 0):
                raise ValueError("the gate must have the sizes of b")
            g.check("gate")
            if None not in (kind, gate_kind) and kind != gate_kind:
                raise ValueError("bias and gate_bias must be of one type")
        if r is not None and (r.shape != out.shape or r.dtype != out.dtype or (r.stride(1) != 1 and r.shape[1] != 1)):
            raise ValueError(f"residual must be a tensor of shape {tuple(out.shape)} and type {out.dtype} with unit "
                             "stride along its rows")
        e = _EpilogueT(_activation(self.activation), None if g is None else g.codes.data_ptr(),
                       None if g is None else g.scales.data_ptr(), bias, gate_bias,
                       (gate_kind or 0) if kind is None else kind, None if r is None else r.data_ptr(),
                       0 if r is None else r.stride(0))
        tensors = (self.bias, self.gate_bias, r) + (() if g is None else (g.codes, g.scales))
        # (alpha is the one float among the arguments)
        at = next(i for i, a in enumerate(args) if type(a) is float) + 1
        return args[:at] + (e,) + args[at:], tensors
