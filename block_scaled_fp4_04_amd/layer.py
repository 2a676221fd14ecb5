"""Python binding of the operators around the MXFP4 products of a transformer
layer (``include/nvfp4_layer.h``): argument marshalling only, like the rest of
the package.

``MxEpilogue`` names what a product adds in its epilogue; ``mx_gemm``,
``mx_gemm_quantized``, ``mx_linear`` and ``mx_grouped_gemm`` take one as
``epilogue``:

    gated = MxEpilogue(activation="silu", gate=w_gate)
    h = mx_linear(x, w_up, epilogue=gated)
    x = mx_linear(h, w_down, epilogue=MxEpilogue(bias=b, residual=x))

``mx_moe`` is a whole layer of experts from a router's choices, in two launches
for few tokens.

``add_norm`` is what stands between two blocks: the norm behind one, its gate
and the residual, and the norm before the next, as rows or as a packed MXFP4
operand; ``rms_norm`` the norm alone.

The products have no backward form, with an epilogue as without.  The gradients
of ``add_norm`` are a function of their own (``add_norm_grad``): nothing here is
recorded by autograd, and results carry no history.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from dataclasses import dataclass

import torch

from . import Nvfp4Error, _i64, _vp, lib
from .mx import (MX_BLOCK, MX_QUANT_ROWS, _GEMM, _GEMM_Q, _GROUPED, _KINDS, MxGroups, MxOperand,
                 _gemm_quantized_args, _kind, _on, _out, _packed, _rows_2d, _run, _type_of)

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}   # NVFP4_ACT_*

LAYER_EXPORTS = ["nvfp4_mx_linear_fused", "nvfp4_mx_gemm_fused", "nvfp4_mx_gemm_quantized_fused",
                 "nvfp4_mx_grouped_gemm_fused",
                 "nvfp4_sequence_add_mx_gemm_fused", "nvfp4_sequence_add_mx_gemm_quantized_fused",
                 "nvfp4_sequence_add_mx_grouped_gemm_fused", "nvfp4_add_norm", "nvfp4_sequence_add_norm",
                 "nvfp4_add_norm_grad", "nvfp4_add_norm_grad_workspace", "nvfp4_mx_moe", "nvfp4_mx_moe_workspace",
                 "nvfp4_sequence_add_mx_moe"]

GATE_NONE, GATE_CHANNEL, GATE_ELEMENT = 0, 1, 2   # NVFP4_GATE_*
NORM_MAX_HIDDEN = 16384

_int, _f32 = ctypes.c_int, ctypes.c_float
_bound = None


class _EpilogueT(ctypes.Structure):
    _fields_ = [("activation", _int), ("gate_packed", _vp), ("gate_scales", _vp), ("bias", _vp), ("gate_bias", _vp),
                ("bias_type", _int), ("residual", _vp), ("ld_residual", _i64)]


class _NormT(ctypes.Structure):
    _fields_ = [("type", _int), ("weight_type", _int), ("rows", _i64), ("hidden", _i64), ("post", _int), ("pre", _int),
                ("post_weight", _vp), ("pre_weight", _vp), ("gate_mode", _int), ("gate", _vp), ("ld_gate", _i64),
                ("scale", _f32), ("residual_scale", _f32), ("eps", _f32)]


class _ExpertsT(ctypes.Structure):
    _fields_ = [("experts", _i64), ("hidden", _i64), ("inner", _i64), ("activation", _int), ("gate_packed", _vp),
                ("gate_scales", _vp), ("up_packed", _vp), ("up_scales", _vp), ("down_packed", _vp), ("down_scales", _vp),
                ("bias_type", _int), ("gate_bias", _vp), ("up_bias", _vp), ("down_bias", _vp)]


_epi, _norm_p, _experts_p = (ctypes.POINTER(t) for t in (_EpilogueT, _NormT, _ExpertsT))
_size = ctypes.c_size_t
_MOE = [_experts_p, _vp, _int, _i64, _vp, _int, _vp, _i64, _i64, _vp, _int, _vp, _size]
_NORM = [_norm_p, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp]
_NORM_GRAD = [_norm_p, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _size]


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
        for name, types in (("nvfp4_mx_linear_fused", _with_epilogue(_GEMM_Q) + [_vp, _size, _vp]),
                            ("nvfp4_add_norm", _NORM + [_vp]), ("nvfp4_sequence_add_norm", [_vp] + _NORM),
                            ("nvfp4_add_norm_grad", _NORM_GRAD + [_vp]),
                            ("nvfp4_add_norm_grad_workspace", [_norm_p, ctypes.POINTER(_size)]),
                            ("nvfp4_mx_moe", _MOE + [_vp]), ("nvfp4_sequence_add_mx_moe", [_vp] + _MOE),
                            ("nvfp4_mx_moe_workspace", [_experts_p, _i64, _i64, _int, ctypes.POINTER(_size)])):
            f = getattr(L, name)
            f.restype, f.argtypes = _int, types
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

    def _marshal(self, b, out, args: tuple, at: int):
        """(C arguments, tensors) for a product of B = b into out whose
        arguments without an epilogue are `args`, the epilogue's place among them
        `at`."""
        groups, g, r = getattr(b, "groups", None), self.gate, self.residual
        bias = gate_bias = gate_codes = gate_scales = kind = gate_kind = residual = None
        ld, tensors = 0, (self.bias, self.gate_bias, r)
        if self.bias is not None or self.gate_bias is not None:
            shape = (b.rows,) if groups is None else (groups, b.rows)
            bias, kind = _bias("bias", self.bias, shape)
            gate_bias, gate_kind = _bias("gate_bias", self.gate_bias, shape)
            if None not in (kind, gate_kind) and kind != gate_kind:
                raise ValueError("bias and gate_bias must be of one type")
        if g is not None:
            _kind(g, "gate", type(b))
            if g.rows != b.rows or g.K != b.K or getattr(g, "groups", None) != groups:
                raise ValueError("the gate must have the sizes of b")
            g.check("gate")
            gate_codes, gate_scales = g.codes.data_ptr(), g.scales.data_ptr()
            tensors += (g.codes, g.scales)
        elif gate_bias is not None:
            raise ValueError("gate_bias needs a gate")
        if r is not None:
            if r.shape != out.shape or r.dtype is not out.dtype or (r.stride(1) != 1 and r.shape[1] != 1):
                raise ValueError(f"residual must be a tensor of shape {tuple(out.shape)} and type {out.dtype} with unit "
                                 "stride along its rows")
            residual, ld = r.data_ptr(), r.stride(0)
        e = _EpilogueT(_activation(self.activation), gate_codes, gate_scales, bias, gate_bias,
                       (gate_kind or 0) if kind is None else kind, residual, ld)
        return args[:at] + (e,) + args[at:], tensors


#: The place of an epilogue among the arguments of a product, behind alpha.
_EPILOGUE_AT = {"nvfp4_mx_gemm": 5, "nvfp4_mx_gemm_quantized": 6, "nvfp4_mx_grouped_gemm": 9}


def _linear(x, b, alpha, out, dtype, epilogue):
    """mx_linear of a 2-D x with an epilogue: one call (nvfp4_mx_linear_fused)."""
    out, args = _gemm_quantized_args(x, b, alpha, out, dtype)
    r = epilogue.residual
    if r is not None and r.dim() == 2 and r.shape[0] > 1 and r.stride(0) < r.shape[1] and 1 in (r.stride(1), r.shape[1]):
        epilogue = dataclasses.replace(epilogue, residual=r.contiguous())   # (one row for all of them, say)
    args, more = epilogue._marshal(b, out, args, 6)
    work, size = None, 0
    if x.shape[0] > MX_QUANT_ROWS or b.K > 8192:   # (below that the call takes no workspace)
        size = sum(_packed(x.shape[0], b.K))
        work = x.new_empty(size, dtype=torch.uint8)
    _run(layer_lib().nvfp4_mx_linear_fused, args + (None if work is None else work.data_ptr(), size),
         (x, b.codes, b.scales, out, work) + more)
    return out


# ---- a whole layer of experts --------------------------------------------------


@functools.lru_cache(maxsize=4096)
def _moe_workspace(experts: int, hidden: int, inner: int, tokens: int, topk: int, out_kind: int) -> int:
    """Bytes of workspace, a function of the sizes alone."""
    size, spec = _size(), _ExpertsT(experts, hidden, inner)
    st = layer_lib().nvfp4_mx_moe_workspace(ctypes.byref(spec), tokens, topk, out_kind, ctypes.byref(size))
    if st:
        raise Nvfp4Error(st, f"nvfp4_mx_moe_workspace({tokens}, {topk})")
    return size.value


def _moe_args(x, ids, weights, up, down, gate, activation, up_bias, gate_bias, down_bias, out, dtype):
    _kind(up, "up", MxGroups)
    _kind(down, "down", MxGroups)
    up.check("up")
    down.check("down")
    if gate is not None:
        _kind(gate, "gate", MxGroups)
        gate.check("gate")
    E, F, H = up.groups, up.rows, up.K
    if (down.groups, down.rows, down.K) != (E, H, F):
        raise ValueError(f"down must be {E} operands of {H} x {F}, not {down.groups} of {down.rows} x {down.K}")
    if gate is not None and (gate.groups, gate.rows, gate.K) != (E, F, H):
        raise ValueError(f"the gate must be {E} operands of {F} x {H}, not {gate.groups} of {gate.rows} x {gate.K}")
    if gate is None and gate_bias is not None:
        raise ValueError("gate_bias needs a gate")
    kind = _rows_2d(x)
    T = x.shape[0]
    if x.shape[1] != H:
        raise ValueError(f"x has rows of {x.shape[1]}, the experts of {H}")
    if ids.dim() != 2 or ids.shape[0] != T or ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise ValueError("expert_ids must be a contiguous [tokens, topk] int32 or int64 tensor")
    if weights is not None and (weights.dtype != torch.float32 or weights.shape != ids.shape or not weights.is_contiguous()):
        raise ValueError(f"weights must be a contiguous float32 tensor of shape {tuple(ids.shape)}")
    bg = bu = bd = bias_type = None
    if not (gate_bias is up_bias is down_bias is None):
        bg, kg = _bias("gate_bias", gate_bias, (E, F))
        bu, ku = _bias("up_bias", up_bias, (E, F))
        bd, kd = _bias("down_bias", down_bias, (E, H))
        bias_type = kg if kg is not None else ku if ku is not None else kd
        if not (kg in (None, bias_type) and ku in (None, bias_type) and kd in (None, bias_type)):
            raise ValueError("the biases must be of one type")
    out, out_kind = _out(out, dtype, T, H, x)
    spec = _ExpertsT(E, H, F, _activation(activation), None if gate is None else gate.codes.data_ptr(),
                     None if gate is None else gate.scales.data_ptr(), up.codes.data_ptr(), up.scales.data_ptr(),
                     down.codes.data_ptr(), down.scales.data_ptr(), bias_type or 0, bg, bu, bd)
    k = ids.shape[1]
    size = _moe_workspace(E, H, F, T, k, out_kind)
    work = x.new_empty(size, dtype=torch.uint8)
    args = (spec, x.data_ptr(), kind, x.stride(0), ids.data_ptr(), 1 if ids.dtype is torch.int64 else 0,
            None if weights is None else weights.data_ptr(), T, k, out.data_ptr(), out_kind, work.data_ptr(), size)
    tensors = (x, ids, weights, out, work, up.codes, up.scales, down.codes, down.scales, up_bias, gate_bias, down_bias)
    return out, args, tensors if gate is None else tensors + (gate.codes, gate.scales)


def mx_moe(x, expert_ids, weights, up: MxGroups, down: MxGroups, gate: MxGroups | None = None, activation="silu",
           up_bias=None, gate_bias=None, down_bias=None, out=None, dtype=None, stream=None):
    """A whole layer of experts (nvfp4_mx_moe): for each token the sum over its
    choices ``expert_ids`` [tokens, topk] (int32 or int64; numbers outside [0,
    experts) are dropped) under ``weights`` (float32, None for ones) of the
    expert's down-projection of

        act(q(x) up^T + up_bias), or act(q(x) gate^T + gate_bias) * (q(x) up^T + up_bias)

    held in bfloat16 and quantised.  x: [tokens, hidden], rows strided as in
    mx_quantize; ``up`` and ``gate`` are [experts, inner, hidden], ``down``
    [experts, hidden, inner]; biases [experts, inner] and [experts, hidden].
    Two launches for up to 4 tokens.  The result is bfloat16 unless
    ``dtype`` or ``out`` says float32."""
    if stream is not None:
        with _on(stream, x):
            return mx_moe(x, expert_ids, weights, up, down, gate, activation, up_bias, gate_bias, down_bias, out, dtype)
    out, args, tensors = _moe_args(x, expert_ids, weights, up, down, gate, activation, up_bias, gate_bias, down_bias, out, dtype)
    _run(layer_lib().nvfp4_mx_moe, args, tensors)
    return out


# ---- norms ------------------------------------------------------------------


def _rows_of(name: str, t, shape, dtype):
    """t (rows may be strided; dimensions in front of the last are rows) as a
    2-D tensor; None for none.  A t whose rows do not follow each other at one
    stride, of a row at least, is copied."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    return _strided(t, shape[-1])


def _strided(t, H: int):
    if t.dim() != 2:
        t = t.reshape(-1, H)
    ld, unit = t.stride()
    return t if (unit == 1 or H == 1) and (ld >= H or t.shape[0] <= 1) else t.contiguous()


def _spec(y, post_weight, gate, pre_weight, scale, residual_scale, eps, post: bool, pre: bool):
    """(the operator's C description, its gate as rows if it has one for every
    element, the tensors that it names)."""
    shape, dtype = y.shape, y.dtype
    if len(shape) < 2:
        raise ValueError("rows must be a tensor of at least two dimensions")
    H, kind = shape[-1], _type_of(dtype, "rows")
    if not 1 <= H <= NORM_MAX_HIDDEN:
        raise ValueError(f"rows must have 1 to {NORM_MAX_HIDDEN} elements, not {H}")
    if post_weight is not None and not post or pre_weight is not None and not pre:
        raise ValueError("a weight without its norm")
    mode, at, channel, ld = GATE_NONE, None, None, 0
    if gate is not None:
        if gate.shape == shape:
            mode, at = GATE_ELEMENT, _rows_of("gate", gate, shape, dtype)
            ld = at.stride(0)
        else:
            mode, at, channel = GATE_CHANNEL, gate, gate
    weight_type = None
    for name, w in (("post_weight", post_weight), ("pre_weight", pre_weight), ("gate", channel)):
        if w is not None:
            of = _KINDS.get(w.dtype)
            if of is None or w.numel() != H or w.dim() != 1 or not w.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 or bfloat16 tensor of shape ({H},)"
                                 + (f" or {tuple(shape)}" if w is channel else ""))
            if weight_type not in (None, of):
                raise ValueError("the weights (and a gate for each channel) must be of one type")
            weight_type = of
    spec = _NormT(kind, weight_type or 0, y.numel() // H, H, post, pre,
                  None if post_weight is None else post_weight.data_ptr(),
                  None if pre_weight is None else pre_weight.data_ptr(), mode, None if at is None else at.data_ptr(),
                  ld, scale, residual_scale, eps)
    return spec, (post_weight, pre_weight, at)


def _at(t):
    return (None, 0) if t is None else (t.data_ptr(), t.stride(0))


def _given(name: str, out, like):
    """`out`, made like `like` if it is None, checked otherwise."""
    if out is None:   # (of a plain tuple: three times as fast as of a torch.Size)
        return torch.empty_like(like) if like.is_contiguous() else like.new_empty((*like.shape,))
    if out.shape != like.shape or out.dtype != like.dtype or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {like.dtype} tensor of shape {tuple(like.shape)}")
    return out


def _norm_args(y, residual, post_weight, gate, pre_weight, scale, residual_scale, eps, post, pre, quantize, h, n, keep):
    post = post_weight is not None if post is None else bool(post)
    spec, named = _spec(y, post_weight, gate, pre_weight, scale, residual_scale, eps, post, bool(pre))
    rows = _strided(y, y.shape[-1])
    res = _rows_of("residual", residual, y.shape, y.dtype)
    h = _given("h", h, y) if keep else None
    codes = scales = None
    if not pre:
        if quantize or n is not None:
            raise ValueError("without the norm before the next block there is no n")
    elif quantize:
        H = y.shape[-1]
        if H % MX_BLOCK:
            raise ValueError(f"packed rows must be a multiple of {MX_BLOCK} long, not {H}")
        if n is None:
            cb, sb = _packed(spec.rows, H)
            n = MxOperand(y.new_empty(cb, dtype=torch.uint8), y.new_empty(sb, dtype=torch.uint8), spec.rows, H)
        else:
            _kind(n, "n", MxOperand)
            if (n.rows, n.K) != (spec.rows, H):
                raise ValueError("n has the wrong shape")
            n.check("n")
        codes, scales = n.codes, n.scales
    else:
        n = _given("n", n, y)
    args = (spec, *_at(rows), *_at(res), None if h is None else h.data_ptr(),
            None if n is None or quantize else n.data_ptr(), None if codes is None else codes.data_ptr(),
            None if scales is None else scales.data_ptr())
    return h, n, args, (rows, res, h, codes if quantize else n, scales, *named)


def add_norm(y, residual=None, post_weight=None, gate=None, pre_weight=None, scale: float = 1.0,
             residual_scale: float = 1.0, eps: float = 1e-6, post=None, pre: bool = True, quantize: bool = False,
             h=None, n=None, stream=None):
    """What stands between two blocks of a layer (nvfp4_add_norm), by rows
    [..., hidden] of float32 or bfloat16, hidden at most NORM_MAX_HIDDEN:

        u = y / rms(y) * post_weight            (``post``; by default if a weight is given; else u = y)
        h = residual_scale * residual + scale * gate * u
        n = h / rms(h) * pre_weight             (``pre``; else n is None)

    Returns (h, n).  Weights are [hidden] or None for ones; the gate is [hidden]
    or has y's shape.  ``quantize``: n as a packed MxOperand of all rows, the bits
    of mx_quantize(n).  ``h`` and ``n`` take given results; h may be the residual
    or y itself."""
    if stream is not None:
        with _on(stream, y):
            return add_norm(y, residual, post_weight, gate, pre_weight, scale, residual_scale, eps, post, pre, quantize, h, n)
    h, n, args, tensors = _norm_args(y, residual, post_weight, gate, pre_weight, scale, residual_scale, eps, post, pre,
                                     quantize, h, n, True)
    _run(layer_lib().nvfp4_add_norm, args, tensors)
    return h, n


def rms_norm(x, weight=None, eps: float = 1e-6, quantize: bool = False, out=None, stream=None):
    """x / rms(x) * weight by rows (nvfp4_add_norm with nothing else), as rows or
    as a packed MxOperand."""
    if stream is not None:
        with _on(stream, x):
            return rms_norm(x, weight, eps, quantize, out)
    _, n, args, tensors = _norm_args(x, None, None, None, weight, 1.0, 1.0, eps, False, True, quantize, None, out, False)
    _run(layer_lib().nvfp4_add_norm, args, tensors)
    return n


@dataclass
class NormGrads:
    """Gradients of add_norm by its inputs (None where there is none): rows
    in the rows' type, those of weights and of a gate for each channel float32."""
    y: "object"
    residual: "object"
    gate: "object"
    post_weight: "object"
    pre_weight: "object"


def add_norm_grad(dh, dn, y, h, post_weight=None, gate=None, pre_weight=None, scale: float = 1.0,
                  residual_scale: float = 1.0, eps: float = 1e-6, post=None, pre=None, residual: bool = True, stream=None):
    """The gradients (NormGrads) of add_norm for those of its results, dh and dn
    (None: zeros), given y and the h that came out (read only with ``pre``, which
    is so by default if dn is given).  ``residual``: whether its gradient is
    wanted.  Weights that are None have no gradient."""
    like = dh if dh is not None else dn
    if like is None:
        raise ValueError("dh or dn must be given")
    if stream is not None:
        with _on(stream, like):
            return add_norm_grad(dh, dn, y, h, post_weight, gate, pre_weight, scale, residual_scale, eps, post, pre, residual)
    pre = dn is not None if pre is None else bool(pre)
    post = post_weight is not None if post is None else bool(post)
    if pre != (dn is not None):
        raise ValueError("dn must be given with the norm before the next block, and only then")
    spec, named = _spec(like, post_weight, gate, pre_weight, scale, residual_scale, eps, post, pre)
    shape, dtype = like.shape, like.dtype
    rows = {name: _rows_of(name, t, shape, dtype) for name, t in
            (("dh", dh), ("dn", dn), ("y", y if post or gate is not None else None), ("h", h if pre else None))}
    for name, used in (("y", post or gate is not None), ("h", pre)):
        if used and rows[name] is None:
            raise ValueError(f"{name} must be given")
    H = shape[-1]
    plain = (*shape,)
    out = NormGrads(like.new_empty(plain), like.new_empty(plain) if residual else None, None, None, None)
    sums = [like.new_empty(H, dtype=torch.float32) if on else None
            for on in (spec.gate_mode == GATE_CHANNEL, post_weight is not None, pre_weight is not None)]
    out.gate, out.post_weight, out.pre_weight = sums
    if spec.gate_mode == GATE_ELEMENT:
        out.gate = like.new_empty(plain)
    work, size = None, _size()
    L = layer_lib()
    if any(s is not None for s in sums):
        st = L.nvfp4_add_norm_grad_workspace(ctypes.byref(spec), ctypes.byref(size))
        if st:
            raise Nvfp4Error(st, "nvfp4_add_norm_grad_workspace")
        work = like.new_empty(size.value, dtype=torch.uint8)
    outs = (out.y, out.residual, out.gate, out.post_weight, out.pre_weight, work)
    args = (spec, *_at(rows["dh"]), *_at(rows["dn"]), *_at(rows["y"]), *_at(rows["h"]),
            *(None if t is None else t.data_ptr() for t in outs), size.value)
    _run(L.nvfp4_add_norm_grad, args, (*(t for t in rows.values()), *outs, *named)[0 if dh is not None else 1:])
    return out
