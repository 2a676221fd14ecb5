"""Python binding of expert routing (``include/nvfp4_moe.h``): a router's
choices sorted by expert, token rows laid out in that order for a grouped
product, added up again under the router's weights, and the gradients.
Argument marshalling only.

    route = moe_sort(expert_ids, experts)
    y = mx_grouped_gemm(mx_quantize(x), w, route.row_offsets, rows=route.tokens)
    out = moe_combine(y, route, weights)

or, for a product that reads its rows in order (``grouped_gemm``), with
``moe_gather(x, route)`` in front of it.

The gradients are functions of their own (``moe_gather_grad``,
``moe_combine_grad``): nothing here is recorded by autograd, and results carry
no history, whatever the inputs require.  A training program calls them from
the backward of its own ``torch.autograd.Function``; the products between them
have no backward form here.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _i64, _vp, lib
from .mx import _on, _rows_2d, _run

INDEX_I32 = 0   # types of expert numbers (nvfp4_moe.h)
INDEX_I64 = 1
MOE_MAX_EXPERTS = 2048

MOE_EXPORTS = ["nvfp4_moe_sort", "nvfp4_moe_gather", "nvfp4_moe_combine",
               "nvfp4_moe_combine_grad", "nvfp4_sequence_add_moe_sort",
               "nvfp4_sequence_add_moe_gather", "nvfp4_sequence_add_moe_combine"]

_int = ctypes.c_int
_SORT = [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp]
_GATHER = [_vp, _int, _i64, _i64, _i64, _i64, _vp, _vp]
_COMBINE = [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp]
_GRAD = [_vp, _i64, _vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp]
_bound = None


def moe_lib() -> ctypes.CDLL:
    """The library with the argument types of its routing functions set."""
    global _bound
    L = lib()
    if _bound is not L:
        for name, types in (("nvfp4_moe_sort", _SORT + [_vp]),
                            ("nvfp4_moe_gather", _GATHER + [_vp]),
                            ("nvfp4_moe_combine", _COMBINE + [_vp]),
                            ("nvfp4_moe_combine_grad", _GRAD + [_vp]),
                            ("nvfp4_sequence_add_moe_sort", [_vp] + _SORT),
                            ("nvfp4_sequence_add_moe_gather", [_vp] + _GATHER),
                            ("nvfp4_sequence_add_moe_combine", [_vp] + _COMBINE)):
            f = getattr(L, name)
            f.restype, f.argtypes = _int, types
        _bound = L
    return L


@dataclass
class MoeRoute:
    """A router's choices sorted by expert (int32 device tensors):
    ``row_offsets`` [experts + 1] where each expert's rows begin, ``slots``
    [tokens, topk] the row of each choice (-1: dropped) and ``tokens``
    [tokens * topk] the token of each row (-1 behind the last one)."""
    row_offsets: "object"
    slots: "object"
    tokens: "object"
    experts: int

    def check(self) -> None:
        off, slots, tokens = self.row_offsets, self.slots, self.tokens
        if not (off.dtype is slots.dtype is tokens.dtype is torch.int32 and slots.dim() == 2
                and off.numel() == self.experts + 1 and tokens.numel() == slots.numel()
                and off.is_contiguous() and slots.is_contiguous() and tokens.is_contiguous()):
            raise ValueError("the tables of a route must be contiguous int32 tensors of their shapes")


def _sort_args(ids, experts, out):
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise ValueError("expert_ids must be a contiguous [tokens, topk] int32 or int64 tensor")
    if not 1 <= experts <= MOE_MAX_EXPERTS:
        raise ValueError(f"experts must be 1 to {MOE_MAX_EXPERTS}, not {experts}")
    T, k = ids.shape
    if out is None:
        tables = ids.new_empty(2 * T * k + experts + 1, dtype=torch.int32)
        slots, tokens, off = tables.split((T * k, T * k, experts + 1))
        out = MoeRoute(off, slots.view(T, k), tokens, experts)
    else:
        out.check()
        if out.experts != experts or tuple(out.slots.shape) != (T, k):
            raise ValueError("out has the wrong shape")
    return out, (ids.data_ptr(), INDEX_I64 if ids.dtype is torch.int64 else INDEX_I32, T, k,
                 experts, out.row_offsets.data_ptr(), out.slots.data_ptr(), out.tokens.data_ptr())


def moe_sort(expert_ids, experts: int, out: MoeRoute | None = None, stream=None) -> MoeRoute:
    """Sort a router's choices, ``expert_ids`` [tokens, topk] (int32 or int64
    device tensor; numbers outside [0, experts) are dropped choices), by
    expert, those of one expert by token (nvfp4_moe_sort).  At most
    MOE_MAX_EXPERTS experts."""
    if stream is not None:
        with _on(stream, expert_ids):
            return moe_sort(expert_ids, experts, out)
    out, args = _sort_args(expert_ids, experts, out)
    _run(moe_lib().nvfp4_moe_sort, args, (expert_ids, out.row_offsets, out.slots, out.tokens))
    return out


def _weights(weights, route):
    if weights is None:
        return None
    if (weights.dtype != torch.float32 or weights.shape != route.slots.shape
            or not weights.is_contiguous()):
        raise ValueError("weights must be a contiguous float32 tensor of shape "
                         f"{tuple(route.slots.shape)}")
    return weights.data_ptr()


def _like(t, name: str, rows: int, hidden: int, dtype, like):
    """`t` made beside `like`, or checked to be a contiguous rows x hidden tensor of `dtype`."""
    if t is None:
        return like.new_empty((rows, hidden), dtype=dtype)
    if tuple(t.shape) != (rows, hidden) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape ({rows}, {hidden})")
    return t


def _gather_args(x, route, out):
    kind = _rows_2d(x)
    route.check()
    T, k = route.slots.shape
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, the route {T} tokens")
    out = _like(out, "out", T * k, x.shape[1], x.dtype, x)
    return out, (x.data_ptr(), kind, T, k, x.shape[1], x.stride(0), route.slots.data_ptr(),
                 out.data_ptr())


def moe_gather(x, route: MoeRoute, out=None, stream=None):
    """The rows of x (tokens x hidden, rows may be strided) in the experts'
    order, one for each kept choice (nvfp4_moe_gather): [tokens * topk,
    hidden].  Rows that no choice owns (behind row_offsets[-1]) are left as
    they were in ``out``: in one that the call makes they hold anything.  Pass a
    zeroed ``out`` to a product or a sum that reads all rows."""
    if stream is not None:
        with _on(stream, x):
            return moe_gather(x, route, out)
    out, args = _gather_args(x, route, out)
    _run(moe_lib().nvfp4_moe_gather, args, (x, route.slots, out))
    return out


def _combine_args(y, route, weights, out):
    kind = _rows_2d(y, "y")
    route.check()
    T, k = route.slots.shape
    y = _like(y, "y", T * k, y.shape[1], y.dtype, y)
    w = _weights(weights, route)
    out = _like(out, "out", T, y.shape[1], y.dtype, y)
    return out, (y.data_ptr(), kind, T, k, y.shape[1], route.slots.data_ptr(), w, out.data_ptr())


def moe_combine(y, route: MoeRoute, weights=None, out=None, stream=None):
    """out[t] = sum over token t's kept choices of weights[t, j] * y[row of the
    choice] (nvfp4_moe_combine), summed in fp32 in the order of j: [tokens,
    hidden].  ``weights``: float32 [tokens, topk]; None for ones."""
    if stream is not None:
        with _on(stream, y):
            return moe_combine(y, route, weights, out)
    out, args = _combine_args(y, route, weights, out)
    _run(moe_lib().nvfp4_moe_combine, args, (y, route.slots, weights, out))
    return out


def moe_gather_grad(dout, route: MoeRoute, out=None, stream=None):
    """The gradient of moe_gather: each token's row is the sum of the
    gradients ``dout`` [tokens * topk, hidden] of its kept choices' rows."""
    return moe_combine(dout, route, None, out, stream)


def moe_combine_grad(dout, y, route: MoeRoute, weights=None, dy=None, dweights=None, stream=None):
    """The gradients (dy, dweights) of moe_combine(y, route, weights) for its
    output's gradient ``dout`` [tokens, hidden] (rows may be strided)
    (nvfp4_moe_combine_grad).  Rows of dy that no choice owns are left as they
    were: in a dy that the call makes they hold anything (their gradient is zero:
    pass a zeroed ``dy`` to what reads all rows); dweights of dropped choices are
    zero.  ``dy`` may be y itself."""
    if stream is not None:
        with _on(stream, dout):
            return moe_combine_grad(dout, y, route, weights, dy, dweights)
    kind = _rows_2d(dout, "dout")
    route.check()
    T, k = route.slots.shape
    if dout.shape[0] != T:
        raise ValueError(f"dout has {dout.shape[0]} rows, the route {T} tokens")
    H = dout.shape[1]
    y = _like(y, "y", T * k, H, dout.dtype, dout)
    w = _weights(weights, route)
    dy = _like(dy, "dy", T * k, H, dout.dtype, dout)
    dweights = _like(dweights, "dweights", T, k, torch.float32, dout)
    args = (dout.data_ptr(), dout.stride(0), y.data_ptr(), kind, T, k, H, route.slots.data_ptr(), w,
            dy.data_ptr(), dweights.data_ptr())
    _run(moe_lib().nvfp4_moe_combine_grad, args, (dout, y, route.slots, weights, dy, dweights))
    return dy, dweights
