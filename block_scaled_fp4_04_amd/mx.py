"""Python binding of the MXFP4 operators (``include/nvfp4_mx.h``): argument
marshalling only, like the rest of the package.

MXFP4 holds 32 consecutive values of a row as E2M1 codes under one
power-of-two scale byte (E8M0).  ``mx_quantize`` makes packed operands from
fp32 or bfloat16 rows, ``mx_to_device`` from the canonical bytes of a
checkpoint, ``mx_gemm`` multiplies two of them, ``mx_linear`` takes plain
activations, and ``mx_grouped_gemm`` serves a layer of experts.

Tensors of one call lie on one GPU; the call runs there, on that GPU's current
stream unless ``stream`` names one.  Results carry no autograd history, whatever
the inputs require: quantisation has no gradient, and the products here have no
backward form.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import numpy as np
import torch

from . import Nvfp4Error, _i64, _u8p, _vp, lib

TYPE_F32 = 0    # element types of rows (nvfp4_mx.h)
TYPE_BF16 = 1
MX_BLOCK = 32   # elements that share a scale
MX_QUANT_ROWS = 16  # most rows of mx_gemm_quantized

MX_EXPORTS = ["nvfp4_mx_packed_size", "nvfp4_mx_pack", "nvfp4_mx_unpack", "nvfp4_mx_quantize",
              "nvfp4_mx_dequantize", "nvfp4_mx_gemm", "nvfp4_mx_gemm_quantized",
              "nvfp4_mx_grouped_gemm", "nvfp4_sequence_add_mx_quantize",
              "nvfp4_sequence_add_mx_gemm", "nvfp4_sequence_add_mx_gemm_quantized",
              "nvfp4_sequence_add_mx_grouped_gemm"]

_int, _f32, _szp = ctypes.c_int, ctypes.c_float, ctypes.POINTER(ctypes.c_size_t)
_QUANT = [_vp, _int, _i64, _i64, _i64, _i64, _i64, _vp, _vp]
_DEQUANT = [_vp, _vp, _i64, _i64, _i64, _vp, _int, _i64, _i64]
_GEMM = [_vp, _vp, _vp, _vp, _f32, _vp, _int, _i64, _i64, _i64]
_GEMM_Q = [_vp, _int, _i64, _vp, _vp, _f32, _vp, _int, _i64, _i64, _i64]
_GROUPED = [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _f32, _vp, _int, _i64, _i64, _i64]
_bound = None


def mx_lib() -> ctypes.CDLL:
    """The library with the argument types of its MXFP4 functions set."""
    global _bound
    L = lib()
    if _bound is not L:
        for name, types in (
                ("nvfp4_mx_packed_size", [_i64, _i64, _szp, _szp]),
                ("nvfp4_mx_pack", [_u8p, _u8p, _i64, _i64, _u8p, _u8p]),
                ("nvfp4_mx_unpack", [_u8p, _u8p, _i64, _i64, _u8p, _u8p]),
                ("nvfp4_mx_quantize", _QUANT + [_vp]),
                ("nvfp4_mx_dequantize", _DEQUANT + [_vp]),
                ("nvfp4_mx_gemm", _GEMM + [_vp]),
                ("nvfp4_mx_gemm_quantized", _GEMM_Q + [_vp]),
                ("nvfp4_mx_grouped_gemm", _GROUPED + [_vp]),
                ("nvfp4_sequence_add_mx_quantize", [_vp, _vp, _int, _i64, _i64, _i64, _vp, _vp]),
                ("nvfp4_sequence_add_mx_gemm", [_vp] + _GEMM),
                ("nvfp4_sequence_add_mx_gemm_quantized", [_vp] + _GEMM_Q),
                ("nvfp4_sequence_add_mx_grouped_gemm", [_vp] + _GROUPED)):
            f = getattr(L, name)
            f.restype, f.argtypes = _int, types
        _bound = L
    return L


def mx_packed_size(rows: int, K: int) -> tuple[int, int]:
    """(code bytes, scale bytes) of a packed rows x K operand."""
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    st = mx_lib().nvfp4_mx_packed_size(rows, K, ctypes.byref(cb), ctypes.byref(sb))
    if st:
        raise Nvfp4Error(st, f"nvfp4_mx_packed_size(rows={rows}, K={K})")
    return cb.value, sb.value


def _packed(rows: int, K: int) -> tuple[int, int]:
    """mx_packed_size without the call (the sizes are checked by the call
    that uses them)."""
    rb, steps = (rows + 15) // 16, (K + 127) // 128
    return rb * steps * 1024, rb * ((steps + 3) // 4) * 256


def _check_canonical(codes: np.ndarray, scales: np.ndarray) -> tuple[int, int]:
    if codes.dtype != np.uint8 or scales.dtype != np.uint8 or codes.ndim != 2 or scales.ndim != 2:
        raise ValueError("codes and scales must be 2-D uint8 arrays")
    rows, K = codes.shape[0], 2 * codes.shape[1]
    if K % MX_BLOCK or scales.shape != (rows, K // MX_BLOCK):
        raise ValueError(f"scales shape {scales.shape} does not match codes {codes.shape} "
                         "(one scale per 32 elements, K % 32 == 0)")
    return rows, K


def mx_pack(codes: np.ndarray, scales: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """Canonical host arrays (codes [rows, K/2], E8M0 scales [rows, K/32]) ->
    packed host arrays (nvfp4_mx_pack)."""
    codes, scales = np.ascontiguousarray(codes), np.ascontiguousarray(scales)
    rows, K = _check_canonical(codes, scales)
    cb, sb = mx_packed_size(rows, K)
    pc, ps = np.empty(cb, np.uint8), np.empty(sb, np.uint8)
    st = mx_lib().nvfp4_mx_pack(codes.ctypes.data_as(_u8p), scales.ctypes.data_as(_u8p), rows, K,
                                pc.ctypes.data_as(_u8p), ps.ctypes.data_as(_u8p))
    if st:
        raise Nvfp4Error(st, "nvfp4_mx_pack")
    return pc, ps


def mx_unpack(packed_codes: np.ndarray, packed_scales: np.ndarray, rows: int, K: int):
    """Packed host arrays -> canonical (codes, scales)."""
    packed_codes = np.ascontiguousarray(packed_codes, dtype=np.uint8)
    packed_scales = np.ascontiguousarray(packed_scales, dtype=np.uint8)
    if (packed_codes.size, packed_scales.size) != mx_packed_size(rows, K):
        raise ValueError("packed buffers have the wrong size")
    codes, scales = np.empty((rows, K // 2), np.uint8), np.empty((rows, K // MX_BLOCK), np.uint8)
    st = mx_lib().nvfp4_mx_unpack(packed_codes.ctypes.data_as(_u8p),
                                  packed_scales.ctypes.data_as(_u8p), rows, K,
                                  codes.ctypes.data_as(_u8p), scales.ctypes.data_as(_u8p))
    if st:
        raise Nvfp4Error(st, "nvfp4_mx_unpack")
    return codes, scales


def _check_packed(name: str, codes, scales, groups: int, rows: int, K: int) -> None:
    cb, sb = _packed(rows, K)
    if (codes.dtype is torch.uint8 and scales.dtype is torch.uint8 and codes.numel() == cb * groups
            and scales.numel() == sb * groups and codes.is_contiguous() and scales.is_contiguous()):
        return
    raise ValueError(f"{name}.codes and {name}.scales must be contiguous uint8 tensors of "
                     f"{cb * groups} and {sb * groups} bytes")


@dataclass
class MxOperand:
    """One MXFP4 operand in the packed layout, resident on a device.
    ``codes``/``scales`` are uint8 torch tensors; ``rows`` x ``K`` is the
    logical shape."""
    block = MX_BLOCK  # elements that share a scale (not a field)
    codes: "object"
    scales: "object"
    rows: int
    K: int

    def check(self, name: str) -> None:
        _check_packed(name, self.codes, self.scales, 1, self.rows, self.K)


@dataclass
class MxGroups:
    """The weight operands of a grouped product, each ``rows`` x ``K``, packed
    and concatenated, resident on a device."""
    block = MX_BLOCK  # elements that share a scale (not a field)
    codes: "object"
    scales: "object"
    groups: int
    rows: int
    K: int

    def check(self, name: str) -> None:
        _check_packed(name, self.codes, self.scales, self.groups, self.rows, self.K)


def _kind(x, name: str, *kinds) -> None:
    """Refuses an operand of another class: groups, and the operands of the
    other format, have the same fields."""
    if type(x) is not kinds[0] and not isinstance(x, kinds):
        raise ValueError(f"{name} must be {' or '.join(k.__name__ for k in kinds)}, not {type(x).__name__}")


def mx_to_device(codes: np.ndarray, scales: np.ndarray, device="cuda") -> MxOperand:
    """Pack canonical host arrays and copy them to ``device``."""
    rows, K = _check_canonical(codes, scales)
    pc, ps = mx_pack(codes, scales)
    return MxOperand(torch.from_numpy(pc).to(device), torch.from_numpy(ps).to(device), rows, K)


def mx_groups_to_device(codes: np.ndarray, scales: np.ndarray, device="cuda") -> MxGroups:
    """Pack canonical weights [G, rows, K/2] and [G, rows, K/32] and copy
    them to ``device``."""
    if codes.ndim != 3 or scales.ndim != 3 or codes.shape[0] != scales.shape[0]:
        raise ValueError("codes and scales must be [G, rows, K/2] and [G, rows, K/32]")
    parts = [mx_pack(c, s) for c, s in zip(codes, scales)]
    pc, ps = np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])
    return MxGroups(torch.from_numpy(pc).to(device), torch.from_numpy(ps).to(device),
                    codes.shape[0], codes.shape[1], 2 * codes.shape[2])


# ---- what the calls share ---------------------------------------------------


def _gpu_of(tensors) -> int:
    """The index of the GPU that all the tensors (None left out) lie on."""
    gpu = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != gpu:
            raise ValueError(f"tensors must be on one device, not on {tensors[0].device} and {t.device}")
    if gpu < 0:
        raise ValueError(f"tensors must be on a GPU, not on {tensors[0].device}")
    return gpu


def _on(stream, like):
    """The context of a stream (a torch stream, or a raw handle of one of the
    GPU that `like` is on): what a call allocates in it belongs to that
    stream."""
    gpu = _gpu_of((like,))
    if not hasattr(stream, "cuda_stream"):
        stream = (torch.cuda.ExternalStream(int(stream), device=gpu) if int(stream)
                  else torch.cuda.default_stream(gpu))
    if stream.device_index != gpu:
        raise ValueError(f"the stream is one of {stream.device}, the tensors are on {like.device}")
    return torch.cuda.stream(stream)


_current_gpu = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _run(fn, args: tuple, tensors: tuple) -> None:
    """Calls the C function on the GPU where the tensors lie, on its current
    stream."""
    gpu = _gpu_of(tensors)
    if gpu == _current_gpu():
        st = fn(*args, _current_stream(gpu))
    else:
        with torch.cuda.device(gpu):
            st = fn(*args, _current_stream(gpu))
    if st:
        sizes = ", ".join(str(a) for a in args if isinstance(a, int) and 0 <= a < 1 << 31)
        raise Nvfp4Error(st, f"{fn.__name__}({sizes})")


_KINDS = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16}


def _type_of(dtype, what: str) -> int:
    kind = _KINDS.get(dtype)
    if kind is None:
        raise ValueError(f"{what} must be float32 or bfloat16, not {dtype}")
    return kind


def _out(out, dtype, M: int, N: int, like):
    """The output tensor (made beside `like`, bfloat16 by default, or the given
    one checked) and its type code."""
    if out is None:
        dtype = dtype or torch.bfloat16
        return like.new_empty((M, N), dtype=dtype), _type_of(dtype, "out")
    if dtype not in (None, out.dtype):
        raise ValueError(f"out is of type {out.dtype}, not {dtype}")
    if tuple(out.shape) != (M, N) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous tensor of shape ({M}, {N})")
    return out, _type_of(out.dtype, "out")


def _rows_2d(x, what: str = "x") -> int:
    """Checks a 2-D float32 / bfloat16 tensor with unit stride along K and
    returns its type code."""
    strides = x.stride()
    if len(strides) != 2 or (strides[1] != 1 and x.shape[1] != 1):
        raise ValueError(f"{what} must be a 2-D tensor with unit stride along its rows")
    return _type_of(x.dtype, what)


def _quantize_args(x, out):
    """(operand, C arguments) of mx_quantize for a 2-D or 3-D x."""
    strides, shape = x.stride(), x.shape
    if len(shape) not in (2, 3) or strides[-1] != 1:
        raise ValueError("x must be a 2-D or 3-D tensor with unit stride along K")
    kind = _type_of(x.dtype, "x")
    grouped = len(shape) == 3
    groups, group_stride = (shape[0], strides[0]) if grouped else (1, 0)
    rows, K = shape[-2:]
    if out is None:
        if K < MX_BLOCK or K % MX_BLOCK:
            raise ValueError(f"K must be a positive multiple of {MX_BLOCK}, not {K}")
        cb, sb = _packed(rows, K)
        codes = x.new_empty(cb * groups, dtype=torch.uint8)
        scales = x.new_empty(sb * groups, dtype=torch.uint8)
        out = MxGroups(codes, scales, groups, rows, K) if grouped else MxOperand(codes, scales, rows, K)
    else:
        _kind(out, "out", MxGroups if grouped else MxOperand)
        if (out.rows, out.K) != (rows, K) or grouped and out.groups != groups:
            raise ValueError("out has the wrong shape")
        out.check("out")
        codes, scales = out.codes, out.scales
    return out, (x.data_ptr(), kind, groups, group_stride, rows, K, strides[-2], codes.data_ptr(),
                 scales.data_ptr())


def mx_quantize(x, out=None, stream=None):
    """Quantise fp32 or bfloat16 device rows to packed MXFP4
    (nvfp4_mx_quantize): a 2-D x (rows x K) gives an MxOperand, a 3-D one
    (groups x rows x K, the weights of a layer of experts) MxGroups; or fills
    ``out``.  K is a multiple of 32; rows and groups may be strided (by whole
    16 bytes)."""
    if stream is not None:
        with _on(stream, x):
            return mx_quantize(x, out)
    out, args = _quantize_args(x, out)
    _run(mx_lib().nvfp4_mx_quantize, args, (x, out.codes, out.scales))
    return out


def mx_dequantize(a, dtype=None, out=None, stream=None):
    """The values of an MxOperand (rows x K) or MxGroups (groups x rows x K)
    as bfloat16 (default) or float32, exact in both but that values from 2^128
    on are infinities (nvfp4_mx_dequantize)."""
    _kind(a, "a", MxOperand, MxGroups)
    if stream is not None:
        with _on(stream, a.codes):
            return mx_dequantize(a, dtype, out)
    groups = getattr(a, "groups", None)
    shape = (a.rows, a.K) if groups is None else (groups, a.rows, a.K)
    if out is None:
        out = torch.empty(shape, dtype=dtype or torch.bfloat16, device=a.codes.device)
    elif tuple(out.shape) != shape or out.stride(-1) != 1 or dtype not in (None, out.dtype):
        raise ValueError(f"out must be a tensor of shape {shape} with unit stride along K")
    a.check("a")
    args = (a.codes.data_ptr(), a.scales.data_ptr(), 1 if groups is None else groups, a.rows, a.K,
            out.data_ptr(), _type_of(out.dtype, "out"), 0 if groups is None else out.stride(0),
            out.stride(-2))
    _run(mx_lib().nvfp4_mx_dequantize, args, (a.codes, a.scales, out))
    return out


def _gemm_args(a, b, alpha, out, dtype):
    _kind(a, "a", MxOperand)
    _kind(b, "b", MxOperand)
    if a.K != b.K:
        raise ValueError(f"K dimension mismatch: A has K={a.K}, B has K={b.K}")
    a.check("a")
    b.check("b")
    out, kind = _out(out, dtype, a.rows, b.rows, a.codes)
    return out, (a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(),
                 float(alpha), out.data_ptr(), kind, a.rows, b.rows, a.K)


def mx_gemm(a: MxOperand, b: MxOperand, alpha: float = 1.0, out=None, dtype=None, stream=None):
    """C = alpha * (A . B^T) of packed MXFP4 operands (nvfp4_mx_gemm): M x N,
    bfloat16 unless ``dtype`` or ``out`` says float32."""
    if stream is not None:
        with _on(stream, a.codes):
            return mx_gemm(a, b, alpha, out, dtype)
    out, args = _gemm_args(a, b, alpha, out, dtype)
    _run(mx_lib().nvfp4_mx_gemm, args, (a.codes, a.scales, b.codes, b.scales, out))
    return out


def _gemm_quantized_args(x, b, alpha, out, dtype):
    _kind(b, "b", MxOperand)
    kind = _rows_2d(x)
    M, K = x.shape
    if K != b.K:
        raise ValueError(f"K dimension mismatch: x has K={K}, B has K={b.K}")
    b.check("b")
    out, out_kind = _out(out, dtype, M, b.rows, x)
    return out, (x.data_ptr(), kind, x.stride(0), b.codes.data_ptr(), b.scales.data_ptr(),
                 float(alpha), out.data_ptr(), out_kind, M, b.rows, K)


def mx_gemm_quantized(x, b: MxOperand, alpha: float = 1.0, out=None, dtype=None, stream=None):
    """mx_gemm(mx_quantize(x), b, alpha) in one launch, bit for bit
    (nvfp4_mx_gemm_quantized): x holds up to MX_QUANT_ROWS rows of fp32 or
    bfloat16 activations."""
    if stream is not None:
        with _on(stream, x):
            return mx_gemm_quantized(x, b, alpha, out, dtype)
    out, args = _gemm_quantized_args(x, b, alpha, out, dtype)
    _run(mx_lib().nvfp4_mx_gemm_quantized, args, (x, b.codes, b.scales, out))
    return out


def mx_linear(x, b: MxOperand, alpha: float = 1.0, out=None, dtype=None, stream=None):
    """C = alpha * (quantise(x) . B^T) for plain activations x (rows x K,
    fp32 or bfloat16): one launch (mx_gemm_quantized) for few rows, else
    mx_quantize and mx_gemm.  Both give the same bits.  Dimensions in front of
    K (batch x sequence x K) are rows, and C has them in front of N; an x whose
    rows do not follow each other at one stride is copied first."""
    if stream is not None:
        with _on(stream, x):
            return mx_linear(x, b, alpha, out, dtype)
    if x.dim() > 2:
        shape = (*x.shape[:-1], b.rows)
        if out is not None and (tuple(out.shape) != shape or not out.is_contiguous()):
            raise ValueError(f"out must be a contiguous tensor of shape {shape}")
        c = mx_linear(x.flatten(0, -2), b, alpha, None if out is None else out.flatten(0, -2), dtype)
        return c.view(shape) if out is None else out
    # (one launch: 16 x 65536 x 8192 52 us, 57 + 2.7 in two; 1 x 6144 x 6144 6.9, 6.4
    # + 2.7.  Behind K = 8192 every 16 columns quantise the rows again, which takes
    # about N K (6 + rows) / 2e8 us: worth it up to the 2.7 us and part of the
    # other call's 8.)
    if x.dim() == 2 and x.shape[0] <= MX_QUANT_ROWS and (
            b.K <= 8192 or b.rows * b.K * (6 + x.shape[0]) <= 800_000_000):
        return mx_gemm_quantized(x, b, alpha, out, dtype)
    _kind(b, "b", MxOperand)
    return mx_gemm(mx_quantize(x), b, alpha, out, dtype)


def _grouped_args(a, b, row_offsets, alpha, rows, out, dtype):
    _kind(a, "a", MxOperand)
    _kind(b, "b", MxGroups)
    if a.K != b.K:
        raise ValueError(f"K dimension mismatch: A has K={a.K}, B has K={b.K}")
    if (row_offsets.dtype != torch.int32 or row_offsets.numel() != b.groups + 1
            or not row_offsets.is_contiguous()):
        raise ValueError(f"row_offsets must be a contiguous int32 tensor of {b.groups + 1} entries")
    if rows is not None and (rows.dtype != torch.int32 or rows.dim() != 1
                             or not rows.is_contiguous()):
        raise ValueError("rows must be a contiguous 1-D int32 tensor")
    a.check("a")
    b.check("b")
    M = a.rows if rows is None else rows.numel()
    out, kind = _out(out, dtype, M, b.rows, a.codes)
    return out, (a.codes.data_ptr(), a.scales.data_ptr(), a.rows,
                 None if rows is None else rows.data_ptr(), b.codes.data_ptr(),
                 b.scales.data_ptr(), row_offsets.data_ptr(), b.groups, float(alpha),
                 out.data_ptr(), kind, M, b.rows, a.K)


def mx_grouped_gemm(a: MxOperand, b: MxGroups, row_offsets, alpha: float = 1.0, rows=None,
                    out=None, dtype=None, stream=None):
    """Grouped product (nvfp4_mx_grouped_gemm): rows row_offsets[g] ..
    row_offsets[g+1]-1 of C belong to group g, whose weights are b's g-th
    operand.  Row r of C takes row rows[r] of A (``MoeRoute.tokens``: the
    activations are quantised once per token and never copied), or row r
    without ``rows``.  Rows behind the last group are left as they were: in an
    ``out`` that the call makes they hold anything."""
    if stream is not None:
        with _on(stream, a.codes):
            return mx_grouped_gemm(a, b, row_offsets, alpha, rows, out, dtype)
    out, args = _grouped_args(a, b, row_offsets, alpha, rows, out, dtype)
    _run(mx_lib().nvfp4_mx_grouped_gemm, args,
         (a.codes, a.scales, b.codes, b.scales, row_offsets, rows, out))
    return out
