"""The operators around the products (include/nvfp4_layer.h) without a GPU:
symbols, and every refusal (all argument checks run before any device work)."""
import ctypes
import os
import re

import pytest

import block_scaled_fp4_04_amd as nv

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, MIS, UNS = nv.ERR_INVALID_VALUE, nv.ERR_MISALIGNED, nv.ERR_UNSUPPORTED
P = 0x100000  # stand-in for an aligned device address: refused calls never use it
U8 = dict(dtype=torch.uint8)


def operand(rows=4, K=64):
    cb, sb = nv.mx_packed_size(rows, K)
    return nv.MxOperand(torch.zeros(cb, **U8), torch.zeros(sb, **U8), rows, K)


def groups(n=2, rows=4, K=64):
    cb, sb = nv.mx_packed_size(rows, K)
    return nv.MxGroups(torch.zeros(cb * n, **U8), torch.zeros(sb * n, **U8), n, rows, K)


def test_library_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "nvfp4_layer.h")).read()
    declared = sorted(set(re.findall(r"^int (nvfp4_\w+)\s*\(", text, re.M)))
    assert declared == sorted(nv.LAYER_EXPORTS)
    for n in declared:
        assert hasattr(nv.lib(), n), n
    assert nv.version() >= 10700 and "nvfp4_version() 10700" in text


def epi(act=0, gate=None, gscale=None, bias=None, gbias=None, btype=0, residual=None, ld=64):
    return nv.layer._EpilogueT(act, gate, gscale, bias, gbias, btype, residual, ld)


BAD_EPILOGUES = [dict(act=5), dict(act=-1), dict(gate=P), dict(gscale=P), dict(gbias=P), dict(bias=P, btype=2),
                 dict(gate=P, gscale=P, gbias=P, btype=-1), dict(residual=P, ld=3), dict(residual=P, ld=-8),
                 dict(residual=P, ld=2 ** 31)]
MISALIGNED = [dict(gate=P + 8, gscale=P), dict(gate=P, gscale=P + 4), dict(bias=P + 2), dict(bias=P + 1, btype=1),
              dict(gate=P, gscale=P, gbias=P + 1, btype=1), dict(residual=P + 1)]


@pytest.mark.parametrize("record", [False, True])
def test_epilogue_refusals(record):
    L = nv.layer.layer_lib()
    h = ctypes.c_void_p()
    assert L.nvfp4_sequence_create(ctypes.byref(h)) == nv.OK

    def call(name, *args):
        if record:
            return getattr(L, "nvfp4_sequence_add_" + name)(h, *args)
        return getattr(L, "nvfp4_" + name)(*args, None)

    def gemm(e, M=4, N=4, K=64, kind=1):
        return call("mx_gemm_fused", P, P, P, P, 1.0, e, P, kind, M, N, K)

    def quantized(e, M=4, N=4, K=64):
        return call("mx_gemm_quantized_fused", P, 1, K, P, P, 1.0, e, P, 1, M, N, K)

    def grouped(e, M=4, N=4, K=64):
        return call("mx_grouped_gemm_fused", P, P, M, None, P, P, P, 2, 1.0, e, P, 1, M, N, K)

    for f in (gemm, quantized, grouped):
        for bad in BAD_EPILOGUES:
            assert f(epi(**bad)) == INV, bad
        for bad in MISALIGNED:
            assert f(epi(**bad)) == MIS, bad
        assert f(epi(), K=48) == INV and f(epi(), N=0) == INV and f(epi(), M=-1) == INV
        assert f(None, K=48) == INV                                     # without one: the plain call's checks
        if record:
            assert f(epi(2, P, P, P, P, 1, P, 4)) == nv.OK
            assert f(epi(residual=P, ld=0), M=1) == nv.OK              # (a single row's stride is not looked at)
            assert f(None) == nv.OK
    assert gemm(epi(residual=P + 2), kind=0) == MIS
    assert quantized(epi(), M=17) == UNS
    assert L.nvfp4_sequence_add_mx_gemm_fused(None, P, P, P, P, 1.0, epi(), P, 1, 4, 4, 64) == INV
    L.nvfp4_sequence_destroy(h)


def test_epilogue_binding_refuses():
    a, w, off = operand(), groups(), torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(4, 64)
    bf = dict(dtype=torch.bfloat16)
    E = nv.MxEpilogue
    cb, sb = nv.packed_size(4, 64)
    other = nv.PackedOperand(torch.zeros(cb, **U8), torch.zeros(sb, **U8), 4, 64)
    cases = [(E("tanh"), "activation"), (E(bias=torch.zeros(5)), "bias"), (E(bias=torch.zeros(4).half()), "bias"),
             (E(bias=torch.zeros(8)[::2]), "bias"), (E(gate_bias=torch.zeros(4)), "gate_bias needs"),
             (E(gate=groups()), "gate must be"), (E(gate=other), "gate must be"), (E(gate=operand(8)), "sizes"),
             (E(gate=operand(4, 96)), "sizes"), (E(gate=operand(), gate_bias=torch.zeros(4), bias=torch.zeros(4, **bf)), "one type"),
             (E(gate=nv.MxOperand(a.codes[:512], a.scales, 4, 64)), "gate.codes"),
             (E(residual=torch.zeros(4, 4)), "residual"), (E(residual=torch.zeros(4, 5, **bf)), "residual"),
             (E(residual=torch.zeros(4, 4, **bf).t().contiguous().t()), "residual")]
    seq = nv.Sequence()
    out = torch.zeros(4, 4, **bf)
    for e, match in cases:
        for f in (lambda: nv.mx_gemm(a, a, epilogue=e), lambda: nv.mx_gemm_quantized(x, a, epilogue=e),
                  lambda: nv.mx_linear(x, a, epilogue=e), lambda: seq.add_mx_gemm(a, a, out, epilogue=e),
                  lambda: seq.add_mx_gemm_quantized(x, a, out, epilogue=e)):
            with pytest.raises(ValueError, match=match):
                f()
    for e, match in [(E(bias=torch.zeros(4)), "bias"), (E(gate=operand()), "gate must be MxGroups"), (E(gate=groups(3)), "sizes")]:
        for f in (lambda: nv.mx_grouped_gemm(a, w, off, epilogue=e),
                  lambda: seq.add_mx_grouped_gemm(a, w, off, out, epilogue=e)):
            with pytest.raises(ValueError, match=match):
                f()
    assert seq.calls == 0
    with pytest.raises(ValueError, match="GPU"):
        nv.mx_gemm(a, a, epilogue=E(bias=torch.zeros(4)))
    with pytest.raises(ValueError, match="residual"):
        nv.mx_linear(torch.zeros(2, 2, 64), a, epilogue=E(residual=torch.zeros(4, 4, **bf)))


def test_epilogue_arguments(monkeypatch):
    """What reaches the C function: every part, for each product, and the leading dimensions of a linear layer."""
    calls = []
    monkeypatch.setattr(nv.mx, "_run", lambda fn, args, tensors: calls.append((fn.__name__, args, tensors)))
    b, g = operand(7), operand(7)
    for lead in ((3,), (2, 3), (4, 100)):
        n = int(torch.tensor(lead).prod())
        r = torch.zeros(*lead, 7, dtype=torch.bfloat16)
        e = nv.MxEpilogue("silu", torch.zeros(7), g, torch.ones(7), r)
        nv.mx_linear(torch.zeros(*lead, 64), b, epilogue=e)
        name, args, tensors = calls[-1]
        assert name == ("nvfp4_mx_gemm_quantized_fused" if n <= 16 else "nvfp4_mx_gemm_fused")
        s = next(a for a in args if isinstance(a, nv.layer._EpilogueT))
        assert args[-3:] == (n, 7, 64) and args[args.index(s) - 1] == 1.0
        assert (s.activation, s.gate_packed, s.gate_scales, s.bias, s.gate_bias, s.bias_type, s.residual, s.ld_residual) == \
            (2, g.codes.data_ptr(), g.scales.data_ptr(), e.bias.data_ptr(), e.gate_bias.data_ptr(), 0, r.data_ptr(), 7)
        assert all(any(t is u for u in tensors) for t in (e.bias, e.gate_bias, g.codes, g.scales))
    nv.mx_gemm(operand(4), b, epilogue=nv.MxEpilogue(gate=g, gate_bias=torch.zeros(7, dtype=torch.bfloat16)))
    s = calls[-1][1][5]
    assert (s.bias, s.bias_type) == (None, 1)
