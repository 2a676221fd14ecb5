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


def test_linear_refusals():
    L = nv.layer.layer_lib()

    def call(e, x=P, kind=1, ld=64, b=P, M=40, N=4, K=64, ws=P, n=1 << 30, out=P):
        return L.nvfp4_mx_linear_fused(x, kind, ld, b, P, 1.0, e, out, 1, M, N, K, ws, n, None)

    for e in (epi(), None):
        for bad in (dict(x=None), dict(kind=2), dict(ld=60), dict(b=None), dict(M=-1), dict(N=0), dict(K=48), dict(ws=None),
                    dict(n=sum(nv.mx_packed_size(40, 64)) - 1), dict(out=None)):
            assert call(e, **bad) == INV, bad
        for bad in (dict(x=P + 8), dict(ws=P + 8), dict(out=P + 2), dict(M=3, x=P + 8)):
            assert call(e, **bad) == MIS, bad
        assert call(e, M=3, K=48) == INV and call(e, M=3, ld=60) == INV
    for bad in BAD_EPILOGUES:
        assert call(epi(**bad)) == INV and call(epi(**bad), M=3, ws=None) == INV, bad


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
    for module in (nv.mx, nv.layer):
        monkeypatch.setattr(module, "_run", lambda fn, args, tensors: calls.append((fn.__name__, args, tensors)))
    b, g = operand(7), operand(7)
    for lead in ((3,), (2, 3), (4, 100)):
        n = int(torch.tensor(lead).prod())
        r = torch.zeros(*lead, 7, dtype=torch.bfloat16)
        e = nv.MxEpilogue("silu", torch.zeros(7), g, torch.ones(7), r)
        nv.mx_linear(torch.zeros(*lead, 64), b, epilogue=e)
        name, args, tensors = calls[-1]
        assert name == "nvfp4_mx_linear_fused"
        s = next(a for a in args if isinstance(a, nv.layer._EpilogueT))
        work = tensors[4]
        size = sum(nv.mx_packed_size(n, 64)) if n > 16 else 0
        assert (work is None) == (size == 0) and args[args.index(s) - 1] == 1.0
        assert args[-5:] == (n, 7, 64, work.data_ptr() if size else None, size)
        assert (s.activation, s.gate_packed, s.gate_scales, s.bias, s.gate_bias, s.bias_type, s.residual, s.ld_residual) == \
            (2, g.codes.data_ptr(), g.scales.data_ptr(), e.bias.data_ptr(), e.gate_bias.data_ptr(), 0, r.data_ptr(), 7)
        assert all(any(t is u for u in tensors) for t in (e.bias, e.gate_bias, g.codes, g.scales))
    nv.mx_gemm(operand(4), b, epilogue=nv.MxEpilogue(gate=g, gate_bias=torch.zeros(7, dtype=torch.bfloat16)))
    s = calls[-1][1][5]
    assert (s.bias, s.bias_type) == (None, 1)


def norm(**kw):
    f = dict(type=1, weight_type=0, rows=4, hidden=64, post=1, pre=1, post_weight=P, pre_weight=P, gate_mode=0, gate=None,
             ld_gate=64, scale=1.0, residual_scale=1.0, eps=1e-6)
    return nv.layer._NormT(**{**f, **kw})


BAD_NORMS = [dict(type=2), dict(weight_type=3), dict(rows=-1), dict(rows=2 ** 31), dict(hidden=0), dict(hidden=16385),
             dict(gate_mode=3), dict(gate_mode=-1), dict(gate_mode=1), dict(gate_mode=2, gate=P, ld_gate=63),
             dict(gate_mode=2, gate=P, ld_gate=2 ** 31), dict(eps=-1.0), dict(eps=float("nan")),
             dict(gate_mode=1, gate=P, post_weight=None, pre_weight=None, weight_type=7)]
MISALIGNED_NORMS = [dict(post_weight=P + 2), dict(pre_weight=P + 1), dict(weight_type=1, pre_weight=P + 1),
                    dict(gate_mode=1, gate=P + 2), dict(gate_mode=2, gate=P + 1)]


@pytest.mark.parametrize("record", [False, True])
def test_norm_refusals(record):
    L = nv.layer.layer_lib()
    seq = ctypes.c_void_p()
    assert L.nvfp4_sequence_create(ctypes.byref(seq)) == nv.OK

    def call(f, y=P, ld=64, res=P, ldr=64, h=P, n=P, c=None, s=None):
        args = (f, y, ld, res, ldr, h, n, c, s)
        return L.nvfp4_sequence_add_norm(seq, *args) if record else L.nvfp4_add_norm(*args, None)

    assert call(None) == INV
    for bad in BAD_NORMS:
        assert call(norm(**bad)) == INV, bad
    for bad in MISALIGNED_NORMS:
        assert call(norm(**bad)) == MIS, bad
    for bad in (dict(y=None), dict(ld=63), dict(ld=-64), dict(ld=2 ** 31), dict(ldr=3), dict(n=None), dict(c=P, s=P),
                dict(n=None, c=P), dict(n=None, s=P), dict(h=None, n=None)):
        assert call(norm(), **bad) == INV, bad
    assert call(norm(pre=0)) == INV and call(norm(pre=0), n=None, c=P, s=P) == INV      # an n without its norm
    assert call(norm(pre=0), n=None, h=None) == INV
    assert call(norm(hidden=72), ld=72, ldr=72, n=None, c=P, s=P) == INV                # not whole blocks
    for bad in (dict(y=P + 1), dict(res=P + 1), dict(h=P + 1), dict(n=P + 1), dict(n=None, c=P + 8, s=P), dict(n=None, c=P, s=P + 4)):
        assert call(norm(), **bad) == MIS, bad
    assert call(norm(type=0), y=P + 2) == MIS
    if record:
        assert call(norm(rows=1), ld=0, ldr=0) == nv.OK
        assert call(norm(gate_mode=2, gate=P), h=None, n=None, c=P, s=P) == nv.OK
        assert call(norm(rows=0), y=None, res=None, h=None, n=None) == nv.OK
        assert L.nvfp4_sequence_add_norm(None, norm(), P, 64, P, 64, P, P, None, None) == INV
    L.nvfp4_sequence_destroy(seq)


def test_norm_grad_refusals():
    L = nv.layer.layer_lib()
    size = ctypes.c_size_t()

    def call(f, dh=P, ldh=64, dn=P, ldn=64, y=P, ldy=64, h=P, ldhh=64, dy=P, dr=P, dg=None, dp=P, dq=P, w=P, n=1 << 30):
        return L.nvfp4_add_norm_grad(f, dh, ldh, dn, ldn, y, ldy, h, ldhh, dy, dr, dg, dp, dq, w, n, None)

    assert call(None) == INV and L.nvfp4_add_norm_grad_workspace(None, ctypes.byref(size)) == INV
    assert L.nvfp4_add_norm_grad_workspace(norm(), None) == INV
    for bad in BAD_NORMS:
        assert call(norm(**bad)) == INV, bad
        assert L.nvfp4_add_norm_grad_workspace(norm(**bad), ctypes.byref(size)) == INV, bad
    for bad in (dict(dn=None), dict(y=None), dict(h=None), dict(ldh=8), dict(ldn=8), dict(ldy=8), dict(ldhh=8), dict(dg=P),
                dict(w=None), dict(n=16)):
        assert call(norm(), **bad) == INV, bad
    assert call(norm(pre=0), dn=None) == INV                                 # a gradient of pre_weight without its norm
    assert call(norm(pre=0), dq=None) == INV                                 # dn without its norm
    assert call(norm(post=0)) == INV                                         # a gradient of post_weight without its norm
    for bad in (dict(dh=P + 1), dict(dn=P + 1), dict(y=P + 1), dict(h=P + 1), dict(dy=P + 1), dict(dr=P + 1), dict(dp=P + 2),
                dict(dq=P + 2), dict(w=P + 8)):
        assert call(norm(), **bad) == MIS, bad
    assert call(norm(gate_mode=1, gate=P), dg=P + 2) == MIS and call(norm(gate_mode=2, gate=P), dg=P + 1) == MIS
    for f, zero in ((norm(), False), (norm(rows=0), True), (norm(post=0, pre=0), True),
                    (norm(post=0, pre=0, gate_mode=1, gate=P), False), (norm(post=0, pre=0, gate_mode=2, gate=P), True)):
        assert L.nvfp4_add_norm_grad_workspace(f, ctypes.byref(size)) == nv.OK and (size.value == 0) == zero


def test_norm_binding_refuses():
    y, w = torch.zeros(4, 64), torch.zeros(64)
    bf = dict(dtype=torch.bfloat16)
    for args, kw, match in [((torch.zeros(64),), {}, "two dimensions"), ((y.half(),), {}, "float32 or bfloat16"),
                            ((torch.zeros(2, 0),), {}, "elements"), ((torch.zeros(2, 16385),), {}, "elements"),
                            ((y, torch.zeros(4, 65)), {}, "residual"), ((y, torch.zeros(4, 64, **bf)), {}, "residual"),
                            ((y,), dict(post_weight=torch.zeros(63)), "post_weight"),
                            ((y,), dict(pre_weight=torch.zeros(64).half()), "pre_weight"),
                            ((y,), dict(post_weight=w, pre_weight=w.to(torch.bfloat16)), "one type"),
                            ((y,), dict(post_weight=w, post=False), "without its norm"),
                            ((y,), dict(pre_weight=w, pre=False), "without its norm"),
                            ((y,), dict(gate=torch.zeros(4, 1)), "gate"), ((y,), dict(gate=torch.zeros(4, 64, **bf)), "gate"),
                            ((y,), dict(pre=False, quantize=True), "no n"), ((y,), dict(pre=False, n=y), "no n"),
                            ((torch.zeros(4, 40),), dict(quantize=True), "multiple"),
                            ((y,), dict(quantize=True, n=y), "n must be"), ((y,), dict(quantize=True, n=operand(5)), "wrong shape"),
                            ((y,), dict(h=torch.zeros(4, 63)), "h must be"), ((y,), dict(n=torch.zeros(64, 4).t()), "n must be")]:
        with pytest.raises(ValueError, match=match):
            nv.add_norm(*args, **kw)
    with pytest.raises(ValueError, match="GPU"):
        nv.rms_norm(y, w)
    for args, kw, match in [((None, None, y, y), {}, "dh or dn"), ((y, y, y, None), {}, "h must be given"),
                            ((y, None, None, None), dict(post=True), "y must be given"), ((y, None, y, y), dict(pre=True), "dn must"),
                            ((y, y, y, y), dict(pre=False), "dn must"), ((y, torch.zeros(4, 65), y, y), {}, "dn"),
                            ((y, y, torch.zeros(3, 64), y), dict(post=True), "y must be"), ((y, None, y, y), dict(pre_weight=w), "without its norm")]:
        with pytest.raises(ValueError, match=match):
            nv.add_norm_grad(*args, **kw)
    seq = nv.Sequence()
    for kw in (dict(h=None), dict(h=None, n=None, pre=False), dict(h=y)):
        with pytest.raises(ValueError, match="out"):
            seq.add_norm(y, None, **kw)
    assert seq.calls == 0


def layer(**kw):
    f = dict(experts=8, hidden=64, inner=96, activation=2, gate_packed=P, gate_scales=P, up_packed=P, up_scales=P,
             down_packed=P, down_scales=P, bias_type=0, gate_bias=P, up_bias=P, down_bias=P)
    return nv.layer._ExpertsT(**{**f, **kw})


@pytest.mark.parametrize("tokens", [4, 500])
@pytest.mark.parametrize("record", [False, True])
def test_moe_refusals(record, tokens):
    L = nv.layer.layer_lib()
    seq = ctypes.c_void_p()
    assert L.nvfp4_sequence_create(ctypes.byref(seq)) == nv.OK

    def call(f, x=P, kind=1, ld=64, ids=P, idt=0, w=P, T=tokens, k=2, out=P, ok=1, ws=P, n=1 << 40):
        args = (f, x, kind, ld, ids, idt, w, T, k, out, ok, ws, n)
        return L.nvfp4_sequence_add_mx_moe(seq, *args) if record else L.nvfp4_mx_moe(*args, None)

    assert call(None) == INV
    for bad in (dict(experts=0), dict(experts=2049), dict(hidden=0), dict(hidden=48), dict(inner=40), dict(inner=-32),
                dict(hidden=2 ** 23), dict(activation=9), dict(gate_packed=None), dict(gate_scales=None), dict(up_packed=None),
                dict(up_scales=None), dict(down_packed=None), dict(down_scales=None), dict(bias_type=2),
                dict(gate_packed=None, gate_scales=None)):                       # (a bias of no gate)
        assert call(layer(**bad)) == INV, bad
    for bad in (dict(x=None), dict(kind=2), dict(ld=32), dict(ld=68), dict(ids=None), dict(idt=2), dict(T=-1), dict(T=2 ** 24),
                dict(k=0), dict(k=2 ** 24), dict(T=2 ** 20, k=2 ** 11), dict(out=None), dict(ok=5), dict(ws=None), dict(n=100)):
        assert call(layer(), **bad) == INV, bad
    for bad in (dict(x=P + 8), dict(ids=P + 2), dict(ids=P + 4, idt=1), dict(w=P + 2), dict(out=P + 8), dict(ws=P + 8)):
        assert call(layer(), **bad) == MIS, bad
    for bad in (dict(gate_packed=P + 8), dict(up_scales=P + 4), dict(down_packed=P + 1), dict(up_bias=P + 2),
                dict(bias_type=1, down_bias=P + 1)):
        assert call(layer(**bad)) == MIS, bad
    size = ctypes.c_size_t()
    assert L.nvfp4_mx_moe_workspace(None, 4, 2, 1, ctypes.byref(size)) == INV
    assert L.nvfp4_mx_moe_workspace(layer(), 4, 2, 1, None) == INV and L.nvfp4_mx_moe_workspace(layer(), -1, 2, 1, ctypes.byref(size)) == INV
    assert L.nvfp4_mx_moe_workspace(layer(), tokens, 2, 1, ctypes.byref(size)) == nv.OK
    need = size.value
    assert call(layer(), n=need - 1) == INV
    assert L.nvfp4_mx_moe_workspace(layer(), 0, 2, 1, ctypes.byref(size)) == nv.OK and size.value == 0
    if record:
        assert call(layer(), n=need) == nv.OK
        assert call(layer(gate_packed=None, gate_scales=None, gate_bias=None), w=None, n=need) == nv.OK
        assert call(layer(), T=0, x=None, ids=None, out=None, ws=None, n=0) == nv.OK
        assert L.nvfp4_sequence_add_mx_moe(None, layer(), P, 1, 64, P, 0, P, 4, 2, P, 1, P, 1 << 40) == INV
    L.nvfp4_sequence_destroy(seq)


def test_moe_binding_refuses():
    up, down, gate = groups(3, 96, 64), groups(3, 64, 96), groups(3, 96, 64)
    x, ids, p = torch.zeros(4, 64), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    seq, out = nv.Sequence(), torch.zeros(4, 64, dtype=torch.bfloat16)
    for args, kw, match in [((x, ids, p, operand(96), down), {}, "up must be"), ((x, ids, p, up, operand(64, 96)), {}, "down must be"),
                            ((x, ids, p, up, down), dict(gate=operand(96)), "gate must be"), ((x, ids, p, up, up), {}, "down must be 3"),
                            ((x, ids, p, up, groups(2, 64, 96)), {}, "down must be 3"), ((x, ids, p, up, down), dict(gate=down), "gate must be 3"),
                            ((x, ids, p, up, down), dict(gate_bias=torch.zeros(3, 96)), "needs a gate"),
                            ((x[:, :32], ids, p, up, down), {}, "rows of 32"), ((x.half(), ids, p, up, down), {}, "float32 or bfloat16"),
                            ((x, ids[:3], p, up, down), {}, "expert_ids"), ((x, ids.float(), p, up, down), {}, "expert_ids"),
                            ((x, ids.t().contiguous().t(), p, up, down), {}, "expert_ids"), ((x, ids, p[:, :1], up, down), {}, "weights"),
                            ((x, ids, p.double(), up, down), {}, "weights"), ((x, ids, p, up, down), dict(activation="elu"), "activation"),
                            ((x, ids, p, up, down), dict(up_bias=torch.zeros(96)), "up_bias"),
                            ((x, ids, p, up, down), dict(down_bias=torch.zeros(3, 96)), "down_bias"),
                            ((x, ids, p, up, down), dict(up_bias=torch.zeros(3, 96), down_bias=torch.zeros(3, 64).bfloat16()), "one type"),
                            ((x, ids, p, nv.MxGroups(up.codes[:-1], up.scales, 3, 96, 64), down), {}, "up.codes")]:
        with pytest.raises(ValueError, match=match):
            nv.mx_moe(*args, **kw)
        with pytest.raises(ValueError, match=match):
            seq.add_mx_moe(*args, out, **kw)
    for kw, match in ((dict(out=torch.zeros(4, 63)), "out"), (dict(dtype=torch.float16), "out"), ({}, "GPU")):
        with pytest.raises(ValueError, match=match):
            nv.mx_moe(x, ids, p, up, down, gate, **kw)
    with pytest.raises(ValueError, match="out"):
        seq.add_mx_moe(x, ids, p, up, down, None)
    assert seq.calls == 0


def test_recorded_rows_are_not_copies():
    """Eager calls copy rows that do not follow each other at one stride; a recorded call would keep what they held."""
    seq, rows, wide = nv.Sequence(), torch.zeros(4, 8), torch.zeros(8, 4).t()
    for y, r, gate, match in ((wide, rows, None, "y does"), (rows, rows[:1].expand(4, 8), None, "residual does"),
                              (rows, wide, None, "residual does"), (rows, None, wide, "gate does"),
                              (torch.zeros(4, 2, 8)[:, :1].expand(4, 2, 8), None, None, "y does")):
        with pytest.raises(ValueError, match=match):
            seq.add_norm(y, r, torch.zeros(*y.shape), torch.zeros(*y.shape), gate=gate)
    with pytest.raises(ValueError, match="GPU"):
        seq.add_norm(torch.zeros(4, 2, 9)[..., 1:], torch.zeros(4, 2, 8), torch.zeros(4, 2, 8), torch.zeros(4, 2, 8), gate=torch.ones(8))
    assert seq.calls == 0


def test_broadcast_residuals_of_a_linear_layer_are_copied(monkeypatch):
    """Rows of a residual that overlap (one row for all of them) reach the call as rows of their own."""
    calls = []
    monkeypatch.setattr(nv.layer, "_run", lambda fn, args, tensors: calls.append((args, tensors)))
    b, row = operand(7), torch.arange(7, dtype=torch.bfloat16)
    for lead in ((6,), (2, 3), (40,), (4, 2, 5)):
        n = int(torch.tensor(lead).prod())
        whole = torch.arange(n * 7, dtype=torch.bfloat16).view(*lead, 7)
        wide = torch.zeros(*lead, 9, dtype=torch.bfloat16)[..., :7]
        some = [row.expand(*lead, 7), whole] + [whole[..., :1, :].expand(*lead, 7)] * (len(lead) > 1)
        for r in some + [wide]:
            nv.mx_linear(torch.zeros(*lead, 64), b, epilogue=nv.MxEpilogue(residual=r))
            args, tensors = calls[-1]
            s = next(a for a in args if isinstance(a, nv.layer._EpilogueT))
            read = next(t for t in tensors if t is not None and t.data_ptr() == s.residual and t.shape == (n, 7))
            assert s.ld_residual == read.stride(0) >= 7 and torch.equal(read.reshape(*lead, 7), r)
            assert (s.residual == r.data_ptr()) == (r is whole or r is wide)
    one = nv.MxEpilogue(residual=torch.zeros(5, 1, dtype=torch.bfloat16)[:1].expand(5, 1))
    nv.mx_linear(torch.zeros(5, 64), operand(1), epilogue=one)
    assert next(a for a in calls[-1][0] if isinstance(a, nv.layer._EpilogueT)).ld_residual == 1
    out = torch.zeros(3, 7, dtype=torch.bfloat16)
    nv.mx_linear(torch.zeros(3, 64), b, out=out, epilogue=nv.MxEpilogue(residual=out))      # (in place: never a copy)
    assert next(a for a in calls[-1][0] if isinstance(a, nv.layer._EpilogueT)).residual == out.data_ptr()


def test_linear_without_rows():
    """No rows: nothing to do and no workspace to do it in, whatever the weight's size (without a GPU the call comes as
    far as looking for one)."""
    L = nv.layer.layer_lib()
    for N, K in ((4, 64), (9000, 16384), (131072, 8192)):
        for e in (None, epi(2, P, P, P, P, 1, P, N)):
            st = L.nvfp4_mx_linear_fused(None, 1, K, P, P, 1.0, e, None, 1, 0, N, K, None, 0, None)
            assert st in (nv.OK, nv.ERR_HIP), (N, K)
            assert L.nvfp4_mx_linear_fused(None, 1, K, P, P, 1.0, e, None, 1, 0, N, K - 16, None, 0, None) == INV


def test_linear_of_few_rows_needs_no_workspace():
    """Up to 16 rows run without one, whatever the weight's size (without a GPU the call comes as far as looking for one)."""
    L = nv.layer.layer_lib()
    for M, N, K in ((1, 4, 64), (16, 9000, 16384), (16, 768, 9984), (5, 131072, 8224)):
        for e in (None, epi(2, P, P, P, P, 1, P, N)):
            for ws, n in ((None, 0), (P, sum(nv.mx_packed_size(M, K)) - 1)):
                if torch.cuda.is_available():
                    continue    # (the addresses stand for nothing)
                assert L.nvfp4_mx_linear_fused(P, 1, K, P, P, 1.0, e, P, 1, M, N, K, ws, n, None) == nv.ERR_HIP, (M, N, K)
    assert L.nvfp4_mx_linear_fused(P, 1, 64, P, P, 1.0, None, P, 1, 17, 4, 64, None, 0, None) == INV
