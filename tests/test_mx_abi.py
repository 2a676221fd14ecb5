"""MXFP4 and routing entry points without a GPU: symbols, the host packer and
every refusal (all argument checks run before any device work)."""
import ctypes
import os
import re

import numpy as np
import pytest

import block_scaled_fp4_04_amd as nv
import mx_ref

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, MIS, UNS = nv.ERR_INVALID_VALUE, nv.ERR_MISALIGNED, nv.ERR_UNSUPPORTED
P = 0x100000  # stand-in for an aligned device address: refused calls never use it


@pytest.mark.parametrize("header,names", [("nvfp4_mx.h", nv.MX_EXPORTS), ("nvfp4_moe.h", nv.MOE_EXPORTS)])
def test_library_exports_every_declared_function(header, names):
    text = open(os.path.join(ROOT, "include", header)).read()
    declared = sorted(set(re.findall(r"^int (nvfp4_\w+)\s*\(", text, re.M)))
    assert declared == sorted(names)
    for n in declared:
        assert hasattr(nv.lib(), n), n


@pytest.mark.parametrize("rows,K", [(0, 32), (1, 32), (16, 128), (17, 160), (100, 6112), (256, 8192)])
def test_packed_size(rows, K):
    rb, c = -(-rows // 16), -(-K // 128)
    assert nv.mx_packed_size(rows, K) == (rb * c * 1024, rb * -(-c // 4) * 256)


@pytest.mark.parametrize("rows,K", [(4, 0), (4, 16), (4, 48), (4, -32), (-1, 64), (2 ** 30 + 1, 32)])
def test_packed_size_rejects(rows, K):
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.mx_packed_size(rows, K)
    assert e.value.status == INV


@pytest.mark.parametrize("rows,K", [(1, 32), (5, 96), (16, 128), (33, 544), (20, 2080)])
def test_pack_roundtrip_and_layout(rows, K):
    g = np.random.default_rng(rows * 1000 + K)
    codes, scales = mx_ref.random_operand(g, rows, K, 0, 256)
    pc, ps = nv.mx_pack(codes, scales)
    c2, s2 = nv.mx_unpack(pc, ps, rows, K)
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)
    rb, c = -(-rows // 16), -(-K // 128)
    q = -(-c // 4)
    wide = np.zeros((rb * 16, c * 64), np.uint8)
    wide[:rows, :K // 2] = codes
    rows_first = wide.reshape(rb, 16, c, 4, 16).transpose(0, 2, 1, 3, 4)
    for r in range(16):
        for b in range(4):                     # block b of a step lies at place b ^ (r / 4)
            assert np.array_equal(pc.reshape(rb, c, 16, 4, 16)[:, :, r, b ^ (r // 4)], rows_first[:, :, r, b])
    wide = np.zeros((rb * 16, q * 16), np.uint8)
    wide[:rows, :K // 32] = scales
    assert np.array_equal(ps.reshape(rb, q, 16, 4, 4),
                          wide.reshape(rb, 16, q, 4, 4).transpose(0, 2, 1, 4, 3))


def test_pack_rejects_bad_shapes():
    with pytest.raises(ValueError):
        nv.mx_pack(np.zeros((2, 16), np.uint8), np.zeros((2, 2), np.uint8))
    with pytest.raises(ValueError):
        nv.mx_pack(np.zeros((2, 8), np.uint8), np.zeros((2, 1), np.uint8))     # K = 16
    with pytest.raises(ValueError):
        nv.mx_unpack(np.zeros(8, np.uint8), np.zeros(8, np.uint8), 1, 32)


def quant(fn="nvfp4_mx_quantize", x=P, kind=1, groups=1, gs=0, rows=4, K=64, ld=64, c=P, s=P):
    L = nv.mx.mx_lib()
    if fn == "nvfp4_mx_quantize":
        return L.nvfp4_mx_quantize(x, kind, groups, gs, rows, K, ld, c, s, None)
    return L.nvfp4_mx_dequantize(c, s, groups, rows, K, x, kind, gs, ld, None)


@pytest.mark.parametrize("fn", ["nvfp4_mx_quantize", "nvfp4_mx_dequantize"])
def test_quantize_refusals(fn):
    for bad in (dict(x=None), dict(c=None), dict(s=None), dict(kind=2), dict(kind=-1), dict(groups=-1),
                dict(rows=-1), dict(K=0), dict(K=48), dict(ld=32), dict(ld=68), dict(groups=2, gs=4), dict(groups=2, gs=-8),
                dict(kind=0, ld=66), dict(groups=2 ** 40), dict(rows=2 ** 30, K=2 ** 20, ld=2 ** 20)):
        assert quant(fn, **bad) == INV, bad
    for bad in (dict(x=P + 8), dict(c=P + 4), dict(s=P + 1)):
        assert quant(fn, **bad) == MIS, bad
    overlap = quant(fn, groups=2, gs=32, x=P + 8)          # one matrix for all groups may be read, not written
    assert overlap == (MIS if fn == "nvfp4_mx_quantize" else INV)
    assert quant(fn, rows=1, ld=3, x=P + 8) == MIS         # (a single row's stride is not looked at)


def gemm(a=P, sa=P, b=P, sb=P, out=P, kind=1, M=4, N=4, K=64):
    return nv.mx.mx_lib().nvfp4_mx_gemm(a, sa, b, sb, 1.0, out, kind, M, N, K, None)


def gemm_q(x=P, kind=1, ld=64, b=P, sb=P, out=P, ok=1, M=4, N=4, K=64):
    return nv.mx.mx_lib().nvfp4_mx_gemm_quantized(x, kind, ld, b, sb, 1.0, out, ok, M, N, K, None)


def grouped(a=P, sa=P, n=4, rows=None, b=P, sb=P, off=P, G=2, out=P, kind=1, M=4, N=4, K=64):
    return nv.mx.mx_lib().nvfp4_mx_grouped_gemm(a, sa, n, rows, b, sb, off, G, 1.0, out, kind, M, N, K, None)


def test_gemm_refusals():
    for bad in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None), dict(kind=2),
                dict(M=-1), dict(N=0), dict(K=0), dict(K=16), dict(K=2 ** 31), dict(M=2 ** 31)):
        assert gemm(**bad) == INV, bad
    for bad in (dict(a=P + 8), dict(sb=P + 4), dict(out=P + 2)):
        assert gemm(**bad) == MIS, bad
    for bad in (dict(x=None), dict(kind=7), dict(ld=32), dict(ld=60), dict(ok=3), dict(N=-1), dict(K=80)):
        assert gemm_q(**bad) == INV, bad
    assert gemm_q(x=P + 2) == MIS
    assert gemm_q(M=17) == UNS
    for bad in (dict(off=None), dict(G=0), dict(G=-1), dict(n=3), dict(n=0), dict(rows=P, n=0), dict(out=None),
                dict(M=-1), dict(N=0), dict(K=100), dict(kind=-1)):
        assert grouped(**bad) == INV, bad
    for bad in (dict(off=P + 2), dict(rows=P + 1, n=9), dict(a=P + 1)):
        assert grouped(**bad) == MIS, bad


def test_moe_refusals():
    L = nv.moe.moe_lib()

    def sort(ids=P, kind=0, T=4, k=2, E=8, off=P, slots=P, tok=P):
        return L.nvfp4_moe_sort(ids, kind, T, k, E, off, slots, tok, None)

    for bad in (dict(ids=None), dict(off=None), dict(slots=None), dict(tok=None), dict(kind=2), dict(T=-1),
                dict(k=0), dict(E=0), dict(E=2049), dict(T=2 ** 24), dict(T=2 ** 23, k=2 ** 9)):
        assert sort(**bad) == INV, bad
    for bad in (dict(ids=P + 2), dict(kind=1, ids=P + 4), dict(off=P + 1), dict(slots=P + 2), dict(tok=P + 3)):
        assert sort(**bad) == MIS, bad

    def gather(x=P, kind=1, T=4, k=2, H=8, ld=8, slots=P, out=P):
        return L.nvfp4_moe_gather(x, kind, T, k, H, ld, slots, out, None)

    for bad in (dict(x=None), dict(slots=None), dict(out=None), dict(kind=5), dict(T=-2), dict(k=0), dict(H=0),
                dict(H=2 ** 23), dict(ld=7), dict(ld=-8), dict(ld=2 ** 31)):
        assert gather(**bad) == INV, bad
    for bad in (dict(x=P + 1), dict(out=P + 1), dict(slots=P + 2), dict(kind=0, x=P + 2)):
        assert gather(**bad) == MIS, bad

    def combine(y=P, kind=1, T=4, k=2, H=8, slots=P, w=P, out=P):
        return L.nvfp4_moe_combine(y, kind, T, k, H, slots, w, out, None)

    for bad in (dict(y=None), dict(slots=None), dict(out=None), dict(kind=-1), dict(H=-1)):
        assert combine(**bad) == INV, bad
    assert combine(w=P + 2) == MIS

    def grad(d=P, ld=8, y=P, kind=1, T=4, k=2, H=8, slots=P, w=P, dy=P, dw=P):
        return L.nvfp4_moe_combine_grad(d, ld, y, kind, T, k, H, slots, w, dy, dw, None)

    for bad in (dict(d=None), dict(y=None), dict(slots=None), dict(dy=None), dict(dw=None), dict(ld=4), dict(kind=3)):
        assert grad(**bad) == INV, bad
    for bad in (dict(dw=P + 2), dict(d=P + 1), dict(y=P + 1), dict(dy=P + 1)):
        assert grad(**bad) == MIS, bad


def test_moe_refuses_long_rows_of_choices():
    """The kernels number a token's choices in 32 bits, some past its last one."""
    L = nv.moe.moe_lib()
    for k in (2 ** 24, 2 ** 31 - 1):
        assert L.nvfp4_moe_sort(P, 0, 1, k, 8, P, P, P, None) == INV
        assert L.nvfp4_moe_gather(P, 1, 1, k, 8, 8, P, P, None) == INV
        assert L.nvfp4_moe_combine(P, 1, 1, k, 8, P, None, P, None) == INV
        assert L.nvfp4_moe_combine_grad(P, 8, P, 1, 1, k, 8, P, None, P, P, None) == INV


def test_sequence_refuses_the_same(tmp_path):
    L, ML = nv.mx.mx_lib(), nv.moe.moe_lib()
    h = ctypes.c_void_p()
    assert L.nvfp4_sequence_create(ctypes.byref(h)) == nv.OK
    try:
        assert L.nvfp4_sequence_add_mx_gemm(h, P, P, P, P, 1.0, P, 1, 4, 4, 40) == INV
        assert L.nvfp4_sequence_add_mx_gemm_quantized(h, P, 1, 64, P, P, 1.0, P, 1, 17, 4, 64) == UNS
        assert L.nvfp4_sequence_add_mx_quantize(h, P + 1, 1, 4, 64, 64, P, P) == MIS
        assert L.nvfp4_sequence_add_mx_grouped_gemm(h, P, P, 4, None, P, P, None, 2, 1.0, P, 1, 4, 4, 64) == INV
        assert ML.nvfp4_sequence_add_moe_sort(h, P, 0, 4, 2, 0, P, P, P) == INV
        assert ML.nvfp4_sequence_add_moe_gather(h, P, 1, 4, 2, 8, 7, P, P) == INV
        assert ML.nvfp4_sequence_add_moe_combine(h, P, 9, 4, 2, 8, P, P, P) == INV
        assert L.nvfp4_sequence_add_mx_gemm(h, P, P, P, P, 1.0, P, 1, 4, 4, 64) == nv.OK
    finally:
        L.nvfp4_sequence_destroy(h)
    assert L.nvfp4_sequence_add_mx_gemm(None, P, P, P, P, 1.0, P, 1, 4, 4, 64) == INV


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        nv.mx_quantize(x)
    with pytest.raises(ValueError, match="GPU"):
        nv.moe_sort(torch.zeros(4, 2, dtype=torch.int32), 8)
    with pytest.raises(ValueError):
        nv.mx_quantize(x.to(torch.float16))
    with pytest.raises(ValueError):
        nv.mx_quantize(x[:, :48])
    with pytest.raises(ValueError):
        nv.mx_quantize(x.t())
    with pytest.raises(ValueError):
        nv.moe_sort(torch.zeros(4, 2), 8)
    u8 = dict(dtype=torch.uint8)
    a = nv.MxOperand(torch.zeros(1024, **u8), torch.zeros(256, **u8), 4, 64)
    b = nv.MxOperand(torch.zeros(1024, **u8), torch.zeros(256, **u8), 4, 96)
    with pytest.raises(ValueError, match="mismatch"):
        nv.mx_gemm(a, b)
    with pytest.raises(ValueError, match="mismatch"):
        nv.mx_linear(x, b)
    with pytest.raises(ValueError):
        nv.mx_gemm(a, nv.MxOperand(torch.zeros(512, **u8), torch.zeros(256, **u8), 4, 64))
    with pytest.raises(ValueError):
        nv.mx_gemm(a, a, out=torch.zeros(4, 5, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        nv.mx_gemm(a, a, dtype=torch.float16)
    with pytest.raises(ValueError):
        nv.mx_dequantize(a, torch.float16)
    with pytest.raises(ValueError, match="float32"):
        nv.mx_gemm(a, a, out=torch.zeros(4, 4, dtype=torch.bfloat16), dtype=torch.float32)
    for experts in (-9, 0, 2049):
        with pytest.raises(ValueError, match="experts"):
            nv.moe_sort(torch.zeros(0, 2, dtype=torch.int32), experts)
    w = nv.MxGroups(torch.zeros(2048, **u8), torch.zeros(512, **u8), 2, 4, 64)
    with pytest.raises(ValueError, match="row_offsets"):
        nv.mx_grouped_gemm(a, w, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="rows"):
        nv.mx_grouped_gemm(a, w, torch.zeros(3, dtype=torch.int32), rows=torch.zeros(4))
    for f in (lambda: nv.mx_quantize(x, stream=0), lambda: nv.mx_gemm(a, a, stream=7),
              lambda: nv.moe_sort(torch.zeros(4, 2, dtype=torch.int32), 8, stream=0)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    i32 = dict(dtype=torch.int32)
    r = nv.MoeRoute(torch.zeros(9, **i32), torch.zeros(4, 2, **i32), torch.zeros(8, **i32), 8)
    with pytest.raises(ValueError):
        nv.moe_gather(x[:3], r)
    with pytest.raises(ValueError):
        nv.moe_combine(x, r)
    with pytest.raises(ValueError, match="weights"):
        nv.moe_combine(torch.zeros(8, 64), r, torch.zeros(4, 3))
    with pytest.raises(ValueError, match="route"):
        nv.moe_gather(x, nv.MoeRoute(r.row_offsets, r.slots, r.tokens.long(), 8))
    with pytest.raises(ValueError):
        nv.moe_combine_grad(x, torch.zeros(8, 64), r)


def test_binding_refuses_operands_of_another_class():
    """Groups where one operand is meant (all but the first would be dropped) and the other way round, and operands
    of the 16-element format, whose buffers have other sizes."""
    u8 = dict(dtype=torch.uint8)
    a = nv.MxOperand(torch.zeros(1024, **u8), torch.zeros(256, **u8), 4, 64)
    w = nv.MxGroups(torch.zeros(3 * 1024, **u8), torch.zeros(768, **u8), 3, 4, 64)
    one = nv.MxGroups(a.codes, a.scales, 1, 4, 64)
    cb, sb = nv.packed_size(4, 64)
    p = nv.PackedOperand(torch.zeros(cb, **u8), torch.zeros(sb, **u8), 4, 64)
    pw = nv.PackedGroups(torch.zeros(3 * cb, **u8), torch.zeros(3 * sb, **u8), 3, 4, 64)
    x, off = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    out = torch.zeros(4, 4, dtype=torch.bfloat16)
    seq = nv.Sequence()
    for bad in (w, one, p, pw):
        for f in (lambda: nv.mx_gemm(bad, a), lambda: nv.mx_gemm(a, bad), lambda: nv.mx_gemm_quantized(x, bad),
                  lambda: nv.mx_linear(x, bad), lambda: nv.mx_linear(x.repeat(9, 1), bad),
                  lambda: nv.mx_linear(x[None], bad), lambda: nv.mx_grouped_gemm(bad, w, off),
                  lambda: nv.mx_quantize(x, out=bad), lambda: seq.add_mx_gemm(bad, a, out),
                  lambda: seq.add_mx_gemm(a, bad, out), lambda: seq.add_mx_gemm_quantized(x, bad, out),
                  lambda: seq.add_mx_grouped_gemm(bad, w, off, out), lambda: seq.add_mx_quantize(x, bad)):
            with pytest.raises(ValueError, match="must be MxOperand"):
                f()
    for bad in (a, p, pw):
        for f in (lambda: nv.mx_grouped_gemm(a, bad, off), lambda: seq.add_mx_grouped_gemm(a, bad, off, out),
                  lambda: nv.mx_quantize(x.expand(3, 4, 64), out=bad)):
            with pytest.raises(ValueError, match="must be MxGroups"):
                f()
    for bad in (p, pw):
        with pytest.raises(ValueError, match="MxOperand or MxGroups"):
            nv.mx_dequantize(bad)
    assert seq.calls == 0


def test_linear_takes_leading_dimensions(monkeypatch):
    """Every row of a batch reaches the product (the calls' arguments, without a GPU)."""
    calls = []
    monkeypatch.setattr(nv.mx, "_run", lambda fn, args, tensors: calls.append((fn.__name__, args)))
    u8 = dict(dtype=torch.uint8)
    b = nv.MxOperand(torch.zeros(1024, **u8), torch.zeros(256, **u8), 7, 64)
    for lead in ((2, 3), (4, 100), (1, 1), (3, 1, 5), (0, 4), (2, 0)):
        rows = int(np.prod(lead))
        out = torch.empty(*lead, 7, dtype=torch.bfloat16)
        for given in (None, out):
            calls.clear()
            c = nv.mx_linear(torch.zeros(*lead, 64), b, out=given)
            assert c.shape == (*lead, 7) and (given is None or c is given)
            name, args = calls[-1]
            assert name == ("nvfp4_mx_gemm_quantized" if rows <= 16 else "nvfp4_mx_gemm")
            assert args[-3:] == (rows, 7, 64)
            assert rows <= 16 or calls[0][1][2:6] == (1, 0, rows, 64)   # one group of all the rows is quantised
            assert given is None or rows == 0 or out.data_ptr() in args
    x = torch.zeros(2, 5, 72)[:, :, :64]                  # rows of a wider buffer: one stride, no copy
    nv.mx_linear(x, b)
    assert calls[-1][1][0] == x.data_ptr() and calls[-1][1][2] == 72
    for bad in (torch.empty(10, 7), torch.empty(2, 5, 8), torch.empty(2, 7, 5).transpose(1, 2)):
        with pytest.raises(ValueError, match="out"):
            nv.mx_linear(x, b, out=bad)
    with pytest.raises(ValueError):
        nv.mx_linear(torch.zeros(64), b)
    with pytest.raises(ValueError, match="mismatch"):
        nv.mx_linear(torch.zeros(2, 5, 96), b)


def test_16_element_calls_refuse_mx_operands():
    """Their scale buffers are half as large: the kernels would read and write past them."""
    u8 = dict(dtype=torch.uint8)
    a = nv.MxOperand(torch.zeros(1024, **u8), torch.zeros(256, **u8), 4, 64)
    w = nv.MxGroups(torch.zeros(3 * 1024, **u8), torch.zeros(768, **u8), 3, 4, 64)
    cb, sb = nv.packed_size(4, 64)
    p = nv.PackedOperand(torch.zeros(cb, **u8), torch.zeros(sb, **u8), 4, 64)
    pw = nv.PackedGroups(torch.zeros(3 * cb, **u8), torch.zeros(3 * sb, **u8), 3, 4, 64)
    x, off = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    out = torch.zeros(4, 4, dtype=torch.bfloat16)
    seq = nv.Sequence()
    for f in (lambda: nv.gemm(a, p, stream=0), lambda: nv.gemm(p, a, stream=0), lambda: nv.gemm(p, w, stream=0),
              lambda: nv.gemm_noalloc(a, p, stream=0), lambda: nv.gemm_noalloc(p, a, stream=0),
              lambda: nv.gemm_quantized(x, a, stream=0), lambda: nv.grouped_gemm(a, pw, off, stream=0),
              lambda: nv.grouped_gemm(p, w, off, stream=0), lambda: nv.quantize(x, out=a, stream=0),
              lambda: seq.add_gemm(a, p, out), lambda: seq.add_gemm(p, a, out),
              lambda: seq.add_gemm_quantized(x, a, 1.0, out), lambda: seq.add_grouped_gemm(a, pw, off, out),
              lambda: seq.add_grouped_gemm(p, w, off, out), lambda: seq.add_quantize(x, a)):
        with pytest.raises(ValueError, match="blocks of 16"):
            f()
    assert seq.calls == 0 and repr(a).count("block") == 0


def test_sequence_runs_on_the_gpu_of_its_tensors(monkeypatch):
    """With the current GPU another one, as the calls by themselves do; a call of another GPU is refused (the GPUs
    are stood in for)."""
    seen, now, where = [], [0], [1]

    class On:
        def __init__(self, gpu):
            self.gpu = gpu

        def __enter__(self):
            self.back, now[0] = now[0], self.gpu

        def __exit__(self, *_):
            now[0] = self.back

    class Lib:
        def nvfp4_sequence_finalize(self, h):
            seen.append(("finalize", now[0]))
            return nv.OK

        def nvfp4_sequence_launch(self, h, stream):
            seen.append(("launch", now[0], stream))
            return nv.OK

    u8 = dict(dtype=torch.uint8)
    a = nv.MxOperand(torch.zeros(1024, **u8), torch.zeros(256, **u8), 4, 64)
    out = torch.zeros(4, 4, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    i32 = dict(dtype=torch.int32)
    r = nv.MoeRoute(torch.zeros(9, **i32), torch.zeros(4, 2, **i32), torch.zeros(8, **i32), 8)
    seq, plain = nv.Sequence(), nv.Sequence()
    monkeypatch.setattr(nv.mx, "_gpu_of", lambda tensors: where[0])
    monkeypatch.setattr(nv.mx, "_current_gpu", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(nv, "_stream_handle", lambda stream: 100 + now[0])
    seq.add_mx_gemm(a, a, out)
    where[0] = 2
    with pytest.raises(ValueError, match="GPU 1.*GPU 2"):
        seq.add_moe_sort(ids, r)
    assert seq.calls == 1
    where[0] = 1
    seq.add_moe_sort(ids, r)
    monkeypatch.setattr(nv, "lib", Lib)
    for s in (seq, plain):
        s.finalize()
        s.launch()
    now[0] = 1
    seq.launch()
    assert now[0] == 1 and seen == [("finalize", 1), ("launch", 1, 101), ("finalize", 0), ("launch", 0, 100),
                                    ("launch", 1, 101)]
    monkeypatch.undo()
    seq.close()
    plain.close()


def test_sequence_refuses_calls_without_an_output(monkeypatch):
    u8, i32 = dict(dtype=torch.uint8), dict(dtype=torch.int32)
    a = nv.MxOperand(torch.zeros(1024, **u8), torch.zeros(256, **u8), 4, 64)
    w = nv.MxGroups(torch.zeros(2048, **u8), torch.zeros(512, **u8), 2, 4, 64)
    r = nv.MoeRoute(torch.zeros(9, **i32), torch.zeros(4, 2, **i32), torch.zeros(8, **i32), 8)
    x, y, off = torch.zeros(4, 64), torch.zeros(8, 64), torch.zeros(3, **i32)
    monkeypatch.setattr(nv.mx, "_gpu_of", lambda tensors: 0)
    seq = nv.Sequence()
    for f in (lambda: seq.add_mx_quantize(x, None), lambda: seq.add_mx_gemm(a, a, None),
              lambda: seq.add_mx_gemm_quantized(x, a, None), lambda: seq.add_mx_grouped_gemm(a, w, off, None),
              lambda: seq.add_moe_gather(x, r, None), lambda: seq.add_moe_combine(y, r, None, None)):
        with pytest.raises(ValueError, match="out"):
            f()
    assert seq.calls == 0


def test_grouped_takes_many_groups():
    """The grid is as large as the rows need, not as the groups (recorded, so that nothing is launched)."""
    L = nv.mx.mx_lib()
    h = ctypes.c_void_p()
    assert L.nvfp4_sequence_create(ctypes.byref(h)) == nv.OK
    try:
        for G, M, N, K in ((2 ** 20, 8, 1024, 64), (2 ** 20, 8, 1024, 8192), (2 ** 22, 1, 65536, 256),
                           (2 ** 16, 4096, 2048, 6144), (2 ** 30, 3, 100, 32)):
            assert L.nvfp4_sequence_add_mx_grouped_gemm(h, P, P, M, None, P, P, P, G, 1.0, P, 1, M, N, K) == nv.OK
    finally:
        L.nvfp4_sequence_destroy(h)


def test_version_tells_of_the_operators():
    """A C caller that looks the functions up at run time can ask for the version first, as the headers say."""
    assert nv.version() >= 10600
    for header in ("nvfp4_mx.h", "nvfp4_moe.h"):
        assert "nvfp4_version() 10600" in open(os.path.join(ROOT, "include", header)).read()
