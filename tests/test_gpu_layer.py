"""Products with an epilogue on the GPU against the 64-bit references of
layer_ref.py.  The values that packed operands stand for come from
mx_dequantize, which is held to every bit elsewhere."""
from __future__ import annotations

import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_04_amd as nv  # noqa: E402
import layer_ref as ref  # noqa: E402

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = list(nv.ACTIVATIONS)


def say(msg: str) -> None:
    print(f"[gpu] {msg}", flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, device=DEV, generator=g)).to(dtype)


def values(q):
    return nv.mx_dequantize(q, torch.float32).double()


def parts(g, M, N, dtype, gate, bias, residual, groups=None, K=None, bias_dtype=torch.float32):
    """An epilogue's tensors; K: of the gate's."""
    lead = () if groups is None else (groups,)
    p = {}
    if gate:
        p["gate"] = nv.mx_quantize(randn(g, *lead, N, K, scale=0.06))
    if bias:
        p["bias"] = randn(g, *lead, N, dtype=bias_dtype)
        if gate:
            p["gate_bias"] = randn(g, *lead, N, dtype=bias_dtype)
    if residual:
        p["residual"] = randn(g, M, N, dtype=dtype)
    return p


def expected(a, w, p, act, alpha, group=None):
    """Reference of rows with the values a by weight values w."""
    pick = (lambda t: t) if group is None else (lambda t: t[group])  # noqa: E731
    more = {k: pick(p[k]).double() for k in ("bias", "gate_bias") if k in p}
    if "gate" in p:
        more["gate"] = ref.product(a, pick(values(p["gate"])), alpha)
    return ref.epilogue(*ref.product(a, w, alpha), activation=act, **more)


# Sizes by the kernel that they reach (gated: two operands' columns).
SIZES = [(1, 768, 6144), (16, 50, 544), (3, 7, 8800), (5, 33, 32), (16, 4100, 160),        # up to 16 rows
         (40, 100, 1024), (64, 17, 8320),                                                  # 17 to 64
         (70, 70, 96), (300, 500, 1024), (200, 333, 6112),                                 # 64 x 64, one and two teams
         (400, 2048, 512), (400, 4001, 256),                                               # 64 x 128
         (512, 2600, 288), (512, 5201, 160),                                               # 128 x 128
         (1024, 3001, 256), (1025, 6000, 128),                                             # 128 x 256
         (4100, 2051, 4224), (4100, 4100, 4128)]                                           # 256 x 256


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, gate):
    g = gen(M * 31 + N)
    for i, dtype in enumerate((torch.bfloat16, torch.float32)):
        act = ACTS[(M + N + i) % len(ACTS)]
        say(f"product {M}x{N}x{K} gate={gate} {act} {dtype}")
        a, b = nv.mx_quantize(randn(g, M, K)), nv.mx_quantize(randn(g, N, K, scale=0.06))
        p = parts(g, M, N, dtype, gate, True, True, K=K, bias_dtype=(torch.float32, torch.bfloat16)[i])
        out = nv.mx_gemm(a, b, 0.75, dtype=dtype, epilogue=nv.MxEpilogue(act, **p))
        want, d = expected(values(a), values(b), p, act, 0.75)
        r = p["residual"].double()
        ref.check(out, want + r, d + 2 * ref.U * ((want + r).abs() + d), f"{M}x{N}x{K}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
def test_every_part_alone(act, gate, bias, residual):
    say(f"parts {act} gate={gate} bias={bias} residual={residual}")
    for M, N, K in ((4, 37, 160), (150, 72, 288)):
        g = gen(M)
        a, b = nv.mx_quantize(randn(g, M, K, scale=2.0)), nv.mx_quantize(randn(g, N, K, scale=0.2))
        for dtype in DT.values():
            p = parts(g, M, N, dtype, gate, bias, residual, K=K)
            out = nv.mx_gemm(a, b, dtype=dtype, epilogue=nv.MxEpilogue(act, **p))
            want, d = expected(values(a), values(b), p, act, 1.0)
            if residual:
                want = want + p["residual"].double()
                d = d + 2 * ref.U * (want.abs() + d)
            ref.check(out, want, d, f"{act} {M}")


def test_without_parts_the_plain_product():
    """An empty epilogue changes nothing: the same bits."""
    for M, N, K in ((1, 768, 1024), (16, 100, 9000 // 32 * 32), (50, 64, 512), (300, 500, 1024), (600, 700, 2048)):
        g = gen(N)
        a, b = nv.mx_quantize(randn(g, M, K)), nv.mx_quantize(randn(g, N, K))
        for dtype in DT.values():
            assert torch.equal(nv.mx_gemm(a, b, 0.5, dtype=dtype, epilogue=nv.MxEpilogue()),
                               nv.mx_gemm(a, b, 0.5, dtype=dtype))


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 768, 6144), (5, 40, 96), (16, 4500, 544), (16, 33, 9984), (7, 9000, 8192)])
def test_from_activations_the_same_bits(M, N, K, gate):
    g = gen(K + M)
    b = nv.mx_quantize(randn(g, N, K, scale=0.06))
    for dtype in DT.values():
        say(f"from activations {M}x{N}x{K} gate={gate} {dtype}")
        x = randn(g, M, K + 8, dtype=dtype)[:, :K]
        e = nv.MxEpilogue("silu", **parts(g, M, N, torch.bfloat16, gate, True, True, K=K))
        one = nv.mx_gemm_quantized(x, b, epilogue=e)
        assert torch.equal(one, nv.mx_gemm(nv.mx_quantize(x), b, epilogue=e))
        assert torch.equal(one, nv.mx_linear(x, b, epilogue=e))


GROUPED = [  # groups, N, K, rows of each group
    (4, 100, 160, (3, 0, 40, 17)), (8, 300, 2080, (5, 0, 0, 64, 1, 200, 16, 3)),      # 64 x 64
    (60, 700, 256, tuple(range(60))),                                                 # 64 x 256
    (100, 60, 288, tuple(50 + i for i in range(100))),                                # 128 x 128 (64 x 64 gated: narrow)
    (4, 2100, 512, (300, 513, 128, 0))]                                               # 128 x 256


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("G,N,K,rows", GROUPED)
def test_grouped(G, N, K, rows, gate):
    M = sum(rows) + 5                                       # five rows behind the last group
    off = torch.tensor([0, *torch.tensor(rows).cumsum(0)], dtype=torch.int32, device=DEV)
    for picked in (False, True):
        for dtype in DT.values():
            g = gen(G + N)
            say(f"grouped {G} x {N} x {K} gate={gate} picked={picked} {dtype}")
            act = ACTS[(G + N + gate) % len(ACTS)]
            a = nv.mx_quantize(randn(g, 77 if picked else M, K))
            w = nv.mx_quantize(randn(g, G, N, K, scale=0.06))
            at = torch.randint(0, 77, (M,), device=DEV, generator=g, dtype=torch.int32) if picked else None
            p = parts(g, M, N, dtype, gate, True, True, groups=G, K=K)
            out = randn(g, M, N, dtype=dtype)
            behind = out[-5:].clone()
            nv.mx_grouped_gemm(a, w, off, 1.25, rows=at, out=out, epilogue=nv.MxEpilogue(act, **p))
            assert torch.equal(out[-5:], behind)
            va, vw, r0 = values(a), values(w), 0
            for i, n in enumerate(rows):
                x = va[at[r0:r0 + n].long()] if picked else va[r0:r0 + n]
                want, d = expected(x, vw[i], p, act, 1.25, i)
                r = p["residual"][r0:r0 + n].double()
                ref.check(out[r0:r0 + n], want + r, d + 2 * ref.U * ((want + r).abs() + d), f"group {i}")
                r0 += n


@pytest.mark.parametrize("gate", [False, True])
def test_grouped_with_packed_rows_of_two_gib(gate):
    """The kernel without 32-bit offsets, from rows at the end of 2 GiB of packed activations."""
    K, R, G, N = 2048, 1 << 21, 3, 50
    cb, sb = nv.mx_packed_size(R, K)
    g = gen(9)
    some = nv.mx_quantize(randn(g, 48, K))
    a = nv.MxOperand(torch.zeros(cb, dtype=torch.uint8, device=DEV), torch.zeros(sb, dtype=torch.uint8, device=DEV), R, K)
    a.codes[-some.codes.numel():] = some.codes
    a.scales[-some.scales.numel():] = some.scales
    w = nv.mx_quantize(randn(g, G, N, K, scale=0.06))
    rows = (40, 0, 33)
    M = sum(rows)
    at = torch.randint(0, 48, (M,), device=DEV, generator=g, dtype=torch.int32)
    off = torch.tensor([0, 40, 40, 73], dtype=torch.int32, device=DEV)
    p = parts(g, M, N, torch.bfloat16, gate, True, True, groups=G, K=K)
    out = nv.mx_grouped_gemm(a, w, off, rows=at + (R - 48), epilogue=nv.MxEpilogue("silu", **p))
    va, vw = values(some), values(w)
    for i, (b, e) in enumerate(((0, 40), (40, 40), (40, 73))):
        want, d = expected(va[at[b:e].long()], vw[i], p, "silu", 1.0, i)
        r = p["residual"][b:e].double()
        ref.check(out[b:e], want + r, d + 2 * ref.U * ((want + r).abs() + d), f"group {i}")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,N,K", [(9, 50, 64), (60, 50, 64), (200, 201, 256), (520, 2600, 128)])
def test_residual_in_place_and_strided(M, N, K, dtype):
    say(f"residual {M}x{N}x{K} {dtype}")
    g = gen(M)
    a, b = nv.mx_quantize(randn(g, M, K)), nv.mx_quantize(randn(g, N, K))
    r = randn(g, M, N, dtype=DT[dtype])
    want = nv.mx_gemm(a, b, dtype=DT[dtype], epilogue=nv.MxEpilogue(residual=r))
    wide = torch.full((M, N + 13), float("nan"), dtype=DT[dtype], device=DEV)   # the gaps must not be read
    wide[:, 5:5 + N] = r
    assert torch.equal(nv.mx_gemm(a, b, dtype=DT[dtype], epilogue=nv.MxEpilogue(residual=wide[:, 5:5 + N])), want)
    nv.mx_gemm(a, b, out=r, epilogue=nv.MxEpilogue(residual=r))
    assert torch.equal(r, want)


@pytest.mark.parametrize("act", ACTS)
def test_large_infinite_and_nan_values(act):
    """Sums far from zero saturate the activations; a NaN row of A, or an infinite bias, reaches its own results only."""
    a = nv.mx_quantize(torch.full((20, 32), 1.0, device=DEV))
    b = nv.mx_quantize(torch.full((6, 32), 1.0, device=DEV))
    bias = torch.tensor([1e30, -1e30, 100.0, -100.0, float("inf"), -40.0], device=DEV)
    for M in (4, 20):
        a_ = nv.mx_quantize(torch.cat([torch.full((M - 1, 32), 1.0, device=DEV), torch.full((1, 32), float("nan"), device=DEV)]))
        out = nv.mx_gemm(a_, b, dtype=torch.float32, epilogue=nv.MxEpilogue(act, bias=bias))
        assert out[M - 1].isnan().all()
        z = (32.0 + bias).double()
        want = ref.act(act, z)
        got = out[:M - 1].double()
        assert torch.equal(got, got[:1].expand_as(got))
        ok = (got[0] - want).abs() <= 1e-5 * want.abs() + 1e-5
        assert (ok | (got[0] == want)).all(), (got[0], want)
    assert torch.equal(nv.mx_gemm(a, b), nv.mx_gemm(a, b, epilogue=nv.MxEpilogue("none")))


def test_leading_dimensions_streams_and_nothing():
    g = gen(4)
    b = nv.mx_quantize(randn(g, 40, 64))
    for lead in ((2, 3), (4, 25), (0, 4)):
        x, r = randn(g, *lead, 64), randn(g, *lead, 40, dtype=torch.bfloat16)
        e = nv.MxEpilogue("gelu", residual=r, bias=randn(g, 40))
        want = nv.mx_linear(x.flatten(0, 1), b, epilogue=nv.MxEpilogue("gelu", residual=r.flatten(0, 1), bias=e.bias))
        assert torch.equal(nv.mx_linear(x, b, epilogue=e), want.view(*lead, 40))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        out = nv.mx_linear(x, b, epilogue=e, stream=s)
        s.synchronize()
        assert torch.equal(out, want.view(*lead, 40))


def test_recorded_and_captured():
    g = gen(6)
    x = randn(g, 16, 256, dtype=torch.bfloat16)
    up, gate, down = (nv.mx_quantize(randn(g, *s, scale=0.06)) for s in ((320, 256), (320, 256), (256, 320)))
    gated, back = nv.MxEpilogue("silu", gate=gate), nv.MxEpilogue(residual=x, bias=randn(g, 256))
    h, y = torch.empty(16, 320, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    q = nv.MxOperand(torch.empty(nv.mx_packed_size(16, 320)[0], dtype=torch.uint8, device=DEV),
                     torch.empty(nv.mx_packed_size(16, 320)[1], dtype=torch.uint8, device=DEV), 16, 320)

    def eager():
        return nv.mx_linear(nv.mx_linear(x, up, epilogue=gated), down, epilogue=back)

    w3 = nv.mx_quantize(randn(g, 2, 48, 256, scale=0.06))
    off = torch.tensor([0, 7, 16], dtype=torch.int32, device=DEV)
    z = torch.empty(16, 48, dtype=torch.bfloat16, device=DEV)
    ge = nv.MxEpilogue("relu", bias=randn(g, 2, 48))
    fixed = nv.mx_quantize(randn(g, 16, 256))
    with nv_sequence() as seq:
        seq.add_mx_gemm_quantized(x, up, h, epilogue=gated)
        seq.add_mx_quantize(h, q)
        seq.add_mx_gemm(q, down, y, epilogue=back)
        seq.add_mx_grouped_gemm(fixed, w3, off, z, epilogue=ge)
        seq.finalize()
        graph = torch.cuda.CUDAGraph()
        eager()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            captured = eager()
        for seed in range(3):
            x.copy_(randn(gen(seed), 16, 256))
            want = eager()
            y.zero_()
            seq.launch()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want) and torch.equal(captured, want)
        assert torch.equal(z, nv.mx_grouped_gemm(fixed, w3, off, epilogue=ge))


def nv_sequence():
    import contextlib
    return contextlib.closing(nv.Sequence())


@pytest.mark.parametrize("M,N,K", [(1, 48, 64), (16, 40, 8192), (16, 33, 8224), (16, 4500, 8224), (17, 64, 96), (100, 257, 544),
                                   (0, 8, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_in_one_call(M, N, K, dtype):
    """nvfp4_mx_linear_fused: the bits of the two calls it is made of, in its workspace, eager and captured."""
    say(f"linear {M}x{N}x{K} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(M + N)
    x = torch.randn(M, K + 16, device=DEV, generator=g).to(DT[dtype])[:, 8:K + 8]
    w, v = (nv.mx_quantize(torch.randn(N, K, device=DEV, generator=g)) for _ in range(2))
    e = nv.MxEpilogue("silu", torch.randn(N, device=DEV, generator=g), v, None,
                      torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16))
    want = nv.mx_gemm(nv.mx_quantize(x), w, 0.5, epilogue=e) if M else x.new_empty(0, N, dtype=torch.bfloat16)
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert nv.mx_linear(x, w, 0.5, out, epilogue=e) is out and torch.equal(out, want)
    if M == 0:
        return
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = nv.mx_linear(x, w, 0.5, epilogue=e)
    for seed in range(3):
        x.copy_(torch.randn(M, K, device=DEV, generator=g))
        want = nv.mx_gemm(nv.mx_quantize(x), w, 0.5, epilogue=e)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("M", [3, 70])
def test_gelu_by_its_own_size(M):
    """gelu keeps its digits where it is small: z comes as it is from the bias of a product of zeros.  With u = 2^-24,
    erfc's factor adds 9 terms of at most 2.2 times their sum and its argument's 3 roundings at a slope below 2.8: 48 u;
    the exponent z^2 / 2 is rounded three times: 1.5 z^2 u."""
    N = 4096
    z = torch.cat([torch.linspace(-12, 12, N - 200, device=DEV), torch.linspace(-1e-3, 1e-3, 200, device=DEV)])
    a, b = nv.mx_quantize(torch.zeros(M, 32, device=DEV)), nv.mx_quantize(torch.zeros(N, 32, device=DEV))
    want = ref.act("gelu", z.double())
    for dtype in DT.values():
        out = nv.mx_gemm(a, b, dtype=dtype, epilogue=nv.MxEpilogue("gelu", bias=z))
        assert torch.equal(out, out[:1].expand_as(out))
        ref.check(out[0], want, (48 + 1.5 * z.double() ** 2) * ref.U * want.abs())


def test_broadcast_residuals():
    """One row of a residual for all rows of a linear layer, with and without leading dimensions."""
    g = gen(12)
    b = nv.mx_quantize(randn(g, 40, 64))
    for lead in ((5,), (30,), (2, 3), (3, 20)):
        x, row = randn(g, *lead, 64), randn(g, 40, dtype=torch.bfloat16)
        for r in (row.expand(*lead, 40), randn(g, *lead, 40, dtype=torch.bfloat16)[..., :1, :].expand(*lead, 40)):
            want = nv.mx_linear(x, b, epilogue=nv.MxEpilogue("silu", residual=r.contiguous()))
            assert torch.equal(nv.mx_linear(x, b, epilogue=nv.MxEpilogue("silu", residual=r)), want)


@pytest.mark.parametrize("N,K", [(40, 64), (9000, 16384)])
def test_linear_without_rows(N, K):
    """An empty batch, also by a weight that more rows would take in two launches."""
    g = gen(13)
    w = nv.mx_quantize(randn(g, N, K, scale=0.06))
    for lead in ((0,), (2, 0)):
        x = torch.empty(*lead, K, dtype=torch.bfloat16, device=DEV)
        out = nv.mx_linear(x, w, epilogue=nv.MxEpilogue("silu", bias=randn(g, N), gate=w))
        assert out.shape == (*lead, N) and torch.equal(out, nv.mx_linear(x, w))


@pytest.mark.parametrize("M,K,gate,two", [(1, 9984, True, False), (4, 9984, True, False), (16, 8192, True, False), (16, 9984, True, True),
                                          (8, 9984, False, False), (8, 9984, True, True), (1, 28672, True, False), (4, 28672, True, True)])
def test_linear_of_few_deep_rows(M, K, gate, two):
    """Rows that one launch would quantise often, twice as often with a gate, are quantised once, in the workspace; the
    same bits, and without a workspace too."""
    import ctypes
    N, g = 768, gen(K + M)
    x = randn(g, M, K, dtype=torch.bfloat16)
    w, v = nv.mx_quantize(randn(g, N, K, scale=0.06)), nv.mx_quantize(randn(g, N, K, scale=0.06))
    want = nv.mx_gemm(nv.mx_quantize(x), w, epilogue=nv.MxEpilogue("silu", gate=v if gate else None))
    e = nv.layer._EpilogueT(2, v.codes.data_ptr() if gate else None, v.scales.data_ptr() if gate else None)
    size = sum(nv.mx_packed_size(M, K))
    work = torch.full((size,), 0xAA, dtype=torch.uint8, device=DEV)
    for ws, n in ((work.data_ptr(), size), (None, 0)):
        out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
        st = nv.layer.layer_lib().nvfp4_mx_linear_fused(x.data_ptr(), 1, K, w.codes.data_ptr(), w.scales.data_ptr(), 1.0,
                                                        ctypes.byref(e), out.data_ptr(), 1, M, N, K, ws, n,
                                                        torch.cuda.current_stream().cuda_stream)
        assert st == nv.OK and torch.equal(out, want)
    assert bool((work != 0xAA).any()) == two


@pytest.mark.parametrize("M,N,K", [(17, 40, 160), (64, 768, 2080), (33, 300, 9024),      # 64 x 64, with one and two teams
                                   (1500, 2051, 224), (4100, 2051, 8192),                # 128 x 256
                                   (4100, 2051, 8224)])                                  # 256 x 256
def test_gated_product_by_size(M, N, K):
    """The sizes at which a gated product takes another kernel than the plain one."""
    say(f"gated {M}x{N}x{K}")
    g = gen(M + K)
    for dtype in DT.values():
        a, b = nv.mx_quantize(randn(g, M, K)), nv.mx_quantize(randn(g, N, K, scale=0.06))
        p = parts(g, M, N, dtype, True, True, True, K=K)
        out = nv.mx_gemm(a, b, 0.75, dtype=dtype, epilogue=nv.MxEpilogue("silu", **p))
        want, d = expected(values(a), values(b), p, "silu", 0.75)
        r = p["residual"].double()
        ref.check(out, want + r, d + 2 * ref.U * ((want + r).abs() + d), f"{M}x{N}x{K}")
