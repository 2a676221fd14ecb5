"""MXFP4 operators on the GPU against the 64-bit references of mx_ref.py.

Quantisation is held to every byte of the packed buffers; products to the
bound of mx_ref.gemm_bound (fp32 sums, one rounding of the output)."""
from __future__ import annotations

import sys

import numpy as np
import pytest

import mx_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_04_amd as nv  # noqa: E402

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = {t: torch.finfo(t).eps for t in DT.values()}


def say(msg: str) -> None:
    print(f"[gpu] {msg}", flush=True)
    sys.stdout.flush()


def rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def host(t):
    return t.to(torch.float32).cpu().numpy()


def equal_bytes(q, x):
    """The packed operand equals the packed reference of the fp32 rows x."""
    pc, ps = nv.mx_pack(*mx_ref.quantize(x))
    gc, gs = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    assert np.array_equal(gs, ps), f"{np.count_nonzero(gs != ps)} scale bytes differ"
    assert np.array_equal(gc, pc), f"{np.count_nonzero(gc != pc)} code bytes differ"


# ---- quantisation ------------------------------------------------------------


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,K,sigma", [(1, 32, 1.0), (16, 128, 1.0), (17, 160, 1e-3), (33, 544, 30.0),
                                          (100, 6112, 1.0), (5, 8192, 0.02)])
def test_quantize(rows, K, sigma, dtype):
    say(f"quantize {rows}x{K} {dtype}")
    x = torch.from_numpy((rng(rows, K).standard_normal((rows, K)) * sigma).astype(np.float32)).to(DT[dtype])
    equal_bytes(nv.mx_quantize(x.to(DEV)), host(x))


@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_every_exponent_and_value(dtype):
    """All finite bfloat16 values beside block maxima of every exponent."""
    bits = np.arange(65536, dtype=np.uint32) << 16
    v = bits.view(np.float32)
    v = v[np.isfinite(v)]
    x = np.zeros((v.size // 32 * 8, 32), np.float32)
    for i in range(8):  # eight shifts of the value list against itself: blocks of mixed exponents
        x[i::8] = np.roll(v, 37 * i)[:v.size // 32 * 32].reshape(32, -1).T if i % 2 else \
            np.roll(v, 11 * i)[:v.size // 32 * 32].reshape(-1, 32)
    equal_bytes(nv.mx_quantize(torch.from_numpy(x).to(DT[dtype]).to(DEV)), x)


@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_edge_blocks(dtype):
    big, tiny = 3.3895313892515355e38, 2.0 ** -133   # largest bfloat16, smallest bfloat16 subnormal
    rows = [np.zeros(32), -np.zeros(32), np.full(32, big), np.full(32, -tiny), np.full(32, 2.0 ** -126),
            np.array([7.0, 5.0, -5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, 6.0, 7.96875] + [0.5] * 20),
            np.array([np.nan] + [1.0] * 31), np.array([1.0] * 31 + [np.inf]), np.array([-np.inf] + [0.0] * 31),
            np.array([big] + [1e-30] * 31), np.array([2.0 ** -125, 2.0 ** -127] * 16)]
    x = np.array(rows, np.float32)
    equal_bytes(nv.mx_quantize(torch.from_numpy(x).to(DT[dtype]).to(DEV)), x)


def test_quantize_strided_rows_and_groups():
    g = rng(3)
    wide = np.full((3, 20, 200), np.nan, np.float32)      # the gaps must not be read
    wide[:, :18, :160] = g.standard_normal((3, 18, 160))
    for dtype in DT.values():
        t = torch.from_numpy(wide).to(dtype).to(DEV)
        equal_bytes(nv.mx_quantize(t[1, :18, :160]), host(t[1, :18, :160]))
        q = nv.mx_quantize(t[:, :18, :160])
        assert (q.groups, q.rows, q.K) == (3, 18, 160)
        cb, sb = nv.mx_packed_size(18, 160)
        for i in range(3):
            one = nv.MxOperand(q.codes[i * cb:(i + 1) * cb], q.scales[i * sb:(i + 1) * sb], 18, 160)
            equal_bytes(one, host(t[i, :18, :160]))


def test_one_row_of_a_wider_buffer():
    """A single row's stride does not matter."""
    x = torch.randn(1, 70, device=DEV).to(torch.bfloat16)[:, :64]
    B = nv.mx_quantize(torch.randn(32, 64, device=DEV))
    equal_bytes(nv.mx_quantize(x), host(x))
    assert torch.equal(nv.mx_gemm_quantized(x, B), nv.mx_gemm(nv.mx_quantize(x.contiguous()), B))


def test_quantize_refuses_misaligned_rows():
    x = torch.zeros(4, 64 + 4, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.mx_quantize(x[:, :64])                          # rows every 136 bytes
    assert e.value.status == nv.ERR_INVALID_VALUE
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.mx_quantize(torch.zeros(4 * 64 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(4, 64))
    assert e.value.status == nv.ERR_MISALIGNED


@pytest.mark.parametrize("dtype", list(DT))
def test_dequantize_every_scale_and_code(dtype):
    codes = np.tile((np.arange(16, dtype=np.uint8) | np.arange(16, dtype=np.uint8)[::-1] << 4)[None], (256, 1))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    got = nv.mx_dequantize(nv.mx_to_device(codes, scales), DT[dtype])
    want = torch.from_numpy(mx_ref.values(codes, scales)).to(torch.float32).to(DT[dtype])  # exact but for 2^129
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.cpu()), torch.nan_to_num(want))


def test_dequantize_strided_and_empty():
    g = rng(4)
    codes, scales = mx_ref.random_operand(g, 2 * 19, 96)
    w = nv.mx_groups_to_device(codes.reshape(2, 19, 48), scales.reshape(2, 19, 3))
    out = torch.full((2, 19, 104), 7.0, device=DEV)
    nv.mx_dequantize(w, out=out[:, :, :96])
    want = mx_ref.values(codes, scales).reshape(2, 19, 96)
    assert np.array_equal(host(out[:, :, :96]), want.astype(np.float32))
    assert (out[:, :, 96:] == 7).all()
    q = nv.mx_quantize(torch.zeros(0, 64, device=DEV))
    assert q.rows == 0 and nv.mx_dequantize(q).shape == (0, 64)


# ---- product -----------------------------------------------------------------

# (every kernel and both of its ends: few rows, one and two teams of waves, 128 and 256 tiles)
SHAPES = [(1, 1, 32), (1, 768, 6144), (2, 17, 128), (16, 256, 6144), (17, 33, 544), (40, 100, 2080), (33, 4500, 160),
          (64, 64, 512), (65, 64, 128), (100, 130, 6112), (130, 200, 640), (257, 260, 1024),
          (300, 1000, 384), (512, 768, 512),
          (1300, 1290, 672), (1285, 1283, 2080), (4010, 3304, 544), (3900, 3301, 128)]


def operands(seed, M, N, K):
    g = rng(seed, M, N, K)
    a, b = mx_ref.random_operand(g, M, K), mx_ref.random_operand(g, N, K)
    return a, b, mx_ref.values(*a), mx_ref.values(*b)


def check(got, va, vb, alpha):
    want = alpha * (va @ vb.T)
    off = np.abs(host(got).astype(np.float64) - want)
    bound = mx_ref.gemm_bound(va, vb, alpha, EPS[got.dtype])
    worst = float((off / bound).max())
    say(f"worst error / bound {worst:.3f}")
    assert worst <= 1.0


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, dtype):
    say(f"gemm {M}x{N}x{K} {dtype}")
    a, b, va, vb = operands(1, M, N, K)
    out = torch.full((M * N + 64,), 3.0, dtype=DT[dtype], device=DEV)
    c = out[:M * N].view(M, N)
    nv.mx_gemm(nv.mx_to_device(*a), nv.mx_to_device(*b), -0.75, out=c)
    check(c, va, vb, -0.75)
    assert (out[M * N:] == 3).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,N,K", [
    (421, 2503, 416), (130, 8190, 4128),        # one round of 64 x 128 tiles
    (1301, 2601, 416), (330, 6144, 672),        # 128 x 128
    (1303, 4701, 288), (3007, 4101, 160),       # 128 x 256
    (4011, 4051, 4192), (8201, 7950, 96)])      # 256 x 256: deep, or many
def test_gemm_large(M, N, K, dtype):
    """The first and the last rows of large products."""
    say(f"gemm {M}x{N}x{K} {dtype}")
    a, b, va, vb = operands(17, M, N, K)
    out = torch.full((M * N + 64,), 3.0, dtype=DT[dtype], device=DEV)
    c = out[:M * N].view(M, N)
    nv.mx_gemm(nv.mx_to_device(*a), nv.mx_to_device(*b), 0.5, out=c)
    w = min(M, 140)
    check(c[:w], va[:w], vb, 0.5)
    check(c[M - w:], va[M - w:], vb, 0.5)
    assert not torch.isnan(c).any() and (out[M * N:] == 3).all()


def test_gemm_nan_blocks_and_extreme_scales():
    """A NaN block reaches its own row (or column) and nothing else; products
    of the largest and smallest scales stay within fp32's rules."""
    for M, N in ((5, 40), (70, 130), (300, 300)):
        a, b, _, _ = operands(2, M, N, 640)
        a[1][3, 7] = 255
        b[1][N - 1, 2] = 255
        c = host(nv.mx_gemm(nv.mx_to_device(*a), nv.mx_to_device(*b)))
        nan = np.zeros((M, N), bool)
        nan[3], nan[:, N - 1] = True, True
        assert np.array_equal(np.isnan(c), nan)
    codes = np.full((16, 64), 0x77, np.uint8)             # 6.0 everywhere
    low, high = np.zeros((16, 4), np.uint8), np.full((16, 4), 254, np.uint8)
    A, B = nv.mx_to_device(codes, low), nv.mx_to_device(codes, high)
    assert (nv.mx_gemm(A, B, dtype=torch.float32) == 128 * 36).all()   # 2^-127 * 2^127
    assert torch.isinf(nv.mx_gemm(B, B)).all()
    assert (nv.mx_gemm(A, A) == 0).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,N,K", [(1, 768, 6144), (3, 50, 160), (16, 256, 2080), (4, 64, 32), (5, 40, 6112),
                                   (13, 128, 8704)])
def test_gemm_quantized_is_the_two_calls(M, N, K, dtype):
    say(f"gemm_quantized {M}x{N}x{K} {dtype}")
    g = rng(5, M, N, K)
    wide = np.full((M, K + 8), np.nan, np.float32)
    wide[:, :K] = g.standard_normal((M, K)) * np.exp(2 * g.standard_normal((M, 1)))
    x = torch.from_numpy(wide).to(DT[dtype]).to(DEV)[:, :K]
    b = mx_ref.random_operand(g, N, K)
    B = nv.mx_to_device(*b)
    for out_type in DT.values():
        two = nv.mx_gemm(nv.mx_quantize(x), B, 0.5, dtype=out_type)
        assert torch.equal(nv.mx_gemm_quantized(x, B, 0.5, dtype=out_type), two)
        assert torch.equal(nv.mx_linear(x, B, 0.5, dtype=out_type), two)
    va = mx_ref.values(*mx_ref.quantize(host(x)))
    check(two, va, mx_ref.values(*b), 0.5)


def test_linear_wide():
    """A few rows by so many columns that a workgroup takes several blocks of them, up to K = 8192 with the rows
    quantised once; behind that they may take a launch of their own."""
    g = rng(16)
    for M, N, K in ((3, 50_000, 2080), (16, 8300, 6112), (5, 4130, 8224), (2, 9000, 16416)):
        x = torch.from_numpy(g.standard_normal((M, K)).astype(np.float32)).to(DEV)
        b = mx_ref.random_operand(g, N, K)
        B = nv.mx_to_device(*b)
        c = nv.mx_gemm_quantized(x, B)
        check(c, mx_ref.values(*mx_ref.quantize(host(x))), mx_ref.values(*b), 1.0)
        assert torch.equal(c, nv.mx_linear(x, B)) and torch.equal(c, nv.mx_gemm(nv.mx_quantize(x), B))
    x = torch.from_numpy(g.standard_normal((3, 2080)).astype(np.float32)).to(DEV)
    b = mx_ref.random_operand(g, 50_000, 2080)
    B = nv.mx_to_device(*b)
    c = nv.mx_linear(x, B)
    check(c, mx_ref.values(*mx_ref.quantize(host(x))), mx_ref.values(*b), 1.0)
    assert torch.equal(c, nv.mx_gemm_quantized(x, B))
    K, N = 8192, 49_200                           # weights beyond the last-level cache
    W = nv.mx_quantize(torch.randn(N, K, device=DEV, dtype=torch.bfloat16))
    for M in (1, 16):
        x = torch.randn(M, K, device=DEV)
        c = nv.mx_linear(x, W)
        assert torch.equal(c, nv.mx_gemm_quantized(x, W))
        c1, s1 = nv.mx_packed_size(16, K)
        for at in (0, N // 16 - 1):               # the first and the last 16 columns by themselves
            part = nv.MxOperand(W.codes[at * c1:(at + 1) * c1], W.scales[at * s1:(at + 1) * s1], 16, K)
            assert torch.equal(c[:, at * 16:at * 16 + 16], nv.mx_linear(x, part))


def test_linear_many_rows_and_none():
    g = rng(6)
    x = torch.from_numpy(g.standard_normal((150, 416)).astype(np.float32)).to(DEV)
    b = mx_ref.random_operand(g, 72, 416)
    B = nv.mx_to_device(*b)
    check(nv.mx_linear(x, B), mx_ref.values(*mx_ref.quantize(host(x))), mx_ref.values(*b), 1.0)
    assert nv.mx_linear(x[:0], B).shape == (0, 72)
    assert nv.mx_gemm(nv.mx_quantize(x[:0]), B).shape == (0, 72)
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.mx_gemm_quantized(x, B)
    assert e.value.status == nv.ERR_UNSUPPORTED


def test_nan_row_of_activations():
    x = torch.ones(20, 256, device=DEV)
    x[7, 100] = float("nan")
    x[9, 3] = float("inf")
    B = nv.mx_quantize(torch.ones(48, 256, device=DEV))
    for c in (nv.mx_linear(x, B), torch.cat([nv.mx_gemm_quantized(x[:10], B), nv.mx_gemm_quantized(x[10:], B)]),
              nv.mx_gemm(nv.mx_quantize(x), B)):
        nan = torch.isnan(c).all(dim=1).cpu()
        assert nan.nonzero().flatten().tolist() == [7, 9]
        assert (c[~nan.to(DEV)] == 256).all()


# ---- grouped product ---------------------------------------------------------


def grouped_reference(va, vb, offsets, rows, alpha, out_eps):
    M, N = len(rows), vb.shape[1]
    want, bound = np.zeros((M, N)), np.zeros((M, N))
    for g in range(vb.shape[0]):
        r = slice(offsets[g], offsets[g + 1])
        if r.stop > r.start:
            want[r] = alpha * (va[rows[r]] @ vb[g].T)
            bound[r] = mx_ref.gemm_bound(va[rows[r]], vb[g], alpha, out_eps)
    return want, bound


@pytest.mark.parametrize("sizes,N,K,tail", [
    ([0, 1, 16, 17, 40], 40, 640, 0),          # empty, one row, whole and broken row blocks
    ([3, 0, 0, 33], 16, 128, 5),                # rows behind the last group
    ([16] * 9, 256, 2080, 0),
    ([5, 27, 2], 73, 4128, 3),                  # odd columns
    ([130, 64, 1, 200], 130, 544, 7),           # dozens of rows each
    ([700, 0, 300], 264, 1152, 2),              # hundreds of rows each
    ([30, 0, 1, 64] * 50, 256, 160, 6),         # many small groups: 64 x 256 tiles
    ([40, 3] * 120, 100, 96, 1),                # the same, narrow: 128 x 128
    ([130, 400] * 40, 290, 224, 4),             # many larger ones: 128 x 256
    ([0, 0, 0], 32, 64, 4),                     # nothing but a tail
    ([150, 0, 200, 110] * 30, 200, 160, 3),     # about a hundred rows each
    ([130, 200, 97, 0, 223] * 13, 520, 3232, 1),  # and deep
    ([66, 47, 80, 130] * 30, 515, 416, 2),      # fewer
])
@pytest.mark.parametrize("indirect", [False, True])
def test_grouped(sizes, N, K, tail, indirect):
    say(f"grouped {sizes} N={N} K={K} tail={tail} indirect={indirect}")
    g = rng(sum(sizes), N, K)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    M = int(off[-1]) + tail
    n = 23 if indirect else M
    a = mx_ref.random_operand(g, n, K)
    b = mx_ref.random_operand(g, len(sizes) * N, K)
    b = b[0].reshape(len(sizes), N, -1), b[1].reshape(len(sizes), N, -1)
    rows = g.integers(0, n, M).astype(np.int32) if indirect else np.arange(M)
    if indirect and tail:
        rows[-tail:] = -1
    A, B = nv.mx_to_device(*a), nv.mx_groups_to_device(*b)
    r = torch.from_numpy(rows.astype(np.int32)).to(DEV) if indirect else None
    for dtype in DT.values():
        out = torch.full((M, N), 5.0, dtype=dtype, device=DEV)
        nv.mx_grouped_gemm(A, B, torch.from_numpy(off).to(DEV), 0.5, rows=r, out=out)
        want, bound = grouped_reference(mx_ref.values(*a), mx_ref.values(*b), off, rows, 0.5, EPS[dtype])
        kept = int(off[-1])
        assert (np.abs(host(out)[:kept] - want[:kept]) <= bound[:kept]).all()
        assert (out[kept:] == 5).all()


def test_operands_past_32_bits():
    """Row blocks of A behind 4 GiB of codes (and, grouped, tables that point
    there), and a quantisation of more than 2^32 values."""
    K, rows = 8192, 1_100_000                                 # 4.5 GB of codes
    cb, sb = nv.mx_packed_size(rows, K)
    g = torch.Generator(device=DEV)
    g.manual_seed(12)
    A = nv.MxOperand(torch.randint(0, 256, (cb,), dtype=torch.uint8, device=DEV, generator=g),
                     torch.randint(120, 130, (sb,), dtype=torch.uint8, device=DEV, generator=g), rows, K)
    b = mx_ref.random_operand(rng(12), 3 * 16, K)
    vb = mx_ref.values(*b)
    c1, s1 = nv.mx_packed_size(16, K)

    def values(block):
        """The 16 rows of a row block, unpacked on the host."""
        return mx_ref.values(*nv.mx_unpack(A.codes[block * c1:(block + 1) * c1].cpu().numpy(),
                                           A.scales[block * s1:(block + 1) * s1].cpu().numpy(), 16, K))

    c = nv.mx_gemm(A, nv.mx_to_device(b[0][:16], b[1][:16]))
    last = rows // 16 - 1
    for block in (0, 40000, last):
        check(c[block * 16:block * 16 + 16], values(block), vb[:16], 1.0)
    del c
    W = nv.mx_groups_to_device(b[0].reshape(3, 16, -1), b[1].reshape(3, 16, -1))
    pick = torch.tensor([rows - 1, 3, 640000, rows - 2, 17], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 2, 2, 5], dtype=torch.int32, device=DEV)
    y = nv.mx_grouped_gemm(A, W, off, rows=pick)
    va = np.stack([values(r // 16)[r % 16] for r in pick.tolist()])
    check(y[:2], va[:2], vb[:16], 1.0)
    check(y[2:], va[2:], vb[32:], 1.0)
    del A
    x = torch.empty(rows // 2, K, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    q = nv.mx_quantize(x)
    tail = nv.MxOperand(q.codes[-c1:], q.scales[-s1:], 16, K)
    equal_bytes(tail, host(x[-16:]))
    assert torch.equal(nv.mx_dequantize(q, x.dtype)[-16:], nv.mx_dequantize(tail, x.dtype))


@pytest.mark.parametrize("K", [131071 * 128, 131073 * 128 - 96])
def test_very_deep_products(K):
    """The deepest operands of the tile kernel's 32-bit offsets, and deeper ones: zeros but for a few blocks,
    whose products are small integers, so that sums are exact in any order."""
    M, N = 80, 72
    say(f"deep K={K}")
    g = torch.Generator(device=DEV)
    g.manual_seed(14)
    at = [0, 4096, K // 2 // 32 * 32, K - 4128, K - 32]

    def rows(n):
        x = torch.zeros(n, K, dtype=torch.bfloat16, device=DEV)
        parts = [torch.randint(-2, 3, (n, 32), device=DEV, generator=g) for _ in at]
        for k, p in zip(at, parts):
            x[:, k:k + 32] = p.to(torch.bfloat16)
        return nv.mx_quantize(x), torch.cat(parts, 1).double().cpu()

    (A, va), (B, vb) = rows(M), rows(N)
    assert torch.equal(nv.mx_gemm(A, B, dtype=torch.float32).double().cpu(), va @ vb.T)
    W = nv.MxGroups(B.codes, B.scales, 1, N, K)
    off = torch.tensor([3, 75], dtype=torch.int32, device=DEV)
    out = torch.zeros(M, N, device=DEV)
    nv.mx_grouped_gemm(A, W, off, out=out)
    assert torch.equal(out[3:75].double().cpu(), (va @ vb.T)[3:75]) and (out[:3] == 0).all() and (out[75:] == 0).all()


@pytest.mark.parametrize("N", [33_000, 33_001])
def test_result_of_more_than_2_31_elements(N):
    M, K = 66_000, 32
    a, b, va, vb = operands(15, M, N, K)
    A, B = nv.mx_to_device(*a), nv.mx_to_device(*b)
    c = nv.mx_gemm(A, B)
    for r in (0, 65_072, M - 16):                 # (behind row 65072: more than 2^31 elements)
        check(c[r:r + 16], va[r:r + 16], vb, 1.0)


def test_grouped_malformed_tables_stay_inside():
    """Offsets and row numbers out of range are clamped: rows may be wrong,
    the memory behind the output is untouched."""
    g = rng(8)
    A, B = nv.mx_to_device(*mx_ref.random_operand(g, 40, 256)), \
        nv.mx_groups_to_device(*(t.reshape(3, 32, -1) for t in mx_ref.random_operand(g, 96, 256)))
    for off in ([0, 10, 5, 60], [-7, 20, 40, 1000], [50, 60, 70, 80]):
        out = torch.full((40 * 32 + 512,), 9.0, device=DEV)
        rows = torch.arange(-20, 60, 2, dtype=torch.int32, device=DEV)
        nv.mx_grouped_gemm(A, B, torch.tensor(off, dtype=torch.int32, device=DEV), rows=rows,
                           out=out[:40 * 32].view(40, 32))
        torch.cuda.synchronize()
        assert (out[40 * 32:] == 9).all()


def test_grouped_without_rows():
    B = nv.mx_quantize(torch.ones(2, 16, 64, device=DEV))
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert nv.mx_grouped_gemm(nv.mx_quantize(torch.zeros(0, 64, device=DEV)), B, off).shape == (0, 16)


# ---- streams, graphs, sequences ------------------------------------------------


def test_streams_and_graph_replays():
    g = rng(9)
    x = torch.from_numpy(g.standard_normal((48, 1056)).astype(np.float32)).to(DEV)
    B = nv.mx_to_device(*mx_ref.random_operand(g, 96, 1056))
    want = nv.mx_gemm(nv.mx_quantize(x), B)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = nv.mx_gemm(nv.mx_quantize(x, stream=s), B, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    q, out = nv.mx_quantize(x), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.mx_quantize(x, out=q)
        nv.mx_gemm(q, B, out=out)
    for i in range(3):
        x.copy_(torch.randn_like(x) * (i + 1))
        want = nv.mx_gemm(nv.mx_quantize(x), B)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_sequence():
    g = rng(10)
    x = torch.from_numpy(g.standard_normal((15, 544)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    B = nv.mx_to_device(*mx_ref.random_operand(g, 64, 544))
    W = nv.mx_groups_to_device(*(t.reshape(2, 32, -1) for t in mx_ref.random_operand(g, 64, 544)))
    off = torch.tensor([0, 9, 15], dtype=torch.int32, device=DEV)
    q = nv.mx_quantize(x)
    c1, c2 = (torch.empty(15, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c3 = torch.empty(15, 32, device=DEV)
    seq = nv.Sequence()
    seq.add_mx_quantize(x, q)
    seq.add_mx_gemm(q, B, c1, 0.5)
    seq.add_mx_gemm_quantized(x, B, c2, 0.5)
    seq.add_mx_grouped_gemm(q, W, off, c3)
    seq.finalize()
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        want = nv.mx_gemm(nv.mx_quantize(x), B, 0.5)
        want3 = nv.mx_grouped_gemm(nv.mx_quantize(x), W, off, dtype=torch.float32)
        seq.launch()
        torch.cuda.synchronize()
        assert torch.equal(c1, want) and torch.equal(c2, want) and torch.equal(c3, want3)
    seq.close()


@pytest.mark.parametrize("lead", [(2, 3), (3, 1, 4), (5, 40)])
@pytest.mark.parametrize("dtype", list(DT))
def test_linear_with_leading_dimensions(lead, dtype):
    """Activations [batch, sequence, K]: every batch, few rows and many, strided rows and ones that need a copy."""
    g = rng(21, *lead)
    n = int(np.prod(lead))
    B = nv.mx_to_device(*mx_ref.random_operand(g, 72, 160))
    wide = torch.from_numpy(g.standard_normal((*lead, 168)).astype(np.float32)).to(DT[dtype]).to(DEV)
    x = wide[..., :160]
    want = nv.mx_linear(x.reshape(n, 160), B, 0.5)
    vb = mx_ref.values(*nv.mx_unpack(B.codes.cpu().numpy(), B.scales.cpu().numpy(), 72, 160))
    check(want, mx_ref.values(*mx_ref.quantize(host(x).reshape(n, 160))), vb, 0.5)
    want = want.view(*lead, 72)
    assert torch.equal(nv.mx_linear(x, B, 0.5), want)
    turned = x.transpose(0, 1).contiguous().transpose(0, 1)      # the same rows at two strides
    out = torch.empty_like(want)
    assert nv.mx_linear(turned, B, 0.5, out=out) is out and torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = nv.mx_linear(turned, B, 0.5, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    assert nv.mx_linear(x[:0], B).shape == (0, *lead[1:], 72)


@pytest.mark.parametrize("G,N,K,rows", [
    (5000, 40, 160, {0: 1, 17: 2, 4999: 5}),      # 64 x 64 tiles, one team of waves
    (700, 300, 4128, {3: 1, 4: 1, 698: 3}),       # two teams
    (300, 16400, 96, {0: 2, 150: 1, 299: 1}),     # 64 x 256
    (65536, 16, 32, {65535: 1}),
])
@pytest.mark.parametrize("tail", [0, 2])
def test_grouped_few_rows_of_many_groups(G, N, K, rows, tail):
    """More groups than rows: the few that have some, wherever they are."""
    say(f"grouped G={G} N={N} K={K} rows={rows} tail={tail}")
    g = rng(G, N, K)
    M = sum(rows.values()) + tail
    sizes = np.zeros(G, np.int64)
    sizes[list(rows)] = list(rows.values())
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(DEV)
    a = mx_ref.random_operand(g, M, K)
    cb, sb = nv.mx_packed_size(N, K)
    B = nv.MxGroups(torch.randint(0, 256, (cb * G,), dtype=torch.uint8, device=DEV),
                    torch.randint(120, 130, (sb * G,), dtype=torch.uint8, device=DEV), G, N, K)
    out = torch.full((M, N), 5.0, device=DEV)
    nv.mx_grouped_gemm(nv.mx_to_device(*a), B, off, out=out)
    va, at = mx_ref.values(*a), 0
    for e, n in rows.items():
        vb = mx_ref.values(*nv.mx_unpack(B.codes[e * cb:(e + 1) * cb].cpu().numpy(),
                                         B.scales[e * sb:(e + 1) * sb].cpu().numpy(), N, K))
        check(out[at:at + n], va[at:at + n], vb, 1.0)
        at += n
    assert (out[at:] == 5).all()


# ---- operands that outgrow the last-level cache (loads and stores with the non-temporal hint) ----


@pytest.mark.parametrize("E,N,K,sizes", [
    (256, 256, 6144, [0, 16, 64, 65, 1, 33, 200, 17]),      # 64 x 256 tiles
    (256, 260, 6112, [128, 129, 5, 0, 300, 256, 200, 61]),  # 128 x 256
    (520, 120, 6112, [0, 16, 128, 129, 1, 33, 257, 17]),    # 128 x 128
    (600, 250, 5216, [1] + [0] * 199),                      # 64 x 64, two teams of waves
    (1500, 250, 2016, [2] + [0] * 499),                     # one team
])
@pytest.mark.parametrize("indirect", [False, True])
def test_grouped_weights_beyond_the_cache(E, N, K, sizes, indirect):
    """Groups of no, one and several row blocks side by side."""
    say(f"grouped E={E} N={N} K={K} sizes={sizes[:8]} indirect={indirect}")
    g = rng(E, N, K)
    sizes = (sizes * E)[:E]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    M, n = int(off[-1]) + 3, 37
    cb, sb = nv.mx_packed_size(N, K)
    assert (cb + sb) * E > 192 << 20
    B = nv.MxGroups(torch.randint(0, 256, (cb * E,), dtype=torch.uint8, device=DEV),
                    torch.randint(120, 130, (sb * E,), dtype=torch.uint8, device=DEV), E, N, K)
    a = mx_ref.random_operand(g, n if indirect else M, K)
    rows = g.integers(0, n, M).astype(np.int32) if indirect else np.arange(M)
    va = mx_ref.values(*a)
    out = torch.full((M, N), 5.0, dtype=torch.bfloat16, device=DEV)
    nv.mx_grouped_gemm(nv.mx_to_device(*a), B, torch.from_numpy(off).to(DEV), out=out,
                       rows=torch.from_numpy(rows).to(DEV) if indirect else None)
    used = [e for e in range(E) if sizes[e]]
    for e in used[:8] + used[len(used) // 2:len(used) // 2 + 8] + used[-8:]:
        vb = mx_ref.values(*nv.mx_unpack(B.codes[e * cb:(e + 1) * cb].cpu().numpy(),
                                         B.scales[e * sb:(e + 1) * sb].cpu().numpy(), N, K))
        check(out[off[e]:off[e + 1]], va[rows[off[e]:off[e + 1]]], vb, 1.0)
    assert not torch.isnan(out).any() and (out[off[-1]:] == 5).all()


def test_few_packed_rows_by_weights_beyond_the_cache():
    """The product of packed rows beside the one that quantises them, whose columns test_linear_wide checks."""
    K, N = 8160, 49_205
    W = nv.mx_quantize(torch.randn(N, K, device=DEV, dtype=torch.bfloat16))
    for M in (1, 7, 16):
        q = nv.mx_quantize(torch.randn(M, K, device=DEV))
        x = nv.mx_dequantize(q)                              # quantising these again gives the same operand
        for dtype in DT.values():
            c = nv.mx_gemm(q, W, dtype=dtype)
            assert torch.equal(c, nv.mx_gemm_quantized(x, W, dtype=dtype))
        c1, s1 = nv.mx_packed_size(N % 16 or 16, K)
        tail = nv.MxOperand(W.codes[-c1:], W.scales[-s1:], N % 16, K)
        check(c[:, N - N % 16:], host(x).astype(np.float64), host(nv.mx_dequantize(tail)).astype(np.float64), 1.0)


@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_and_back_beyond_the_cache(dtype):
    """The same rows in parts, which take the plain loads and stores."""
    rows, K = (6205, 8224) if dtype == "fp32" else (12_301, 8224)
    x = torch.randn(rows, K, device=DEV).to(DT[dtype]) * torch.rand(rows, 1, device=DEV).to(DT[dtype]) * 8
    assert x.numel() * x.element_size() > 192 << 20
    q = nv.mx_quantize(x)
    back = {t: nv.mx_dequantize(q, t) for t in DT.values()}
    assert torch.equal(back[torch.float32], back[torch.bfloat16].float())
    for r in range(0, rows, 2048):
        part = nv.mx_quantize(x[r:r + 2048])
        cb, sb = nv.mx_packed_size(r, K)
        assert torch.equal(q.codes[cb:cb + part.codes.numel()], part.codes)
        assert torch.equal(q.scales[sb:sb + part.scales.numel()], part.scales)
        for t in DT.values():
            assert torch.equal(back[t][r:r + 2048], nv.mx_dequantize(part, t))
    equal_bytes(part, host(x[r:]))


# ---- rounding and range ---------------------------------------------------------


def test_quantize_fp32_beside_the_borders():
    """fp32 values one step below, on and above every border between codes, under every scale."""
    tops = [np.float32(1.5) * np.float32(2.0) ** e for e in range(-140, 127)] + [np.float32(2.0 ** -149)]
    blocks = []
    for top in tops:
        _, e = np.frexp(np.float64(top))
        scale = 2.0 ** max(e - 3, -127)
        for sign in (1.0, -1.0):
            v = np.array([sign * edge * scale for edge in mx_ref.EDGES], np.float64).astype(np.float32)
            inf = np.float32(np.inf)
            row = np.concatenate([v, np.nextafter(v, inf), np.nextafter(v, -inf), [top, -top, 0.0, -0.0]])
            row = np.where(np.abs(row) <= np.float32(top) * np.float32(1.3), row, 0.0)   # (none above the top)
            blocks.append(np.concatenate([row, np.zeros(32 - row.size)]).astype(np.float32))
    equal_bytes(nv.mx_quantize(torch.from_numpy(np.stack(blocks)).to(DEV)), np.stack(blocks))


@pytest.mark.parametrize("dtype", list(DT))
def test_dequantize_past_the_largest_value(dtype):
    """A code times its scale is exact where the type holds it; 2^128 and more are infinities."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (6, 2))
    codes = (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)
    scales = np.array([[0], [1], [251], [252], [253], [254]], np.uint8)
    got = nv.mx_dequantize(nv.mx_to_device(codes, scales), DT[dtype]).double().cpu().numpy()
    want = mx_ref.values(codes, scales)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))
    assert np.isinf(want).sum() == 2 * (2 * 2 + 2 * 4)       # +-4, 6 under byte 253; +-2, 3, 4, 6 under 254; twice
