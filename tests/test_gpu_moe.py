"""Expert routing on the GPU against the 64-bit references of mx_ref.py, and
a whole layer of experts through it."""
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


def say(msg: str) -> None:
    print(f"[gpu] {msg}", flush=True)
    sys.stdout.flush()


def rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def host(t):
    return t.to(torch.float32).cpu().numpy()


def choices(g, T, k, E, drop=0.0):
    ids = g.integers(0, E, (T, k)).astype(np.int32)       # the same expert twice in a row happens
    bad = g.random((T, k)) < drop
    return np.where(bad, g.choice([-1, E, E + 5, -2 ** 31], (T, k)), ids).astype(np.int32)


def check_sort(ids, E, wide=False):
    t = torch.from_numpy(ids).to(DEV)
    r = nv.moe_sort(t.to(torch.int64) if wide else t, E)
    off, slots, tokens = mx_ref.sort(ids, E)
    assert np.array_equal(r.row_offsets.cpu().numpy(), off)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    assert np.array_equal(r.tokens.cpu().numpy(), tokens)
    return r


@pytest.mark.parametrize("T,k,E,drop", [
    (1, 1, 1, 0.0), (1, 8, 256, 0.0), (64, 8, 256, 0.0), (7, 3, 2, 0.5), (512, 8, 256, 0.1), (33, 1, 2048, 0.0),
    (513, 8, 64, 0.0), (1024, 4, 300, 0.05), (3000, 7, 257, 0.3), (9001, 2, 1, 0.5), (100, 6, 40, 1.0),
    (4096, 1, 7, 0.0), (700, 64, 512, 0.2), (2048, 8, 256, 0.0), (2049, 8, 2048, 0.1),
    (20000, 3, 5, 0.3), (8192, 8, 256, 0.05)])
@pytest.mark.parametrize("wide", [False, True])
def test_sort(T, k, E, drop, wide):
    say(f"sort T={T} k={k} E={E} drop={drop} wide={wide}")
    check_sort(choices(rng(T, k, E), T, k, E, drop), E, wide)


def test_sort_one_expert_takes_all_and_wide_numbers():
    check_sort(np.full((5000, 2), 3, np.int32), 5)
    ids = torch.tensor([[2 ** 32 + 1, 1], [-2 ** 40, 0]], device=DEV)   # low words that look like experts
    r = nv.moe_sort(ids, 4)
    assert r.row_offsets.tolist() == [0, 1, 2, 2, 2] and r.slots.tolist() == [[-1, 1], [-1, 0]]


def test_sort_a_long_list():
    """More than 1024 chunks: larger ones, sorted against torch."""
    E, ids = 37, torch.from_numpy(choices(rng(1), 600_001, 8, 37, 0.1)).to(DEV)
    r = nv.moe_sort(ids, E)
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    kept = int((key < E).sum())
    assert torch.equal(r.row_offsets.long(), torch.searchsorted(key[order], torch.arange(E + 1, device=DEV)))
    assert torch.equal(r.tokens[:kept].long(), order[:kept] // 8) and (r.tokens[kept:] == -1).all()
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel(), device=DEV)
    assert torch.equal(r.slots.flatten().long(), torch.where(key < E, slots, -1))


def test_sort_no_tokens():
    r = nv.moe_sort(torch.empty(0, 8, dtype=torch.int32, device=DEV), 16)
    assert r.row_offsets.tolist() == [0] * 17
    x = torch.empty(0, 64, device=DEV)
    assert nv.moe_gather(x, r).shape == (0, 64) and nv.moe_combine(x, r).shape == (0, 64)
    dy, dw = nv.moe_combine_grad(x, x, r)
    assert dy.shape == (0, 64) and dw.shape == (0, 8)


ROWS = [(1, 1, 1, 1), (5, 3, 4, 7), (64, 8, 256, 6144), (33, 2, 8, 973), (200, 8, 32, 514), (17, 9, 5, 2050),
        (40, 17, 64, 132)]


def case(T, k, E, H, dtype, drop=0.2):
    g = rng(T, k, E, H)
    ids = choices(g, T, k, E, drop)
    r = nv.moe_sort(torch.from_numpy(ids).to(DEV), E)
    make = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32)).to(DT[dtype])  # noqa: E731
    w = torch.from_numpy(g.random((T, k)).astype(np.float32))
    return ids, r, make, w


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,k,E,H", ROWS)
def test_gather(T, k, E, H, dtype):
    ids, r, make, _ = case(T, k, E, H, dtype)
    x = make(T, H)
    out = torch.full((T * k, H), 7.0, dtype=DT[dtype], device=DEV)
    nv.moe_gather(x.to(DEV), r, out=out)
    _, slots, tokens = mx_ref.sort(ids, E)
    want = host(x)[np.maximum(tokens, 0)]
    want[tokens < 0] = 7.0                                  # rows that no choice owns stay
    assert np.array_equal(host(out), want)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,k,E,H", ROWS)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, E, H, dtype, weighted):
    ids, r, make, w = case(T, k, E, H, dtype)
    off, slots, _ = mx_ref.sort(ids, E)
    y = make(T * k, H)
    y[off[-1]:] = float("nan")                              # behind the last row: never read
    w[torch.from_numpy(slots < 0)] = float("nan")           # of dropped choices: ignored
    out = nv.moe_combine(y.to(DEV), r, w.to(DEV) if weighted else None)
    wn = w.numpy() if weighted else None
    want = mx_ref.combine(host(y), slots, wn)
    mag = mx_ref.combine(np.abs(host(y)), slots, np.abs(wn) if weighted else None)
    # k products and k sums rounded to fp32 (2^-24 each), the result once by half a step
    bound = 2 * k * 2.0 ** -24 * mag + torch.finfo(DT[dtype]).eps / 2 * np.abs(want) * 1.001 + 1e-40
    assert (np.abs(host(out) - want) <= bound).all()
    if not weighted:
        assert torch.equal(out, nv.moe_gather_grad(y.to(DEV), r))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,k,E,H", ROWS)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad(T, k, E, H, dtype, weighted):
    ids, r, make, w = case(T, k, E, H, dtype)
    off, slots, _ = mx_ref.sort(ids, E)
    y, d = make(T * k, H), make(T, H)
    y[off[-1]:] = float("nan")
    dy0 = torch.full((T * k, H), 7.0, dtype=DT[dtype], device=DEV)
    dy, dw = nv.moe_combine_grad(d.to(DEV), y.to(DEV), r, w.to(DEV) if weighted else None, dy=dy0)
    wn = w.numpy() if weighted else None
    want, dwant = mx_ref.combine_grad(host(d), host(y), slots, wn)
    kept = int(off[-1])
    half = torch.finfo(DT[dtype]).eps / 2
    assert (np.abs(host(dy)[:kept] - want[:kept]) <= (half + 2.0 ** -24) * np.abs(want[:kept]) * 1.001 + 1e-40).all()
    assert (dy[kept:] == 7).all()
    # H products and sums of fp32, in any order
    _, mag = mx_ref.combine_grad(np.abs(host(d)), np.abs(host(y)), slots, None)
    assert (np.abs(dw.cpu().numpy() - dwant) <= (H + 1) * 2.0 ** -24 * mag).all()
    assert (dw.cpu().numpy()[slots < 0] == 0).all()
    # the gradient may take y's place
    y2 = y.to(DEV)
    _, dw2 = nv.moe_combine_grad(d.to(DEV), y2, r, w.to(DEV) if weighted else None, dy=y2)
    assert torch.equal(y2[:kept], dy[:kept]) and torch.equal(dw2, dw)


def test_gradients_against_differences():
    """combine is linear in y and in the weights: a difference along any
    direction is the gradient's product with it, up to fp32 rounding."""
    T, k, E, H = 30, 4, 8, 96
    ids, r, make, w = case(T, k, E, H, "fp32")
    y, dy, d, dw = make(T * k, H).to(DEV), make(T * k, H).to(DEV), make(T, H).to(DEV), torch.randn(T, k).to(DEV)
    w = w.to(DEV)
    kept = int(r.row_offsets[-1])
    dy[kept:] = 0
    y[kept:] = 0
    loss = lambda y, w: float((nv.moe_combine(y, r, w).double() * d.double()).sum())  # noqa: E731
    gy, gw = nv.moe_combine_grad(d, y, r, w, dy=torch.zeros_like(y))
    size = float(nv.moe_combine(y.abs() + dy.abs(), r, w.abs() + dw.abs()).double().mul(d.abs().double()).sum())
    tol = 64 * 2.0 ** -24 * size      # a few fp32 roundings (steps, products, sums) of every term
    assert abs((loss(y + dy, w) - loss(y - dy, w)) / 2 - float((gy.double() * dy.double()).sum())) <= tol
    assert abs((loss(y, w + dw) - loss(y, w - dw)) / 2 - float((gw.double() * dw.double()).sum())) <= tol
    x = make(T, H).to(DEV)
    gx = nv.moe_gather_grad(dy, r)
    rows = nv.moe_gather(x, r, out=torch.zeros_like(y))
    assert abs(float((rows.double() * dy.double()).sum()) - float((gx.double() * x.double()).sum())) <= \
        8 * 2.0 ** -24 * float((rows.abs().double() * dy.abs().double()).sum())


def test_strided_and_unaligned_rows():
    for dtype in DT.values():
        ids, r, make, w = case(20, 3, 4, 64, "fp32", drop=0.0)
        wide = torch.randn(20, 70, device=DEV).to(dtype)
        x = wide[:, 3:67]                                   # rows start on odd addresses, 70 elements apart
        assert torch.equal(nv.moe_gather(x, r), nv.moe_gather(x.contiguous(), r))
        y = torch.randn(60, 64, device=DEV).to(dtype)
        a = nv.moe_combine_grad(x, y, r, w.to(DEV))
        b = nv.moe_combine_grad(x.contiguous(), y, r, w.to(DEV))
        assert torch.equal(a[0], b[0])
        assert torch.allclose(a[1], b[1], rtol=0, atol=64 * 2.0 ** -23 * 64)   # another order of 64 terms of about 1
        flat = torch.randn(60 * 64 + 1, device=DEV).to(dtype)[1:].view(60, 64)  # an odd base address
        assert torch.equal(nv.moe_combine(flat, r), nv.moe_combine(flat.clone(), r))


def test_more_than_2_31_elements():
    """Rows behind 2^32 bytes and 2^31 elements of the experts' order."""
    T, k, E, H = 300_000, 8, 16, 1024
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    ids = torch.randint(0, E, (T, k), device=DEV, generator=g)
    r = nv.moe_sort(ids, E)
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    rows = nv.moe_gather(x, r)
    for i in (0, T * k // 2, T * k - 1):
        assert torch.equal(rows[i], x[r.tokens[i].long()])
    dy, dw = nv.moe_combine_grad(x, rows, r)
    assert torch.equal(dy[-1000:], rows[-1000:])              # every row holds its token's gradient
    want = (x[-50:].double() ** 2).sum(1, keepdim=True).expand(50, k)
    assert ((dw[-50:].double() - want).abs() <= (H + 1) * 2.0 ** -24 * want).all()
    back = nv.moe_gather_grad(rows, r)
    # k equal values of 8 bits: their sums are exact in fp32, and rounded once
    assert torch.equal(back, (k * x.float()).to(torch.bfloat16))


def test_other_streams_and_shared_tables():
    """Two streams at once with the same route: no call keeps anything."""
    T, k, E, H = 128, 4, 8, 512
    ids, r, make, w = case(T, k, E, H, "bf16")
    x, wd, idt = make(T, H).to(DEV), w.to(DEV), torch.from_numpy(ids).to(DEV)
    want = nv.moe_combine(nv.moe_gather(x, r, out=torch.zeros(T * k, H, dtype=x.dtype, device=DEV)), r, wd)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in streams:
            route = nv.moe_sort(idt, E, stream=s)
            got.append(nv.moe_combine(nv.moe_gather(x, route, stream=s), route, wd, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)


@pytest.mark.parametrize("T,k,E", [(9000, 2, 40), (3000, 7, 2048)])
def test_a_long_sort_replayed(T, k, E):
    """Three launches, the histograms in row_tokens: every replay starts from what the last one left there."""
    g = rng(13)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    ids.copy_(torch.from_numpy(choices(g, T, k, E, 0.1)))
    r = nv.moe_sort(ids, E)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.moe_sort(ids, E, out=r)
    for _ in range(3):
        new = choices(g, T, k, E, 0.2)
        ids.copy_(torch.from_numpy(new))
        want = nv.moe_sort(ids, E)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((r.row_offsets, want.row_offsets), (r.slots, want.slots), (r.tokens, want.tokens)):
            assert torch.equal(a, b)
        check_sort(new, E)


def test_raw_stream_handles():
    g = rng(14)
    x = torch.randn(40, 128, device=DEV)
    ids = torch.from_numpy(choices(g, 40, 3, 6, 0.0)).to(DEV)
    s = torch.cuda.Stream()
    want = nv.mx_quantize(x)
    torch.cuda.synchronize()
    for handle in (0, s.cuda_stream, s):
        q = nv.mx_quantize(x, stream=handle)
        r = nv.moe_sort(ids, 6, stream=handle)
        y = nv.moe_gather(x, r, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
        assert torch.equal(y, x[r.tokens.long()])


def test_malformed_slots_stay_inside():
    ids, r, make, w = case(16, 2, 4, 32, "fp32", drop=0.0)
    bad = nv.MoeRoute(r.row_offsets, torch.full_like(r.slots, 1 << 30), r.tokens, 4)
    bad.slots[3, 1] = 5
    buf = torch.full((32 * 32 + 256,), 4.0, device=DEV)
    out = buf[:32 * 32].view(32, 32)
    nv.moe_gather(make(16, 32).to(DEV), bad, out=out)
    y = torch.ones(32, 32, device=DEV)
    c = nv.moe_combine(y, bad)
    torch.cuda.synchronize()
    assert (buf[32 * 32:] == 4).all() and (out[:5] == 4).all() and (out[6:] == 4).all()
    assert float(c[3].sum()) == 32 and float(c.sum()) == 32


def swiglu(h):
    g, u = h.float().chunk(2, dim=1)
    return (torch.nn.functional.silu(g) * u).to(torch.bfloat16)


def layer(x, ids, w, up, down, E):
    """A layer of experts in MXFP4, as a serving program runs it."""
    r = nv.moe_sort(ids, E)
    h = nv.mx_grouped_gemm(nv.mx_quantize(x), up, r.row_offsets, rows=r.tokens)
    y = nv.mx_grouped_gemm(nv.mx_quantize(swiglu(h)), down, r.row_offsets)
    return r, y, nv.moe_combine(y, r, w)


@pytest.mark.parametrize("T,E,k,H,I,drop", [(1, 8, 2, 256, 64, 0.0), (64, 16, 4, 512, 96, 0.1),
                                            (300, 4, 2, 256, 160, 0.0)])
def test_a_layer_of_experts(T, E, k, H, I, drop):  # noqa: E741
    """Sort, quantise, product, activation, product, combine and the way back:
    every step against the 64-bit reference on the step's own inputs."""
    say(f"layer T={T} E={E} k={k} H={H} I={I}")
    g = rng(T, E, k, H)
    ids = choices(g, T, k, E, drop)
    x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    w = torch.softmax(torch.from_numpy(g.standard_normal((T, k)).astype(np.float32)), 1).to(DEV)
    up = torch.from_numpy(g.standard_normal((E, 2 * I, H)).astype(np.float32) * 0.05).to(DEV)
    down = torch.from_numpy(g.standard_normal((E, H, I)).astype(np.float32) * 0.05).to(DEV)
    idt = torch.from_numpy(ids).to(DEV)
    r, y, out = layer(x, idt, w, nv.mx_quantize(up), nv.mx_quantize(down), E)
    off, slots, tokens = mx_ref.sort(ids, E)
    kept = int(off[-1])
    val = lambda t: mx_ref.values(*mx_ref.quantize(host(t)))  # noqa: E731
    eps = torch.finfo(torch.bfloat16).eps
    h = nv.mx_grouped_gemm(nv.mx_quantize(x), nv.mx_quantize(up), r.row_offsets, rows=r.tokens)
    act = swiglu(h)
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        if off[e + 1] == off[e]:
            continue
        va, vb = val(x)[tokens[rows]], val(up[e])
        assert (np.abs(host(h)[rows] - va @ vb.T) <= mx_ref.gemm_bound(va, vb, 1.0, eps)).all()
        va, vb = val(act)[rows], val(down[e])
        assert (np.abs(host(y)[rows] - va @ vb.T) <= mx_ref.gemm_bound(va, vb, 1.0, eps)).all()
    want = mx_ref.combine(host(y), slots, w.cpu().numpy())
    mag = mx_ref.combine(np.abs(host(y)), slots, w.cpu().numpy())
    assert (np.abs(host(out) - want) <= 2 * k * 2.0 ** -24 * mag + eps / 2 * np.abs(want) * 1.001 + 1e-40).all()
    # the way back to the experts' outputs and to the tokens
    d = torch.randn_like(out)
    dy, dw = nv.moe_combine_grad(d, y, r, w)
    dx = nv.moe_gather_grad(dy, r)
    wy, ww = mx_ref.combine_grad(host(d), host(y), slots, w.cpu().numpy())
    assert (np.abs(host(dy)[:kept] - wy[:kept]) <= eps / 2 * np.abs(wy[:kept]) * 1.01 + 1e-40).all()
    assert np.abs(dw.cpu().numpy() - ww).max() <= (H + 1) * 2.0 ** -24 * mx_ref.combine_grad(
        np.abs(host(d)), np.abs(host(y)), slots, None)[1].max()
    wx = mx_ref.combine(host(dy), slots, None)
    assert (np.abs(host(dx) - wx) <= eps / 2 * np.abs(wx) * 1.01 + k * 2.0 ** -23 * mx_ref.combine(
        np.abs(host(dy)), slots, None) + 1e-40).all()


def test_the_16_element_format_behind_the_same_routing():
    """moe_sort and moe_gather in front of the library's grouped GEMM of
    E4M3-scaled blocks: each expert's rows equal a GEMM of their own."""
    g = rng(77)
    T, k, E, H, N = 40, 2, 4, 256, 48
    idt = torch.from_numpy(choices(g, T, k, E)).to(DEV)
    x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    w = torch.from_numpy(g.standard_normal((E * N, H)).astype(np.float32)).to(DEV)
    parts = [nv.quantize(w[e * N:(e + 1) * N]) for e in range(E)]
    W = nv.PackedGroups(torch.cat([p.codes for p in parts]), torch.cat([p.scales for p in parts]), E, N, H)
    r = nv.moe_sort(idt, E)
    rows = nv.moe_gather(x, r)
    c = nv.grouped_gemm(nv.quantize(rows), W, r.row_offsets)
    off = r.row_offsets.tolist()
    for e in range(E):
        if off[e + 1] > off[e]:
            one = nv.gemm(nv.quantize(rows[off[e]:off[e + 1]]), parts[e])
            # both sum exact products in fp32, in another order, and round once
            assert torch.allclose(c[off[e]:off[e + 1]].float(), one.float(), rtol=2.0 ** -7, atol=1e-3)
    assert nv.moe_combine(c, r).shape == (T, N)


def test_graph_replays_and_sequence():
    T, E, k, H, N = 48, 16, 4, 512, 64
    g = rng(11)
    ids = torch.from_numpy(choices(g, T, k, E, 0.1)).to(DEV)
    x = torch.randn(T, H, device=DEV).to(torch.bfloat16)
    w = torch.rand(T, k, device=DEV)
    W = nv.mx_quantize(torch.randn(E, N, H, device=DEV))

    def step():
        r = nv.moe_sort(ids, E)
        y = nv.mx_grouped_gemm(nv.mx_quantize(x), W, r.row_offsets, rows=r.tokens)
        return nv.moe_combine(y, r, w)

    r, q = nv.moe_sort(ids, E), nv.mx_quantize(x)
    y, out = torch.empty(T * k, N, dtype=torch.bfloat16, device=DEV), torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    xs = torch.zeros(T * k, H, dtype=torch.bfloat16, device=DEV)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    seq = nv.Sequence()
    seq.add_moe_sort(ids, r)
    seq.add_moe_gather(x, r, xs)
    seq.add_mx_quantize(x, q)
    seq.add_mx_grouped_gemm(q, W, r.row_offsets, y, rows=r.tokens)
    seq.add_moe_combine(y, r, w, out)
    seq.finalize()
    for i in range(3):
        ids.copy_(torch.from_numpy(choices(g, T, k, E, 0.3)).to(DEV))
        x.copy_(torch.randn_like(x))
        w.copy_(torch.rand_like(w))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        seq.launch()
        torch.cuda.synchronize()
        assert torch.equal(captured, want) and torch.equal(out, want)
        rr = nv.moe_sort(ids, E)
        kept = int(rr.row_offsets[-1])
        assert torch.equal(xs[:kept], nv.moe_gather(x, rr)[:kept])
    seq.close()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("k,H", [(1, 1021), (2, 1024), (4, 1021), (8, 1020)])
def test_rows_beyond_the_cache(k, H, dtype):
    """Stores with the non-temporal hint, for each number of rows that are read at a time."""
    say(f"rows beyond the cache k={k} H={H} {dtype}")
    size = torch.finfo(DT[dtype]).bits // 8
    T, E = (200 << 20) // (k * H * size) + 1, 11
    g = torch.Generator(device=DEV)
    g.manual_seed(k)
    ids = torch.randint(-1, E, (T, k), device=DEV, generator=g, dtype=torch.int32)      # some dropped
    r = nv.moe_sort(ids, E)
    kept = int(r.row_offsets[-1])
    make = lambda n: torch.randn(n, H, device=DEV, generator=g).to(DT[dtype])  # noqa: E731
    x, w = make(T), torch.rand(T, k, device=DEV, generator=g)
    rows = torch.full((T * k + 1, H), 7.0, dtype=DT[dtype], device=DEV)
    nv.moe_gather(x, r, out=rows[:-1])
    assert torch.equal(rows[:kept], x[r.tokens[:kept].long()]) and (rows[kept:] == 7).all()
    y, d = make(T * k), make(T)
    out, back = nv.moe_combine(y, r, w), nv.moe_gather_grad(y, r)
    dy = torch.full((T * k + 1, H), 7.0, dtype=DT[dtype], device=DEV)
    _, dw = nv.moe_combine_grad(d, y, r, w, dy=dy[:-1])
    assert (dy[kept:] == 7).all()
    half = torch.finfo(DT[dtype]).eps / 2 * 1.001
    for t in range(0, T, 4096):
        at = r.slots[t:t + 4096].long()
        on = (at >= 0)[:, :, None]
        wt, gt = w[t:t + 4096, :, None].double(), d[t:t + 4096, None].double()
        yt = torch.where(on, y[at.clamp(min=0)].double(), 0.0)
        # k products and k sums rounded to fp32 (2^-24 each), the result once by half a step
        for got, p in ((out, wt * yt), (back, yt)):
            want = p.sum(1)
            assert ((got[t:t + 4096].double() - want).abs()
                    <= 2 * k * 2.0 ** -24 * p.abs().sum(1) + half * want.abs() + 1e-40).all()
        want = (wt * gt).expand(-1, -1, H)                    # rounded to fp32, then to the type
        off = torch.where(on, (dy[at.clamp(min=0)].double() - want).abs(), 0.0)
        assert (off <= (half + 2.0 ** -24) * want.abs() * 1.001 + 1e-40).all()
        p = yt * gt                                           # H products and sums of fp32, in any order
        assert ((dw[t:t + 4096].double() - p.sum(2)).abs() <= (H + 1) * 2.0 ** -24 * p.abs().sum(2)).all()
