"""The norms around a block's residual and their gradients on the GPU, against
the 64-bit formulas of layer_ref.py and against differences."""
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


def say(msg: str) -> None:
    print(f"[gpu] {msg}", flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    return (shift + scale * torch.randn(*shape, device=DEV, generator=g)).to(dtype)


def dbl(t):
    return None if t is None else t.double()


def make(g, rows, H, dtype, wdtype, post, gate, pre, residual=True):
    how = dict(post=post, post_weight=randn(g, H, dtype=wdtype, scale=0.3, shift=1.0) if post else None,
               pre_weight=randn(g, H, dtype=wdtype, scale=0.3, shift=1.0) if pre else None, scale=0.75,
               residual_scale=1.25, eps=1e-5, gate=None)
    if gate == "channel":
        how["gate"] = randn(g, H, dtype=wdtype)
    elif gate == "element":
        how["gate"] = randn(g, rows, H, dtype=dtype)
    y = randn(g, rows, H, dtype=dtype, scale=3.0)
    return y, randn(g, rows, H, dtype=dtype) if residual else None, how


def check_forward(y, res, how, pre, h, n, what):
    want, b = ref.norm_h(dbl(y), dbl(res), how["post"], dbl(how["post_weight"]), dbl(how["gate"]), how["scale"],
                         how["residual_scale"], how["eps"])
    ref.check(h, want, b, what + " h")
    if pre:
        want, b = ref.norm_n(dbl(h), dbl(how["pre_weight"]), how["eps"])
        ref.check(n, want, b, what + " n")
    else:
        assert n is None


def check_grads(dh, dn, y, h, how, gr, what):
    names = {k: how[k] for k in ("post", "scale", "residual_scale", "eps")}
    gate = how["gate"]
    want = ref.norm_grads(dbl(dh), dbl(dn), dbl(y), dbl(h), post_weight=dbl(how["post_weight"]), gate=dbl(gate),
                          pre_weight=dbl(how["pre_weight"]), channel=gate is not None and gate.dim() == 1, **names)
    for name in ("y", "residual", "gate", "post_weight", "pre_weight"):
        got = getattr(gr, name)
        if got is None:
            assert name == "residual" or name not in want or name in ("post_weight", "pre_weight") and how[name] is None, name
        else:
            ref.check(got, *want[name], f"{what} d{name}")


# Every number of waves to a row and of pieces to a lane, rows cut short and shorter than a piece.
WIDTHS = [1, 3, 4, 7, 8, 9, 31, 64, 100, 255, 512, 513, 1000, 1024, 1025, 2047, 2048, 4096, 4100, 5003, 6144, 8192, 8200, 12289, 16384]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(H, dtype):
    say(f"norm width {H} {dtype}")
    g = gen(H)
    forms = [(True, "element", True), (False, "channel", True), (True, "none", False), (True, "channel", True)]
    for i, (post, gate, pre) in enumerate(forms):
        wdtype = torch.float32 if (H + i) % 2 else torch.bfloat16
        y, res, how = make(g, 7 if H > 64 else 70, H, DT[dtype], wdtype, post, gate, pre)
        h, n = nv.add_norm(y, res, pre=pre, **how)
        check_forward(y, res, how, pre, h, n, f"{H}")
        dh, dn = randn(g, *y.shape, dtype=y.dtype), randn(g, *y.shape, dtype=y.dtype) if pre else None
        check_grads(dh, dn, y, h, how, nv.add_norm_grad(dh, dn, y, h, **how), f"{H}")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "element"])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_every_form(post, gate, pre, residual, dtype):
    for rows, H in ((1, 6144), (33, 200)):
        g = gen(rows)
        y, res, how = make(g, rows, H, DT[dtype], torch.float32, post, gate, pre, residual)
        h, n = nv.add_norm(y, res, pre=pre, **how)
        check_forward(y, res, how, pre, h, n, "form")
        dn = randn(g, rows, H, dtype=y.dtype) if pre else None
        for dh in (randn(g, rows, H, dtype=y.dtype), None):
            if dh is None and dn is None:
                continue
            gr = nv.add_norm_grad(dh, dn, y, h, residual=residual, **how)
            check_grads(dh, dn, y, h, how, gr, "form")
            assert (gr.residual is None) == (not residual)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,H", [(5000, 64), (3000, 1030), (1500, 4104), (700, 9000)])
def test_many_rows(rows, H, dtype):
    """More rows than the workgroups of a launch take at once; the same bits every time."""
    say(f"norm {rows} rows of {H} {dtype}")
    g = gen(rows)
    y, res, how = make(g, rows, H, DT[dtype], DT[dtype], True, "channel", True)
    h, n = nv.add_norm(y, res, **how)
    check_forward(y, res, how, True, h, n, "many")
    dh, dn = randn(g, rows, H, dtype=y.dtype), randn(g, rows, H, dtype=y.dtype)
    gr = nv.add_norm_grad(dh, dn, y, h, **how)
    check_grads(dh, dn, y, h, how, gr, "many")
    again = nv.add_norm_grad(dh, dn, y, h, **how)
    for name in ("y", "residual", "gate", "post_weight", "pre_weight"):
        assert torch.equal(getattr(gr, name), getattr(again, name))


def test_rows_past_the_grid():
    """More rows than one launch has workgroups for."""
    rows = (1 << 22) + 1000
    x = torch.arange(rows * 3, device=DEV, dtype=torch.float32).view(rows, 3) % 1000 + 1
    want, b = ref.norm_n(x.double())
    ref.check(nv.rms_norm(x), want, b)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,H", [(1, 32), (5, 64), (16, 128), (17, 160), (33, 544), (100, 2080), (3, 6112), (20, 8192), (2, 16384)])
def test_packed_result(rows, H, dtype):
    """n as an operand: every byte of mx_quantize(n), padding among them; and the whole way into a product."""
    say(f"packed norm {rows}x{H} {dtype}")
    g = gen(H + rows)
    y, res, how = make(g, rows, H, DT[dtype], torch.float32, True, "element", True)
    h, n = nv.add_norm(y, res, **how)
    cb, sb = nv.mx_packed_size(rows, H)
    into = nv.MxOperand(torch.full((cb,), 0xAA, dtype=torch.uint8, device=DEV), torch.full((sb,), 0xAA, dtype=torch.uint8, device=DEV), rows, H)
    for given in (None, into):
        h2, q = nv.add_norm(y, res, quantize=True, n=given, **how)
        want = nv.mx_quantize(n)
        assert torch.equal(h, h2) and (q.rows, q.K) == (rows, H)
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    w = nv.mx_quantize(randn(g, 40, H))
    assert torch.equal(nv.mx_gemm(q, w), nv.mx_linear(n, w))
    assert torch.equal(nv.rms_norm(y, how["pre_weight"], quantize=True).codes, nv.mx_quantize(nv.rms_norm(y, how["pre_weight"])).codes)


@pytest.mark.parametrize("dtype", list(DT))
def test_strides_places_and_leading_dimensions(dtype):
    dt = DT[dtype]
    for H in (72, 201, 1500):
        g = gen(H)
        y, res, how = make(g, 24, H, dt, dt, True, "element", True)
        h, n = nv.add_norm(y, res, **how)
        dh, dn = randn(g, 24, H, dtype=dt), randn(g, 24, H, dtype=dt)
        want = nv.add_norm_grad(dh, dn, y, h, **how)

        def wide(t):                                       # the gaps must not be read
            w = torch.full((24, H + 11), float("nan"), dtype=dt, device=DEV)
            w[:, 3:3 + H] = t
            return w[:, 3:3 + H]

        how2 = dict(how, gate=wide(how["gate"]))
        h2, n2 = nv.add_norm(wide(y), wide(res), **how2)
        assert torch.equal(h, h2) and torch.equal(n, n2)
        got = nv.add_norm_grad(wide(dh), wide(dn), wide(y), wide(h), **how2)
        lead = dict(how, gate=how["gate"].view(2, 3, 4, H))
        h3, n3 = nv.add_norm(y.view(2, 3, 4, H), res.view(2, 3, 4, H), **lead)
        assert torch.equal(h3.view(24, H), h) and torch.equal(n3.view(24, H), n)
        got3 = nv.add_norm_grad(*(t.view(2, 3, 4, H) for t in (dh, dn, y, h)), **lead)
        for name in ("y", "residual", "gate", "post_weight", "pre_weight"):
            assert torch.equal(getattr(got, name), getattr(want, name))
            assert torch.equal(getattr(got3, name).reshape(getattr(want, name).shape), getattr(want, name))
        # the residual stream updated in place, and y overwritten
        for place in (res.clone(), y.clone()):
            a, b = (y, place) if place.data_ptr() != y.data_ptr() and torch.equal(place, res) else (place, res)
            h4, n4 = nv.add_norm(a, b, h=place, **how)
            assert h4 is place and torch.equal(h4, h) and torch.equal(n4, n)
        # one row of the residual for all of them
        one = res[:1].expand(24, H)
        assert torch.equal(nv.add_norm(y, one, **how)[0], nv.add_norm(y, one.contiguous(), **how)[0])


def test_gradients_against_differences():
    """Central differences of the 64-bit formulas, along random directions."""
    rows, H = 6, 40
    g = gen(1)
    y, res, how = make(g, rows, H, torch.float32, torch.float32, True, "channel", True)
    dh, dn = randn(g, rows, H), randn(g, rows, H)
    h, _ = nv.add_norm(y, res, **how)
    gr = nv.add_norm_grad(dh, dn, y, h, **how)
    inputs = {"y": y, "residual": res, "gate": how["gate"], "post_weight": how["post_weight"], "pre_weight": how["pre_weight"]}

    def loss(**v):
        hh, _ = ref.norm_h(v["y"], v["residual"], True, v["post_weight"], v["gate"], how["scale"], how["residual_scale"], how["eps"])
        nn, _ = ref.norm_n(hh, v["pre_weight"], how["eps"])
        return (hh * dh.double()).sum() + (nn * dn.double()).sum()

    base = {k: v.double() for k, v in inputs.items()}
    for name in inputs:
        way = torch.randn(base[name].shape, device=DEV, generator=g, dtype=torch.float64)
        step = 1e-5
        up = loss(**dict(base, **{name: base[name] + step * way}))
        down = loss(**dict(base, **{name: base[name] - step * way}))
        slope = float((up - down) / (2 * step))
        got = float((getattr(gr, name).double() * way).sum())
        # (the difference's own error is step^2 times a third derivative, below 1e-7 of
        # the sum of magnitudes; the gradient's fp32 error below 1e-5 of it)
        size = float((getattr(gr, name).double() * way).abs().sum())
        assert abs(slope - got) <= 2e-5 * size, (name, slope, got)


def test_zero_rows_infinities_and_no_rows():
    for dt in DT.values():
        x = torch.zeros(5, 64, dtype=dt, device=DEV)
        x[1] = 1.0
        x[2, 3] = float("inf")
        x[3, 4] = float("nan")
        h, n = nv.add_norm(x, x, eps=1e-6)
        assert torch.equal(n[0], torch.zeros_like(n[0]))
        ref.check(n[1], *ref.norm_n(h[1].double()))        # (2 / sqrt(4 + 1e-6), not 1)
        assert n[2].isnan().sum() == 1 and n[2, 3].isnan() and (n[2][n[2].isfinite()] == 0).all()
        assert n[3].isnan().all() and torch.equal(n[4], n[0])
        _, q = nv.add_norm(x, x, quantize=True)
        want = nv.mx_quantize(n)
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
        # no rows: nothing but zero sums
        e = torch.empty(0, 64, dtype=dt, device=DEV)
        w = torch.ones(64, device=DEV)
        h, n = nv.add_norm(e, e, w, w, w)
        assert h.shape == n.shape == (0, 64)
        gr = nv.add_norm_grad(e, e, e, e, w, w, w)
        for t in (gr.gate, gr.post_weight, gr.pre_weight):
            assert torch.equal(t, torch.zeros(64, device=DEV))


def test_streams_graphs_and_sequences():
    g = gen(8)
    y, res, how = make(g, 40, 320, torch.bfloat16, torch.float32, True, "channel", True)
    dh, dn = randn(g, 40, 320, dtype=y.dtype), randn(g, 40, 320, dtype=y.dtype)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h, n = nv.add_norm(y, res, stream=s, **how)
    with torch.cuda.stream(s):
        gs = nv.add_norm_grad(dh, dn, y, h, **how)
    s.synchronize()
    h1, n1 = nv.add_norm(y, res, **how)
    g1 = nv.add_norm_grad(dh, dn, y, h1, **how)
    torch.cuda.synchronize()
    assert torch.equal(h, h1) and torch.equal(n, n1) and torch.equal(gs.post_weight, g1.post_weight)

    def step():
        h, n = nv.add_norm(y, res, **how)
        return h, n, nv.add_norm_grad(dh, dn, y, h, **how)

    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ch, cn, cg = step()
    with torch.cuda.graph(other):
        oh, on, og = step()
    seq = nv.Sequence()
    sh, sq = torch.empty_like(y), nv.mx_quantize(y)
    seq.add_norm(y, res, sh, sq, quantize=True, **how)
    seq.add_norm(y, None, None, n1, pre_weight=how["pre_weight"])
    seq.finalize()
    for seed in range(3):
        y.copy_(randn(gen(seed), 40, 320))
        dn.copy_(randn(gen(seed + 9), 40, 320))
        want = step()
        graph.replay()
        other.replay()
        seq.launch()
        torch.cuda.synchronize()
        for a, b, c in ((ch, cn, cg), (oh, on, og)):
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])
            for name in ("y", "residual", "gate", "post_weight", "pre_weight"):
                assert torch.equal(getattr(c, name), getattr(want[2], name))
        q = nv.mx_quantize(want[1])
        assert torch.equal(sh, want[0]) and torch.equal(sq.codes, q.codes) and torch.equal(sq.scales, q.scales)
        assert torch.equal(n1, nv.rms_norm(y, how["pre_weight"]))
    seq.close()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("H", [3, 64, 201, 2048, 2050, 4100, 6144, 9000, 16384])
def test_rows_up_to_the_largest_mean_of_squares(H, dtype):
    """Rows whose sum of squares passes fp32's range while its mean does not, side by side with others: the limit is the
    mean's, 2^128, from which on rows are zeros."""
    say(f"rows of {H} up to 2^64 {dtype}")
    g = gen(H)
    rows = 45
    size = torch.exp2(torch.randint(-20, 63, (rows, 1), device=DEV, generator=g).float())
    size[::3] = 2.0 ** 62.5
    size[5:8] = 1.0
    sign = lambda: torch.where(torch.rand(rows, H, device=DEV, generator=g) < 0.5, -1.0, 1.0)  # noqa: E731
    x = (size * sign() * (1 + 0.25 * torch.rand(rows, H, device=DEV, generator=g))).to(DT[dtype])    # (the mean stays below 2^126)
    wide = dict(scale=0.75, residual_scale=1.25, eps=1e-6)
    for post, pre in ((False, True), (True, False)):
        w = randn(g, H, scale=0.3, shift=1.0)
        how = dict(wide, post=post, post_weight=w if post else None, pre_weight=w if pre else None, gate=randn(g, H) if post else None)
        # the norm before the next block of large rows h, and the norm behind a block of large rows y
        y, res = (x, (sign() * 2.0 ** -3).to(x.dtype)) if post else ((sign() * 2.0 ** -3).to(x.dtype), (x * 0.5).to(x.dtype))
        h, n = nv.add_norm(y, res, pre=pre, **how)
        check_forward(y, res, how, pre, h, n, f"{H} {post}")
        # what the weights' gradients add of these rows
        dh, dn = randn(g, rows, H, dtype=x.dtype), None
        if pre:
            dh, dn = None, randn(g, rows, H, dtype=x.dtype)
        gr = nv.add_norm_grad(dh, dn, y, h, **how)
        want = ref.norm_grads(dbl(dh), dbl(dn), dbl(y), dbl(h), post, dbl(how["post_weight"]), dbl(how["gate"]), dbl(how["pre_weight"]),
                              0.75, 1.25, 1e-6, channel=True)
        for name in ("gate", "post_weight") if post else ("pre_weight",):
            ref.check(getattr(gr, name), *want[name], f"{H} d{name}")
    # and past it
    x[4], x[9] = 2.0 ** 64.5, -(2.0 ** 90)
    n = nv.rms_norm(x)
    assert (n[4] == 0).all() and (n[9] == 0).all()
    keep = [r for r in range(rows) if r not in (4, 9)]
    ref.check(n[keep], *ref.norm_n(x[keep].double(), None, 1e-6))
    # an eps beside which small squares count
    x = torch.ones(4, H, device=DEV, dtype=DT[dtype])
    x[0], x[1], x[2] = 2.0 ** -61, 2.0 ** 63 / H ** 0.5, 2.0 ** 60
    n = nv.rms_norm(x, eps=0.0)
    past = H > 256
    ref.check(n[[0, 1, 3] if past else [0, 1, 2, 3]], *ref.norm_n(x[[0, 1, 3] if past else [0, 1, 2, 3]].double(), None, 0.0))
    assert not past or (n[2] == 0).all()



@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("size,eps", [(1e-15, 0.0), (1e12, 1e-6), (1e15, 1e-6), (1e17, 0.0), (1e17, 1e-6)])
@pytest.mark.parametrize("H", [40, 96, 2048, 6001])
def test_gradients_of_rows_far_from_one(H, size, eps, dtype):
    """The part of a gradient along the row: of a size with the rest whatever the row's."""
    if H * (3 * size) ** 2 > 2.0 ** 128 and eps < 1e-30:
        pytest.skip("values of 3e17 are past the header's limit for such an eps, 2^64 / sqrt(6001) = 2.4e17")
    say(f"gradients of rows of {H}, {size} {dtype}")
    g = gen(H)
    for post, pre in ((False, True), (True, False), (True, True)):
        y, res, how = make(g, 9, H, DT[dtype], torch.float32, post, "channel", pre)
        y, res, how = (y * size).to(y.dtype), (res * size).to(y.dtype), dict(how, eps=eps)
        h, n = nv.add_norm(y, res, pre=pre, **how)
        check_forward(y, res, how, pre, h, n, f"{H} {size}")
        # gradients that point along the rows, beside what does not
        dh, dn = (randn(g, 9, H) + 2 * y.float() / size).to(y.dtype), None
        if pre:
            dh, dn = None, (randn(g, 9, H) + 2 * h.float() / h.float().square().mean(1, keepdim=True).sqrt()).to(y.dtype)
        check_grads(dh, dn, y, h, how, nv.add_norm_grad(dh, dn, y, h, **how), f"{H} {size} {post} {pre}")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("H", [3, 64, 201, 2048, 2050, 4100, 6144, 9000, 16384])
def test_gradients_up_to_the_largest_mean_of_squares(H, dtype):
    """Rows of 2^-20 to 2^62.5 side by side."""
    say(f"gradients of rows of {H} up to 2^64 {dtype}")
    g = gen(H + 1)
    rows = 45
    size = torch.exp2(torch.randint(-20, 63, (rows, 1), device=DEV, generator=g).float())
    size[::3] = 2.0 ** 62.5
    sign = lambda: torch.where(torch.rand(rows, H, device=DEV, generator=g) < 0.5, -1.0, 1.0)  # noqa: E731
    x = (size * sign() * (1 + 0.25 * torch.rand(rows, H, device=DEV, generator=g))).to(DT[dtype])
    w = randn(g, H, scale=0.3, shift=1.0)
    along = (randn(g, rows, H) + x.float() / size).to(x.dtype)
    for post, pre in ((False, True), (True, False)):
        how = dict(post=post, post_weight=w if post else None, pre_weight=w if pre else None, gate=randn(g, H) if post else None,
                   scale=0.75, residual_scale=1.25, eps=1e-6)
        y, h = (x, randn(g, rows, H, dtype=x.dtype)) if post else (randn(g, rows, H, dtype=x.dtype), x)
        dh, dn = (None, along) if pre else (along, None)
        check_grads(dh, dn, y, h, how, nv.add_norm_grad(dh, dn, y, h, **how), f"{H} {post}")


def test_a_gate_of_mode_none_is_not_read():
    """A description used again with NVFP4_GATE_NONE may still name the gate of another call."""
    import ctypes
    L = nv.layer.layer_lib()
    for dtype in DT.values():
        for post in (False, True):
            g = gen(5)
            y, res, how = make(g, 6, 200, dtype, torch.float32, post, "none", True)
            want_h, want_n = nv.add_norm(y, res, **how)
            left = randn(g, 200)
            spec = nv.layer._NormT(0 if dtype is torch.float32 else 1, 0, 6, 200, post, 1,
                                   how["post_weight"].data_ptr() if post else None, how["pre_weight"].data_ptr(), 0, left.data_ptr(),
                                   200, how["scale"], how["residual_scale"], how["eps"])
            h, n = torch.empty_like(y), torch.empty_like(y)
            args = (ctypes.byref(spec), y.data_ptr(), 200, res.data_ptr(), 200, h.data_ptr(), n.data_ptr(), None, None)
            assert L.nvfp4_add_norm(*args, torch.cuda.current_stream().cuda_stream) == nv.OK
            assert torch.equal(h, want_h) and torch.equal(n, want_n)


@pytest.mark.parametrize("H", [7, 640, 16384])
@pytest.mark.parametrize("eps", [0.0, 0.9e-30, 1e-30, 1e-29])
def test_small_rows_beside_a_small_eps(eps, H):
    """Squares that the scale makes subnormal do not count beside the eps that they are scaled for."""
    g = gen(H)
    x = randn(g, 40, H) * torch.exp2(torch.linspace(-58, -40, 40, device=DEV))[:, None]
    dn = randn(g, 40, H)
    n = nv.rms_norm(x, eps=eps)
    ref.check(n, *ref.norm_n(x.double(), None, eps), f"{H} {eps}")
    how = dict(post=False, post_weight=None, gate=None, pre_weight=torch.ones(H, device=DEV), scale=1.0, residual_scale=1.0, eps=eps)
    check_grads(None, dn, x, x, how, nv.add_norm_grad(None, dn, x, x, **how), f"{H} {eps}")
