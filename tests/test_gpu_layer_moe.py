"""A whole layer of experts on the GPU.

The rounding of h to four bits turns an error of fp32 sums into a step where a
value lies next to a border between codes, so the result cannot be held to a
bound by elements.  Two tests together hold it: with weights whose products are
exact in fp32 (small integers) nothing is near a border by accident, and the
result is compared with the definition in 64 bits; and with weights as they
come, with the definition under the bound that those few steps leave."""
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


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, device=DEV, generator=g)).to(dtype)


def values(q):
    return nv.mx_dequantize(q, torch.float32).double()


def held(x):
    """What MXFP4 holds for rows, float64 (mx_quantize and its inverse are tested byte for byte elsewhere)."""
    return values(nv.mx_quantize(x))


def choices(g, T, k, E, drop=0.2, again=0.2):
    ids = torch.randint(0, E, (T, k), device=DEV, generator=g)
    if k > 1:                                                     # the same expert twice
        twice = torch.rand(T, device=DEV, generator=g) < again
        ids[twice, 1] = ids[twice, 0]
    gone = torch.rand(T, k, device=DEV, generator=g)
    ids = torch.where(gone < drop / 2, -1, torch.where(gone < drop, E + 3, ids))
    return ids


def expected(x, ids, p, up, down, act, gate=None, up_bias=None, gate_bias=None, down_bias=None):
    """The definition: (result, sum of the magnitudes of its terms)."""
    E = up.groups
    dbl = lambda t: None if t is None else t.double()  # noqa: E731
    vu, vd, vg = values(up), values(down), None if gate is None else values(gate)
    vx = held(x)
    out = torch.zeros(x.shape[0], x.shape[1], dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(out)
    for e in range(E):
        at = torch.nonzero(ids == e)
        if not len(at):
            continue
        t, j = at[:, 0], at[:, 1]
        z = vx[t] @ vu[e].T
        if up_bias is not None:
            z = z + dbl(up_bias[e])
        if gate is not None:
            v = vx[t] @ vg[e].T
            if gate_bias is not None:
                v = v + dbl(gate_bias[e])
            h = ref.act(act, v) * z
        else:
            h = ref.act(act, z)
        vh = held(h.to(torch.bfloat16))
        y = vh @ vd[e].T
        m = vh.abs() @ vd[e].abs().T
        if down_bias is not None:
            y, m = y + dbl(down_bias[e]), m + dbl(down_bias[e]).abs()
        w = torch.ones(len(at), 1, dtype=torch.float64, device=DEV) if p is None else p[t, j].double()[:, None]
        out.index_add_(0, t, w * y)
        mag.index_add_(0, t, (w * m).abs())
    return out, mag


def experts(g, E, F, H, gate, bias, exact, dtype=torch.float32):
    """Weights (small integers where products are to be exact) and biases."""
    def w(*shape):
        if exact:                                                 # codes 0, +-0.5, +-1 under scale 1: exact in MXFP4
            return nv.mx_quantize(torch.randint(-1, 2, shape, device=DEV, generator=g).float() * 4)
        return nv.mx_quantize(randn(g, *shape, scale=0.06))

    b = (lambda *s: torch.randint(-3, 4, s, device=DEV, generator=g).to(dtype)) if exact else (lambda *s: randn(g, *s, dtype=dtype))  # noqa: E731
    more = {}
    if gate:
        more["gate"] = w(E, F, H)
    if bias:
        more.update(up_bias=b(E, F), down_bias=b(E, H))
        if gate:
            more["gate_bias"] = b(E, F)
    return w(E, F, H), w(E, H, F), more


# tokens, topk, experts, inner, hidden: few tokens (two launches), then more, or rows too long for that
SIZES = [(1, 8, 256, 256, 6144), (1, 1, 1, 32, 32), (3, 2, 5, 96, 160), (4, 8, 64, 256, 544), (2, 128, 300, 64, 96),
         (3, 4, 8, 1056, 2080), (4, 1, 2, 2048, 32), (1, 100, 7, 64, 64), (2, 3, 4, 96, 30016), (16, 8, 64, 256, 544), (17, 4, 8, 160, 2080),
         (33, 3, 2, 64, 4192), (64, 8, 16, 512, 256), (64, 1, 3, 2048, 96), (5, 100, 7, 64, 64), (64, 8, 300, 32, 1024),
         (65, 2, 4, 96, 160), (20, 30, 9, 64, 96), (130, 8, 32, 288, 544),
         # choices sorted beside the quantisation and not, short products of up to 16 rows an expert
         (128, 2, 16, 352, 128), (257, 1, 20, 416, 160), (20, 12, 15, 480, 96), (20, 12, 14, 512, 96),
         # h packed by the products of 64 x 256, 128 x 128 and 128 x 256 tiles, with broken steps behind the last block
         (100, 8, 256, 288, 256), (90, 9, 200, 160, 64), (100, 8, 640, 32, 64), (100, 8, 700, 64, 96), (4096, 8, 16, 160, 64),
         (2500, 4, 9, 544, 96)]


@pytest.mark.parametrize("T,k,E,F,H", SIZES)
@pytest.mark.parametrize("gate,act", [(True, "relu"), (False, "none")])
def test_exact_sums(T, k, E, F, H, gate, act):
    """Integer activations and weights: every sum is exact in fp32, so only the roundings of the definition happen."""
    for bias, idt, xdt, odt in ((False, torch.int32, "bf16", "fp32"), (True, torch.int64, "fp32", "bf16")):
        say(f"moe exact {T}x{k} of {E}, {F} x {H} gate={gate} bias={bias}")
        g = gen(T * 100 + F)
        up, down, more = experts(g, E, F, H, gate, bias, True)
        ids = choices(g, T, k, E)
        x = torch.randint(-2, 3, (T, H), device=DEV, generator=g).to(DT[xdt])
        p = torch.randint(1, 5, (T, k), device=DEV, generator=g).float() / 4
        out = nv.mx_moe(x, ids.to(idt), p, up, down, activation=act, dtype=DT[odt], **more)
        want, mag = expected(x, ids, p, up, down, act, **more)
        # (sums of h's values, which have up to 2^24 times their smallest step, round: a bound as of any
        # product)
        ref.check(out, want, (F / 64 + 20 + k) * 4 * ref.U * mag, f"{T} {E}")


@pytest.mark.parametrize("T,k,E,F,H", SIZES)
@pytest.mark.parametrize("act", list(nv.ACTIVATIONS))
def test_random(T, k, E, F, H, act):
    """Errors of the sums of up to 2^-19 of h's size move one value in 2^-16 over a border between codes, by up to a
    third of itself, which over a row of F >= 32 products is sqrt(2^-16) / 3 = 2^-9.6 of the result; its rounding is 2^-9.
    A token of few values may hold one of those steps: elements stay within a tenth of the terms' magnitudes."""
    for gate in (True, False):
        say(f"moe random {T}x{k} of {E}, {F} x {H} {act} gate={gate}")
        g = gen(T + F + len(act))
        up, down, more = experts(g, E, F, H, gate, True, False, torch.bfloat16)
        ids = choices(g, T, k, E)
        x, p = randn(g, T, H, dtype=torch.bfloat16), torch.rand(T, k, device=DEV, generator=g)
        out = nv.mx_moe(x, ids, p, up, down, activation=act, **more).double()
        want, mag = expected(x, ids, p, up, down, act, **more)
        assert float((out - want).norm()) <= 2.0 ** -7 * float(want.norm()) + 1e-30
        assert ((out - want).abs() <= 0.1 * mag + 2.0 ** -8 * want.abs()).all()
        none = ((ids < 0) | (ids >= E)).all(1)
        assert (out[none] == 0).all()


def test_both_forms_agree():
    """Four tokens in two launches and the same tokens among 65 by the general form: the same h, so the results differ by
    fp32 sums only, but for steps of h as above."""
    g = gen(3)
    up, down, more = experts(g, 16, 256, 512, True, True, True)
    x = torch.randint(-2, 3, (65, 512), device=DEV, generator=g).to(torch.bfloat16)
    ids, p = choices(g, 65, 4, 16), torch.rand(65, 4, device=DEV, generator=g)
    a = nv.mx_moe(x[:4], ids[:4].contiguous(), p[:4].contiguous(), up, down, activation="relu", dtype=torch.float32, **more)
    b = nv.mx_moe(x, ids, p, up, down, activation="relu", dtype=torch.float32, **more)
    _, mag = expected(x, ids, p, up, down, "relu", **more)
    ref.check(a, b[:4], (256 / 64 + 24) * 8 * ref.U * mag[:4])


def test_nothing_kept_strides_and_no_weights():
    g = gen(5)
    up, down, more = experts(g, 6, 64, 96, True, True, False)
    for T in (1, 4, 20, 100):
        x = randn(g, T, 96, dtype=torch.bfloat16)
        none = torch.full((T, 3), -1, device=DEV, dtype=torch.int32)
        out = torch.full((T, 96), float("nan"), dtype=torch.bfloat16, device=DEV)
        assert nv.mx_moe(x, none, None, up, down, out=out, **more) is out and (out == 0).all()
        ids = choices(g, T, 3, 6)
        wide = torch.full((T, 120), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, 8:104] = x
        want = nv.mx_moe(x, ids, None, up, down, **more)
        assert torch.equal(nv.mx_moe(wide[:, 8:104], ids, torch.ones(T, 3, device=DEV), up, down, **more), want)
        p = torch.rand(T, 3, device=DEV, generator=g)
        dirty = torch.where((ids < 0) | (ids >= 6), float("nan"), p)   # weights of dropped choices are ignored
        assert torch.equal(nv.mx_moe(x, ids, dirty, up, down, **more), nv.mx_moe(x, ids, p, up, down, **more))
    assert nv.mx_moe(x[:0], ids[:0], None, up, down, **more).shape == (0, 96)


def test_nan_rows_stay_their_own():
    g = gen(6)
    up, down, more = experts(g, 4, 64, 96, True, False, False)
    for T in (4, 90):
        x, ids = randn(g, T, 96), torch.randint(0, 4, (T, 2), device=DEV, generator=g)
        want = nv.mx_moe(x, ids, None, up, down, **more)
        x[1, 40] = float("nan")
        x[3, 0] = float("inf")
        got = nv.mx_moe(x, ids, None, up, down, **more)
        assert got[1].isnan().all() and got[3].isnan().all()
        rest = [t for t in range(T) if t not in (1, 3)]
        assert torch.equal(got[rest], want[rest])


def test_streams_graphs_and_sequences():
    g = gen(7)
    up, down, more = experts(g, 12, 128, 256, True, True, False)
    for T in (3, 80):
        x, p = randn(g, T, 256, dtype=torch.bfloat16), torch.rand(T, 2, device=DEV, generator=g)
        ids = choices(g, T, 2, 12).to(torch.int32)
        want = nv.mx_moe(x, ids, p, up, down, **more)
        streams = [torch.cuda.Stream() for _ in range(3)]
        torch.cuda.synchronize()
        got = [nv.mx_moe(x, ids, p, up, down, stream=s, **more) for s in streams for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in got)
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        outs = []
        for gr in graphs:
            with torch.cuda.graph(gr):
                outs.append(nv.mx_moe(x, ids, p, up, down, **more))
        seq, so = nv.Sequence(), torch.empty_like(want)
        seq.add_mx_moe(x, ids, p, up, down, so, **more)
        seq.finalize()
        for seed in range(3):
            x.copy_(randn(gen(seed), T, 256))
            ids.copy_(choices(gen(seed), T, 2, 12))
            want = nv.mx_moe(x, ids, p, up, down, **more)
            for s, gr in zip(streams, graphs):                         # at the same time, on two streams
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s):
                    gr.replay()
            seq.launch()
            torch.cuda.synchronize()
            assert all(torch.equal(o, want) for o in (*outs, so))
        seq.close()


@pytest.mark.parametrize("T", [4, 100])
def test_a_whole_layer(T):
    """The operators together, as a layer runs them: norm into a packed operand and gated feed-forward, its result
    normed and added, then the experts, their result gated and added; recorded and eager; held against the same steps
    from plain calls."""
    g = gen(T)
    H, F, E, k = 256, 192, 8, 2
    x = randn(g, T, H, dtype=torch.bfloat16)
    w = [1 + 0.1 * randn(g, H) for _ in range(4)]
    wg, wu, wd = (nv.mx_quantize(randn(g, *s, scale=0.08)) for s in ((F, H), (F, H), (H, F)))
    up, down, more = experts(g, E, F, H, True, True, False)
    ids, p = choices(g, T, k, E).to(torch.int32), torch.rand(T, k, device=DEV, generator=g)
    layer_scale = 0.5 * randn(g, H)
    q = nv.rms_norm(x, w[0], quantize=True)
    f = nv.mx_gemm(q, wu, epilogue=nv.MxEpilogue("silu", gate=wg))
    y = nv.mx_linear(f, wd)
    h1, n1 = nv.add_norm(y, x, post_weight=w[1], pre_weight=w[2])
    m = nv.mx_moe(n1, ids, p, up, down, **more)
    h2, n2 = nv.add_norm(m, h1, post_weight=w[3], gate=layer_scale, pre_weight=w[0])
    # the same from plain steps
    n0, _ = ref.norm_n(x.double(), w[0].double())
    assert torch.equal(q.codes, nv.mx_quantize(nv.rms_norm(x, w[0])).codes)
    v, z = nv.mx_gemm(q, wg, dtype=torch.float32), nv.mx_gemm(q, wu, dtype=torch.float32)
    fr = (ref.act("silu", v.double()) * z.double())
    ref.check(f, fr, 2.0 ** -18 * fr.abs())
    hr, b = ref.norm_h(y.double(), x.double(), True, w[1].double(), eps=1e-6)
    ref.check(h1, hr, b)
    want, _ = expected(n1, ids, p, up, down, "silu", **more)
    assert float((m.double() - want).norm()) <= 2.0 ** -7 * float(want.norm())
    hr, b = ref.norm_h(m.double(), h1.double(), True, w[3].double(), layer_scale.double(), eps=1e-6)
    ref.check(h2, hr, b)
    ref.check(n2, *ref.norm_n(h2.double(), w[0].double()))
    assert n0.shape == n2.shape and n2.isfinite().all()
    # recorded
    seq = nv.Sequence()
    sf, sy, sh1, sn1, sm, sh2, sn2 = (torch.zeros_like(t) for t in (f, y, h1, n1, m, h2, n2))
    sq, sq2 = nv.mx_quantize(torch.zeros_like(x)), nv.mx_quantize(torch.zeros_like(f))
    seq.add_norm(x, None, None, sq, pre_weight=w[0], quantize=True)
    seq.add_mx_gemm(sq, wu, sf, epilogue=nv.MxEpilogue("silu", gate=wg))
    seq.add_mx_quantize(sf, sq2)
    seq.add_mx_gemm(sq2, wd, sy)
    seq.add_norm(sy, x, sh1, sn1, post_weight=w[1], pre_weight=w[2])
    seq.add_mx_moe(sn1, ids, p, up, down, sm, **more)
    seq.add_norm(sm, sh1, sh2, sn2, post_weight=w[3], gate=layer_scale, pre_weight=w[0])
    seq.finalize()
    for _ in range(3):
        seq.launch()
        torch.cuda.synchronize()
        for a, b in ((sf, f), (sy, y), (sh1, h1), (sn1, n1), (sm, m), (sh2, h2), (sn2, n2)):
            assert torch.equal(a, b)
    seq.close()


@pytest.mark.parametrize("T,k,E,F,H", SIZES)
@pytest.mark.parametrize("gated", [True, False])
def test_whatever_the_workspace_holds(T, k, E, F, H, gated):
    """The same bits from a workspace full of NaN scales (0xFF) as from one of zeros: all that counts is written."""
    say(f"moe workspace {T}x{k} of {E}, {F} x {H}")
    g = gen(T + E)
    up, down, more = experts(g, E, F, H, gated, True, False)
    x, ids = randn(g, T, H, dtype=torch.bfloat16), choices(g, T, k, E)
    outs = []
    for fill in (0, 255):
        out, args, tensors = nv.layer._moe_args(x, ids, None, up, down, more.get("gate"), "silu", more["up_bias"],
                                                more.get("gate_bias"), more["down_bias"], None, None)
        work = tensors[4]
        assert work.dtype == torch.uint8 and args[-2:] == (work.data_ptr(), work.numel())
        work.fill_(fill)
        nv.mx._run(nv.layer.layer_lib().nvfp4_mx_moe, args, tensors)
        outs.append(out)
    assert outs[0].isfinite().all() and torch.equal(*outs)
