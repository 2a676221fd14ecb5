"""What is measured of the operators that stand around the MXFP4 products of a transformer layer.

  linear   activations, quantised on the way, times a weight held in MXFP4, with bias, activation, gate and
           residual in the product's epilogue:
             out = act(q(x) . Wg^T + bg) * (q(x) . W^T + b) + residual, or without a gate act(q(x) . W^T + b) + residual
  moe      a whole layer of experts for few tokens:
             out[t] = sum_j p[t, j] * (q(h[t, j]) . Wd_e^T + bd_e), e = ids[t, j],
             h[t, j] = act(q(x[t]) . Wg_e^T + bg_e) * (q(x[t]) . Wu_e^T + bu_e), held in bfloat16
  norm     the norms behind one block and before the next, with the block's gate and the residual between them:
             u = y / rms(y) * w_post, h = residual_scale * residual + scale * gate * u, n = h / rms(h) * w_pre
  norm_grad  the gradients of the same

q() is MXFP4 (OCP Microscaling Formats v1.0): 32 consecutive values of a row as E2M1 codes with one power-of-two
scale byte (E8M0).  `run` computes the operators in their plain form or, where `own` is true, through the package.
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token through the gated first half of a feed-forward block, an eighth of its columns: latency
        {"name": "gate_decode", "op": "linear", "M": 1, "N": 768, "K": 6144, "dtype": "bf16", "act": "silu", "gate": True, "bias": False, "residual": False},
        # 512 requests through the second half, added to the residual stream
        {"name": "down_batch", "op": "linear", "M": 512, "N": 6144, "K": 2048, "dtype": "bf16", "act": "none", "gate": False, "bias": True, "residual": True},
        # a ragged prefill in fp32 with every part of the epilogue: no size a multiple of a tile
        {"name": "gelu_ragged_fp32", "op": "linear", "M": 1237, "N": 2056, "K": 6112, "dtype": "fp32", "act": "gelu", "gate": False, "bias": True, "residual": True},
        # a long prefill through the gated first half: compute
        {"name": "gate_prefill", "op": "linear", "M": 16384, "N": 4096, "K": 8192, "dtype": "bf16", "act": "silu", "gate": True, "bias": False, "residual": False},
        # one request decoding, top 8 of 256 experts, an eighth of each expert's columns: latency
        {"name": "moe_token", "op": "moe", "tokens": 1, "topk": 8, "experts": 256, "inner": 256, "hidden": 6144, "dtype": "bf16", "act": "silu", "gate": True, "bias": False, "drop": 0.0},
        # sixteen requests: most choices have an expert of their own
        {"name": "moe_decode", "op": "moe", "tokens": 16, "topk": 8, "experts": 256, "inner": 256, "hidden": 6144, "dtype": "bf16", "act": "silu", "gate": True, "bias": False, "drop": 0.0},
        # sixty-one requests by few wide experts with biases, some choices on another GPU
        {"name": "moe_wide_bias", "op": "moe", "tokens": 61, "topk": 4, "experts": 32, "inner": 1024, "hidden": 2048, "dtype": "bf16", "act": "gelu_tanh", "gate": True, "bias": True, "drop": 0.25},
        # one decode step's residual and norm, 16 requests: latency
        {"name": "norm_decode", "op": "norm", "rows": 16, "cols": 6144, "dtype": "bf16", "post": False, "gate": "none", "pre": True, "residual": True},
        # a long prefill with the norms on both sides of the residual and a gate from the activations: bandwidth
        {"name": "norm_prefill", "op": "norm", "rows": 16384, "cols": 6144, "dtype": "bf16", "post": True, "gate": "element", "pre": True, "residual": True},
        # odd rows in fp32 with a learned gate for each channel
        {"name": "norm_odd_fp32", "op": "norm", "rows": 4099, "cols": 2047, "dtype": "fp32", "post": True, "gate": "channel", "pre": True, "residual": True},
        # a training step's backward pass, weights and gates learned
        {"name": "norm_train", "op": "norm_grad", "rows": 8192, "cols": 2048, "dtype": "bf16", "post": True, "gate": "channel", "pre": True, "residual": True},
        # the same in fp32 with odd rows, a gate from the activations, no norm behind the block
        {"name": "norm_train_odd_fp32", "op": "norm_grad", "rows": 2053, "cols": 5003, "dtype": "fp32", "post": False, "gate": "element", "pre": True, "residual": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def draw(rng):
    op = rng.choice(("linear", "linear", "moe", "moe", "norm", "norm_grad"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    while True:
        if op == "linear":
            c = {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 16, 8192), "K": BLOCK * _log(rng, 4, 256), "dtype": dtype,
                 "act": rng.choice(ACTS), "gate": rng.random() < 0.5, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
            if c["M"] * c["N"] * c["K"] * (2 if c["gate"] else 1) > 2 * 16384 * 4096 * 8192:
                continue
        elif op == "moe":
            experts = _log(rng, 2, 256)
            c = {"op": op, "tokens": _log(rng, 1, 512), "topk": rng.randint(1, min(8, experts)), "experts": experts, "inner": BLOCK * _log(rng, 2, 64),
                 "hidden": BLOCK * _log(rng, 8, 192), "dtype": dtype, "act": rng.choice(ACTS), "gate": rng.random() < 0.7, "bias": rng.random() < 0.5,
                 "drop": rng.choice((0.0, 0.25))}
            if experts * c["inner"] * c["hidden"] > 256 * 256 * 6144:
                continue
        else:
            c = {"op": op, "rows": _log(rng, 1, 16384), "cols": _log(rng, 32, 8192), "dtype": dtype, "post": rng.random() < 0.5,
                 "gate": rng.choice(("none", "channel", "element")), "pre": rng.random() < 0.8, "residual": rng.random() < 0.8}
            if c["rows"] * c["cols"] * (2 if dtype == "fp32" else 1) > 16384 * 6144 or not (c["post"] or c["gate"] != "none" or c["pre"]):
                continue
        return c


def work(case):
    c, size = case, 4 if case["dtype"] == "fp32" else 2
    if c["op"] == "linear":
        M, N, K, n = c["M"], c["N"], c["K"], 2 if c["gate"] else 1
        return {"bytes": size * M * K + n * N * K * 17 / 32 + size * M * N * (2 if c["residual"] else 1) + 4 * N * n * c["bias"], "flops": 2 * n * M * N * K}
    if c["op"] == "moe":
        pairs, n = c["tokens"] * c["topk"] * (1 - c["drop"]), 3 if c["gate"] else 2
        used = min(c["experts"], pairs)
        return {"bytes": used * n * c["inner"] * c["hidden"] * 17 / 32 + (size + 2) * c["tokens"] * c["hidden"] + 8 * pairs, "flops": 2 * pairs * n * c["inner"] * c["hidden"]}
    row = size * c["rows"] * c["cols"]
    streams = 2 + c["residual"] + (c["gate"] == "element") + c["pre"]   # y and h; residual, gate, n
    if c["op"] == "norm_grad":                                          # dh and dy; y, h, gate; dn; dresidual, dgate
        streams = 2 + (c["post"] or c["gate"] != "none") + 2 * c["pre"] + c["residual"] + 2 * (c["gate"] == "element")
    return {"bytes": streams * row, "flops": c["rows"] * c["cols"] * (12 if c["op"] == "norm" else 30)}


# ---- inputs ---------------------------------------------------------------------------------


def _activations(g, rows, cols, dtype):
    """Rows of a unit normal with one channel in a hundred twenty times as large, as the residual stream has them."""
    loud = 1 + 19 * (torch.rand(cols, device="cuda", generator=g) < 0.01).float()
    x = torch.empty(rows, cols, dtype=TYPES[dtype], device="cuda")
    for r in range(0, rows, 4096):
        x[r:r + 4096] = torch.randn(min(4096, rows - r), cols, device="cuda", generator=g) * loud
    return x


def _normal(g, shape, dtype, scale=1.0, shift=0.0):
    return (shift + scale * torch.randn(shape, device="cuda", generator=g)).to(dtype)


def _weights(g, shape):
    w = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for e in range(shape[0]):
        w[e] = 0.02 * torch.randn(shape[1:], device="cuda", generator=g)
    return w


def _inputs(case, seed):
    """The inputs of a case by name, the same for every form."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 29)
    c, s, dt = case, {}, TYPES[case["dtype"]]
    if c["op"] == "linear":
        s["x"] = _activations(g, c["M"], c["K"], c["dtype"])
        s["w"] = _normal(g, (c["N"], c["K"]), torch.bfloat16, 0.02)
        s["wg"] = _normal(g, (c["N"], c["K"]), torch.bfloat16, 0.02) if c["gate"] else None
        s["b"] = _normal(g, (c["N"],), torch.float32, 0.5) if c["bias"] else None
        s["bg"] = _normal(g, (c["N"],), torch.float32, 0.5) if c["bias"] and c["gate"] else None
        s["residual"] = _normal(g, (c["M"], c["N"]), dt) if c["residual"] else None
    elif c["op"] == "moe":
        E, F, H = c["experts"], c["inner"], c["hidden"]
        popular = 0.5 * torch.randn(E, device="cuda", generator=g)
        logits, ids = (torch.randn(c["tokens"], E, device="cuda", generator=g) + popular).topk(c["topk"], dim=1)
        gone = torch.rand(ids.shape, device="cuda", generator=g) < c["drop"]
        s["ids"] = torch.where(gone, -1, ids).to(torch.int32).contiguous()
        s["p"] = torch.softmax(logits, dim=1).contiguous()
        s["x"] = _activations(g, c["tokens"], H, c["dtype"])
        s["wg"] = _weights(g, (E, F, H)) if c["gate"] else None
        s["wu"] = _weights(g, (E, F, H))
        s["wd"] = _weights(g, (E, H, F))
        s["bg"] = _normal(g, (E, F), torch.float32, 0.5) if c["bias"] and c["gate"] else None
        s["bu"] = _normal(g, (E, F), torch.float32, 0.5) if c["bias"] else None
        s["bd"] = _normal(g, (E, H), torch.float32, 0.5) if c["bias"] else None
    else:
        R, C = c["rows"], c["cols"]
        s["y"] = _normal(g, (R, C), dt)
        s["residual"] = _activations(g, R, C, c["dtype"]) if c["residual"] else None
        s["w_post"] = _normal(g, (C,), dt, 0.2, 1.0) if c["post"] else None
        s["w_pre"] = _normal(g, (C,), dt, 0.2, 1.0) if c["pre"] else None
        s["gate"] = None if c["gate"] == "none" else torch.sigmoid(_normal(g, (C,) if c["gate"] == "channel" else (R, C), dt))
        # (a branch scaled for a deep stack)
        s["scale"], s["residual_scale"] = 0.5, 1.0
        if c["op"] == "norm_grad":
            # what the forward pass left, and the gradients that come back
            h = _forward(s, torch.float32)[0].to(dt)
            s["h"] = h
            s["dh"] = _normal(g, (R, C), dt)
            s["dn"] = _normal(g, (R, C), dt) if c["pre"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import block_scaled_fp4_04_amd as nv
        s["nv"] = nv
    # the weights as their program keeps them: packed, or as the values that their codes stand for
    for name in ("w", "wg", "wu", "wd"):
        if s.get(name) is not None:
            s[name] = s["nv"].mx_quantize(s[name]) if own else _rounded(s[name])
    if case["op"] == "moe" and not own:
        # rows that the largest expert has, as a program that pads its experts keeps it
        s["most"] = max(1, int(torch.bincount(s["ids"].flatten().long() + 1, minlength=2)[1:].max()))
    return s


# ---- the operators --------------------------------------------------------------------------


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        nv = s["nv"]
        if op == "linear":
            e = nv.MxEpilogue(activation=c["act"], bias=s["b"], gate=s["wg"], gate_bias=s["bg"], residual=s["residual"])
            return nv.mx_linear(s["x"], s["w"], dtype=s["x"].dtype, epilogue=e)
        if op == "moe":
            return nv.mx_moe(s["x"], s["ids"], s["p"], s["wu"], s["wd"], gate=s["wg"], activation=c["act"], up_bias=s["bu"], gate_bias=s["bg"], down_bias=s["bd"])
        how = dict(post_weight=s["w_post"], gate=s["gate"], pre_weight=s["w_pre"], scale=s["scale"], residual_scale=s["residual_scale"], eps=EPS)
        if op == "norm":
            h, n = nv.add_norm(s["y"], s["residual"], pre=c["pre"], post=c["post"], **how)
            return {"h": h, "n": n}
        d = nv.add_norm_grad(s["dh"], s["dn"], s["y"], s["h"], pre=c["pre"], post=c["post"], residual=c["residual"], **how)
        return {"dy": d.y, "dresidual": d.residual, "dgate": d.gate, "dw_post": d.post_weight, "dw_pre": d.pre_weight}
    if op == "linear":
        x = _rounded(s["x"])
        z = x @ s["w"].t()
        if c["bias"]:
            z = z + s["b"]
        if c["gate"]:
            v = x @ s["wg"].t()
            if c["bias"]:
                v = v + s["bg"]
            z = _act(v, c["act"]) * z
        else:
            z = _act(z, c["act"])
        if c["residual"]:
            z = z + s["residual"].float()
        return z.to(s["x"].dtype)
    if op == "moe":
        return _experts(s, c)
    if op == "norm":
        h, n = _forward(s, s["y"].dtype)
        return {"h": h, "n": n}
    return _backward(s)


def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _rounded(x):
    """The values, in 32 bits, that MXFP4 holds for x: in each 32 values of a row the scale is
    2^(floor(log2(largest magnitude)) - 2), from 2^-127 on, and each value over the scale is rounded to
    the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), at most 6."""
    v = x.float().reshape(*x.shape[:-1], -1, BLOCK)
    top = v.abs().amax(-1, keepdim=True)
    byte = ((top.view(torch.int32) >> 23) - 2).clamp(min=0)
    y = v * ((254 - byte) << 23).view(torch.float32)
    size = y.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    q = (torch.round(y / step) * step).clamp(-6, 6)
    scale = torch.where(byte > 0, byte << 23, 1 << 22).view(torch.float32)
    return (q * scale).reshape(x.shape)


def _experts(s, c):
    ids, E, T, k = s["ids"].long(), c["experts"], c["tokens"], c["topk"]
    flat, x = ids.reshape(-1), _rounded(s["x"])
    kept = (flat >= 0)[:, None]
    if flat.numel() <= E:
        # few choices: each multiplies by a copy of its expert's weights
        e = flat.clamp(min=0)
        a = x.repeat_interleave(k, 0)[:, :, None]

        def by(w, v, b):
            z = torch.bmm(w[e], v)[:, :, 0]
            return z if b is None else z + b[e]

        z = by(s["wu"], a, s["bu"])
        z = _act(by(s["wg"], a, s["bg"]), c["act"]) * z if c["gate"] else _act(z, c["act"])
        h = _rounded(z.to(torch.bfloat16))
        y = by(s["wd"], h[:, :, None], s["bd"])
    else:
        # rows sorted by expert and padded to the largest one's, and batched products
        key = torch.where(flat >= 0, flat, E)
        order = torch.argsort(key, stable=True)
        off = torch.searchsorted(key[order], torch.arange(E + 1, device="cuda"))
        at = off[:-1, None] + torch.arange(s["most"], device="cuda")
        pad = (at >= off[1:, None])[:, :, None]
        a = torch.where(pad, 0.0, x[order[at.clamp(max=flat.numel() - 1)] // k])

        def by(w, v, b):
            z = torch.bmm(v, w.transpose(1, 2))
            return z if b is None else z + b[:, None, :]

        z = by(s["wu"], a, s["bu"])
        z = _act(by(s["wg"], a, s["bg"]), c["act"]) * z if c["gate"] else _act(z, c["act"])
        y = by(s["wd"], _rounded(z.to(torch.bfloat16)), s["bd"])
        place = torch.empty_like(order)
        place[order] = torch.arange(order.numel(), device="cuda")
        e = flat.clamp(min=0)
        y = y[e, (place - off[e]).clamp(0, s["most"] - 1)]
    y = torch.where(kept, y, 0.0).reshape(T, k, -1)
    return (y * s["p"][:, :, None]).sum(1).to(torch.bfloat16)


def _forward(s, kept):
    """(h, n), h rounded to the type `kept` before it is normed."""
    u = s["y"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = s["scale"] * u
    if s["residual"] is not None:
        h = s["residual_scale"] * s["residual"].float() + h
    h = h.to(kept)
    if s["w_pre"] is None:
        return h, None
    v = h.float()
    return h, (v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["w_pre"].float()).to(kept)


def _norm_back(d, x, w):
    """The gradients of x / rms(x) * w by x and by w, for the result's gradient d."""
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    g = d * w
    return r * g - x * r * r * r * (g * x).mean(1, keepdim=True), (d * x * r).sum(0)


def _backward(s):
    c, dt = s["case"], s["y"].dtype
    out = {"dy": None, "dresidual": None, "dgate": None, "dw_post": None, "dw_pre": None}
    d, y = s["dh"].float(), s["y"].float()
    if c["pre"]:
        dx, out["dw_pre"] = _norm_back(s["dn"].float(), s["h"].float(), s["w_pre"].float())
        d = d + dx
    if c["residual"]:
        out["dresidual"] = (s["residual_scale"] * d).to(dt)
    d = s["scale"] * d
    if s["gate"] is not None:
        u = y
        if c["post"]:
            u = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["w_post"].float()
        out["dgate"] = (d * u).sum(0) if c["gate"] == "channel" else (d * u).to(dt)
        d = d * s["gate"].float()
    if c["post"]:
        d, out["dw_post"] = _norm_back(d, y, s["w_post"].float())
    out["dy"] = d.to(dt)
    return out


# ---- the definition in 64 bits ----------------------------------------------------------------

EDGES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _held(x):
    """What MXFP4 holds for x: a value's code counts the borders that its magnitude passes; one on a border goes
    to the even code."""
    v = x.double().reshape(-1, BLOCK)
    top = v.abs().max(1).values
    e = torch.where(top > 0, torch.frexp(top).exponent - 1, -1000) - 2
    scale = torch.exp2(e.clamp(min=-127).double())[:, None]
    m, code = v.abs() / scale, torch.zeros(v.shape, dtype=torch.long, device=x.device)
    for k, edge in enumerate(EDGES):
        code += (m >= edge) if k % 2 else (m > edge)
    grid = torch.tensor(CODES, dtype=torch.float64, device=x.device)
    return (grid[code] * torch.sign(v) * scale).reshape(x.shape)


def _activate(name, z):
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * 0.5 * torch.erfc(-z / math.sqrt(2)),
            "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))}[name]()


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "linear":
        w = _held(s["w"]).t().contiguous()
        wg = _held(s["wg"]).t().contiguous() if c["gate"] else None
        parts = []
        for r in range(0, c["M"], 4096):
            x = _held(s["x"][r:r + 4096])
            z = x @ w + (s["b"].double() if c["bias"] else 0.0)
            if c["gate"]:
                z = z * _activate(c["act"], x @ wg + (s["bg"].double() if c["bias"] else 0.0))
            else:
                z = _activate(c["act"], z)
            parts.append(z + s["residual"][r:r + 4096].double() if c["residual"] else z)
        return torch.cat(parts)
    if c["op"] == "moe":
        ids, x = s["ids"].cpu(), _held(s["x"])
        out = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            t, j = [v.to("cuda") for v in torch.nonzero(ids == e, as_tuple=True)]
            if not t.numel():
                continue
            z = x[t] @ _held(s["wu"][e]).t() + (s["bu"][e].double() if c["bias"] else 0.0)
            if c["gate"]:
                z = z * _activate(c["act"], x[t] @ _held(s["wg"][e]).t() + (s["bg"][e].double() if c["bias"] else 0.0))
            else:
                z = _activate(c["act"], z)
            y = _held(z.to(torch.bfloat16)) @ _held(s["wd"][e]).t() + (s["bd"][e].double() if c["bias"] else 0.0)
            out.index_add_(0, t, y * s["p"][t, j].double()[:, None])
        return out
    y = s["y"].double()
    rms = lambda v: (v.square().sum(1, keepdim=True) / v.shape[1] + EPS).sqrt()  # noqa: E731
    gate = 1.0 if s["gate"] is None else s["gate"].double()
    unit = y / rms(y) if c["post"] else y
    u = unit * s["w_post"].double() if c["post"] else y
    if c["op"] == "norm":
        h = s["scale"] * gate * u
        if c["residual"]:
            h = h + s["residual_scale"] * s["residual"].double()
        v = h.to(s["y"].dtype).double()
        return {"h": h, "n": v / rms(v) * s["w_pre"].double() if c["pre"] else None}
    out = {"dy": None, "dresidual": None, "dgate": None, "dw_post": None, "dw_pre": None}
    total = s["dh"].double()
    if c["pre"]:
        h, dn = s["h"].double(), s["dn"].double()
        hat = h / rms(h)
        out["dw_pre"] = (dn * hat).sum(0)
        t = dn * s["w_pre"].double()
        total = total + (t - hat * (t * hat).mean(1, keepdim=True)) / rms(h)
    if c["residual"]:
        out["dresidual"] = s["residual_scale"] * total
    branch = s["scale"] * total
    if c["gate"] != "none":
        out["dgate"] = (branch * u).sum(0) if c["gate"] == "channel" else branch * u
    du = branch * gate
    if c["post"]:
        out["dw_post"] = (du * unit).sum(0)
        t = du * s["w_post"].double()
        out["dy"] = (t - unit * (t * unit).mean(1, keepdim=True)) / rms(y)
    else:
        out["dy"] = du
    return out
