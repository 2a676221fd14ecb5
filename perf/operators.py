"""What is measured of the MXFP4 product and of the expert routing around it.

MXFP4 (OCP Microscaling Formats v1.0) holds 32 consecutive values of a row as E2M1 codes with one
power-of-two scale byte (E8M0).  Five operators:

  quantize  rows of activations or weights into MXFP4, and back to values
  linear    activations, quantised on the way, times a weight held in MXFP4
  experts   the same for a layer of experts: rows sorted by expert, one weight for each
  dispatch  tokens sorted by expert (a router's choices) and their rows laid out in that order,
            with the gradient of the rows
  combine   the experts' rows added up again for each token under the router's weights, with the
            gradients of rows and weights

`run` computes them in their plain form or, where `own` is true, through the package.
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decode step's activations, 16 rows of the hidden size: latency
        {"name": "quantize_decode", "op": "quantize", "rows": 16, "cols": 6144, "dtype": "bf16"},
        # a weight matrix or a long prefill in fp32: bandwidth; odd sizes, the last step cut short
        {"name": "quantize_weight_fp32", "op": "quantize", "rows": 16381, "cols": 8160, "dtype": "fp32"},
        # the attention projection of one token, an eighth of the heads: latency
        {"name": "linear_decode", "op": "linear", "M": 1, "N": 768, "K": 6144, "dtype": "bf16"},
        # 512 requests through the up-projection
        {"name": "linear_batch", "op": "linear", "M": 512, "N": 2048, "K": 6144, "dtype": "bf16"},
        # a ragged prefill from fp32 activations: no size a multiple of a tile
        {"name": "linear_ragged_fp32", "op": "linear", "M": 1237, "N": 2056, "K": 6112, "dtype": "fp32"},
        # the largest product of the benchmark's size sweep: compute
        {"name": "linear_saturation", "op": "linear", "M": 16384, "N": 8192, "K": 8192, "dtype": "bf16"},
        # 512 requests decoding, top 8 of 256 experts: about 16 rows each, every weight streamed once
        {"name": "experts_decode", "op": "experts", "tokens": 512, "topk": 8, "experts": 256, "N": 256, "K": 6144, "dtype": "bf16"},
        # 4096 prompt tokens through the same layer: about 128 rows each
        {"name": "experts_prefill", "op": "experts", "tokens": 4096, "topk": 8, "experts": 256, "N": 256, "K": 6144, "dtype": "bf16"},
        # 64 requests' dispatch in a decode step: latency
        {"name": "dispatch_decode", "op": "dispatch", "tokens": 64, "topk": 8, "experts": 256, "hidden": 6144, "dtype": "bf16", "drop": 0.0, "grad": False},
        # a training step's dispatch and its gradient, some choices dropped over capacity
        {"name": "dispatch_train", "op": "dispatch", "tokens": 8192, "topk": 8, "experts": 256, "hidden": 2048, "dtype": "bf16", "drop": 0.05, "grad": True},
        # the way back in the same decode step: latency
        {"name": "combine_decode", "op": "combine", "tokens": 64, "topk": 8, "experts": 256, "hidden": 6144, "dtype": "bf16", "drop": 0.0, "grad": False},
        # the way back in a training step, with the gradients of rows and weights
        {"name": "combine_train", "op": "combine", "tokens": 8192, "topk": 8, "experts": 256, "hidden": 2048, "dtype": "bf16", "drop": 0.05, "grad": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "experts", "dispatch", "combine"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    while True:
        if op == "quantize":
            c = {"op": op, "rows": _log(rng, 1, 16384), "cols": BLOCK * _log(rng, 1, 256), "dtype": dtype}
        elif op == "linear":
            c = {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 16, 8192), "K": BLOCK * _log(rng, 4, 256), "dtype": dtype}
        elif op == "experts":
            experts = _log(rng, 2, 256)
            c = {"op": op, "tokens": _log(rng, 1, 4096), "topk": rng.randint(1, min(8, experts)), "experts": experts,
                 "N": _log(rng, 16, 2048), "K": BLOCK * _log(rng, 4, 192), "dtype": dtype}
            if experts * c["N"] * c["K"] > 256 * 256 * 6144 or c["tokens"] * c["topk"] * c["N"] * c["K"] > 4096 * 8 * 256 * 6144:
                continue
        else:
            experts = _log(rng, 2, 512)
            c = {"op": op, "tokens": _log(rng, 1, 8192), "topk": rng.randint(1, min(8, experts)), "experts": experts,
                 "hidden": _log(rng, 32, 6144), "dtype": dtype, "drop": rng.choice((0.0, 0.05, 0.5)), "grad": rng.random() < 0.6}
            if c["tokens"] * c["topk"] * c["hidden"] * (2 if dtype == "fp32" else 1) > 8192 * 8 * 2048:
                continue
        return c


def work(case):
    c, size = case, 4 if case["dtype"] == "fp32" else 2
    op = c["op"]
    if op == "quantize":
        return {"bytes": 2 * size * c["rows"] * c["cols"], "flops": 0}
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": size * M * K + N * K * 17 / 32 + 2 * M * N, "flops": 2 * M * N * K}
    pairs = c["tokens"] * c["topk"]
    if op == "experts":
        N, K, used = c["N"], c["K"], min(c["experts"], pairs)
        return {"bytes": size * c["tokens"] * K + used * N * K * 17 / 32 + 2 * pairs * N + 4 * pairs, "flops": 2 * pairs * N * K}
    row, kept = size * c["hidden"], pairs * (1 - c["drop"])
    if op == "dispatch":
        once = (c["tokens"] + kept) * row
        return {"bytes": once * (2 if c["grad"] else 1) + 16 * pairs, "flops": kept * c["hidden"] if c["grad"] else 0}
    b = (kept + c["tokens"]) * row + 8 * pairs
    if c["grad"]:
        b += (kept + c["tokens"]) * row + 4 * pairs
    return {"bytes": b, "flops": kept * c["hidden"] * (5 if c["grad"] else 2)}


# ---- inputs ---------------------------------------------------------------------------------


def _activations(g, rows, cols, dtype):
    """Rows of a unit normal with one channel in a hundred twenty times as large, as the residual stream has them."""
    loud = 1 + 19 * (torch.rand(cols, device="cuda", generator=g) < 0.01).float()
    x = torch.empty(rows, cols, dtype=TYPES[dtype], device="cuda")
    for r in range(0, rows, 4096):
        x[r:r + 4096] = torch.randn(min(4096, rows - r), cols, device="cuda", generator=g) * loud
    return x


def _choices(g, case):
    """Each token's experts, some more popular than others; -1 where a choice was dropped."""
    popular = 0.5 * torch.randn(case["experts"], device="cuda", generator=g)
    logits = torch.randn(case["tokens"], case["experts"], device="cuda", generator=g) + popular
    ids = logits.topk(case["topk"], dim=1).indices
    if case.get("drop"):
        ids = torch.where(torch.rand(ids.shape, device="cuda", generator=g) < case["drop"], -1, ids)
    return ids.to(torch.int32).contiguous()


def _inputs(case, seed):
    """The inputs of a case by name, the same for every form."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    c, s = case, {}
    if c["op"] == "quantize":
        s["x"] = _activations(g, c["rows"], c["cols"], c["dtype"])
    elif c["op"] == "linear":
        s["x"] = _activations(g, c["M"], c["K"], c["dtype"])
        s["w"] = (0.02 * torch.randn(c["N"], c["K"], device="cuda", generator=g)).to(torch.bfloat16)
    elif c["op"] == "experts":
        s["ids"] = _choices(g, c)
        s["x"] = _activations(g, c["tokens"], c["K"], c["dtype"])
        s["w"] = torch.empty(c["experts"], c["N"], c["K"], dtype=torch.bfloat16, device="cuda")
        for e in range(c["experts"]):
            s["w"][e] = 0.02 * torch.randn(c["N"], c["K"], device="cuda", generator=g)
    else:
        s["ids"] = _choices(g, c)
        pairs = c["tokens"] * c["topk"]
        if c["op"] == "dispatch":
            s["x"] = _activations(g, c["tokens"], c["hidden"], c["dtype"])
            if c["grad"]:
                s["grad"] = torch.randn(pairs, c["hidden"], device="cuda", generator=g).to(TYPES[c["dtype"]])
        else:
            s["y"] = torch.randn(pairs, c["hidden"], device="cuda", generator=g).to(TYPES[c["dtype"]])
            s["weights"] = torch.softmax(torch.randn(c["tokens"], c["topk"], device="cuda", generator=g), dim=1)
            if c["grad"]:
                s["grad"] = torch.randn(c["tokens"], c["hidden"], device="cuda", generator=g).to(TYPES[c["dtype"]])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if own:
        import block_scaled_fp4_04_amd as nv
        s["nv"] = nv
    if op in ("linear", "experts"):
        # the weight as its program keeps it: packed, or as the values that its codes stand for
        s["w"] = s["nv"].mx_quantize(s["w"]) if own else _rounded(s["w"])
    if op in ("experts", "combine"):
        # the router's choices are sorted before the experts' product and kept for the way back
        s["route"] = s["nv"].moe_sort(s["ids"], case["experts"]) if own else _sorted(s["ids"], case["experts"])
    if op == "experts" and not own:
        # rows that the largest expert has, as a program that pads its experts keeps it
        off = s["route"]["row_offsets"]
        s["most"] = int((off[1:] - off[:-1]).max())
    if op == "dispatch" or op == "combine" and case["grad"]:
        # the buffer of the rows in the experts' order; those of dropped choices stay zero
        s["rows"] = torch.zeros(case["tokens"] * case["topk"], case["hidden"], dtype=TYPES[case["dtype"]], device="cuda")
    return s


# ---- the operators --------------------------------------------------------------------------


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        nv = s["nv"]
        if op == "quantize":
            return nv.mx_dequantize(nv.mx_quantize(s["x"]), s["x"].dtype)
        if op == "linear":
            return nv.mx_linear(s["x"], s["w"])
        if op == "experts":
            r = s["route"]
            return nv.mx_grouped_gemm(nv.mx_quantize(s["x"]), s["w"], r.row_offsets, rows=r.tokens)
        if op == "dispatch":
            r = nv.moe_sort(s["ids"], c["experts"])
            out = {"row_offsets": r.row_offsets, "slots": r.slots, "tokens": r.tokens, "rows": nv.moe_gather(s["x"], r, out=s["rows"])}
            if c["grad"]:
                out["dx"] = nv.moe_gather_grad(s["grad"], r)
            return out
        out = {"out": nv.moe_combine(s["y"], s["route"], s["weights"])}
        if c["grad"]:
            out["dy"], out["dweights"] = nv.moe_combine_grad(s["grad"], s["y"], s["route"], s["weights"], dy=s["rows"])
        return out
    if op == "quantize":
        return _rounded(s["x"]).to(s["x"].dtype)
    if op == "linear":
        return (_rounded(s["x"]) @ s["w"].t()).to(torch.bfloat16)
    if op == "experts":
        # rows padded to the largest expert's, one batched product, and back
        r, E = s["route"], c["experts"]
        off = r["row_offsets"].long()
        at = off[:-1, None] + torch.arange(s["most"], device="cuda")
        pad = (at >= off[1:, None])[:, :, None]
        at = at.clamp(max=r["tokens"].numel() - 1)
        a = torch.where(pad, 0.0, _rounded(s["x"])[r["tokens"].long()[at]])
        y = torch.bmm(a, s["w"].transpose(1, 2))
        e = torch.searchsorted(off[1:], torch.arange(r["tokens"].numel(), device="cuda"), right=True).clamp(max=E - 1)
        return y[e, torch.arange(r["tokens"].numel(), device="cuda") - off[e]].to(torch.bfloat16)
    if op == "dispatch":
        r = _sorted(s["ids"], c["experts"])
        kept = (r["tokens"] >= 0)[:, None]
        out = dict(r, rows=torch.where(kept, s["x"][r["tokens"].long().clamp(min=0)], 0))
        if c["grad"]:
            out["dx"] = _back(s["grad"], r["slots"], None).to(s["x"].dtype)
        return out
    r = s["route"]
    out = {"out": _back(s["y"], r["slots"], s["weights"]).to(s["y"].dtype)}
    if c["grad"]:
        slots, g = r["slots"].long(), s["grad"].float()
        kept = slots >= 0
        w = torch.where(kept, s["weights"], 0.0)
        y = s["y"][slots.clamp(min=0)].float()
        out["dweights"] = torch.where(kept, (y * g[:, None, :]).sum(2), 0.0)
        back = torch.zeros(slots.numel() + 1, g.shape[1], dtype=s["y"].dtype, device="cuda")
        back[torch.where(kept, slots, slots.numel())] = (w[:, :, None] * g[:, None, :]).to(s["y"].dtype)
        out["dy"] = back[:-1]
    return out


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


def _sorted(ids, experts):
    """A router's choices in the experts' order, those of one expert by token: where each expert's rows
    begin, the row of each choice (-1: dropped) and the token of each row (-1: no row)."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    byrow = key[order]
    off = torch.searchsorted(byrow, torch.arange(experts + 1, device=ids.device))
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel(), device=ids.device)
    slots = torch.where(key < experts, slots, -1).reshape(ids.shape)
    tokens = torch.where(byrow < experts, order // ids.shape[1], -1)
    return {"row_offsets": off.to(torch.int32), "slots": slots.to(torch.int32), "tokens": tokens.to(torch.int32)}


def _back(y, slots, weights):
    """For each token the sum over its choices of their rows, weighted or not; dropped choices give nothing."""
    at = slots.long()
    w = (at >= 0).float() if weights is None else torch.where(at >= 0, weights, 0.0)
    return (y[at.clamp(min=0)].float() * w[:, :, None]).sum(1)


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


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    op = c["op"]
    if op == "quantize":
        return torch.cat([_held(p) for p in s["x"].split(4096)])
    if op == "linear":
        w = _held(s["w"]).t().contiguous()
        return torch.cat([_held(p) @ w for p in s["x"].split(4096)])
    ids = s["ids"].cpu().tolist()
    E, k = c["experts"], c["topk"]
    chosen = [[] for _ in range(E)]
    for t, row in enumerate(ids):
        for j, e in enumerate(row):
            if 0 <= e < E:
                chosen[e].append((t, j))
    off, tokens, slots = [0], [], [[-1] * k for _ in ids]
    for pairs in chosen:
        for t, j in pairs:
            slots[t][j] = len(tokens)
            tokens.append(t)
        off.append(len(tokens))
    if op == "experts":
        a = _held(s["x"])
        return torch.cat([a[tokens[b:e]] @ _held(s["w"][i]).t() for i, (b, e) in enumerate(zip(off, off[1:])) if e > b])
    kept = len(tokens)
    at = torch.tensor(slots, device="cuda")
    if op == "dispatch":
        rows = torch.zeros(len(ids) * k, c["hidden"], dtype=torch.float64, device="cuda")
        rows[:kept] = s["x"][tokens].double()
        out = {"row_offsets": torch.tensor(off, dtype=torch.int32), "slots": at.to(torch.int32),
               "tokens": torch.tensor(tokens + [-1] * (len(ids) * k - kept), dtype=torch.int32), "rows": rows}
        if c["grad"]:
            out["dx"] = sum(torch.where(at[:, j, None] >= 0, s["grad"].double()[at[:, j]], 0.0) for j in range(k))
        return out
    y, w = s["y"].double(), s["weights"].double()
    picked = [torch.where(at[:, j, None] >= 0, y[at[:, j]], 0.0) for j in range(k)]
    out = {"out": sum(w[:, j, None] * p for j, p in enumerate(picked))}
    if c["grad"]:
        g = s["grad"].double()
        out["dweights"] = torch.stack([(p * g).sum(1) for p in picked], dim=1)
        out["dy"] = torch.zeros_like(y)
        for j in range(k):
            t = torch.nonzero(at[:, j] >= 0).flatten()
            out["dy"][at[t, j]] = w[t, j, None] * g[t]
    return out
