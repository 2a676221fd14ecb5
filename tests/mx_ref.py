"""Plain references, in 64 bits, of the MXFP4 operators and of the expert
routing: written from the definitions, sharing nothing with the library."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EDGES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def quantize(x):
    """fp32 [rows, K] -> (codes [rows, K/2], scale bytes [rows, K/32])."""
    rows, K = x.shape
    v = x.astype(np.float64).reshape(rows, K // 32, 32)
    bad = ~np.isfinite(v).all(axis=2)
    a = np.where(bad[:, :, None], 0.0, np.abs(v))
    top = a.max(axis=2)
    _, e = np.frexp(top)                      # top = m * 2^e, m in [0.5, 1)
    byte = np.where(top > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    y = np.ldexp(a, (127 - byte)[:, :, None])
    code = np.zeros(y.shape, np.uint8)
    for i, edge in enumerate(EDGES):          # a tie goes to the even code
        code += (y >= edge) if i % 2 else (y > edge)
    code |= (np.signbit(v) << 3).astype(np.uint8)
    code = np.where(bad[:, :, None], 0, code).astype(np.uint8).reshape(rows, K)
    byte = np.where(bad, 255, byte).astype(np.uint8)
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8), byte


def values(codes, scales):
    """Canonical codes and scale bytes -> float64 [..., K]."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    s = np.ldexp(1.0, scales.astype(np.int64) - 127)
    s = np.where(scales == 255, np.nan, s)
    return v * np.repeat(s, 32, axis=-1)


def random_operand(g, rows, K, lo=118, hi=132):
    """Random codes of all 16 kinds under random scales."""
    return (g.integers(0, 256, (rows, K // 2), dtype=np.uint8),
            g.integers(lo, hi, (rows, K // 32), dtype=np.uint8))


def gemm_bound(a, b, alpha, out_eps):
    """How far the product of values a [M, K], b [N, K] may be off: each
    matrix instruction (64 elements deep at least) and each of at most 16
    partial sums adds with at most two units in the last place of fp32
    (2^-22 of the magnitudes), alpha rounds once (2^-24), the output once by
    half a step (out_eps / 2)."""
    mag = abs(alpha) * (np.abs(a) @ np.abs(b).T)
    adds = a.shape[1] / 64 + 17
    return adds * 2.0 ** -22 * mag + (2.0 ** -24 + out_eps / 2) * abs(alpha) * np.abs(a @ b.T) + 1e-40


def sort(ids, experts):
    """(row_offsets, slots, tokens) by the definition."""
    T, k = ids.shape
    lists = [[] for _ in range(experts)]
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < experts:
                lists[ids[t, j]].append((t, j))
    off = np.zeros(experts + 1, np.int32)
    slots = np.full((T, k), -1, np.int32)
    tokens = np.full(T * k, -1, np.int32)
    n = 0
    for e in range(experts):
        for t, j in lists[e]:
            slots[t, j], tokens[n] = n, t
            n += 1
        off[e + 1] = n
    return off, slots, tokens


def combine(y, slots, weights):
    """float64 [T, H]."""
    T, k = slots.shape
    out = np.zeros((T, y.shape[1]))
    for j in range(k):
        on = slots[:, j] >= 0
        w = 1.0 if weights is None else weights[on, j, None].astype(np.float64)
        out[on] += w * y[slots[on, j]].astype(np.float64)
    return out


def combine_grad(dout, y, slots, weights):
    """(dy with NaN in rows that no choice owns, dweights), float64."""
    T, k = slots.shape
    dy = np.full(y.shape, np.nan)
    dw = np.zeros((T, k))
    for j in range(k):
        on = slots[:, j] >= 0
        w = 1.0 if weights is None else weights[on, j, None].astype(np.float64)
        dy[slots[on, j]] = w * dout[on].astype(np.float64)
        dw[on, j] = (dout[on].astype(np.float64) * y[slots[on, j]].astype(np.float64)).sum(1)
    return dy, dw
