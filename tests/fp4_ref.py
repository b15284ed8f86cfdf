"""Plain float64 forms of the 4-bit quantisation and of routing from logits (test infrastructure only)."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def e4m3_grid():
    """The non-negative finite E4M3 values by code."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


E4M3 = e4m3_grid()


def nearest(v, grid):
    """Index of the nearest grid value, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    below, above = v - grid[lo], grid[hi] - v
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def quantize(x, fmt, ts=None):
    """(codes [rows, K/2], scale codes, values) of x [rows, K] float64 (finite)."""
    rows, K = x.shape
    b = x.reshape(rows, K // BLOCK[fmt], BLOCK[fmt])
    amax = np.abs(b).max(2)
    if fmt == "mxfp4":
        e = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))), -1000)
        # log2 may round up to the next power: step back where it did
        e = np.where((amax > 0) & (2.0 ** e > amax), e - 1, e)
        sh = np.clip(e - 2, -127, 127)
        sc = (sh + 127).astype(np.uint8)
        unit = 2.0 ** sh
    else:
        g = 1.0 if ts is None else float(np.float32(ts))
        sc = nearest(amax / (6.0 * g), E4M3).astype(np.uint8)
        unit = (E4M3[sc].astype(np.float32) * np.float32(g)).astype(np.float64)
    u = unit[:, :, None]
    # |x| against border * unit in extended precision of exact products: 53 bits hold 24 + 24 + 3
    a = np.abs(b)
    code = np.zeros(b.shape, dtype=np.uint8)
    for border, closed in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        code += (a >= border * u) if closed else (a > border * u)
    code = np.where(u > 0, code, 0).astype(np.uint8)
    vals = np.where(np.signbit(b), -1.0, 1.0) * GRID[code] * u
    code = code | (np.signbit(b).astype(np.uint8) << 3)
    code = np.where(u > 0, code, 0).astype(np.uint8)   # a block whose scale is 0 has no signs either
    c = code.reshape(rows, K // 2, 2)
    return (c[:, :, 0] | (c[:, :, 1] << 4)), sc, vals.reshape(rows, K)


def values(codes, scales, fmt, ts=None):
    """float64 values of codes [..., K/2] with scales [..., K/block]."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    v = GRID[n & 7] * np.where(n >> 3, -1.0, 1.0)
    d = 2.0 ** (scales.astype(np.float64) - 127) if fmt == "mxfp4" else E4M3[scales & 127]
    if ts is not None:
        d = d * np.asarray(ts, dtype=np.float64)
    return v * np.repeat(d, BLOCK[fmt], -1)


def score(z, kind):
    with np.errstate(all="ignore"):
        if kind == "softmax":
            m = z.max(1, keepdims=True)
            e = np.where(np.isneginf(z), 0.0, np.exp(z - np.where(np.isfinite(m), m, 0.0)))
            return e / np.where(e.sum(1, keepdims=True) > 0, e.sum(1, keepdims=True), 1.0)
        if kind == "sigmoid":
            return np.where(z >= 0, 1 / (1 + np.exp(-z)), np.exp(z) / (1 + np.exp(z)))
        return np.sqrt(np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z))))


def route(z, k, kind, bias=None, G=1, kept=1, group="top2", renorm=True, scale=1.0):
    """Row by row, in plain loops: (idx [T, k], w [T, k]) from float64 logits."""
    T, E = z.shape
    s = score(z, kind)
    idx, w = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T):
        key = [s[t, e] + (0.0 if bias is None else float(bias[e])) for e in range(E)]
        live = [not np.isneginf(z[t, e]) for e in range(E)]
        worth = []
        for g in range(G):
            ks = sorted((key[e] for e in range(g * E // G, (g + 1) * E // G) if live[e]), reverse=True)
            worth.append(-np.inf if not ks else sum(ks[:2]) if group == "top2" else ks[0])
        best = sorted(range(G), key=lambda g: (-worth[g], g))[:kept]
        cand = [e for e in range(E) if live[e] and e // (E // G) in best]
        sel = sorted(cand, key=lambda e: (-key[e], e))[:k]
        ws = np.array([s[t, e] for e in sel])
        if len(sel):
            idx[t, :len(sel)] = sel
            w[t, :len(sel)] = scale * (ws / ws.sum() if renorm else ws)
    return idx, w


def route_weights(z, idx, kind, renorm, scale):
    """The weights of a fixed selection as a function of the logits (for differences)."""
    s = score(z, kind)
    T, k = idx.shape
    w = np.zeros((T, k))
    for t in range(T):
        ws = np.array([s[t, e] if e >= 0 else 0.0 for e in idx[t]])
        w[t] = scale * (ws / ws.sum() if renorm and ws.sum() > 0 else ws)
    return w
