"""The block operators' definitions in 64 bits, for the tests (CPU, numpy).

Written from include/llmoe_block.h; shares no code with the library.
"""
import numpy as np


def e4m3_values():
    """The 256 values of e4m3 by code, from the format: sign, 4 exponent bits
    (bias 7), 3 mantissa bits; no infinities, S.1111.111 is NaN."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, c >> 3 & 15, c & 7
        a = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if e == 15 and m == 7 else -a if s else a
    return v


E4M3 = e4m3_values()
_POS = E4M3[:127]  # 0 .. 448, ascending


def nearest_e4m3(q):
    """Largest magnitude 448: the nearest e4m3 value of each q, ties to the even code."""
    a = np.minimum(np.abs(q), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    up = _POS[hi] - a
    down = a - _POS[lo]
    code = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    return np.copysign(_POS[code], q)


def scale_exponent(amax):
    """Smallest k >= -126 with amax <= 448 * 2^k."""
    k = np.full(amax.shape, -126)
    some = amax > 0
    k[some] = np.maximum(-126, np.ceil(np.log2(amax[some] / 448)).astype(int))
    # log2 is rounded: settle the exact powers by comparison
    k = np.where(amax > 448.0 * np.exp2(k.astype(float)), k + 1, k)
    lower = (k > -126) & (amax <= 448.0 * np.exp2(k - 1.0))
    return np.where(lower, k - 1, k)


def row_bytes(n):
    return n + -(-(n // 32) // 16) * 16


def split_mx8(rows, n):
    """uint8 rows -> (codes' values [.., n], scale codes [.., n / 32], padding)."""
    return E4M3[rows[..., :n]], rows[..., n:n + n // 32], rows[..., n + n // 32:]


def mx8_values(rows, n):
    v, s, _ = split_mx8(rows, n)
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(float) - 127))
    return v * np.repeat(scale, 32, axis=-1)


def pack_mx8(v):
    """64-bit values [rows, n] (finite) as MX8 rows."""
    rows, n = v.shape
    g = v.reshape(rows, n // 32, 32)
    k = scale_exponent(np.abs(g).max(-1))
    q = nearest_e4m3(g / np.exp2(k.astype(float))[..., None]).reshape(rows, n)
    code = np.searchsorted(_POS, np.abs(q)).astype(np.uint8) | np.where(np.signbit(q), 128, 0).astype(np.uint8)
    out = np.zeros((rows, row_bytes(n)), np.uint8)
    out[:, :n] = code
    out[:, n:n + n // 32] = k + 127
    return out


def check_mx8(rows, v, err):
    """MX8 rows against 64-bit values v [rows, n] that the kernel holds to
    within err: the scale is the definition's for some value within err of the
    group's largest, every code is as near to its value as the nearest code
    allows for, and the padding is zero."""
    n = v.shape[1]
    q, s, pad = split_mx8(rows, n)
    assert not pad.any()
    g = np.abs(v).reshape(len(v), n // 32, 32)
    e = err.reshape(g.shape)
    lo, hi = np.maximum(0, g - e).max(-1), (g + e).max(-1)
    k = s.astype(int) - 127
    assert ((scale_exponent(lo) <= k) & (k <= scale_exponent(hi))).all()
    scale = np.repeat(np.exp2(k.astype(float)), 32, axis=-1)
    # a value moved by err moves past the midpoint of two codes by at most err
    off = np.abs(q * scale - v)
    best = np.abs(nearest_e4m3(v / scale) * scale - v)
    assert (off <= best + 2 * err).all()


def rmsnorm(h, w, eps):
    h, w = h.astype(np.float64), w.astype(np.float64)
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def router(logits, bias, active, K, scoring, renorm, scale):
    """idx, w and the smallest gap between distinct keys near the selection."""
    l = logits.astype(np.float64)
    rows, E = l.shape
    idx = np.full((rows, K), -1, np.int64)
    w = np.zeros((rows, K))
    gap = np.inf
    for r in range(rows):
        if active is not None and not active[r]:
            continue
        can = l[r] > -np.inf
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                s = np.where(can, 1 / (1 + np.exp(-np.where(can, l[r], 0))), 0)
            key = s.copy()
        else:
            top = l[r][can].max() if can.any() else 0.0
            if top == np.inf:
                s = (l[r] == np.inf).astype(float)
            else:
                s = np.where(can, np.exp(np.where(can, l[r] - top, 0)), 0)
            s = s / s.sum() if s.sum() > 0 else s
            key = l[r].copy()
        if bias is not None:
            key = key + bias.astype(np.float64)
        can &= key > -np.inf
        key = np.where(can, key, -np.inf)
        order = sorted(np.flatnonzero(can), key=lambda e: (-key[e], e))
        chosen = order[:K]
        near = np.array([key[e] for e in order[:K + 1]])
        d = -np.diff(near[np.isfinite(near)])
        if (d > 0).any():
            gap = min(gap, d[d > 0].min())
        total = sum(s[e] for e in chosen)
        for j, e in enumerate(chosen):
            idx[r, j] = e
            w[r, j] = s[e] * (scale / total if renorm and total > 0 else 0.0 if renorm else scale)
    return idx, w, gap


def product(x, w, counts, T, swiglu):
    """Received rows, their 64-bit results and a bound of what fp32 sums of
    `in` products may be off (each addition by 2^-23 of the sum of magnitudes)."""
    E, R = counts.shape
    n_in = x.shape[1]
    rows, vals, errs = [], [], []
    for e in range(E):
        at = np.concatenate([np.arange((e * R + s) * T, (e * R + s) * T + counts[e, s]) for s in range(R)]).astype(int)
        a, b = x[at].astype(np.float64), w[e].astype(np.float64)
        r, m = a @ b.T, (np.abs(a) @ np.abs(b).T) * n_in * 2.0 ** -23
        if swiglu:
            h = b.shape[0] // 2
            g, u, mg, mu = r[:, :h], r[:, h:], m[:, :h], m[:, h:]
            with np.errstate(over="ignore"):
                silu = g / (1 + np.exp(-g))
            r = silu * u
            # |silu'| <= 1.1; the division, exponential and products add a few fp32 roundings
            m = (1.1 * mg * (np.abs(u) + mu) + np.abs(silu) * mu) + np.abs(r) * (8 + np.abs(g)) * 2.0 ** -23
        rows.append(at)
        vals.append(r)
        errs.append(m)
    return np.concatenate(rows), np.concatenate(vals), np.concatenate(errs)
