"""Definitions of the block-scaled operators and of the router with groups, for
the tests (CPU, numpy).  Written from include/llmoe_block.h; shares no code with
the library."""
import numpy as np

import block_reference as ref

BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def row_bytes(n):
    return n + -(-4 * blocks(n) // 16) * 16


def scale_of(amax):
    """fp32: amax / 448, at least 2^-126; NaN where amax is not finite."""
    amax = amax.astype(np.float32)
    with np.errstate(all="ignore"):
        s = np.maximum(amax / np.float32(448), np.float32(2.0 ** -126))
    return np.where(np.isfinite(amax), s, np.float32("nan"))


def codes_of(v, scale):
    """The codes' values of v (fp32) at these scales: nearest to the fp32 product v * (1 / scale)."""
    q = v.astype(np.float32) * (np.float32(1) / scale.astype(np.float32))
    return ref.nearest_e4m3(q.astype(np.float64))


def as_codes(q):
    return np.searchsorted(ref._POS, np.abs(q)).astype(np.uint8) | np.where(np.signbit(q), 128, 0).astype(np.uint8)


def spread(scale, n):
    return np.repeat(scale, BLOCK, axis=-1)[..., :n]


def block_max(v):
    """Largest magnitude of each block of the last axis; NaN where a block holds one."""
    pad = np.zeros((*v.shape[:-1], blocks(v.shape[-1]) * BLOCK - v.shape[-1]), v.dtype)
    return np.abs(np.concatenate([v, pad], -1)).reshape(*v.shape[:-1], -1, BLOCK).max(-1)


def split(rows, n):
    """uint8 rows -> (codes' values, fp32 scales, padding)."""
    b = 4 * blocks(n)
    return ref.E4M3[rows[..., :n]], np.ascontiguousarray(rows[..., n:n + b]).view(np.float32), rows[..., n + b:]


def values(rows, n):
    q, s, _ = split(rows, n)
    return q * spread(s.astype(np.float64), n)


def pack(v):
    """fp32 values [rows, n] (finite) as FP8B rows."""
    n = v.shape[-1]
    s = scale_of(block_max(v))
    out = np.zeros((*v.shape[:-1], row_bytes(n)), np.uint8)
    out[..., :n] = as_codes(codes_of(v, spread(s, n)))
    out[..., n:n + 4 * blocks(n)] = np.ascontiguousarray(s, np.float32).view(np.uint8)
    return out


def check(rows, v, err):
    """FP8B rows against 64-bit values v [rows, n] that the kernel holds to within
    err: a scale is within its block's largest err and a half unit of fp32 of
    amax / 448, a code as near to its value as the nearest allows for."""
    n = v.shape[1]
    q, s, pad = split(rows, n)
    assert not pad.any()
    lo, hi = block_max(np.maximum(0, np.abs(v) - err)), block_max(np.abs(v) + err)
    s = s.astype(np.float64)
    assert (np.maximum(lo / 448 * (1 - 2.0 ** -24), 2.0 ** -126) <= s).all()
    assert (s <= np.maximum(hi / 448 * (1 + 2.0 ** -24), 2.0 ** -126)).all()
    wide = spread(s, n)
    off = np.abs(q * wide - v)
    best = np.abs(ref.nearest_e4m3(v / wide) * wide - v)
    # a value moved by err, and its quotient by two roundings of fp32 (1 / s and
    # the product, 2^-24 each), passes the midpoint of two codes by at most that
    assert (off <= best + 2 * err + 2 * np.abs(v) * 2.0 ** -23).all()


def pack_weights(w):
    """fp32 values [..., rows, cols] (finite) as codes and block scales."""
    r, c = w.shape[-2:]
    s = scale_of(np.swapaxes(block_max(np.swapaxes(block_max(w), -1, -2)), -1, -2))
    return as_codes(codes_of(w, spread_weights(s, r, c))), s


def spread_weights(s, r, c):
    return np.repeat(np.repeat(s, BLOCK, -2)[..., :r, :], BLOCK, -1)[..., :c]


def weight_values(codes, s):
    return ref.E4M3[codes] * spread_weights(s.astype(np.float64), *codes.shape[-2:])


def product_error(n_in):
    """A product's error over the sum of its magnitudes: block_reference.product
    has `in` additions of 2^-23; a block's scales are multiplied (one rounding)
    and applied (another), both 2^-24, and joined (one of in / 128 additions)."""
    return (n_in + blocks(n_in) + 2) / n_in


def group_router(logits, bias, active, K, groups, kept, top2, scoring, renorm, scale, same=1e-12):
    """idx, w and the smallest gap, over distinct values, of the group scores at
    the border of the kept and of the keys near the choice."""
    l = logits.astype(np.float64)
    rows, E = l.shape
    S = E // groups
    masked = l.copy()
    keys = l.copy()
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            keys = 1 / (1 + np.exp(-l))
    if bias is not None:
        keys = keys + bias.astype(np.float64)
    can = (l > -np.inf) & (keys > -np.inf)
    gap = np.inf
    for r in range(rows):
        score = []
        for g in range(groups):
            k = np.sort(keys[r, g * S:(g + 1) * S][can[r, g * S:(g + 1) * S]])[::-1]
            score.append(k[:2].sum() if top2 and len(k) else k[0] if len(k) else None)
        order = sorted(range(groups), key=lambda g: (score[g] is None, -(score[g] or 0), g))
        if kept < groups and score[order[kept]] is not None:
            d = score[order[kept - 1]] - score[order[kept]]
            if d > same:
                gap = min(gap, d)
            elif not d == 0:
                gap = 0.0  # equal but for 64 bits' rounding: either may lead
        for g in order[kept:]:
            masked[r, g * S:(g + 1) * S] = -np.inf
    idx, w, near = ref.router(masked, bias, active, K, scoring, True, scale)
    if not renorm:  # an unrenormalised softmax is over the experts of all groups
        for r in range(rows):
            score = np.zeros(E)
            if scoring == "sigmoid":
                with np.errstate(over="ignore"):
                    score = 1 / (1 + np.exp(-l[r]))
            elif can[r].any():
                top = l[r][can[r]].max()
                score[can[r]] = np.exp(l[r][can[r]] - top) if top < np.inf else l[r][can[r]] == np.inf
                score /= score.sum()
            w[r] = np.where(idx[r] >= 0, score[np.maximum(idx[r], 0)] * scale, 0)
    return idx, w, min(gap, near)
