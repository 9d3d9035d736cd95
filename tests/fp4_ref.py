"""The 4-bit form and the mixture-of-experts layer in NumPy float64, from the
definitions in include/wc_fp4.h and include/wc_moe.h, with bounds on what a
32-bit computation of them may be off by.  Shares no code with the library."""
import math

import numpy as np

GROUP = 32
MAGS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
U32 = 2.0 ** -24  # half a step of fp32, relative
U16 = 2.0 ** -8   # half a step of BF16, relative


def bf16_round(v):
    """float64 -> the nearest BF16 as float64, ties to even, infinite past the range."""
    v = np.asarray(v, dtype=np.float64)
    m, e = np.frexp(v)
    e = np.maximum(e, -125)  # subnormals share the smallest normal's step
    step = np.ldexp(1.0, e - 8)
    with np.errstate(invalid="ignore"):
        r = np.rint(v / step) * step
    r = np.where(np.isfinite(v), r, v)
    return np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, v), r)


def to_bits(v):
    """BF16 bit patterns of float64 values that BF16 holds."""
    with np.errstate(over="ignore", invalid="ignore"):
        return (np.asarray(v, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def of_bits(b):
    return (np.asarray(b, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def groups_of(cols):
    return -(-cols // GROUP)


def encode(bits):
    """(codes, scales) of BF16 bit patterns [rows, cols], group by group."""
    rows, cols = bits.shape
    G = groups_of(cols)
    w = np.zeros((rows, G * GROUP))
    w[:, :cols] = of_bits(bits)
    sign = np.zeros((rows, G * GROUP), dtype=np.uint8)
    sign[:, :cols] = bits >> 15
    w = w.reshape(rows, G, GROUP)
    top = np.abs(w).max(-1)
    bad = ~np.isfinite(top)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(top > 0, np.ceil(np.log2(np.where(bad | (top == 0), 1.0, top) / 7)), -126)
    e = np.maximum(e, -126)
    e = np.where(np.ldexp(7.0, (e - 1).astype(int)) >= np.where(bad, 0, top), e - 1, e)
    e = np.where(np.ldexp(7.0, e.astype(int)) < np.where(bad, 0, top), e + 1, e)
    e = np.maximum(e, -126).astype(int)
    mags = np.broadcast_to(MAGS, (rows, G, 8)) * np.ldexp(1.0, e)[..., None]
    ok = bf16_round(mags) == mags
    ok &= np.isfinite(bf16_round(mags))
    best = np.full(w.shape, np.inf)
    code = np.zeros(w.shape, dtype=np.uint8)
    with np.errstate(invalid="ignore"):
        for k in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they keep ties
            d = np.where(ok[..., k:k + 1], np.abs(np.abs(w) - mags[..., k:k + 1]), np.inf)
            near = d < best
            best, code = np.where(near, d, best), np.where(near, k, code).astype(np.uint8)
    code = (code.reshape(rows, -1) | sign << 3).reshape(w.shape)
    code = np.where(bad[..., None], 0, code).reshape(rows, -1)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8), scales


def values(codes, scales, cols):
    """float64 values of codes [rows, 16 G] and scales [rows, G]."""
    q = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    s = np.ldexp(1.0, scales.astype(int) - 127)
    s = np.where(scales == 255, np.nan, s).repeat(GROUP, -1)
    v = np.where(q & 8, -1.0, 1.0) * MAGS[q & 7] * s
    return bf16_round(v)[:, :cols]


def chain(cols):
    """An addend of a row's sum goes through at most this many fp32 additions:
    32 inside a matrix instruction, one for each of the cols / 32 instructions
    and fewer than 32 where waves and column splits are joined.  Each is off by
    at most a whole step (an addition that truncates)."""
    return cols / 32 + 64


def gemv(w, x):
    """(y, bound) of y[b][r] = sum_c w[r][c] x[b][c]."""
    y = x @ w.T
    return y, chain(w.shape[1]) * 2 * U32 * (np.abs(x) @ np.abs(w).T)


def route(x, router, k, scoring, bias, renorm, scale=1.0):
    """(ids, weights, weights' relative bound, gap): gap is the smallest
    distance between a chosen expert's value and the next one's, over twice the
    error of both; choices are the same in 32 bits where it is above 1."""
    _, lb = gemv(router, x)
    T, E = lb.shape
    # row by row, so that equal router rows give equal logits
    logits = np.stack([(x * router[e]).sum(-1) for e in range(E)], -1)
    with np.errstate(all="ignore"):
        if scoring == "sigmoid":
            p = 1 / (1 + np.exp(-logits))
        else:
            p = np.exp(logits - logits.max(-1, keepdims=True))
            p = p / p.sum(-1, keepdims=True)
    # exp, the division and a sum of E terms, next to the logits' own error
    prel = 2 * lb.max(-1) + (E + 32) * 2 * U32
    ids = np.full((T, k), -1, dtype=np.int32)
    weights = np.zeros((T, k))
    gap = math.inf
    for t in range(T):
        v = logits[t] if bias is None else p[t] + bias
        verr = lb[t].max() if bias is None else prel[t] + 2 * U32 * np.abs(v[np.isfinite(v)]).max(initial=0)
        left = [e for e in range(E) if bias is None or bias[e] != -np.inf]
        left.sort(key=lambda e: (not np.isnan(v[e]), -v[e] if not np.isnan(v[e]) else 0, e))
        row = left[:k]
        for j in range(min(len(row), len(left) - 1)):
            d = v[left[j]] - v[left[j + 1]]
            if d > 0:  # equal values go by index on both sides
                gap = min(gap, d / (2 * verr))
        w = p[t, row]
        if renorm:
            w = w / w.sum() if w.sum() != 0 else w * 0
        ids[t, :len(row)], weights[t, :len(row)] = row, w * scale
    return ids, weights, (2 * prel + (k + 4) * 2 * U32), gap


def moe(x, router, gate_up, down, k, scoring="softmax", bias=None, renorm=True, scale=1.0):
    """(y, bound, ids, weights, weights' relative bound, gap): gate_up
    [E, 2 I, H] and down [E, H, I] as float64 arrays or indexable by expert."""
    ids, weights, wrel, gap = route(x, router, k, scoring, bias, renorm, scale)
    T, H = x.shape
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    with np.errstate(all="ignore"):
        for t in range(T):
            terms = 0
            for e, p in zip(ids[t], weights[t]):
                if e < 0:
                    continue
                gu, gb = gemv(gate_up[e], x[t:t + 1])
                I = gu.shape[1] // 2
                terms += I
                g, u, db, ub = gu[0, :I], gu[0, I:], gb[0, :I], gb[0, I:]
                act = g / (1 + np.exp(-g))
                h = act * u * p
                # |silu'| <= 1.1; exp, division and two products; BF16 once
                hb = np.abs(p) * (1.1 * db * (np.abs(u) + ub) + np.abs(act) * ub)
                hb += np.abs(h) * (wrel[t] + 16 * 2 * U32)
                hb += U16 * (np.abs(h) + hb)
                y[t] += down[e] @ h
                bound[t] += np.abs(down[e]) @ (hb + chain(I * k) * 2 * U32 * np.abs(h))
        bound += U16 * (np.abs(y) + bound)
    return y, bound, ids, weights, wrel, gap
