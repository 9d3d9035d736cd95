"""The mixture-of-experts layer in NumPy float64 with the bound that
include/wc_moe.h's arithmetic allows: weight * silu(gate) * up enters the second
product as two BF16 numbers, so it is off by at most half a step of half a step
of BF16 (2^-16 of it) beside fp32's errors.  tests/fp4_ref.py allows one BF16
rounding there.  With inputs of two numbers per token the first products' own
bound is small, and the loss of the low parts does not fit the whole one."""
import numpy as np

from tests import fp4_ref
from tests.fp4_ref import U16, U32, chain, gemv


def inputs(rng, T, H):
    """x of two numbers per token, as BF16 values."""
    x = np.zeros((T, H))
    for row in x:
        at = rng.permutation(H)[:2]
        row[at] = fp4_ref.bf16_round(rng.standard_normal(at.size))
    return x


def split(v):
    """The two BF16 numbers whose sum stands for v."""
    hi = fp4_ref.bf16_round(v)
    return hi, fp4_ref.bf16_round(v - hi)


def moe(x, router, gate_up, down, k, scoring="softmax", bias=None, renorm=True, scale=1.0, parts=None):
    """(y before its rounding, bound of the rounded y, ids, gap); `parts`: what
    to put in place of an activation v, for the bound's own tests."""
    ids, weights, wrel, gap = fp4_ref.route(x, router, k, scoring, bias, renorm, scale)
    T, H = x.shape
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for e, p in zip(ids[t], weights[t]):
            if e < 0:
                continue
            gu, gb = gemv(gate_up[e], x[t:t + 1])
            I = gu.shape[1] // 2
            g, u, db, ub = gu[0, :I], gu[0, I:], gb[0, :I], gb[0, I:]
            act = g / (1 + np.exp(-g))
            h = act * u * p
            # |silu'| <= 1.1; exp, division and two products; then the two parts
            hb = np.abs(p) * (1.1 * db * (np.abs(u) + ub) + np.abs(act) * ub)
            hb += np.abs(h) * (wrel[t] + 16 * 2 * U32)
            hb += U16 * U16 * (np.abs(h) + hb)
            y[t] += down[e] @ (h if parts is None else parts(h))
            # the parts' sums go on their own: |hi| + |lo| <= (1 + 2 U16) |h|
            bound[t] += np.abs(down[e]) @ (hb + chain(I * k) * 2 * U32 * (1 + 2 * U16) * np.abs(h))
    bound += U16 * (np.abs(y) + bound)
    return y, bound, ids, gap
