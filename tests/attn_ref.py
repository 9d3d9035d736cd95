"""Attention in NumPy float64, from the definitions in include/wc_attn.h, with
bounds on what a computation in 32 bits may be off by.  Shares no code with the
library."""
import numpy as np

from tests import fp4_ref
from tests.fp4_ref import U16, U32, chain

STEP = 2 * U32  # one fp32 operation, were it to truncate


def held(bits):
    """float64 values that a 4-bit cache holds for BF16 rows [.., dim]."""
    rows = bits.reshape(-1, bits.shape[-1])
    return fp4_ref.values(*fp4_ref.encode(rows), rows.shape[1]).reshape(bits.shape)


def attend(q, k, v, positions, scale, window, split_weights):
    """One head: (out, its bound, lse, its bound) of q [n, d] at `positions` over
    k, v [L, d].  split_weights: the weights enter the second product as two BF16
    numbers (16 bits), else as one (8 bits).

    A score is off by its sum's error, the factor's two roundings, the offset's
    subtraction and the exponential's, which together are relative errors of the
    weight; numerator and denominator each carry the largest of them.  The result
    is rounded to BF16 once."""
    n, d = q.shape
    L = k.shape[0]
    at = np.arange(L)
    out, bound = np.zeros((n, d)), np.zeros((n, d))
    lse, lbound = np.full(n, -np.inf), np.zeros(n)
    with np.errstate(all="ignore"):
        for i, p in enumerate(positions):
            ok = at <= p
            if window:
                ok &= at > p - window
            if not ok.any():
                continue
            kk, vv = k[ok], v[ok]
            s = kk @ q[i] * scale
            top = s.max()
            if top == -np.inf:
                continue
            ds = abs(scale) * chain(d) * STEP * (np.abs(kk) @ np.abs(q[i]))
            ds = (ds + 8 * STEP * (np.abs(s) + abs(top) + 32)).max() * 1.01  # the offset is within 16 / log2(e) of top
            w = np.exp(s - top)
            total = w.sum()
            m = len(w)
            rel = 2 * ds + (m / 4 + 128) * STEP  # weights, and the sums of both
            part = U16 ** 2 * 4 if split_weights else 2 * U16
            o = w @ vv / total
            a = w @ np.abs(vv) / total
            out[i] = o
            bound[i] = (2 * rel + part) * a
            bound[i] += U16 * (np.abs(o) + bound[i]) + 1e-37
            lse[i] = top + np.log(total)
            lbound[i] = rel + 8 * STEP * (abs(lse[i]) + abs(top) + 1)
    return out, bound, lse, lbound


def compare(got, ref, bound, what):
    got = np.asarray(got, dtype=np.float64)
    same = (np.isnan(got) & np.isnan(ref)) | (got == ref)
    with np.errstate(invalid="ignore"):
        err = np.where(same, 0.0, np.abs(got - ref))
        bad = ~(err <= bound) & ~same
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {tuple(np.argwhere(bad)[0])}: "
                           f"{got[bad][0]} for {ref[bad][0]}, bound {np.broadcast_to(bound, bad.shape)[bad][0]}")
