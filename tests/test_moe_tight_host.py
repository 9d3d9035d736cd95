"""The bound of tests/moe_tight.py, without a GPU: two parts of an activation
stay within it, one part, or the low parts of other columns, do not."""
import numpy as np
import pytest

from tests import fp4_ref, moe_tight


def layer(T, H, I, E, seed):
    rng = np.random.default_rng([seed, T, H, I, E])
    r = fp4_ref.bf16_round
    return (moe_tight.inputs(rng, T, H), r(rng.standard_normal((E, H))), r(rng.standard_normal((E, 2 * I, H))),
            r(rng.standard_normal((E, H, I)) / np.sqrt(I)))


def two(h):
    return sum(moe_tight.split(h))


def one(h):
    return moe_tight.split(h)[0]


def others(h):
    hi, lo = moe_tight.split(h)
    return hi + np.roll(lo, 1)


@pytest.mark.parametrize("T,H,I,E,k", [(9, 256, 96, 12, 3), (5, 1000, 264, 6, 2), (3, 128, 700, 8, 4)])
def test_bound_tells_the_parts_apart(T, H, I, E, k):
    args = layer(T, H, I, E, 1)
    y, bound, _, _ = moe_tight.moe(*args, k)
    for parts, fits in ((two, True), (one, False), (others, False)):
        got = fp4_ref.bf16_round(moe_tight.moe(*args, k, parts=parts)[0])
        over = np.abs(got - y) > bound
        assert over.any() != fits, parts.__name__
        assert fits or over.mean() > 0.02  # dozens of outputs


def test_two_parts_hold_sixteen_bits():
    v = np.random.default_rng(2).standard_normal(20000) * np.exp2(np.random.default_rng(3).integers(-30, 30, 20000))
    assert (np.abs(two(v) - v) <= 2.0 ** -16 * np.abs(v)).all()
    assert (np.abs(one(v) - v) > 2.0 ** -12 * np.abs(v)).mean() > 0.5
