"""Queries that are not finite, beside others: nobody else's results change, in the
attention of prompts and in that over the 4-bit cache."""
import numpy as np
import pytest

import synth
from tests import fp4_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests import test_gpu_cache as of_cache, test_gpu_prompt as of_prompt  # noqa: E402

NAN, INF, MINUS_INF = 0x7FC0, 0x7F80, 0xFF80


def scaled(bits, size):
    return synth.bf16_bits((fp4_ref.of_bits(bits) * size[:, None, None]).astype(np.float32))


def prompt(dim, heads, lengths, steepness):
    """Scores that grow along the first sequence and fall along the others, whose
    largest ones then come last, as tiles are taken from the end on."""
    c = of_prompt.Case(lengths, heads, 1, dim, seed=21)
    size = np.concatenate([np.arange(n)[::1 if i == 0 else -1] * steepness + 0.1 for i, n in enumerate(lengths)])
    c.k = scaled(c.k, size)
    c.k[:, :, 0] &= 0x7FFF  # not negative: an infinite query has scores of its sign
    return c


def spoil(q, value):
    q[...] = value if value == NAN else 0
    if value != NAN:
        q[..., 0] = value


def expect(out, lse, value, what):
    if value == MINUS_INF:  # every score is -inf
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all()), what
    else:
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all()), what


@pytest.mark.parametrize("dim", [32, 64, 128, 160, 256])
@pytest.mark.parametrize("window", [0, 400])
@pytest.mark.parametrize("value", [NAN, INF, MINUS_INF])
@pytest.mark.parametrize("steepness", [0.05, 0.004])  # rises past fp32's exponents, and by a few dozen
def test_prompt(dim, window, value, steepness):
    c = prompt(dim, 2, [700, 699, 40], steepness)
    clean, clean_lse = (t.clone() for t in c.run(scale=1.0, window=window))
    assert bool(torch.isfinite(clean).all()) and bool(torch.isfinite(clean_lse).all())
    rows = [0, 5, 333, 690, 700, 731, 1000, 1031, 1398, 1420]  # one in a wave's 32 queries, or two
    for r in rows:
        spoil(c.q[r, 0], value)
    out, lse = c.run(scale=1.0, window=window)
    mine = torch.zeros(len(c.q), 2, dtype=torch.bool, device=of_prompt.DEV)
    mine[rows, 0] = True
    expect(out[mine], lse[mine], value, "the spoilt rows")
    assert torch.equal(out[~mine], clean[~mine])
    assert torch.equal(lse[~mine], clean_lse[~mine])


@pytest.mark.parametrize("value", [NAN, MINUS_INF])
def test_prompt_in_the_largest_blocks(value):
    """As many rows and heads as take blocks of eight waves."""
    c = prompt(64, 16, [8300], 0.005)
    c.k = scaled(c.k[::-1], np.ones(8300))  # the largest in the oldest tiles
    clean, clean_lse = (t.clone() for t in c.run(scale=1.0))
    assert bool(torch.isfinite(clean).all())
    for r in (33, 4099, 8299):
        spoil(c.q[r, 3], value)
    out, lse = c.run(scale=1.0)
    mine = torch.zeros(8300, 16, dtype=torch.bool, device=of_prompt.DEV)
    mine[[33, 4099, 8299], 3] = True
    expect(out[mine], lse[mine], value, "the spoilt rows")
    assert torch.equal(out[~mine], clean[~mine]) and torch.equal(lse[~mine], clean_lse[~mine])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv,new", [(8, 2, 1), (4, 2, 5), (4, 1, 16)])
@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("value", [NAN, INF, MINUS_INF])
def test_cache(dim, heads, kv, new, window, value):
    c = of_cache.Case([1500, 1499, 60], new, heads, kv, dim, 64, seed=22)
    size = np.ones(len(c.k))
    for i, n in enumerate(c.lengths):
        p = np.arange(n)
        at = c.table[i, p // c.page].astype(np.int64) * c.page + p % c.page
        size[at] = (p if i == 0 else n - p) / 20 + 0.1
    c.k = scaled(c.k, size)
    c.k[:, :, :32] &= 0x7FFF
    c.k[:, :, 0] = np.maximum(c.k[:, :, :32].max(-1), 0x3F80)  # coded to a number above 0: no 0 times infinity
    cache = c.cache()
    clean, clean_lse = (t.clone() for t in c.run(cache, scale=1.0, window=window))
    assert bool(torch.isfinite(clean).all())
    mine = torch.zeros(3, new, heads, dtype=torch.bool, device=of_cache.DEV)
    for seq, i, h in ((0, 0, 1), (1, new - 1, heads - 1), (2, new // 2, 0)):
        spoil(c.q[seq, i, h], value)
        mine[seq, i, h] = True
    out, lse = c.run(cache, scale=1.0, window=window)
    expect(out[mine], lse[mine], value, "the spoilt queries")
    assert torch.equal(out[~mine], clean[~mine]) and torch.equal(lse[~mine], clean_lse[~mine])
