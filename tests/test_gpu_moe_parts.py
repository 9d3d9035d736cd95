"""What the mixture-of-experts layer keeps of weight * silu(gate) * up between
its two products: the sum of two BF16 numbers, each in its place."""
import numpy as np
import pytest

from tests import fp4_ref, moe_tight

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402
from tests.test_gpu_moe import Layer  # noqa: E402

DEV = "cuda:0"
KINDS = [("bf16", "bf16"), ("fp4", "fp4"), ("fp4", "bf16"), ("bf16", "fp4")]


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 96, 12, 3), (9, 256, 96, 12, 3), (17, 130, 72, 5, 2),
                                       (40, 100, 129, 3, 1), (64, 128, 48, 8, 4), (30, 520, 700, 8, 4)])
@pytest.mark.parametrize("kinds", KINDS)
def test_within_the_bound_of_two_parts(T, H, I, E, k, kinds):
    layer = Layer(T, H, I, E, kinds, seed=22, rows=4.0)
    layer.x = fp4_ref.to_bits(moe_tight.inputs(np.random.default_rng([T, H]), T, H))
    y, ids, _ = wc.moe(*layer.device(), k)
    ref, bound, rids, gap = moe_tight.moe(*layer.real(), k)
    assert gap > 1, "the seed gives a choice that 32 bits do not settle"
    assert np.array_equal(ids.cpu().numpy(), rids)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= bound).all(), f"{np.max(err / bound):.3g} of the bound"


@pytest.mark.parametrize("counts,k", [([1], 1), ([8], 1), ([9], 1), ([17], 1), ([64], 1), ([1, 8, 9, 17, 29], 1),
                                      ([1, 8, 9, 17, 29], 2), ([16, 0, 24, 7], 1), ([16, 0, 24, 7], 2)])
@pytest.mark.parametrize("H,I", [(128, 48), (109, 37), (128, 1300), (2176, 136)])
@pytest.mark.parametrize("kinds", KINDS)
def test_high_parts_cancel(counts, k, H, I, kinds):
    """Activation j of a token is 32 (1 + m_j n 2^-12) for whole m_j and n: 32
    is its high part.  Rows of the second matrix take pairs of them with opposite
    signs, so that y is made of low parts alone, and exact.  Expert e takes the
    next counts[e] tokens; with k = 2 also those of the expert before it, at
    weights of a half each."""
    E, T = len(counts), sum(counts)
    rng = np.random.default_rng([H, I, T, k])
    A, B, C = 0, 40, 64  # columns of 1, of n, and of the experts' marks
    m = rng.integers(-3, 4, (E, I))
    gu = np.zeros((E, 2 * I, H))
    gu[:, :I, A], gu[:, I:, A], gu[:, I:, B] = 32, 1, m * 2.0 ** -12
    down = np.zeros((E, H, I))
    for e in range(E):
        for r in range(H):
            j = rng.permutation(I)[:6]
            down[e, r, j] = np.array([1, -1, 1, -1, 2, -2])
    n = rng.integers(1, 5, T)
    x, router = np.zeros((T, H)), np.zeros((E, H))
    x[:, A], x[:, B] = 1, n
    mine = np.repeat(np.arange(E), counts)
    x[np.arange(T), C + mine] = 1
    router[np.arange(E), C + np.arange(E)] = 40
    if k == 2:
        router[np.arange(E), C + (np.arange(E) + 1) % E] = 40
    dev = [torch.from_numpy(v).to(torch.bfloat16).to(DEV) for v in (x, router, gu, down)]
    for i, kind in zip((2, 3), kinds):
        if kind == "fp4":
            q = wc.fp4_encode(dev[i])
            assert torch.equal(wc.fp4_decode(q), dev[i])
            dev[i] = q
    y, ids, weights = wc.moe(*dev, k)
    ref = np.zeros((T, H))
    for t in range(T):
        chosen = sorted({int(mine[t]), int(mine[t] - 1) % E} if k == 2 else {int(mine[t])})
        assert ids[t].tolist() == chosen
        for e in chosen:
            ref[t] += down[e] @ m[e] * (n[t] * 32 * 2.0 ** -12 / k)
    assert bool((weights == 1 / k).all())
    assert (ref != 0).mean() > 0.7
    assert np.array_equal(fp4_ref.bf16_round(ref), ref)
    assert np.array_equal(y.double().cpu().numpy(), ref)
