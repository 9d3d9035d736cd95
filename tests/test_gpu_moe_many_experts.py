"""Mixture-of-experts layers of more than 128 experts (a wave for each token's
choice) and of rows so long that a wave of the router has several steps, at sizes
near those in use.  The seeds give choices that 32 bits settle."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_moe import Layer, check  # noqa: E402


@pytest.mark.parametrize("T,H,I,E,k,seed", [(4, 5120, 32, 256, 8, 41), (16, 1024, 64, 256, 8, 41),
                                            (64, 768, 40, 160, 4, 40)])
@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("fp4", "fp4")])
def test_softmax(T, H, I, E, k, seed, kinds):
    check(Layer(T, H, I, E, kinds, seed), k)


@pytest.mark.parametrize("T,H,I,E,k,seed", [(2, 7168, 16, 256, 8, 65), (9, 512, 48, 512, 6, 50)])
@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("fp4", "fp4")])
def test_biased_sigmoid(T, H, I, E, k, seed, kinds):
    bias = np.random.default_rng(seed).standard_normal(E) * 0.3
    bias[[1, E - 1]] = -np.inf
    _, ids, _ = check(Layer(T, H, I, E, kinds, seed), k, "sigmoid", bias)
    assert not bool(((ids == 1) | (ids == E - 1)).any())
