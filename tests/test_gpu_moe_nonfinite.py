"""The mixture-of-experts layer at the ends of the number range: activations
past BF16's largest number, and infinite weights of the second product."""
import math

import numpy as np
import pytest

from tests import fp4_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402

DEV = "cuda:0"
H, I = 64, 48


def layer(kind, gates, ups, down):
    """One expert that every token chooses with weight 1, whose activation j of
    token t is silu(gates[t]) * ups[t] for j = 5 and 0 for every other j."""
    x = torch.zeros(len(gates), H, dtype=torch.bfloat16, device=DEV)
    x[:, 3] = torch.tensor(gates, dtype=torch.float64).to(torch.bfloat16)
    x[:, 40] = torch.tensor(ups, dtype=torch.float64).to(torch.bfloat16)
    gu = torch.zeros(1, 2 * I, H, dtype=torch.bfloat16, device=DEV)
    gu[0, 5, 3] = 1.0
    gu[0, I + 5, 40] = 1.0
    router = torch.zeros(1, H, dtype=torch.bfloat16, device=DEV)
    if kind == "fp4":
        gu = wc.fp4_encode(gu)
    y, ids, weights = wc.moe(x, router, gu, down, 1)
    assert bool((ids == 0).all()) and bool((weights == 1).all())
    return y.double().cpu().numpy(), x.double().cpu().numpy()


def silu(v):
    return v / (1 + np.exp(-v))


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("T", [1, 8, 9, 33])
def test_finite_activations_past_bf16(kind, T):
    """159/128 2^63 * 206/128 2^64 = 1.99915 * 2^127 is a float, but rounds to
    infinity in BF16; half and a quarter of it are finite there."""
    a, b = 159 / 128 * 2.0 ** 63, 206 / 128 * 2.0 ** 64
    sign = [1.0 if t % 3 else -1.0 for t in range(T)]
    down = torch.zeros(1, H, I, dtype=torch.bfloat16, device=DEV)
    down[0, 7, 5], down[0, 21, 5] = 0.5, -0.25
    y, _ = layer(kind, [a] * T, [b * s for s in sign], wc.fp4_encode(down) if kind == "fp4" else down)
    v = a * b * np.array(sign)  # silu(a) = a this far out
    ref = np.zeros((T, H))
    ref[:, 7], ref[:, 21] = 0.5 * v, -0.25 * v
    # the activation's two parts, y's rounding, and a few fp32 operations
    tol = 2.0 ** -16 + fp4_ref.U16 + 16 * fp4_ref.U32
    assert np.isfinite(y).all()
    assert (np.abs(y - ref) <= tol * np.abs(ref)).all()


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("T", [1, 8, 9, 33])
def test_infinite_second_weights(kind, T):
    """An infinite weight times an activation is an infinity of their sign,
    whether the activation's low part is positive, 0 or negative, and NaN only
    where the activation is 0; the other outputs do not notice."""
    rng = np.random.default_rng(T)
    gates = (rng.integers(1, 65, T) / 8.0).tolist()
    ups = (rng.integers(1, 65, T) / 8.0 * rng.choice([-1.0, 1.0], T)).tolist()
    if T > 8:
        ups[4] = 0.0
    if T > 1:
        gates[2], ups[2] = 40.0, 2.0  # 80: the low part is 0
    down = torch.zeros(1, H, I, dtype=torch.bfloat16, device=DEV)
    down[0, 7, 5], down[0, 21, 5], down[0, 30, 5] = math.inf, -math.inf, 1.5
    if kind == "fp4":
        q = wc.fp4_encode(torch.where(torch.isinf(down), torch.sign(down) * 6.0, down))
        q.scales[0, 7, 0] = 254   # 6 * 2^127
        q.scales[0, 21, 0] = 253  # -6 * 2^126
        down = q
        back = wc.fp4_decode(q)
        assert bool(torch.isinf(back[0, [7, 21], 5]).all())
    y, x = layer(kind, gates, ups, down)
    v = silu(x[:, 3]) * x[:, 40]
    for row, w in ((7, 1.0), (21, -1.0)):
        for t in range(T):
            if v[t] == 0:
                assert math.isnan(y[t, row])
            else:
                assert y[t, row] == math.copysign(math.inf, w * v[t]), (t, row, v[t], y[t, row])
    tol = 2.0 ** -16 + fp4_ref.U16 + 16 * fp4_ref.U32
    assert (np.abs(y[:, 30] - 1.5 * v) <= tol * np.abs(1.5 * v)).all()
    rest = np.delete(y, [7, 21, 30], 1)
    assert (rest == 0).all()
