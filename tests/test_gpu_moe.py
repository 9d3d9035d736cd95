"""The mixture-of-experts layer on the GPU against its definition in 64 bits
(tests/fp4_ref.py): the same experts, weights and outputs within what 32-bit
sums and the two BF16 roundings may be off by."""
import numpy as np
import pytest

import synth
from tests import fp4_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402

DEV = "cuda:0"


def bits(rng, *shape, sigma=1.0):
    return synth.bf16_bits((rng.standard_normal(shape) * sigma).astype(np.float32))


def dev16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(DEV)


class Layer:
    """Seeded weights of one layer, on the device and as float64."""

    def __init__(self, T, H, I, E, kinds=("bf16", "bf16"), seed=0, rows=1.0):
        rng = np.random.default_rng([seed, T, H, I, E])
        self.x = bits(rng, T, H)
        self.router = bits(rng, E, H, sigma=1 / np.sqrt(H))
        self.w = [bits(rng, E, 2 * I, H, sigma=rows / np.sqrt(H)), bits(rng, E, H, I, sigma=rows / np.sqrt(I))]
        self.kinds = kinds

    def device(self):
        out = [dev16(self.x), dev16(self.router)]
        for w, kind in zip(self.w, self.kinds):
            out.append(wc.fp4_encode(dev16(w)) if kind == "fp4" else dev16(w))
        return out

    def real(self):
        out = [fp4_ref.of_bits(self.x), fp4_ref.of_bits(self.router)]
        for w, kind in zip(self.w, self.kinds):
            if kind == "fp4":
                q = fp4_ref.encode(w.reshape(-1, w.shape[-1]))
                out.append(fp4_ref.values(*q, w.shape[-1]).reshape(w.shape))
            else:
                out.append(fp4_ref.of_bits(w))
        return out


SCORING = {"softmax": wc.SOFTMAX, "sigmoid": wc.SIGMOID}


def check(layer, k, scoring="softmax", bias=None, renorm=True, scale=1.0):
    d = layer.device()
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).to(DEV)
    T, H = layer.x.shape
    E, _, I = layer.w[1].shape
    work = torch.full((wc.moe_workspace_bytes(T, H, I, E, k),), 0xFF, dtype=torch.uint8, device=DEV)
    room = torch.full((T * H + 16,), 5.0, dtype=torch.bfloat16, device=DEV)
    y, ids, weights = wc.moe(*d, k, scoring=SCORING[scoring], bias=b, renorm=renorm, scale=scale,
                             work=work, out=room[:T * H].view(T, H))
    torch.cuda.synchronize()
    assert bool((room[T * H:] == 5.0).all()), "written past y"
    ry, bound, rids, rw, wrel, gap = fp4_ref.moe(
        *layer.real(), k, scoring, None if bias is None else bias.astype(np.float32).astype(np.float64),
        renorm, scale)
    assert gap > 1, "the seed gives a choice that 32 bits do not settle"
    assert np.array_equal(ids.cpu().numpy(), rids)
    werr = np.abs(weights.cpu().numpy().astype(np.float64) - rw)
    assert (werr <= wrel[:, None] * np.abs(rw)).all(), f"weights: {werr.max():.3g}"
    err = np.abs(y.double().cpu().numpy() - ry)
    assert (err <= bound).all(), f"y: {np.max(err / np.where(bound > 0, bound, 1)):.3g} of the bound"
    return y, ids, weights


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 31, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("fp4", "fp4")])
def test_tokens(T, kinds):
    check(Layer(T, 256, 96, 12, kinds), 3)


@pytest.mark.parametrize("H,I", [(1, 1), (8, 5), (31, 33), (32, 16), (100, 72), (127, 129), (128, 128),
                                 (130, 17), (1000, 264), (1031, 40), (2048, 200)])
@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("fp4", "fp4"), ("fp4", "bf16"), ("bf16", "fp4")])
def test_sizes(H, I, kinds):
    check(Layer(5, H, I, 6, kinds, seed=2), 2)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (2, 2), (16, 16), (17, 5), (64, 6), (65, 8), (128, 8),
                                 (129, 4), (200, 16), (512, 16)])
def test_experts(E, k):
    check(Layer(4, 64, 32, E, seed=3), k)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_scoring(scoring, renorm, with_bias):
    bias = np.random.default_rng(8).standard_normal(24) * 0.3 if with_bias else None
    check(Layer(9, 192, 64, 24, ("fp4", "fp4"), seed=22), 5, scoring, bias, renorm, 2.5)


@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("fp4", "fp4")])
def test_ordinary_layer(kinds):
    check(Layer(9, 1024, 512, 32, kinds, seed=5), 4)


def test_all_tokens_choose_the_same_experts():
    bias = np.full(10, 0.0)
    bias[[2, 7]] = 2.0
    for T in (16, 17, 40, 64):
        _, ids, _ = check(Layer(T, 128, 48, 10, seed=22), 2, bias=bias)
        assert bool(((ids == 2) | (ids == 7)).all())


@pytest.mark.parametrize("T,H,I,k", [(9, 20000, 20, 2), (4, 65536, 8, 1), (64, 8200, 24, 2), (33, 4104, 72, 3),
                                     (1, 12000, 40, 1)])
@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("fp4", "fp4")])
def test_wide_inputs(T, H, I, k, kinds):
    """Inputs of which only some tokens' fit the LDS of a block at a time."""
    check(Layer(T, H, I, 3, kinds, seed=30), k)


@pytest.mark.parametrize("T,H,I", [(64, 96, 700), (30, 520, 1300), (8, 40, 4100), (64, 5000, 48)])
@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("fp4", "fp4"), ("fp4", "bf16"), ("bf16", "fp4")])
def test_long_second_products(T, H, I, kinds):
    """Few and many output rows, each with a long sum over the chosen experts."""
    check(Layer(T, H, I, 8, kinds, seed=30), 4)


def test_ties_go_to_the_lowest_index():
    layer = Layer(6, 160, 32, 70, seed=7)
    layer.router[:] = layer.router[3]  # every logit of a token is the same
    _, ids, weights = check(layer, 4)
    assert ids.cpu().tolist() == [[0, 1, 2, 3]] * 6
    layer = Layer(6, 160, 32, 70, seed=7)
    layer.router[66] = layer.router[2]
    check(layer, 70 - 54)


def test_masked_experts_and_tokens_without_any():
    layer = Layer(19, 128, 64, 9, seed=8)
    bias = np.full(9, -np.inf)
    y, ids, weights = check(layer, 3, bias=bias)
    assert bool((y == 0).all()) and bool((ids == -1).all()) and bool((weights == 0).all())
    bias[[4, 6]] = [0.1, -0.2]  # two experts for three places
    y, ids, weights = check(layer, 3, bias=bias)
    assert bool((ids[:, 2] == -1).all()) and bool((weights[:, 2] == 0).all())
    check(layer, 3, "sigmoid", bias=bias, renorm=False)


def test_weights_that_vanish():
    """Sigmoid scores that underflow to 0: their sum is 0 and so is y."""
    layer = Layer(2, 64, 32, 4, seed=9)
    layer.x[:] = synth.bf16_bits(np.full(layer.x.shape, 16.0, dtype=np.float32))
    layer.router[:] = synth.bf16_bits(np.full(layer.router.shape, -1.0, dtype=np.float32))
    y, ids, weights = wc.moe(*layer.device(), 2, scoring=wc.SIGMOID)
    assert ids.cpu().tolist() == [[0, 1]] * 2
    assert bool((weights == 0).all()) and bool((y == 0).all())


@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("fp4", "fp4")])
def test_infinities_and_nan_stay_where_they_belong(kinds):
    """A NaN token gives a NaN row, an expert with infinities spoils the tokens
    that chose it; every other row keeps its bits."""
    T, k = 40, 2
    layer = Layer(T, 256, 64, 8, kinds, seed=10)
    clean, ids, _ = wc.moe(*layer.device(), k)
    layer.x[11, 3] = 0x7FC0
    layer.w[0][5, 9, 17] = 0x7F80
    layer.w[1][6, 30, 2] = 0xFF80
    y, ids2, w2 = wc.moe(*layer.device(), k)
    assert bool(torch.isnan(y[11]).all()) and bool(torch.isnan(w2[11]).all())
    chose = (ids == 5).any(1) | (ids == 6).any(1)
    other = ~chose
    other[11] = False
    assert int(other.sum()) > 4 and int(chose.sum()) > 4
    keep = torch.arange(T, device=DEV) != 11
    assert torch.equal(ids[keep], ids2[keep])
    assert torch.equal(y[other], clean[other])
    assert not bool(torch.isfinite(y[(ids == 6).any(1)][:, 30]).any())


def test_offsets_past_32_bits():
    """A stack of more than 2^32 weights, with everything in its last experts."""
    E, H, I = 260, 4096, 2048
    gu = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device=DEV)
    dn = torch.zeros((E, H, I), dtype=torch.bfloat16, device=DEV)
    assert gu.numel() > 1 << 32
    gu[E - 1, I - 1, H - 1] = 2.0          # gate row I - 1
    gu[E - 1, 2 * I - 1, H - 1] = 3.0      # its up row
    dn[E - 1, H - 1, I - 1] = 1.0
    x = torch.zeros((2, H), dtype=torch.bfloat16, device=DEV)
    x[:, H - 1] = torch.tensor([1.0, 4.0])
    bias = torch.zeros(E, device=DEV)
    bias[E - 2:] = 1.0
    y, ids, w = wc.moe(x, torch.zeros((E, H), dtype=torch.bfloat16, device=DEV), gu, dn, 2, bias=bias)
    assert ids.cpu().tolist() == [[E - 2, E - 1]] * 2
    g = torch.tensor([2.0, 8.0], dtype=torch.float64)
    ref = 0.5 * g * torch.sigmoid(g) * torch.tensor([3.0, 12.0], dtype=torch.float64)
    err = (y[:, H - 1].double().cpu() - ref).abs()
    assert bool((err <= 2.1 * fp4_ref.U16 * ref).all())  # two roundings to BF16
    assert int((y != 0).sum()) == 2


@pytest.mark.parametrize("T", [1, 20, 64])
def test_repeats_its_bits_on_streams_and_in_graphs(T):
    layer = Layer(T, 512, 160, 16, ("fp4", "fp4"), seed=11)
    d = layer.device()
    ref = [v.clone() for v in wc.moe(*d, 4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = wc.moe(*d, 4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    work = torch.empty(wc.moe_workspace_bytes(T, 512, 160, 16, 4), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(ref[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, ids, weights = wc.moe(*d, 4, work=work, out=out)
    for _ in range(4):
        d[0].copy_(d[0].flip(1))
        ref = wc.moe(*d, 4)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, ids, weights), ref))
