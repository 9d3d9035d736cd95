"""Log probabilities, entropy and top alternatives on the GPU against their
definition in 64 bits.

What 32 bits may be off by: an exponent x - m is off by half a step of itself and
its product with log2(e) by two of them, the exponential by two steps, a sum of n
terms by a step for each addition that a term goes through (n / 256 in a lane and
fewer than 64 where lanes, waves and parts are joined, each with a factor of its
own).  Terms are positive, so that the sum's relative error is that of its terms:
U (4 |x - m| + n / 64 + 256) for U = 2^-24 and the terms that matter, |x - m| < 90;
weighted by p, with |x - m| exp(x - m) summed to at most log n + the entropy."""
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
U = 2.0 ** -24


def reference(x, tokens, top):
    """x float64 [rows, vocab]: logprobs, entropy, ids, alternatives, bound of them, bound of the entropy."""
    rows, n = x.shape
    with np.errstate(all="ignore"):
        m = x.max(-1, keepdims=True)
        m = np.where(m == -np.inf, 0.0, m)
        e = np.exp(x - m)
        s = e.sum(-1, keepdims=True)
        p = e / s
        lp = x - m - np.log(s)
        h = -np.where(p > 0, p * lp, 0.0).sum(-1)
        spread = np.where(e > 0, p * np.abs(x - m), 0.0).sum(-1)
    lp[np.isneginf(x)] = -np.inf
    h[(s == 0)[:, 0]] = 0.0
    rel = U * (4 * spread + n / 64 + 256)                       # of s, and of the sum of u exp(u)
    bound = rel[:, None] + 4 * U * (np.abs(lp) + np.abs(np.where(np.isfinite(x), x - m, 0.0)) + 1)
    hb = 2 * rel * (1 + spread) + 8 * U * (np.abs(h) + spread + 1)
    got = np.array([lp[r, t] if 0 <= t < n else np.nan for r, t in enumerate(tokens)])
    gb = np.array([bound[r, t] if 0 <= t < n else 0 for r, t in enumerate(tokens)])
    ids = np.full((rows, top), -1)
    best, bb = np.full((rows, top), -np.inf), np.zeros((rows, top))
    for r in range(rows):
        left = np.flatnonzero(~np.isneginf(x[r]))
        left = left[np.lexsort((left, -x[r, left]))][:top]
        ids[r, :len(left)], best[r, :len(left)], bb[r, :len(left)] = left, lp[r, left], bound[r, left]
    return got, gb, h, hb, ids, best, bb


def near(got, ref, bound, what):
    got = got.double().cpu().numpy()
    ref = np.where(np.abs(ref) >= 2.0 ** 128, np.copysign(np.inf, ref), ref)  # past fp32: its infinity
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= bound) & ~same
    assert not bad.any(), (f"{what}: first at {tuple(np.argwhere(bad)[0])}: {got[bad][0]} for {ref[bad][0]}, bound "
                           f"{bound[bad][0]}")


def check(x, tokens, top, **more):
    """x: a device tensor of fp32 or BF16."""
    t = torch.as_tensor(tokens, dtype=torch.int64, device=DEV)
    lp, h, ids, best = wc.token_logprobs(x, t, top, **more)
    torch.cuda.synchronize()
    rlp, lb, rh, hb, rids, rbest, bb = reference(x.double().cpu().numpy(), t.tolist(), top)
    assert np.array_equal(ids.cpu().numpy(), rids)
    near(lp, rlp, lb, "logprobs")
    near(h, rh, hb, "entropy")
    near(best, rbest, bb, "top logprobs")
    return lp, h, ids, best


def logits(rows, vocab, kind, seed=0, sigma=2.5):
    rng = np.random.default_rng([seed, rows, vocab])
    x = torch.from_numpy((rng.standard_normal((rows, vocab)) * sigma).astype(np.float32)).to(DEV)
    return (x if kind == "f32" else x.bfloat16()), rng.integers(0, vocab, rows)


KINDS = ["f32", "bf16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 63, 64, 65, 1000, 1023, 1024, 1025, 4095, 4096, 4097, 5003, 8192, 50001])
def test_sizes(vocab, kind):
    for rows, top in ((1, 5), (3, 20), (2, 0)):
        check(*logits(rows, vocab, kind), top)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("top", [0, 1, 2, 5, 16, 20, 31, 32])
def test_tops(top, kind):
    check(*logits(4, 32000, kind, seed=1), top)
    check(*logits(300, 2500, kind, seed=2), top)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [1, 2, 5, 64, 255, 1023, 1024, 1025, 3000])
def test_rows(rows, kind):
    """Every number of parts that a row is split into."""
    check(*logits(rows, 4500, kind, seed=3), 4)
    if rows < 100:
        check(*logits(rows, 100003, kind, seed=4), 8)
        check(*logits(rows, 140001, kind, seed=4), 8)


@pytest.mark.parametrize("kind", KINDS)
def test_ties_go_to_the_lowest_index(kind):
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    for rows, vocab in ((2, 20000), (1500, 3000), (1, 70), (600, 9000), (2, 140000)):
        x = torch.zeros(rows, vocab, dtype=dtype, device=DEV)
        check(x, [vocab - 1] * rows, 20)
        x[:, 1::2] = -0.0  # equal to 0
        check(x, [1] * rows, 20)
        x[:, vocab // 2:] = 1.0
        check(x, [0] * rows, 32)
        x = torch.arange(vocab, device=DEV).remainder(7).to(dtype).expand(rows, -1).contiguous()
        check(x, [3] * rows, 32)
        # rising and falling values: every batch, or only the first, has better ones
        x = (torch.arange(vocab, device=DEV) // 40).float().div(64).to(dtype).expand(rows, -1).contiguous()
        check(x, [3] * rows, 32)
        check(x.flip(1), [3] * rows, 32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("top", [1, 20, 32])
def test_rising_rows(kind, top):
    """Every batch of a row holds more values above the list's least than there is room for."""
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    for rows, vocab in ((2, 50003), (1200, 20000)):
        g = torch.Generator().manual_seed(top)
        at = torch.arange(vocab).float().div(vocab).expand(rows, -1)
        noise = torch.randn(rows, vocab, generator=g)
        for x in (12 * at, 12 * at + noise / 64, 12 * at + noise, 6 * at * noise,
                  torch.where(torch.arange(vocab) % 3 == 0, 12 * at, float("-inf"))):
            check(x.to(dtype).to(DEV), [vocab - 2] * rows, top)


@pytest.mark.parametrize("kind", KINDS)
def test_masked_tokens(kind):
    for rows, vocab in ((3, 20000), (1500, 3000)):
        x, tokens = logits(rows, vocab, kind, seed=5)
        x[:, : vocab // 2] = -float("inf")
        x[1, :] = -float("inf")        # nothing left
        x[2, :] = -float("inf")
        x[2, [7, vocab - 1]] = torch.tensor([1.0, 3.0], dtype=x.dtype, device=DEV)
        tokens[:3] = [5, 5, 7]
        lp, h, ids, best = check(x, tokens, 6)
        assert lp[1] == -float("inf") and h[1] == 0 and ids[1].tolist() == [-1] * 6
        assert ids[2].tolist() == [vocab - 1, 7, -1, -1, -1, -1]


@pytest.mark.parametrize("kind", KINDS)
def test_the_lowest_numbers_as_a_mask(kind):
    x, tokens = logits(3, 9000, kind, seed=6)
    low = torch.finfo(x.dtype).min
    x[0, 100:] = low
    x[1, :] = low  # all equal
    x[2, :] = low
    x[2, 8999] = torch.finfo(x.dtype).max
    tokens[:] = [50, 8999, 8999]
    lp, h, ids, _ = check(x, tokens, 5)
    assert ids[1].tolist() == [0, 1, 2, 3, 4] and lp[2] == 0 and h[2] == 0


@pytest.mark.parametrize("kind", KINDS)
def test_nan_and_infinity(kind):
    for rows, vocab in ((4, 20000), (1500, 3000)):
        x, tokens = logits(rows, vocab, kind, seed=7)
        clean = [t.clone() for t in wc.token_logprobs(x, torch.as_tensor(tokens, device=DEV), 5)]
        order = torch.sort(x[:3].float(), dim=-1, descending=True, stable=True).indices
        x[0, [vocab - 3, 40]] = float("nan")
        x[1, 2000] = float("inf")
        x[2, :] = float("nan")
        lp, h, ids, best = wc.token_logprobs(x, torch.as_tensor(tokens, device=DEV), 5)
        assert bool(torch.isnan(lp[:3]).all()) and bool(torch.isnan(h[:3]).all()) and bool(torch.isnan(best[:3]).all())
        rest = [i for i in order[0].tolist() if i not in (vocab - 3, 40)]
        assert ids[0].tolist() == [40, vocab - 3] + rest[:3]
        assert ids[1].tolist() == [2000] + [i for i in order[1].tolist() if i != 2000][:4]
        assert ids[2].tolist() == [0, 1, 2, 3, 4]
        assert all(torch.equal(a[3:], b[3:]) for a, b in zip((lp, h, ids, best), clean))


@pytest.mark.parametrize("kind", KINDS)
def test_certain_and_even_rows(kind):
    """One token that is all but certain, and a row in which all are alike."""
    x, _ = logits(2, 30000, kind, seed=8, sigma=1.0)
    x[0, 777] = 60.0
    x[1] = 4.0
    lp, h, _, _ = check(x, [777, 9], 3)
    # 30000 tokens of about exp(-60) sqrt(e), each times 60: 2.6e-20, which log s - w / s keeps
    assert 2e-20 < h[0] < 4e-20


@pytest.mark.parametrize("kind", KINDS)
def test_strides_and_odd_starts(kind):
    x, tokens = logits(5, 7001, kind, seed=9)
    want = check(x, tokens, 7)
    wide = torch.full((5, 7100), float("nan"), dtype=x.dtype, device=DEV)
    for at in (0, 1, 3, 99):
        part = wide[:, at:at + 7001]
        wide.fill_(float("nan"))
        part.copy_(x)
        got = wc.token_logprobs(part, torch.as_tensor(tokens, device=DEV), 7)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_tokens_outside_the_vocabulary():
    x, tokens = logits(4, 3000, "f32", seed=10)
    tokens[:] = [-1, 3000, 1 << 40, 5]
    lp, *_ = check(x, tokens, 2)
    assert torch.isnan(lp).tolist() == [True, True, True, False]


def test_no_rows():
    x = torch.zeros(0, 100, device=DEV)
    lp, h, ids, best = wc.token_logprobs(x, torch.zeros(0, dtype=torch.int64, device=DEV), 3)
    assert lp.shape == h.shape == (0,) and ids.shape == best.shape == (0, 3)


def test_offsets_past_32_bits():
    rows, stride = 70, 1 << 25
    x = torch.empty(rows * stride, dtype=torch.bfloat16, device=DEV)
    part = x.view(rows, stride)[:, -3000:]
    src, tokens = logits(rows, 3000, "bf16", seed=11)
    part.copy_(src)
    assert (rows - 1) * stride * 2 > 1 << 32
    got = wc.token_logprobs(part, torch.as_tensor(tokens, device=DEV), 4)
    want = check(src, tokens, 4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_workspace_of_the_callers():
    x, tokens = logits(3, 40000, "f32", seed=12)
    x, tokens = logits(3, 140000, "f32", seed=12)
    need = wc.token_logprobs_workspace_bytes(3, 140000, 9)
    assert need > 0
    work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    check(x, tokens, 9, work=work)
    assert bool((work[need:] == 0xFF).all())
    assert wc.token_logprobs_workspace_bytes(3000, 40000, 9) == 0


@pytest.mark.parametrize("rows,vocab", [(3, 9001), (1200, 9001), (2, 150001)])
def test_repeats_its_bits_on_streams_and_in_graphs(rows, vocab):
    x, tokens = logits(rows, vocab, "f32", seed=13)
    t = torch.as_tensor(tokens, device=DEV)
    ref = [v.clone() for v in wc.token_logprobs(x, t, 6)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = wc.token_logprobs(x, t, 6, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = wc.token_logprobs(x, t, 6)
    for i in range(4):
        x.copy_(x.roll(1, 0) * 1.1)
        g.replay()
        torch.cuda.synchronize()
        want = wc.token_logprobs(x, t, 6)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
