"""Attention of packed prompts on the GPU against its definition in 64 bits
(tests/attn_ref.py)."""
import numpy as np
import pytest

import synth
from tests import attn_ref, fp4_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402

DEV = "cuda:0"
DIMS = [32, 64, 96, 128, 160, 192, 224, 256]


def bits(rng, *shape, sigma=1.0):
    return synth.bf16_bits((rng.standard_normal(shape) * sigma).astype(np.float32))


def dev16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(DEV)


def of(t):
    return t.view(torch.bfloat16).double().cpu().numpy()


def starts_of(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)


class Case:
    def __init__(self, lengths, heads=4, kv=2, dim=64, seed=0, spare=0):
        n = sum(lengths) + spare
        rng = np.random.default_rng([seed, n, heads, kv, dim])
        self.lengths, self.heads, self.kv, self.dim = lengths, heads, kv, dim
        self.q, self.k, self.v = bits(rng, n, heads, dim, sigma=1.5), bits(rng, n, kv, dim), bits(rng, n, kv, dim)

    def run(self, **more):
        return wc.prompt_attention(dev16(self.q), dev16(self.k), dev16(self.v), starts_of(self.lengths), **more)

    def check(self, scale=None, window=0, rows=None):
        """Every row, or those of `rows` in each sequence."""
        out, lse = self.run(scale=scale, window=window)
        torch.cuda.synchronize()
        out, lse = of(out), lse.cpu().numpy()
        q, k, v = (fp4_ref.of_bits(x) for x in (self.q, self.k, self.v))
        scale = self.dim ** -0.5 if scale is None else float(np.float32(scale))
        at = 0
        for i, n in enumerate(self.lengths):
            p = np.arange(n) if rows is None else np.unique(np.clip(rows, 0, max(0, n - 1)))[:n]
            for h in range(self.heads):
                j = h // (self.heads // self.kv)
                o, ob, l, lb = attn_ref.attend(q[at + p, h], k[at:at + n, j], v[at:at + n, j], p, scale, window, False)
                attn_ref.compare(out[at + p, h], o, ob, f"out of sequence {i} (length {n}), head {h}")
                attn_ref.compare(lse[at + p, h], l, lb, f"lse of sequence {i} (length {n}), head {h}")
            at += n
        return out, lse


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("lengths", [[1], [0, 2, 0, 31, 32, 33], [63, 64, 65], [127, 1, 130], [257]])
def test_dims_and_lengths(dim, lengths):
    Case(lengths, 2, 1, dim).check()


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (6, 2), (8, 1), (16, 2), (10, 5)])
def test_heads(heads, kv):
    Case([40, 150], heads, kv, 64, seed=1).check()


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 63, 64, 65, 100, 130, 5000])
@pytest.mark.parametrize("dim", [64, 128])
def test_windows(window, dim):
    Case([5, 300, 129], 2, 1, dim, seed=2).check(window=window)


@pytest.mark.parametrize("dim", [32, 64, 128, 192, 256])
@pytest.mark.parametrize("window", [0, 500])
def test_long(dim, window):
    """Enough rows for every block shape; some rows of each sequence."""
    rows = np.array([0, 1, 31, 32, 63, 64, 100, 127, 128, 255, 256, 257, 511, 512, 1000, 1279, 1280, 1535, 2047, 2048, 4000])
    Case([4001, 1280, 2050], 2, 1, dim, seed=3).check(window=window, rows=rows)


def test_many_blocks():
    """More heads and rows than fill the card, in blocks of the largest kind."""
    rows = np.array([0, 33, 255, 256, 300, 511, 700, 1023])
    Case([1024, 1000, 700, 900, 1, 1024], 32, 8, 128, seed=4).check(rows=rows)


def test_many_sequences():
    rng = np.random.default_rng(5)
    Case([int(x) for x in rng.integers(0, 40, 200)], 2, 1, 32, seed=5).check()


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 1e-4])
def test_scales(scale):
    Case([70, 200], 2, 1, 64, seed=6).check(scale=scale)


def test_scores_that_rise_and_fall_far():
    c = Case([700, 699], 2, 1, 64, seed=7)
    size = np.concatenate([np.arange(700) / 20, np.arange(699)[::-1] / 20]) + 0.1
    c.k = synth.bf16_bits((fp4_ref.of_bits(c.k) * size[:, None, None]).astype(np.float32))
    c.check(scale=1.0)


def test_slices_and_rows_behind_the_last_sequence():
    c = Case([70, 33], 4, 2, 96, seed=8, spare=21)
    n = 70 + 33
    want = [t[:n].clone() for t in c.run()]
    wide = torch.zeros(n + 21, 10, 96, dtype=torch.int16, device=DEV)
    wide[:, 1:5], wide[:, 5:7], wide[:, 8:10] = dev16(c.q), dev16(c.k), dev16(c.v)
    room = torch.full(((n + 21) * 4 * 96 + 64,), 5.0, dtype=torch.bfloat16, device=DEV)
    out = room[:-64].view(n + 21, 4, 96)
    got, lse = wc.prompt_attention(wide[:, 1:5], wide[:, 5:7], wide[:, 8:10], starts_of(c.lengths), out=out)
    assert got is out and torch.equal(out[:n], want[0]) and torch.equal(lse[:n], want[1])
    assert bool((out[n:] == 5.0).all()) and bool((room[-64:] == 5.0).all())
    # rows before the first and behind the last of the starts
    out.fill_(5.0)
    s = torch.tensor([70, 103], dtype=torch.int32, device=DEV)
    _, lse = wc.prompt_attention(wide[:, 1:5], wide[:, 5:7], wide[:, 8:10], s, out=out)
    assert torch.equal(out[70:n], want[0][70:]) and torch.equal(lse[70:n], want[1][70:])
    assert bool((out[:70] == 5.0).all()) and bool((out[n:] == 5.0).all())


def test_starts_out_of_range_count_as_the_nearer_end():
    c = Case([50, 40], 2, 1, 64, seed=9)
    want = c.run()
    for starts in ([-7, 50, 1 << 30], [0, 50, 40, 90], [0, 50, 90, 90, 95]):
        s = torch.tensor(starts, dtype=torch.int32, device=DEV)
        got = wc.prompt_attention(dev16(c.q), dev16(c.k), dev16(c.v), s)
        # falling starts: rows 40 .. 49 belong to two sequences, and either may write them last
        own = 40 if starts[2] == 40 else 50
        assert torch.equal(got[0][:own], want[0][:own])
        if own == 50:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_tokens_and_no_sequences():
    e = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = wc.prompt_attention(e, e, e, torch.zeros(3, dtype=torch.int32, device=DEV))
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    x = torch.ones(5, 2, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(x, 3.0)
    wc.prompt_attention(x, x, x, torch.zeros(1, dtype=torch.int32, device=DEV), out=out)
    wc.prompt_attention(x, x, x, torch.zeros(4, dtype=torch.int32, device=DEV), out=out)
    assert bool((out == 3.0).all())


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("value", [0x7F80, 0xFF80, 0x7FC0])
@pytest.mark.parametrize("window,dim", [(0, 64), (40, 64), (90, 128), (0, 256)])
def test_nan_and_infinities_reach_those_who_attend_to_them(what, value, window, dim):
    c = Case([130, 60, 20], 2, 1, dim, seed=10)
    clean, clean_lse = (t.clone() for t in c.run(window=window))
    for seq, start, n in ((0, 0, 130), (1, 130, 60), (2, 190, 20)):
        for p in sorted({0, 1, n // 2, 63, 64, n - 1}):
            if p >= n:
                continue
            src = getattr(c, what)
            keep = src[start + p].copy()
            src[start + p, 0, 3] = value
            out, lse = c.run(window=window)
            src[start + p] = keep
            rows = np.arange(210) - start
            hit = torch.from_numpy((rows >= p) & (rows < n) & ((rows - p < window) if window else True)).to(DEV)
            near = (out.float() - clean.float()).abs() <= 2.1 * 2.0 ** -8 * clean.float().abs() + 2.0 ** -8
            if what == "v":
                got = out[hit][:, :, 3]
                assert bool((torch.isnan(got) if value == 0x7FC0 else torch.isinf(got)).all()), (seq, p)
                if value != 0x7FC0:
                    assert bool((torch.signbit(got) == (value == 0xFF80)).all())
                near[:, :, 3] |= hit[:, None]
                assert torch.equal(lse, clean_lse)
            else:
                near |= hit[:, None, None]
                assert torch.equal(lse[~hit], clean_lse[~hit])
                if value == 0x7FC0:
                    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[hit]).all())
            assert bool(near.all()), (seq, p, torch.nonzero(~near)[:3])


def test_all_values_not_finite():
    c = Case([100, 70], 2, 1, 64, seed=11)
    c.v[:] = 0x7FC0
    out, lse = c.run()
    assert bool(torch.isnan(out).all()) and bool(torch.isfinite(lse).all())


def test_offsets_past_32_bits():
    """Rows far apart, so that the last ones' offsets pass 2^32 bytes."""
    n, width = 300, 1 << 23
    x = torch.zeros(n * width, dtype=torch.bfloat16, device=DEV).view(n, width)
    assert (n - 1) * width * 2 > 1 << 32
    c = Case([200, 100], 2, 1, 64, seed=12)
    parts = []
    for at, src in ((width - 128, c.q), (0, c.k), (64, c.v)):
        y = x[:, at:at + src.shape[1] * 64].unflatten(1, (-1, 64))
        y.copy_(dev16(src).view(torch.bfloat16))
        parts.append(y)
    got = wc.prompt_attention(*parts, starts_of(c.lengths))
    want = c.run()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_repeats_its_bits_on_streams_and_in_graphs(dim):
    c = Case([300, 33, 450], 8, 2, dim, seed=13)
    q, k, v, s = dev16(c.q), dev16(c.k), dev16(c.v), starts_of(c.lengths)
    ref = [t.clone() for t in wc.prompt_attention(q, k, v, s)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = wc.prompt_attention(q, k, v, s, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = wc.prompt_attention(q, k, v, s)
    for i in range(4):
        q.copy_(q.flip(0))
        s[1] = 250 + 10 * i
        g.replay()
        torch.cuda.synchronize()
        want = wc.prompt_attention(q, k, v, s)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_a_first_call_that_is_captured():
    """Head dims whose blocks need more than 64 KB of LDS, first called in a graph."""
    c = Case([100, 61], 2, 1, 224, seed=14)
    q, k, v, s = dev16(c.q), dev16(c.k), dev16(c.v), starts_of(c.lengths)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = wc.prompt_attention(q, k, v, s)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = wc.prompt_attention(q, k, v, s)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
