"""The 4-bit cache and the attention over it on the GPU, against their
definitions in 64 bits (tests/attn_ref.py, tests/fp4_ref.py)."""
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
    """float64 of a device tensor of BF16 (or its bits)."""
    return t.view(torch.bfloat16).double().cpu().numpy()


# ---- append and read-back ----------------------------------------------------

@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("heads,page", [(1, 32), (3, 64), (8, 96), (2, 256)])
def test_append_and_read(dim, heads, page):
    rng = np.random.default_rng([dim, heads, page])
    pages, n = 5, 77
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    k, v = bits(rng, n, heads, dim), bits(rng, n, heads, dim, sigma=100.0)
    cache = wc.fp4_cache(pages, page, heads, dim, DEV)
    before = cache.clone()
    at = torch.from_numpy(slots).to(DEV)
    wc.fp4_cache_append(cache, dev16(k), dev16(v), at)
    for got, src in zip(wc.fp4_cache_read(cache, at), (k, v)):
        assert np.array_equal(of(got), attn_ref.held(src))
    # everything else is as it was
    rest = np.setdiff1d(np.arange(pages * page), slots)
    for got in wc.fp4_cache_read(cache, torch.from_numpy(rest).to(DEV)):
        assert bool((got == 0).all())
    wc.fp4_cache_append(cache, torch.zeros_like(dev16(k)), torch.zeros_like(dev16(v)), at)
    # zero rows have the smallest scale, 1; the rest of a tile keeps its bytes
    assert int((cache != before).sum()) == int((cache == 1).sum()) == 2 * n * heads * dim // 32


@pytest.mark.parametrize("kind", ["normal", "uniform", "wide"])
def test_append_rounds_as_the_encoder(kind):
    """Every kind of group: infinities, NaN, subnormals, the largest numbers."""
    n, heads, dim = 64, 2, 128
    w = [synth.random_bits(n * heads * dim, 3 + i, kind if kind != "wide" else "uniform").reshape(n, heads, dim)
         for i in range(2)]
    if kind == "wide":
        for x in w:
            x[::3] &= 0x807F  # subnormals
            x[1::3] = (x[1::3] & 0x807F) | 0x7F00  # next to the largest
    cache = wc.fp4_cache(2, 32, heads, dim, DEV)
    slots = torch.arange(n, device=DEV)
    wc.fp4_cache_append(cache, dev16(w[0]), dev16(w[1]), slots)
    for got, src in zip(wc.fp4_cache_read(cache, slots), w):
        q = wc.fp4_encode(dev16(src).view(-1, dim))
        want = wc.fp4_decode(q).view(n, heads, dim)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_append_takes_slices_and_leaves_out_slots():
    rng = np.random.default_rng(5)
    n, heads, dim, page = 41, 4, 64, 32
    fused = dev16(bits(rng, n, 10, dim))
    k, v = fused[:, 2:6], fused[:, 6:]
    slots = torch.arange(n, device=DEV) + 7
    slots[[0, 5, 40]] = torch.tensor([-1, 3 * page, 1 << 62], device=DEV)
    cache = wc.fp4_cache(3, page, heads, dim, DEV)
    guard = torch.full((cache.numel() + 8192,), 7, dtype=torch.uint8, device=DEV)
    inside = guard[4096:4096 + cache.numel()].view(cache.shape)
    inside.zero_()
    wc.fp4_cache_append(inside, k, v, slots)
    assert bool((guard[:4096] == 7).all()) and bool((guard[4096 + cache.numel():] == 7).all())
    gk, gv = wc.fp4_cache_read(inside, slots)
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[[0, 5, 40]] = False
    for got, src in ((gk, k), (gv, v)):
        want = attn_ref.held(src.cpu().numpy().view(np.uint16))
        assert np.array_equal(of(got[keep]), want[keep.cpu().numpy()])
        assert bool(torch.isnan(got[~keep]).all())
    one = wc.fp4_cache_read(inside, slots[1:2])
    assert torch.equal(one[0], gk[1:2]) and torch.equal(one[1], gv[1:2])
    assert wc.fp4_cache_read(inside, slots[:0])[0].shape == (0, heads, dim)
    wc.fp4_cache_append(inside, k[:0], v[:0], slots[:0])


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("heads,tokens", [(16, 700), (3, 130), (1, 40)])
def test_append_runs_of_slots(dim, heads, tokens):
    """Runs of slots of any length from any place on, in order, falling, and with gaps
    and unused places between: whole aligned fours and parts of them."""
    rng = np.random.default_rng([dim, heads, tokens])
    page, pages = 64, 40
    free = list(rng.permutation(pages))
    slots = []
    while len(slots) < tokens:
        n, at = int(rng.integers(1, 40)), int(rng.integers(0, 25))
        run = free.pop() * page + at + np.arange(n)
        kind = rng.integers(0, 5)
        run = run[::-1] if kind == 0 else run[rng.random(n) < 0.8] if kind == 1 else run
        slots += run.tolist() + [-1] * int(rng.integers(0, 3) if kind == 2 else 0)
    slots = np.array(slots[:tokens], dtype=np.int64)
    k, v = bits(rng, tokens, heads, dim), bits(rng, tokens, heads, dim)
    cache = wc.fp4_cache(pages, page, heads, dim, DEV)
    at = torch.from_numpy(slots).to(DEV)
    wc.fp4_cache_append(cache, dev16(k), dev16(v), at)
    real = slots >= 0
    for got, src in zip(wc.fp4_cache_read(cache, at), (k, v)):
        assert np.array_equal(of(got)[real], attn_ref.held(src)[real])
        assert np.isnan(of(got)[~real]).all()
    rest = torch.from_numpy(np.setdiff1d(np.arange(pages * page), slots)).to(DEV)
    for got in wc.fp4_cache_read(cache, rest):
        assert bool((got == 0).all())
    # one by one, the same bytes
    other = wc.fp4_cache(pages, page, heads, dim, DEV)
    for part in np.array_split(np.arange(tokens), 7):
        p = torch.from_numpy(part).to(DEV)
        wc.fp4_cache_append(other, dev16(k)[p], dev16(v)[p], at[p])
    assert torch.equal(cache, other)


# ---- attention ---------------------------------------------------------------

class Case:
    def __init__(self, lengths, new=1, heads=8, kv=2, dim=128, page=32, seed=0, spare=2, width=None):
        rng = np.random.default_rng([seed, new, heads, kv, dim, page, len(lengths)])
        self.lengths, self.new, self.heads, self.kv, self.dim, self.page = lengths, new, heads, kv, dim, page
        need = [-(-max(0, n) // page) for n in lengths]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(lengths), max([1] + need) if width is None else width), -7, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        shape = (self.pages * page, kv, dim)
        self.k, self.v = bits(rng, *shape), bits(rng, *shape)
        self.q = bits(rng, len(lengths), new, heads, dim, sigma=1.5)

    def cache(self):
        c = wc.fp4_cache(self.pages, self.page, self.kv, self.dim, DEV)
        # what no sequence holds is all NaN
        c.fill_(255)
        slots = self.slots()
        at = torch.from_numpy(slots).to(DEV)
        wc.fp4_cache_append(c, dev16(self.k[slots]), dev16(self.v[slots]), at)
        return c

    def slots(self):
        out = [np.zeros(0, dtype=np.int64)]
        for i, n in enumerate(self.lengths):
            p = np.arange(max(0, n))
            out.append(self.table[i, p // self.page].astype(np.int64) * self.page + p % self.page)
        return np.concatenate(out)

    def run(self, cache=None, **more):
        q = dev16(self.q)
        return wc.fp4_attention(q, self.cache() if cache is None else cache, torch.from_numpy(self.table).to(DEV),
                                torch.tensor(self.lengths, dtype=torch.int32, device=DEV), **more)

    def check(self, scale=None, window=0, change=None, **more):
        k, v = attn_ref.held(self.k), attn_ref.held(self.v)
        cache = self.cache()
        out, lse = self.run(cache, scale=scale, window=window, **more)
        torch.cuda.synchronize()
        out, lse = of(out), lse.cpu().numpy()
        q = fp4_ref.of_bits(self.q)
        scale = self.dim ** -0.5 if scale is None else float(np.float32(scale))
        for i, n in enumerate(self.lengths):
            p = np.arange(max(0, n))
            at = self.table[i, p // self.page].astype(np.int64) * self.page + p % self.page
            for h in range(self.heads):
                j = h // (self.heads // self.kv)
                o, ob, l, lb = attn_ref.attend(q[i, :, h], k[at, j], v[at, j], n - self.new + np.arange(self.new),
                                               scale, window, True)
                attn_ref.compare(out[i, :, h], o, ob, f"out of sequence {i} (length {n}), head {h}")
                attn_ref.compare(lse[i, :, h], l, lb, f"lse of sequence {i} (length {n}), head {h}")
        return out, lse


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("heads,kv,new", [(8, 2, 1), (4, 4, 1), (16, 1, 1), (6, 2, 4), (3, 1, 16), (10, 2, 3)])
def test_dims_and_heads(dim, heads, kv, new):
    Case([0, 1, 2, 31, 32, 33, 95, 161], new, heads, kv, dim).check()


@pytest.mark.parametrize("page", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 2, 31, 32, 33, 100, 5000])
def test_pages_and_windows(page, window):
    Case([1, 17, 64, 100, 127, 128, 129, 300], 1, 4, 1, 64, page, seed=1).check(window=window)
    Case([3, 8, 40, 290], 5, 4, 1, 64, page, seed=2).check(window=window)


@pytest.mark.parametrize("length", [500, 1500, 4095, 4096, 4097, 20000])
@pytest.mark.parametrize("new", [1, 4])
def test_long(length, new):
    Case([length, 7, length // 3], new, 4, 2, 128, 64, seed=3).check()


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("heads,kv,new", [(4, 2, 1), (3, 1, 7)])
def test_sequences_in_several_blocks(dim, heads, kv, new):
    """Sequences that are split and joined, beside one that is not and an empty one."""
    Case([2300, 0, 40, 1200], new, heads, kv, dim, 64, seed=14).check()


@pytest.mark.parametrize("seqs", [63, 64, 65, 130])
@pytest.mark.parametrize("window", [0, 2500])
def test_many_sequences_in_several_blocks(seqs, window):
    """More sequences than a wave has lanes, the long ones among the last."""
    lengths = [int(x) for x in np.random.default_rng(15).integers(0, 60, seqs)]
    lengths[-1], lengths[-3], lengths[seqs // 2] = 3000, 2600, 2200
    Case(lengths, 1, 2, 1, 32, 64, seed=15).check(window=window)


@pytest.mark.parametrize("window", [0, 700])
def test_many_sequences(window):
    lengths = [int(x) for x in np.random.default_rng(4).integers(0, 900, 70)]
    Case(lengths, 1, 4, 2, 32, 64, seed=4).check(window=window)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 1e-4])
def test_scales(scale):
    Case([70, 300], 2, 4, 2, 64, seed=5).check(scale=scale)


def test_scores_that_rise_and_fall_far():
    """Largest scores that move by hundreds, up and down, along the sequence."""
    c = Case([1500, 1499], 2, 4, 2, 64, 64, seed=6)
    size = np.ones(c.k.shape[0], dtype=np.float32)
    for i, n in enumerate(c.lengths):
        p = np.arange(n)
        at = c.table[i, p // c.page].astype(np.int64) * c.page + p % c.page
        size[at] = (p / 20 if i == 0 else (n - p) / 20) + 0.1
    c.k = synth.bf16_bits((fp4_ref.of_bits(c.k) * size[:, None, None]).astype(np.float32))
    c.check(scale=1.0)


def test_a_strided_query_and_outputs_of_the_callers():
    c = Case([65, 3, 200], 3, 4, 2, 96, 64, seed=7)
    cache = c.cache()
    want = c.run(cache)
    wide = torch.zeros(3, 3, 9, 96, dtype=torch.int16, device=DEV)
    wide[:, :, 2:6] = dev16(c.q)
    room = torch.full((3 * 3 * 4 * 96 + 64,), 5.0, dtype=torch.bfloat16, device=DEV)
    out = room[:-64].view(3, 3, 4, 96)
    table = torch.from_numpy(c.table).to(DEV)
    lengths = torch.tensor(c.lengths, dtype=torch.int32, device=DEV)
    need = wc.fp4_attention_workspace_bytes(cache, 3, 3, 4, table.shape[1])
    work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    got = wc.fp4_attention(wide[:, :, 2:6], cache, table, lengths, out=out, work=work)
    assert got[0] is out and all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((room[-64:] == 5.0).all()) and bool((work[need:] == 0xFF).all())
    # a sequence's first token alone, as three-dimensional queries
    one = wc.fp4_attention(wide[:, 2, 2:6], cache, table, lengths)
    assert torch.equal(one[0], want[0][:, 2]) and torch.equal(one[1], want[1][:, 2])


def test_no_sequences_and_no_pages():
    cache = wc.fp4_cache(1, 32, 2, 64, DEV)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = wc.fp4_attention(q[:0], cache, z(0, 3), z(0))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = wc.fp4_attention(q, cache, z(2, 0), z(2))
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    out, lse = wc.fp4_attention(q, cache, z(2, 0), z(2) - 5)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def spoil(c, cache, seq, position, what, rows):
    """NaN (an infinity in the source) as the key or value of one position."""
    slot = c.table[seq, position // c.page].astype(np.int64) * c.page + position % c.page
    k, v = c.k[slot:slot + 1].copy(), c.v[slot:slot + 1].copy()
    (k if what == "k" else v)[:, rows] = 0x7F80
    wc.fp4_cache_append(cache, dev16(k), dev16(v), torch.tensor([slot], device=DEV))


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("new,heads,kv", [(1, 4, 2), (5, 4, 2), (16, 4, 1)])
def test_nan_reaches_those_who_attend_to_it(what, window, new, heads, kv):
    """NaN at each position near the end and the window's start: queries that
    attend to it get NaN, all others keep their bits."""
    n = 130
    c = Case([n, 60], new, heads, kv, 64, seed=8)
    cache = c.cache()
    clean, clean_lse = (t.clone() for t in c.run(cache, window=window))
    places = sorted({n - 1, n - 2, n - new, max(0, n - new - 1), 100, 96, 95, 0,
                     max(0, n - new - window), max(0, n - window), max(0, n - window - 1)})
    for position in places:
        bad = c.cache()
        spoil(c, bad, 0, position, what, 0)
        out, lse = c.run(bad, window=window)
        group = heads // kv
        for i in range(new):
            p = n - new + i
            hit = position <= p and (window == 0 or position > p - window)
            for h in range(heads):
                if hit and h < group:
                    o = out[0, i, h]
                    # a NaN value spoils its group of 32 columns, a NaN key everything
                    assert bool(torch.isnan(o).all()), (position, i, h)
                    assert bool(torch.isnan(lse[0, i, h])) == (what == "k")
                else:
                    assert torch.equal(out[0, i, h], clean[0, i, h]), (position, i, h)
                    assert lse[0, i, h] == clean_lse[0, i, h]
        assert torch.equal(out[1], clean[1]) and torch.equal(lse[1], clean_lse[1])


def test_pages_outside_the_cache_give_nan():
    c = Case([130, 130, 40], 4, 4, 2, 64, seed=9)
    cache = c.cache()
    clean, _ = c.run(cache)
    c.table[0, 2] = c.pages  # positions 64 .. 95
    c.table[1, 0] = -1
    out, lse = c.run(cache)
    assert bool(torch.isnan(out[:2]).all()) and bool(torch.isnan(lse[:2]).all())
    assert torch.equal(out[2], clean[2])
    # a window that starts behind them
    out, lse = c.run(cache, window=30)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())


def test_nan_in_sequences_of_several_blocks():
    """A NaN key and a NaN value in the middle of a long sequence, a page that is not
    there in another: all their queries; the third sequence keeps its bits."""
    c = Case([2500, 2500, 2400], 2, 4, 2, 64, 64, seed=16)
    clean, _ = c.run(c.cache())
    for what in ("k", "v"):
        cache = c.cache()
        spoil(c, cache, 0, 1100, what, 0)
        table = c.table.copy()
        c.table[1, 20] = c.pages + 5
        out, lse = c.run(cache)
        c.table = table
        assert bool(torch.isnan(out[0, :, :2]).all()) and torch.equal(out[0, :, 2:], clean[0, :, 2:])
        assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
        assert torch.equal(out[2], clean[2])


def test_lengths_past_the_table_give_nan():
    c = Case([64, 64], 3, 4, 2, 64, seed=10)
    cache = c.cache()
    clean, _ = c.run(cache)
    table, q = torch.from_numpy(c.table).to(DEV), dev16(c.q)
    for window in (0, 20):
        clean, _ = c.run(cache, window=window)
        out, lse = wc.fp4_attention(q, cache, table, torch.tensor([66, 64], dtype=torch.int32, device=DEV), window=window)
        assert bool(torch.isnan(out[0, 1:]).all()) and bool(torch.isnan(lse[0, 1:]).all())  # positions 64 and 65
        assert bool(torch.isfinite(out[0, 0]).all())                                        # position 63
        assert torch.equal(out[1], clean[1])
        out, lse = wc.fp4_attention(q, cache, table, torch.tensor([2 ** 31 - 1, 64], dtype=torch.int32, device=DEV),
                                    window=window)
        assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all()) and torch.equal(out[1], clean[1])


def test_offsets_past_32_bits():
    """A cache of more than 4 GiB with the sequence in its last pages."""
    page, heads, dim = 256, 8, 128
    pages = (1 << 32) // (page * heads * 34 * dim // 32) + 4
    cache = wc.fp4_cache(pages, page, heads, dim, DEV)
    assert (pages - 2) * cache[0].numel() > 1 << 32
    c = Case([300], 1, 8, 8, 128, page, seed=11, spare=0)
    at = np.array([pages - 1, pages - 2])
    p = np.arange(300)
    slots = torch.from_numpy(at[p // page] * page + p % page).to(DEV)
    src = torch.from_numpy(c.slots())
    wc.fp4_cache_append(cache, dev16(c.k)[src.to(DEV)], dev16(c.v)[src.to(DEV)], slots)
    got = wc.fp4_attention(dev16(c.q), cache, torch.tensor([at.tolist()], dtype=torch.int32, device=DEV),
                           torch.tensor([300], dtype=torch.int32, device=DEV))
    want = c.run()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("new", [1, 6])
@pytest.mark.parametrize("length", [900, 4000])
def test_repeats_its_bits_on_streams_and_in_graphs(new, length):
    c = Case([length, 33, 450], new, 8, 2, 128, 64, seed=12)
    cache = c.cache()
    ref = [t.clone() for t in c.run(cache)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.run(cache, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    q, table = dev16(c.q), torch.from_numpy(c.table).to(DEV)
    lengths = torch.tensor(c.lengths, dtype=torch.int32, device=DEV)
    k, v = dev16(c.k[:3]), dev16(c.v[:3])
    spots = torch.from_numpy(np.array([c.table[i, (n - 1) // c.page].astype(np.int64) * c.page + (n - 1) % c.page
                                       for i, n in enumerate(c.lengths)])).to(DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wc.fp4_cache_append(cache, k, v, spots)
        out, lse = wc.fp4_attention(q, cache, table, lengths)
    for i in range(4):
        k.copy_(k.flip(0))
        q.copy_(q.flip(2))
        g.replay()
        torch.cuda.synchronize()
        want = wc.fp4_attention(q, cache, table, lengths)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        other = wc.fp4_cache(c.pages, c.page, c.kv, c.dim, DEV)
        wc.fp4_cache_append(other, k, v, spots)
        for a, b in zip(wc.fp4_cache_read(cache, spots), wc.fp4_cache_read(other, spots)):
            assert torch.equal(a, b)
