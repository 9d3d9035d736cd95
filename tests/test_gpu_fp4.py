"""The 4-bit tier on the GPU against its definition in 64 bits
(tests/fp4_ref.py): codes and scales are equal, values read back are equal,
products are within what 32-bit sums may be off by."""
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


def dev16(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(DEV)


def guarded(shape, dtype, fill):
    """A tensor of `shape` inside a larger one, and a check that what lies
    around it still holds `fill`."""
    n = int(np.prod(shape))
    pad = 64 // dtype.itemsize
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device=DEV)

    def check():
        assert bool((buf[:pad] == fill).all()) and bool((buf[pad + n:] == fill).all()), "written outside"
    return buf[pad:pad + n].view(shape), check


def encode_guarded(bits):
    rows, cols = bits.shape
    G = fp4_ref.groups_of(cols)
    codes, c1 = guarded((rows, 16 * G), torch.uint8, 0xA5)
    scales, c2 = guarded((rows, G), torch.uint8, 0x5A)
    q = wc.fp4_encode(dev16(bits), out=wc.Fp4(codes, scales, cols))
    torch.cuda.synchronize()
    c1(), c2()
    return q


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (5, 33), (2, 63), (7, 64), (4, 129),
                                       (33, 257), (16, 4096), (65, 4100), (1000, 96)])
@pytest.mark.parametrize("kind", ["normal", "uniform"])
def test_encode_and_decode_equal_the_definition(rows, cols, kind):
    """'uniform' holds every kind of BF16 pattern: most of its groups have an
    infinity or a NaN or span the whole range."""
    bits = synth.random_bits(rows * cols, 11 * rows + cols, kind).reshape(rows, cols)
    if kind == "uniform":  # keep most groups free of exponent 255
        keep = np.random.default_rng(cols).random(bits.shape) < 0.99
        bits = np.where(keep & (bits >> 7 & 0xFF == 0xFF), bits & 0xBFFF, bits).astype(np.uint16)
    q = encode_guarded(bits)
    codes, scales = fp4_ref.encode(bits)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    out, check = guarded((rows, cols), torch.bfloat16, 1.0)
    wc.fp4_decode(q, out=out)
    torch.cuda.synchronize()
    check()
    got = fp4_ref.of_bits(out.view(torch.int16).cpu().numpy().view(np.uint16))
    np.testing.assert_array_equal(got, fp4_ref.values(codes, scales, cols))


def test_every_pattern_at_every_scale():
    """Every finite BF16 value in a group whose maximum is up to two octaves
    above it, and all-zero and smallest groups."""
    v = np.arange(1 << 16, dtype=np.uint32)
    v = v[(v >> 7 & 0xFF) != 0xFF].astype(np.uint16)
    rows = []
    for d in range(4):
        top = np.minimum((v & 0x7FFF) + (d << 7) + (37 * d), 0x7F7F).astype(np.uint16)
        g = np.zeros((v.size, 32), dtype=np.uint16)
        g[:, 5], g[:, 31], g[:, 6] = v, top, v ^ 0x8000
        rows.append(g.reshape(-1, 64))
    bits = np.concatenate([r[: r.shape[0] // 2 * 2] for r in rows])
    q = encode_guarded(bits)
    codes, scales = fp4_ref.encode(bits)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.isfinite(fp4_ref.values(codes, scales, 64)).all()


def test_decode_takes_any_codes_and_scales():
    """All 256 scales with all 16 codes: the BF16 of the value, infinite past
    the range, NaN at scale 255."""
    codes = np.tile(np.arange(16, dtype=np.uint8) | (15 - np.arange(16, dtype=np.uint8)) << 4, (256, 1))
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    out = wc.fp4_decode(wc.Fp4(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), 32))
    got = fp4_ref.of_bits(out.view(torch.int16).cpu().numpy().view(np.uint16))
    np.testing.assert_array_equal(got, fp4_ref.values(codes, scales, 32))


def test_encode_of_a_stack_is_that_of_its_matrices():
    bits = synth.random_bits(3 * 40 * 70, 3).reshape(3, 40, 70)
    q = wc.fp4_encode(dev16(bits))
    for i in range(3):
        codes, scales = fp4_ref.encode(bits[i])
        assert np.array_equal(q.codes[i].cpu().numpy(), codes)
        assert np.array_equal(q.scales[i].cpu().numpy(), scales)
    assert tuple(wc.fp4_decode(q).shape) == (3, 40, 70)


def check_gemv(rows, cols, batch, seed=0):
    rng = np.random.default_rng([seed, rows, cols, batch])
    w = synth.bf16_bits((rng.standard_normal((rows, cols)) * 0.05 *
                         np.exp(rng.standard_normal((rows, 1)))).astype(np.float32))
    x = synth.bf16_bits(rng.standard_normal((batch, cols)).astype(np.float32))
    codes, scales = fp4_ref.encode(w)
    q = wc.Fp4(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), cols)
    out, check = guarded((batch, rows), torch.float32, 7.0)
    wc.fp4_gemv(q, dev16(x), out=out)
    torch.cuda.synchronize()
    check()
    y, bound = fp4_ref.gemv(fp4_ref.values(codes, scales, cols), fp4_ref.of_bits(x))
    err = np.abs(out.cpu().numpy().astype(np.float64) - y)
    assert (err <= bound).all(), f"{(rows, cols, batch)}: {np.max(err / bound):.3g} of the bound"


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (16, 32), (17, 33), (15, 127), (16, 128),
                                       (40, 129), (64, 1000), (33, 1024), (100, 1031), (19, 4100),
                                       (256, 4096), (48, 24576)])
@pytest.mark.parametrize("batch", [1, 2, 5, 16, 17, 32, 33, 64, 65, 130, 256])
def test_gemv(rows, cols, batch):
    check_gemv(rows, cols, batch)


@pytest.mark.parametrize("rows,cols,batch", [(4096, 4096, 1), (4096, 4096, 4), (5003, 4100, 7),
                                             (1024, 14336, 16), (4097, 1056, 48), (2000, 2048, 200)])
def test_gemv_at_ordinary_sizes(rows, cols, batch):
    check_gemv(rows, cols, batch)


@pytest.mark.parametrize("rows,cols,batch", [(10300, 1000, 9), (10241, 512, 16), (10270, 8, 5), (10300, 520, 20),
                                             (10250, 520, 40), (2600, 1056, 250), (5130, 1032, 50),
                                             (5200, 648, 31), (10241, 100, 64)])
def test_gemv_of_tall_matrices(rows, cols, batch):
    """Rows and batches at which each of the taller blocks is taken, with a last
    one that is not whole."""
    check_gemv(rows, cols, batch)


def test_gemv_integers_are_exact():
    """Sums of small whole numbers are exact in fp32 whatever their order."""
    rng = np.random.default_rng(5)
    for rows, cols, batch in [(37, 100, 1), (64, 640, 20), (130, 2048, 70)]:
        w = fp4_ref.MAGS[rng.integers(0, 8, (rows, cols))] * 2 * rng.choice([-1, 1], (rows, cols))
        x = rng.integers(-8, 9, (batch, cols)).astype(np.float64)
        q = wc.fp4_encode(dev16(fp4_ref.to_bits(w)))
        got = wc.fp4_gemv(q, dev16(fp4_ref.to_bits(x))).cpu().numpy()
        ref = wc.fp4_decode(q).double().cpu().numpy()
        assert np.array_equal(got, x @ ref.T)


def test_gemv_keeps_infinities_and_nan_to_their_rows():
    rows, cols, batch = 40, 300, 18
    rng = np.random.default_rng(9)
    w = synth.random_bits(rows * cols, 4).reshape(rows, cols)
    x = synth.bf16_bits(rng.standard_normal((batch, cols)).astype(np.float32))
    clean = wc.fp4_gemv(wc.fp4_encode(dev16(w)), dev16(x)).cpu().numpy()
    w[7, 299] = 0x7F80          # a group of NaN in the last, short group of row 7
    x[3, 10], x[17, 299] = 0x7FC0, 0xFF80
    got = wc.fp4_gemv(wc.fp4_encode(dev16(w)), dev16(x)).cpu().numpy()
    assert np.isnan(got[:, 7]).all()
    assert np.isnan(got[3]).all() and not np.isfinite(got[17]).any()
    r, b = np.delete(np.arange(rows), 7), np.delete(np.arange(batch), [3, 17])
    assert np.array_equal(got[np.ix_(b, r)], clean[np.ix_(b, r)])


def test_gemv_empty_sizes():
    e = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    x = torch.empty((2, 64), dtype=torch.bfloat16, device=DEV)
    assert tuple(wc.fp4_gemv(wc.Fp4(e(0, 32), e(0, 2), 64), x).shape) == (2, 0)
    out = torch.full((2, 5), 3.0, device=DEV)
    wc.fp4_gemv(wc.Fp4(e(5, 0), e(5, 0), 0), x[:, :0].contiguous(), out=out)  # an empty sum is 0
    assert bool((out == 0).all())
    assert tuple(wc.fp4_decode(wc.fp4_encode(x[:0])).shape) == (0, 64)
    assert tuple(wc.fp4_decode(wc.fp4_encode(x[:, :0].contiguous())).shape) == (2, 0)


def test_gemv_offsets_past_32_bits():
    """Codes of more than 2^32 bytes: rows at both ends, with a one-hot x."""
    rows, cols = 270000, 32768
    G = cols // 32
    codes = torch.zeros((rows, 16 * G), dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, G), 127, dtype=torch.uint8, device=DEV)
    assert codes.numel() > 1 << 32
    codes[0, 16 * G - 1] = 0x70    # column cols - 1: 6
    codes[rows - 1, 16 * G - 1] = 0xB0  # -1.5
    codes[rows - 2, 0] = 0x05      # column 0: 3
    x = torch.zeros((1, cols), dtype=torch.bfloat16, device=DEV)
    x[0, cols - 1], x[0, 0] = 1.0, 2.0
    y = wc.fp4_gemv(wc.Fp4(codes, scales, cols), x)[0]
    assert [y[i].item() for i in (0, 1, rows - 2, rows - 1)] == [6.0, 0.0, 6.0, -1.5]
    assert int((y != 0).sum()) == 3


def test_gemv_repeats_its_bits_and_runs_in_a_graph():
    q = wc.fp4_encode(dev16(synth.random_bits(512 * 2080, 6).reshape(512, 2080)))
    for batch in (1, 24, 100):
        x = dev16(synth.vectors(6, batch, 2080))
        out = torch.empty((batch, 512), device=DEV)
        ref = wc.fp4_gemv(q, x).clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            wc.fp4_gemv(q, x, out=out)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, ref)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            wc.fp4_gemv(q, x, out=out)
        for _ in range(4):
            x.copy_(x.flip(1))
            ref = wc.fp4_gemv(q, x)
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
