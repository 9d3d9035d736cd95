"""Slices of the inputs' rows: with rows of a length that is no multiple of 8
they start at any 2-byte address, and give the bits of an aligned copy."""
import pytest

import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402

DEV = "cuda:0"


def dev16(a):
    return torch.from_numpy(a.view("int16")).to(DEV)


@pytest.mark.parametrize("cols", [1, 7, 33, 100, 516, 1031, 4100, 4101])
@pytest.mark.parametrize("batch", [1, 4, 5, 16, 17, 70])
def test_fp4_gemv(cols, batch):
    q = wc.fp4_encode(dev16(synth.random_bits(83 * cols, cols).reshape(83, cols)))
    x = dev16(synth.vectors(cols + batch, batch + 9, cols))
    for first in (1, 2, 3, 9):
        part = x[first:first + batch]
        assert torch.equal(wc.fp4_gemv(q, part), wc.fp4_gemv(q, part.clone())), first


@pytest.mark.parametrize("hidden,inter", [(1, 1), (7, 16), (33, 20), (1031, 48), (4100, 33)])
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
@pytest.mark.parametrize("tokens", [1, 9, 17])
def test_moe(hidden, inter, kind, tokens):
    w = [dev16(synth.random_bits(6 * r * c, 7 + r).reshape(6, r, c))
         for r, c in ((2 * inter, hidden), (hidden, inter))]
    if kind == "fp4":
        w = [wc.fp4_encode(v) for v in w]
    router = dev16(synth.vectors(8, 6, hidden))
    x = dev16(synth.vectors(hidden, tokens + 9, hidden))
    for first in (1, 3, 9):
        part = x[first:first + tokens]
        got, ref = wc.moe(part, router, *w, 2), wc.moe(part.clone(), router, *w, 2)
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), first


def test_rows_of_whole_pieces_keep_their_alignment():
    """Rows of a multiple of 8 must start at 16-byte boundaries, as they do in
    every slice of whole rows; a view that starts elsewhere is refused."""
    q = wc.fp4_encode(dev16(synth.random_bits(20 * 64, 1).reshape(20, 64)))
    flat = dev16(synth.vectors(2, 1, 64 * 4 + 8)).flatten()
    wc.fp4_gemv(q, flat[:192].view(3, 64)[1:])
    with pytest.raises(wc.WCError):
        wc.fp4_gemv(q, flat[4:196].view(3, 64))
    odd = wc.fp4_encode(dev16(synth.random_bits(20 * 33, 1).reshape(20, 33)))
    assert wc._lib.wc_fp4_gemv(odd.codes.data_ptr(), odd.scales.data_ptr(), 20, 33, flat.data_ptr() + 1, 1,
                               torch.empty(20, device=DEV).data_ptr(), None) == -1
