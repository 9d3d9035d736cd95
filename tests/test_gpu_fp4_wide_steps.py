"""Every tile of the 4-bit product for larger batches over several whole steps of
512 columns per wave, where inputs and codes are loaded while earlier ones are
multiplied.  Weights and inputs are small whole numbers, so that fp32 sums are
exact in any order and one value from a wrong place shows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402

DEV = "cuda:0"
ENOUGH = torch.cuda.get_device_properties(0).multi_processor_count * 5 // 8  # blocks that a tile must give
# (rows of a block, inputs of a block, batch that takes it)
TILES = [(64, 64, 40), (64, 64, 64), (64, 32, 20), (64, 32, 32), (32, 32, 31), (32, 16, 9), (32, 16, 16)]


def blocks(rows, batch, mt, nt):
    return -(-rows // mt) * -(-batch // nt)


def tile_of(rows, batch):
    """The tile that the dispatch rule gives."""
    if batch > 32 and blocks(rows, batch, 64, 64) >= ENOUGH:
        return 64, 64
    if batch > 16 and blocks(rows, batch, 64, 32) >= ENOUGH:
        return 64, 32
    if batch > 16 and blocks(rows, batch, 32, 32) >= ENOUGH:
        return 32, 32
    return (32, 16) if blocks(rows, batch, 32, 16) >= ENOUGH else None


def whole_numbers(g, *shape, most):
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV).to(torch.bfloat16)


# 13 steps: 3 or 4 per wave; none, one piece or nearly a whole step left over; 20 steps and a ragged end
@pytest.mark.parametrize("cols", [6656, 6664, 7160, 10312])
@pytest.mark.parametrize("mt,nt,batch", TILES)
def test_every_tile(mt, nt, batch, cols):
    rows = mt * ENOUGH + 5  # the last block is not whole
    assert tile_of(rows, batch) == (mt, nt)
    g = torch.Generator(DEV).manual_seed(cols + batch)
    magnitude = torch.tensor([0.0, 1, 2, 3, 4, 6], device=DEV)[torch.randint(6, (rows, cols), generator=g, device=DEV)]
    w = magnitude * (torch.randint(2, (rows, cols), generator=g, device=DEV) * 2 - 1)
    w[:, ::32] = 6.0  # every group's scale is 1
    q = wc.fp4_encode(w.to(torch.bfloat16))
    w = w.double()
    out = torch.empty(batch, rows, device=DEV)
    for _ in range(3):
        x = whole_numbers(g, batch, cols, most=8)
        assert 6 * 8 * cols < 1 << 24
        wc.fp4_gemv(q, x, out=out)
        assert torch.equal(out.double(), x.double() @ w.T)


@pytest.mark.parametrize("batch", [33, 100, 256])
def test_several_batch_tiles(batch):
    """Batches of more than one tile of inputs, the last one not whole."""
    rows, cols = 64 * (ENOUGH // -(-batch // 64) + 1) + 37, 4616
    assert tile_of(rows, batch) == (64, 64)
    g = torch.Generator(DEV).manual_seed(batch)
    w = whole_numbers(g, rows, cols, most=4)
    w[:, ::32] = 6.0
    q = wc.fp4_encode(w)
    x = whole_numbers(g, batch, cols, most=8)
    assert torch.equal(wc.fp4_gemv(q, x).double(), x.double() @ wc.fp4_decode(q).double().T)
