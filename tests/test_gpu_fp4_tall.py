"""4-bit products of more rows than one launch's grid takes."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("batch", [1, 5, 17])
def test_rows_past_a_grid(batch):
    """2^29 + 53 rows of 32 columns: more than 2^32 threads in one launch, so
    the rows go in parts; both ends of every part are set, the others are 0."""
    rows, cols = (1 << 29) + 53, 32
    codes = torch.zeros((rows, 16), dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, 1), 127, dtype=torch.uint8, device=DEV)
    at = [0, 1, (1 << 28) - 1, 1 << 28, (1 << 28) + 17, (1 << 29) - 1, 1 << 29, rows - 2, rows - 1]
    for n, r in enumerate(at):
        codes[r, n] = 0x70  # column 2 n + 1: 6
        codes[r, 15] = 0x0A  # column 30: -1
    x = torch.zeros((batch, cols), dtype=torch.bfloat16, device=DEV)
    x[:, 1:18:2] = torch.arange(2.0, 11.0, device=DEV).to(torch.bfloat16)
    x[:, 30] = torch.arange(batch, device=DEV).to(torch.bfloat16)
    y = wc.fp4_gemv(wc.Fp4(codes, scales, cols), x)
    ref = 6.0 * torch.arange(2.0, 11.0)[None] - torch.arange(batch).float()[:, None]
    assert torch.equal(y[:, at].cpu(), ref)
    for b in range(batch):
        assert int((y[b] != 0).sum()) == int((ref[b] != 0).sum())
