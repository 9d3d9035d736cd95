"""GEMV at the most rows that the entry points take: every row is computed, and
none past them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("rows,cols,batch", [((1 << 26) - 16, 5, 1), ((1 << 26) - 16, 9, 2), ((1 << 28) - 16, 8, 1),
                                             ((1 << 28) - 16, 32, 5), ((1 << 32) - 256, 0, 1)])
def test_plain_gemv(rows, cols, batch):
    w = torch.ones(rows, cols, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(batch, cols, dtype=torch.bfloat16, device=DEV)
    y = torch.full((batch * rows + 64,), 77.0, device=DEV)
    wc.gemv_bf16(w, x, out=y[:batch * rows].view(batch, rows))
    assert bool((y[:batch * rows] == cols).all()) and bool((y[batch * rows:] == 77).all())


@pytest.mark.parametrize("rows,cols", [((1 << 26) - 16, 5), ((1 << 28) - 16, 8)])
def test_decode_gemv(rows, cols):
    w = torch.ones(rows, cols, dtype=torch.bfloat16, device=DEV)
    h, c = wc.encode(w, wc.BYTESPLIT)
    del w
    y = wc.decode_gemv(h, c, rows, cols, torch.ones(1, cols, dtype=torch.bfloat16, device=DEV))
    assert bool((y == cols).all())
