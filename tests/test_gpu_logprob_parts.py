"""Log probabilities of rows in every number of parts up to 64, where the parts of a row
are as many as the lanes that join them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402
from tests.test_gpu_logprob import DEV, KINDS, check, logits  # noqa: E402


def parts_of(rows, vocab, top, dtype):
    need = wc.token_logprobs_workspace_bytes(rows, vocab, top, dtype)  # a row's part: 16 bytes and a key for each
    return max(1, need // (rows * (16 + 8 * top)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("top", [0, 1, 32])
@pytest.mark.parametrize("rows,vocab,parts", [(1, 262144, 64), (16, 262144, 64), (17, 262144, 32), (1, 262145, 33),
                                              (16, 262145, 33), (1, 258049, 64), (1, 258048, 63), (2, 131073, 33),
                                              (1, 1000003, 62)])
def test_parts(kind, top, rows, vocab, parts):
    x, tokens = logits(rows, vocab, kind, seed=41)
    assert parts_of(rows, vocab, top, x.dtype) == parts
    check(x, tokens, top)
    x[:, -40:] += 30.0  # the best in the last part
    check(x, tokens, top)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("vocab", [262144, 262145])
def test_ties_masks_and_nan_over_the_parts(kind, vocab):
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    x = torch.zeros(3, vocab, dtype=dtype, device=DEV)
    x[1] = (torch.arange(vocab, device=DEV) // 5000).to(dtype) / 8          # equal ones, larger from part to part
    x[2] = -float("inf")
    x[2, [5, vocab // 2, vocab - 1]] = torch.tensor([1.0, 2.0, 1.0], dtype=dtype, device=DEV)
    check(x, [vocab - 1, 0, vocab - 1], 32)
    x[2] = -float("inf")
    lp, h, ids, best = check(x, [0, 0, 0], 32)
    assert lp[2] == -float("inf") and h[2] == 0 and bool((ids[2] == -1).all())
    x[0, vocab - 3] = float("nan")
    lp, h, ids, best = wc.token_logprobs(x, torch.zeros(3, dtype=torch.int64, device=DEV), 32)
    assert bool(torch.isnan(lp[0])) and bool(torch.isnan(h[0])) and bool(torch.isnan(best[0]).all())
    assert ids[0].tolist() == [vocab - 3] + list(range(31))
    assert np.isfinite(lp[1].item())
