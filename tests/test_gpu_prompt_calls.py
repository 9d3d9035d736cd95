"""Calls of the prompt attention at the edges of what its header allows."""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import decode_gemv_sign_amd as wc  # noqa: E402
from tests.test_gpu_prompt import DEV, Case, dev16, starts_of  # noqa: E402


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("stride", [0, 8, 32, 64])
def test_one_token_of_any_stride(dim, stride):
    """Strides lie between tokens: of one token they say nothing."""
    c = Case([1], 4, 2, dim, seed=31)
    q, k, v = (dev16(x) for x in (c.q, c.k, c.v))
    want, want_lse = wc.prompt_attention(q, k, v, starts_of([1]))
    assert torch.equal(want[0].view(torch.int16), v[0].repeat_interleave(2, 0))
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    shape = wc.PromptShape(1, stride, stride, stride, 1, 4, 2, dim, 0, dim ** -0.5)
    assert wc._lib.wc_prompt_attention(ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                       starts_of([1]).data_ptr(), out.data_ptr(), lse.data_ptr(),
                                       torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("scale", [0.0, -0.0])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_scale_of_zero_of_large_scores(dim, scale):
    """Every score is 0, however large the product: the mean of the values.  Scores of
    2^118 dim and more differ from token to token."""
    c = Case([200, 70], 2, 1, dim, seed=32)
    small = c.run(scale=scale)
    c.q = (c.q & 0x807F) | 0x5D80  # 2^60 and up, of either sign
    c.k = (c.k & 0x807F) | 0x5C80  # 2^58 and up
    got = c.run(scale=scale)
    # The products are below 2^127: where the factor is fp32's least number, 2^-149, weights are
    # within 2^-22 of 1, BF16 rounds them to 1, and the outputs are the same sums over a divisor
    # off by 2^-22 at most: one step of BF16, in a rare tie.
    near = (got[0].float() - small[0].float()).abs() <= 2.0 ** -7 * small[0].float().abs()
    assert bool(near.all())
    count = np.concatenate([np.arange(1, 201), np.arange(1, 71)])
    want = torch.from_numpy(np.log(count)).to(DEV)[:, None]
    # the sum is off by 2^-22 at most, its offset by as much, the logarithm by two of its steps
    assert bool(((got[1].double() - want).abs() <= 2.0 ** -22 * (2 + want)).all())
