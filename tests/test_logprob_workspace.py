"""The scratch size of token_logprobs without a GPU: numbers and types that a call
refuses are refused here too."""
import pytest
import torch

import decode_gemv_sign_amd as wc


class _Lib:
    def __init__(self):
        self.shapes = []

    def wc_token_logprobs_workspace_bytes(self, shape):
        s = shape._obj
        self.shapes.append((s.rows, s.vocab, s.kind, s.top))
        return 48


@pytest.fixture
def stub(monkeypatch):
    lib = _Lib()
    monkeypatch.setattr(wc, "_lib", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    wc._logprob_need.cache_clear()
    yield lib
    wc._logprob_need.cache_clear()


def test_sizes_are_looked_up_once(stub):
    for _ in range(2):
        assert wc.token_logprobs_workspace_bytes(4, 200000, 5) == 48
        assert wc.token_logprobs_workspace_bytes(4, 200000, 5, torch.bfloat16) == 48
        assert wc.token_logprobs_workspace_bytes(0, 1) == 48
    assert stub.shapes == [(4, 200000, 1, 5), (4, 200000, 0, 5), (0, 1, 1, 0)]


@pytest.mark.parametrize("args", [((1 << 32) + 4, 200000), (4, (1 << 32) + 200000), (-4, 200000), (4, 200000, (1 << 32) + 5),
                                  (4, 200000, -1), (4, 200000, 33), (1 << 31, 10), (10, 1 << 31), (4, 0)])
def test_numbers_out_of_range(stub, args):
    """Not taken modulo 2^32."""
    with pytest.raises(ValueError):
        wc.token_logprobs_workspace_bytes(*args)
    assert stub.shapes == []


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32])
def test_types(stub, dtype):
    """Not taken for BF16."""
    with pytest.raises(TypeError):
        wc.token_logprobs_workspace_bytes(4, 200000, 5, dtype)
    assert stub.shapes == []
