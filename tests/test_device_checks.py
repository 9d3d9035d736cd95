"""The 4-bit calls and the mixture of experts refuse tensors or a stream of
another device than the current one, before any device work: checked without a
GPU, on meta tensors that say they are on a device."""
import pytest
import torch

import decode_gemv_sign_amd as wc


class _Stream:
    cuda_stream = 0

    def __init__(self, device):
        self.device_index = device


class _Lib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("wc_"):
            raise AttributeError(name)

        def call(*args):
            if name == "wc_moe_workspace_bytes":
                return 4096
            self.calls.append(name)
            return 0
        return call


def t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="meta")


def b16(*shape):
    return t(torch.bfloat16, *shape)


Q = wc.Fp4(t(torch.uint8, 6, 48), t(torch.uint8, 6, 3), 70)
CALLS = {
    "fp4_encode": lambda s: wc.fp4_encode(b16(6, 70), stream=s),
    "fp4_encode out": lambda s: wc.fp4_encode(b16(6, 70), out=Q, stream=s),
    "fp4_decode": lambda s: wc.fp4_decode(Q, stream=s),
    "fp4_gemv": lambda s: wc.fp4_gemv(Q, b16(3, 70), stream=s),
    "moe": lambda s: wc.moe(b16(3, 64), b16(5, 64), b16(5, 80, 64), b16(5, 64, 40), 2, stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("tensors,current,stream,ok", [
    (0, 0, None, True), (1, 1, None, True), (1, 1, 1, True),
    (1, 0, None, False), (0, 1, None, False), (1, 0, 1, False), (0, 0, 1, False)])
def test_device_of_the_tensors(monkeypatch, name, tensors, current, stream, ok):
    lib = _Lib()
    monkeypatch.setattr(wc, "_lib", lib)
    monkeypatch.setattr(wc, "_on_device", lambda v: True)
    monkeypatch.setattr(wc, "_ptr", lambda v: None)
    monkeypatch.setattr(wc, "_stream", lambda s=None: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda v: tensors)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)
    s = None if stream is None else _Stream(stream)
    if ok:
        CALLS[name](s)
        assert lib.calls == ["wc_" + name.split()[0]]
    else:
        with pytest.raises(ValueError, match="device"):
            CALLS[name](s)
        assert lib.calls == []
