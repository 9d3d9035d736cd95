"""Numbers that do not fit a field of wc_moe_shape are refused: they are not
taken modulo 2^32, which would make another layer of them.  The workspace's size
is that of the library in use."""
import pytest
import torch

import decode_gemv_sign_amd as wc


def b16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="meta")


class _Lib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("wc_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append(name)
            return 4096 if name == "wc_moe_workspace_bytes" else 0
        return call


@pytest.mark.parametrize("change", [
    dict(scoring=1 << 32), dict(scoring=(1 << 32) + 1), dict(scoring=-1), dict(top_k=(1 << 32) + 2),
    dict(top_k=-2), dict(top_k=2 - (1 << 32))])
def test_moe_refuses(monkeypatch, change):
    lib = _Lib()
    monkeypatch.setattr(wc, "_lib", lib)
    monkeypatch.setattr(wc, "_on_device", lambda t: True)
    monkeypatch.setattr(wc, "_ptr", lambda t: None)
    monkeypatch.setattr(wc, "_stream", lambda s=None: 0)
    a = dict(x=b16(3, 64), router=b16(5, 64), gate_up=b16(5, 80, 64), down=b16(5, 64, 40), top_k=2)
    with pytest.raises(ValueError, match="outside"):
        wc.moe(**{**a, **change})
    assert "wc_moe" not in lib.calls


@pytest.mark.parametrize("at", range(5))
@pytest.mark.parametrize("wrap", [1 << 32, -(1 << 32)])
def test_workspace_refuses(at, wrap):
    shape = [3, 64, 40, 5, 2]
    assert wc.moe_workspace_bytes(*shape) > 0
    shape[at] += wrap
    with pytest.raises(ValueError, match="outside"):
        wc.moe_workspace_bytes(*shape)


def test_workspace_size_follows_the_library(monkeypatch):
    class Other:
        @staticmethod
        def wc_moe_workspace_bytes(shape):
            return 12345

    here, lib = wc.moe_workspace_bytes(3, 64, 40, 5, 2), wc._lib
    assert here != 12345
    monkeypatch.setattr(wc, "_load", lambda path: Other if path == "other" else lib)
    try:
        wc.use_library("other")
        assert wc.moe_workspace_bytes(3, 64, 40, 5, 2) == 12345
    finally:
        wc.use_library(wc.LIB_PATH)
    assert wc.moe_workspace_bytes(3, 64, 40, 5, 2) == here and wc._lib is lib
