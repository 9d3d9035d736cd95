"""Refusals of the prompt attention without a GPU: the binding's checks (before any
library call, on meta tensors) and the C ABI's (before any device work)."""
import contextlib
import ctypes
import os
import subprocess

import pytest
import torch

import decode_gemv_sign_amd as wc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
META = torch.device("meta")


class _Lib:
    def __init__(self):
        self.calls = []

    def wc_prompt_attention(self, *args):
        self.calls.append(args)
        return 0


class _Stream:
    def __init__(self, device, handle=0):
        self.device_index, self.cuda_stream = device, handle


@pytest.fixture
def stub(monkeypatch):
    lib = _Lib()
    monkeypatch.setattr(wc, "_lib", lib)
    monkeypatch.setattr(wc, "_on_device", lambda t: t.device.type == "meta")
    monkeypatch.setattr(wc, "_ptr", lambda t: None)
    monkeypatch.setattr(wc, "_stream", lambda s=None: 0 if s is None else s.cuda_stream)
    return lib


def t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device=META)


def b16(*shape):
    return t(torch.bfloat16, *shape)


def call(**more):
    return wc.prompt_attention(**{"q": b16(70, 4, 64), "k": b16(70, 2, 64), "v": b16(70, 2, 64),
                                  "starts": t(torch.int32, 4), **more})


def test_the_plain_calls_pass(stub):
    call()
    fused = b16(70, 9, 64)
    out, lse = call(q=fused[:, :4], k=fused[:, 4:6], v=fused[:, 6:8], window=5, scale=2.0)
    assert out.shape == (70, 4, 64) and out.dtype == torch.bfloat16
    assert lse.shape == (70, 4) and lse.dtype == torch.float32
    shape = stub.calls[1][0]._obj
    assert [getattr(shape, n) for n, _ in shape._fields_] == [70, 576, 576, 576, 3, 4, 2, 64, 5, 2.0]
    assert stub.calls[0][0]._obj.scale == 0.125
    call(q=b16(0, 4, 64), k=b16(0, 2, 64), v=b16(0, 2, 64), starts=t(torch.int32, 1))
    assert len(stub.calls) == 3


@pytest.mark.parametrize("more", [
    {"q": b16(70, 4, 48)}, {"q": b16(70, 4, 288)}, {"q": b16(70, 256)}, {"q": b16(1, 70, 4, 64)}, {"q": b16(69, 4, 64)},
    {"q": b16(70, 3, 64)}, {"q": b16(70, 4, 32)}, {"q": t(torch.float16, 70, 4, 64)},
    {"q": torch.empty(70, 4, 64, dtype=torch.bfloat16)}, {"q": b16(70, 64, 4).transpose(1, 2)},
    {"q": b16(4, 70, 64).transpose(0, 1)}, {"q": b16(70, 4, 66)[:, :, :64]}, {"q": b16(1, 4, 64).expand(70, 4, 64)},
    {"k": b16(71, 2, 64)}, {"k": b16(70, 1, 64)}, {"k": b16(70, 2, 32)}, {"v": b16(70, 4, 64)}, {"v": b16(69, 2, 64)},
    {"v": b16(70, 2, 128)[:, :, ::2]}, {"k": b16(70, 0, 64)}, {"k": b16(70, 2, 1, 64)},
    {"starts": t(torch.int64, 4)}, {"starts": t(torch.int32, 0)}, {"starts": t(torch.int32, 2, 2)},
    {"starts": t(torch.int32, 8)[::2]}, {"starts": torch.empty(4, dtype=torch.int32)},
    {"out": b16(69, 4, 64)}, {"out": t(torch.float32, 70, 4, 64)}, {"out": b16(70, 8, 64)[:, :4]},
    {"window": -1}, {"window": 1 << 32}])
def test_refuses(stub, more):
    with pytest.raises((ValueError, TypeError)):
        call(**more)
    assert stub.calls == []


@pytest.mark.parametrize("tensors,current,stream,ok", [
    (0, 0, None, True), (1, 1, None, True), (1, 1, 1, True),
    (1, 0, None, False), (0, 1, None, False), (1, 0, 1, False), (0, 0, 1, False)])
def test_device_of_the_tensors(stub, monkeypatch, tensors, current, stream, ok):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda v: tensors)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)
    s = None if stream is None else _Stream(stream)
    if ok:
        call(stream=s)
    else:
        with pytest.raises(ValueError, match="device"):
            call(stream=s)
    assert len(stub.calls) == ok


def test_memory_of_another_stream(stub, monkeypatch):
    now, made, kept = [3], [], []
    empty = torch.empty

    @contextlib.contextmanager
    def on(s):
        now.append(s.cuda_stream)
        yield
        now.pop()

    monkeypatch.setattr(wc, "_stream", lambda s=None: now[-1] if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Stream(-1))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda v, s: kept.append(v))
    args = {"q": b16(70, 4, 64), "k": b16(70, 2, 64), "v": b16(70, 2, 64), "starts": t(torch.int32, 4)}
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(now[-1]) or empty(*a, **k))
    out = wc.prompt_attention(**args, stream=_Stream(-1, 7))
    assert made == [7, 7] and all(any(k is o for k in kept) for o in out)


P = 1 << 20  # a pointer that is aligned, and never followed


def abi(q=P, k=P, v=P, starts=P, out=P, lse=None, **more):
    s = {"tokens": 70, "q_stride": 256, "k_stride": 128, "v_stride": 128, "seqs": 3, "heads": 4, "kv_heads": 2,
         "head_dim": 64, "window": 0, "scale": 1.0, **more}
    shape = wc.PromptShape(*(s[n] for n, _ in wc.PromptShape._fields_))
    return wc._lib.wc_prompt_attention(ctypes.byref(shape), q, k, v, starts, out, lse, None)


def test_abi():
    assert wc._lib.wc_prompt_attention(None, P, P, P, P, P, None, None) == -1
    for more in ({"tokens": 0}, {"seqs": 0}):
        assert abi(None, None, None, None, None, **more) == 0
    for more, code in [({"head_dim": 0}, -1), ({"head_dim": 48}, -1), ({"head_dim": 288}, -1), ({"heads": 0}, -1),
                       ({"kv_heads": 0}, -1), ({"heads": 5}, -1), ({"heads": 1026}, -1), ({"q_stride": 248}, -1),
                       ({"q_stride": 260}, -1), ({"k_stride": 120}, -1), ({"v_stride": 132}, -1),
                       ({"q_stride": 1 << 24}, -2), ({"k_stride": 1 << 24}, -2), ({"v_stride": 1 << 24}, -2),
                       ({"tokens": 1 << 31}, -2), ({"seqs": 1 << 31}, -2), ({"seqs": 1 << 23}, -2)]:
        assert abi(**more) == code, more
    for name in ("q", "k", "v", "starts", "out"):
        assert abi(**{name: None}) == -1, name
    for more in ({"q": P + 8}, {"k": P + 2}, {"v": P + 4}, {"starts": P + 2}, {"out": P + 8}, {"lse": P + 2}):
        assert abi(**more) == -1, more


def test_struct_matches_the_header(tmp_path):
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "wc_attn.h"\nint main(void){\n' + "".join(
        f'printf("%zu\\n", offsetof(wc_prompt_shape, {n}));' for n, _ in wc.PromptShape._fields_) +
        'printf("%zu\\n", sizeof(wc_prompt_shape));return 0;}\n')
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                           str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [getattr(wc.PromptShape, n).offset for n, _ in wc.PromptShape._fields_] + [
        ctypes.sizeof(wc.PromptShape)]
