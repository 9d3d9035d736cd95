"""Refusals of token_logprobs without a GPU: the binding's checks (before any
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
        self.calls, self.need = [], 0

    def wc_token_logprobs_workspace_bytes(self, *args):
        return self.need

    def wc_token_logprobs(self, *args):
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
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    wc._logprob_need.cache_clear()
    yield lib
    wc._logprob_need.cache_clear()


def t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device=META)


def f32(*shape):
    return t(torch.float32, *shape)


def call(**more):
    return wc.token_logprobs(**{"logits": f32(7, 100), "tokens": t(torch.int64, 7), **more})


def test_the_plain_calls_pass(stub):
    out = call(top=5)
    assert [tuple(v.shape) for v in out] == [(7,), (7,), (7, 5), (7, 5)]
    assert [v.dtype for v in out] == [torch.float32, torch.float32, torch.int32, torch.float32]
    call(logits=t(torch.bfloat16, 7, 130)[:, 3:103])
    call(logits=f32(0, 100), tokens=t(torch.int64, 0))
    shapes = [a[0]._obj for a in stub.calls]
    assert [(s.stride, s.rows, s.vocab, s.kind, s.top) for s in shapes] == [
        (100, 7, 100, 1, 5), (130, 7, 100, 0, 0), (100, 0, 100, 1, 0)]


@pytest.mark.parametrize("more", [
    {"logits": t(torch.float16, 7, 100)}, {"logits": torch.empty(7, 100)}, {"logits": f32(700)}, {"logits": f32(7, 0)},
    {"logits": f32(1, 7, 100)}, {"logits": f32(100, 7).T}, {"logits": f32(7, 200)[:, ::2]},
    {"logits": f32(1, 100).expand(7, 100)}, {"logits": f32(6, 100)}, {"top": -1}, {"top": 33},
    {"tokens": t(torch.int32, 7)}, {"tokens": t(torch.int64, 8)}, {"tokens": t(torch.int64, 7, 1)},
    {"tokens": t(torch.int64, 14)[::2]}, {"tokens": torch.empty(7, dtype=torch.int64)}])
def test_refuses(stub, more):
    with pytest.raises((ValueError, TypeError)):
        call(**more)
    assert stub.calls == []


def test_workspace(stub):
    stub.need = 100
    for work in (t(torch.uint8, 99), t(torch.int8, 100), t(torch.uint8, 200)[::2], torch.empty(100, dtype=torch.uint8)):
        with pytest.raises((ValueError, TypeError)):
            call(work=work)
    assert stub.calls == []
    call(work=t(torch.uint8, 100))
    assert stub.calls[0][8] == 100


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

    stub.need = 64
    monkeypatch.setattr(wc, "_stream", lambda s=None: now[-1] if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Stream(-1))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda v, s: kept.append(v))
    args = {"logits": f32(7, 100), "tokens": t(torch.int64, 7)}
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(now[-1]) or empty(*a, **k))
    out = wc.token_logprobs(**args, top=2, stream=_Stream(-1, 7))
    assert set(made) == {7} and all(any(k is o or k is o._base for k in kept) for o in out)


P = 1 << 20  # a pointer that is aligned, and never followed


def abi(logits=P, tokens=P, lp=P, entropy=P, ids=P, best=P, work=P, size=1 << 30, **more):
    s = {"stride": 200000, "rows": 7, "vocab": 200000, "kind": 1, "top": 3, **more}
    shape = wc.LogprobShape(*(s[n] for n, _ in wc.LogprobShape._fields_))
    need = wc._lib.wc_token_logprobs_workspace_bytes(ctypes.byref(shape))
    return need, wc._lib.wc_token_logprobs(ctypes.byref(shape), logits, tokens, lp, entropy, ids, best, work,
                                           need - 1 if size is None else size, None)


def test_abi():
    assert wc._lib.wc_token_logprobs(None, P, P, P, P, P, P, P, 1, None) == -1
    assert wc._lib.wc_token_logprobs_workspace_bytes(None) == 0
    assert abi(None, None, None, None, None, None, None, rows=0)[1] == 0
    for more, code in [({"vocab": 0}, -1), ({"vocab": 1 << 31}, -1), ({"kind": 2}, -1), ({"top": 33}, -5),
                       ({"rows": 1 << 24}, -2)]:
        assert abi(**more) == (0, code), more
    for more, code in [({"stride": 199999}, -1), ({"stride": 1 << 40}, -2), ({"logits": None}, -1), ({"logits": P + 2}, -1),
                       ({"logits": P + 1, "kind": 0}, -1), ({"tokens": None}, -1), ({"tokens": P + 4}, -1),
                       ({"lp": None}, -1), ({"lp": P + 2}, -1), ({"entropy": None}, -1), ({"entropy": P + 1}, -1),
                       ({"ids": None}, -1), ({"ids": P + 2}, -1), ({"best": None}, -1), ({"best": P + 2}, -1),
                       ({"work": None}, -1), ({"work": P + 8}, -1), ({"size": None}, -2)]:
        need, got = abi(**more)
        assert need > 0 and got == code, more


def test_struct_matches_the_header(tmp_path):
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "wc_logprob.h"\nint main(void){\n' + "".join(
        f'printf("%zu\\n", offsetof(wc_logprob_shape, {n}));' for n, _ in wc.LogprobShape._fields_) +
        'printf("%zu\\n", sizeof(wc_logprob_shape));return 0;}\n')
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                           str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [getattr(wc.LogprobShape, n).offset for n, _ in wc.LogprobShape._fields_] + [
        ctypes.sizeof(wc.LogprobShape)]
