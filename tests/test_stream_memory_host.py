"""Memory that a call with stream= allocates comes from that stream's pool, and
what it returns is kept from reuse while the caller's stream reads it: checked
without a GPU, on meta tensors, against stand-ins for torch's streams."""
import contextlib

import pytest
import torch

import decode_gemv_sign_amd as wc

META = torch.device("meta")
HERE, SIDE = 3, 7  # handles of the current and of the other stream


class _Handle:
    """A stream that is not torch's own."""

    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class _Stream(_Handle):
    device_index = 0


class _Lib:
    def __getattr__(self, name):
        if not name.startswith("wc_"):
            raise AttributeError(name)

        def call(*args):
            if name == "wc_build_dict":
                args[-1]._obj.n, args[-1]._obj.total_bytes = args[2], 2048
            return 4096 if name == "wc_moe_workspace_bytes" else 0
        return call


@pytest.fixture
def record(monkeypatch):
    """What was allocated, as (handle of the stream, tensor), and which tensors
    were recorded for which other stream."""
    now, made, kept = [HERE], [], []
    empty = torch.empty

    @contextlib.contextmanager
    def stream(s):
        assert isinstance(s, _Stream)
        now.append(s.cuda_stream)
        yield
        now.pop()

    def alloc(*a, **k):
        t = empty(*a, **k)
        made.append((now[-1], t))
        return t

    monkeypatch.setattr(wc, "_lib", _Lib())
    monkeypatch.setattr(wc, "_on_device", lambda t: t.device.type == "meta")
    monkeypatch.setattr(wc, "_ptr", lambda t: None)
    monkeypatch.setattr(wc, "_stream", lambda s=None: now[-1] if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", _Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Stream(now[-1]))
    monkeypatch.setattr(torch, "empty", alloc)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((s.cuda_stream, t)))
    return made, kept


def b16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=META)


def u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device=META)


W, X, Q = b16(6, 70), b16(3, 70), wc.Fp4(u8(6, 48), u8(6, 3), 70)
N = 6 * 70
HEAD, COPY = wc.Header(), u8(2048)
HEAD.n, HEAD.total_bytes = N, 2048
MOE = b16(3, 64), b16(5, 64), b16(5, 80, 64), b16(5, 64, 40), 2
CALLS = {  # the outputs of each call
    "fp4_encode": lambda s: list(wc.fp4_encode(W, stream=s)[:2]),
    "fp4_decode": lambda s: [wc.fp4_decode(Q, stream=s)],
    "fp4_gemv": lambda s: [wc.fp4_gemv(Q, X, stream=s)],
    "moe": lambda s: list(wc.moe(*MOE, stream=s)),
    "build_dict": lambda s: [wc.build_dict(W, wc.K15, stream=s)][:0],  # a workspace alone
    "encode_into": lambda s: [wc.encode_into(HEAD, W, COPY, stream=s)][:0],
    "encode": lambda s: [wc.encode(W, wc.K15, stream=s)[1]],
    "decode": lambda s: [wc.decode(HEAD, COPY, stream=s)],
    "decode_gemv": lambda s: [wc.decode_gemv(HEAD, COPY, 6, 70, X, stream=s)],
    "gemv_bf16": lambda s: [wc.gemv_bf16(W, X, stream=s)],
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("kind", [_Stream, _Handle])
def test_memory_comes_from_the_streams_pool(record, name, kind):
    made, kept = record
    out = CALLS[name](kind(SIDE))
    assert made and all(h == SIDE for h, _ in made)
    assert all(any(t is o for _, t in made) for o in out)
    assert all(any(t is o and h == HERE for h, t in kept) for o in out)


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("stream", [None, _Stream(HERE), _Handle(HERE)])
def test_memory_of_the_current_stream(record, name, stream):
    made, kept = record
    CALLS[name](stream)
    assert made and all(h == HERE for h, _ in made) and not kept
