"""Refusals of the 4-bit cache's calls without a GPU: the binding's checks (before
any library call, on meta tensors) and the C ABI's (before any device work)."""
import ctypes
import re
import subprocess
import os

import pytest
import torch

import decode_gemv_sign_amd as wc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
META = torch.device("meta")


class _Lib:
    def __init__(self, need=0):
        self.calls, self.need = [], need

    def __getattr__(self, name):
        if not name.startswith("wc_"):
            raise AttributeError(name)

        def call(*args):
            if name.endswith("workspace_bytes"):
                return self.need
            self.calls.append((name, args))
            return 0
        return call


class _Stream:
    cuda_stream = 0

    def __init__(self, device):
        self.device_index = device


@pytest.fixture
def stub(monkeypatch):
    lib = _Lib()
    monkeypatch.setattr(wc, "_lib", lib)
    monkeypatch.setattr(wc, "_on_device", lambda t: t.device.type == "meta")
    monkeypatch.setattr(wc, "_ptr", lambda t: None)
    monkeypatch.setattr(wc, "_stream", lambda s=None: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    wc._attention_need.cache_clear()
    yield lib
    wc._attention_need.cache_clear()


def t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device=META)


def b16(*shape):
    return t(torch.bfloat16, *shape)


def cache(pages=5, heads=2, tiles=2, dim=64):
    return t(torch.uint8, pages, heads, tiles, 34 * dim)


def i32(*shape):
    return t(torch.int32, *shape)


def i64(*shape):
    return t(torch.int64, *shape)


APPEND_OK = lambda **k: wc.fp4_cache_append(**{"cache": cache(), "k": b16(7, 2, 64), "v": b16(7, 2, 64),  # noqa: E731
                                               "slots": i64(7), **k})
READ_OK = lambda **k: wc.fp4_cache_read(**{"cache": cache(), "slots": i64(7), **k})  # noqa: E731
ATTEND_OK = lambda **k: wc.fp4_attention(**{"q": b16(3, 4, 64), "cache": cache(), "table": i32(3, 9),  # noqa: E731
                                            "lengths": i32(3), **k})


def test_the_plain_calls_pass(stub):
    APPEND_OK()
    READ_OK()
    ATTEND_OK()
    ATTEND_OK(q=b16(3, 16, 4, 64))
    ATTEND_OK(q=b16(3, 9, 64)[:, 2:6])
    ATTEND_OK(q=b16(3, 5, 9, 64)[:, :, 2:6])
    APPEND_OK(k=b16(7, 5, 64)[:, 1:3], v=b16(7, 64, 64)[:, 7:9])
    assert [n for n, _ in stub.calls] == ["wc_fp4_cache_append", "wc_fp4_cache_read"] + ["wc_fp4_attention"] * 4 + [
        "wc_fp4_cache_append"]
    strides = [args[1]._obj.q_stride for n, args in stub.calls if n == "wc_fp4_attention"]
    assert strides == [256, 256, 9 * 64, 9 * 64]
    assert stub.calls[-1][1][2] == 5 * 64 and stub.calls[-1][1][4] == 64 * 64


@pytest.mark.parametrize("more", [
    {"cache": torch.empty(5, 2, 2, 34 * 64, dtype=torch.uint8)},
    {"cache": t(torch.int8, 5, 2, 2, 34 * 64)},
    {"cache": cache()[0]},
    {"cache": cache()[:, :1]},
    {"cache": t(torch.uint8, 5, 2, 2, 34 * 48)},
    {"cache": t(torch.uint8, 5, 2, 2, 34 * 288)},
    {"cache": t(torch.uint8, 5, 2, 2, 0)},
    {"cache": t(torch.uint8, 1, 2, 1 << 27, 34 * 64)},
    {"k": b16(7, 2, 32)}, {"k": b16(7, 3, 64)}, {"k": b16(6, 2, 64)}, {"v": b16(8, 2, 64)},
    {"k": t(torch.float32, 7, 2, 64)}, {"v": torch.empty(7, 2, 64, dtype=torch.bfloat16)},
    {"k": b16(7, 64, 2).transpose(1, 2)}, {"k": b16(2, 7, 64).transpose(0, 1)},
    {"k": b16(1, 2, 64).expand(7, 2, 64)}, {"k": b16(7, 2, 128)[:, :, ::2]}, {"k": b16(7, 2, 65)[:, :, :64]},
    {"k": t(torch.bfloat16, 7 * 132)[:7 * 132].view(7, 132)[:, :128].unflatten(1, (2, 64))},  # 132 apart
    {"slots": i32(7)}, {"slots": i64(8)}, {"slots": i64(7, 1)}, {"slots": i64(14)[::2]},
    {"slots": torch.empty(7, dtype=torch.int64)},
])
def test_append_refuses(stub, more):
    with pytest.raises((ValueError, TypeError)):
        APPEND_OK(**more)
    assert stub.calls == []


@pytest.mark.parametrize("more", [
    {"slots": i64(7, 1)}, {"slots": i32(7)}, {"out": (b16(7, 2, 64), b16(6, 2, 64))},
    {"out": (b16(7, 2, 64), t(torch.float16, 7, 2, 64))}, {"out": (b16(7, 4, 64)[:, :2], b16(7, 2, 64))},
])
def test_read_refuses(stub, more):
    with pytest.raises((ValueError, TypeError)):
        READ_OK(**more)
    assert stub.calls == []


@pytest.mark.parametrize("more", [
    {"q": b16(3, 4, 32)}, {"q": b16(4, 64)}, {"q": b16(3, 3, 64)}, {"q": b16(3, 1, 1, 4, 64)},
    {"q": b16(3, 0, 4, 64)}, {"q": b16(3, 17, 4, 64)}, {"q": b16(2, 4, 64)}, {"q": b16(3, 4, 128)[:, :, ::2]},
    {"q": b16(5, 3, 4, 64).transpose(0, 1)[:3, :5]}, {"q": t(torch.float32, 3, 4, 64)},
    {"table": i32(2, 9)}, {"table": i32(27)}, {"table": i64(3, 9)}, {"table": i32(3, 18)[:, ::2]},
    {"lengths": i32(2)}, {"lengths": i64(3)}, {"lengths": i32(3, 1)},
    {"out": b16(3, 4, 32)}, {"out": t(torch.float32, 3, 4, 64)}, {"out": b16(3, 8, 64)[:, :4]},
    {"window": -1}, {"window": 1 << 32},
])
def test_attention_refuses(stub, more):
    with pytest.raises((ValueError, TypeError)):
        ATTEND_OK(**more)
    assert stub.calls == []


def test_attention_workspace(stub):
    stub.need = 1000
    for work in (t(torch.uint8, 999), t(torch.int8, 1000), t(torch.uint8, 2000)[::2],
                 torch.empty(1000, dtype=torch.uint8)):
        with pytest.raises((ValueError, TypeError)):
            ATTEND_OK(work=work)
    assert stub.calls == []
    ATTEND_OK(work=t(torch.uint8, 1000))
    ATTEND_OK()
    assert len(stub.calls) == 2


@pytest.mark.parametrize("args", [(5, 0, 2, 64), (5, 33, 2, 64), (5, 32, 2, 0), (5, 32, 2, 48), (5, 32, 2, 288)])
def test_cache_sizes(args):
    with pytest.raises(ValueError):
        wc.fp4_cache(*args, device=META)
    assert wc.fp4_cache(5, 96, 2, 160, META).shape == (5, 2, 3, 34 * 160)


CALLS = {"fp4_cache_append": APPEND_OK, "fp4_cache_read": READ_OK, "fp4_attention": ATTEND_OK}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("tensors,current,stream,ok", [
    (0, 0, None, True), (1, 1, None, True), (1, 1, 1, True),
    (1, 0, None, False), (0, 1, None, False), (1, 0, 1, False), (0, 0, 1, False)])
def test_device_of_the_tensors(stub, monkeypatch, name, tensors, current, stream, ok):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda v: tensors)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)
    s = None if stream is None else _Stream(stream)
    if ok:
        CALLS[name](stream=s)
        assert [n for n, _ in stub.calls] == ["wc_" + name]
    else:
        with pytest.raises(ValueError, match="device"):
            CALLS[name](stream=s)
        assert stub.calls == []


def test_memory_of_another_stream(stub, monkeypatch):
    """What a call with stream= allocates comes from that stream's pool."""
    import contextlib
    now, made, kept = [3], [], []
    empty = torch.empty

    class Side:
        cuda_stream, device_index = 7, -1

    @contextlib.contextmanager
    def on(s):
        now.append(s.cuda_stream)
        yield
        now.pop()

    def alloc(*a, **k):
        v = empty(*a, **k)
        made.append((now[-1], v))
        return v

    stub.need = 512
    monkeypatch.setattr(wc, "_stream", lambda s=None: now[-1] if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Stream(0))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda v, s: kept.append(v))
    args = {"q": b16(3, 4, 64), "cache": cache(), "table": i32(3, 9), "lengths": i32(3)}
    slots, c = i64(7), cache()
    monkeypatch.setattr(torch, "empty", alloc)
    for call, outputs, all_of in ((lambda: wc.fp4_attention(**args, stream=Side()), 2, 3),
                                  (lambda: wc.fp4_cache_read(c, slots, stream=Side()), 2, 2)):
        made.clear()
        kept.clear()
        out = call()
        assert len(made) == all_of and all(h == 7 for h, _ in made)
        assert len(kept) == outputs and all(any(k is o for k in kept) for o in out)


# ---- the C ABI ---------------------------------------------------------------

def cache_struct(**more):
    v = {"data": 1 << 20, "pages": 5, "page_size": 64, "kv_heads": 2, "head_dim": 64, **more}
    return wc.CacheStruct(*(v[k] for k in ("data", "pages", "page_size", "kv_heads", "head_dim")))


def shape_struct(**more):
    v = {"q_stride": 256, "seqs": 3, "new_tokens": 1, "heads": 4, "table_width": 9, "window": 0, "scale": 1.0, **more}
    return wc.AttentionShape(*(v[f] for f, _ in wc.AttentionShape._fields_))


P = 1 << 20  # a pointer that is aligned, and never followed


def append(c, k=P, ks=128, v=P, vs=128, slots=P, tokens=7):
    return wc._lib.wc_fp4_cache_append(ctypes.byref(c), k, ks, v, vs, slots, tokens, None)


def attend(c, s, q=P, table=P, lengths=P, out=P, lse=None, work=P, size=1 << 40):
    return wc._lib.wc_fp4_attention(ctypes.byref(c), ctypes.byref(s), q, table, lengths, out, lse, work, size, None)


@pytest.mark.parametrize("more,code", [
    ({"data": None}, -1), ({"data": P + 8}, -1), ({"pages": 0}, -1), ({"pages": 1 << 31}, -2),
    ({"pages": 1 << 30, "page_size": 64}, -2), ({"page_size": 0}, -1), ({"page_size": 48}, -1),
    ({"page_size": (1 << 20) + 32}, -1), ({"kv_heads": 0}, -1), ({"kv_heads": 1025}, -1), ({"head_dim": 0}, -1),
    ({"head_dim": 16}, -1), ({"head_dim": 288}, -1)])
def test_abi_caches(more, code):
    c = cache_struct(**more)
    assert append(c) == code
    assert wc._lib.wc_fp4_cache_read(ctypes.byref(c), P, 7, P, P, None) == code
    assert attend(c, shape_struct()) == code
    assert wc._lib.wc_fp4_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(shape_struct())) == 0


def test_abi_append():
    c = cache_struct()
    assert append(c, tokens=0, k=None, v=None, slots=None) == 0
    for more, code in [({"k": None}, -1), ({"k": P + 2}, -1), ({"v": None}, -1), ({"v": P + 8}, -1), ({"slots": None}, -1),
                       ({"slots": P + 4}, -1), ({"ks": 120}, -1), ({"ks": 132}, -1), ({"vs": 64}, -1),
                       ({"vs": 129}, -1), ({"ks": 1 << 31}, -2), ({"tokens": 1 << 31}, -2)]:
        assert append(c, **more) == code, more
    assert wc._lib.wc_fp4_cache_append(None, P, 128, P, 128, P, 7, None) == -1
    for args, code in [((P, 0, None, None), 0), ((None, 7, P, P), -1), ((P + 4, 7, P, P), -1), ((P, 7, None, P), -1),
                       ((P, 7, P, P + 8), -1), ((P, 1 << 31, P, P), -2)]:
        assert wc._lib.wc_fp4_cache_read(ctypes.byref(c), *args, None) == code, args


def test_abi_attention():
    c = cache_struct()
    assert attend(c, shape_struct(seqs=0), q=None, table=None, lengths=None, out=None, work=None) == 0
    for more, code in [({"new_tokens": 0}, -5), ({"new_tokens": 17}, -5), ({"heads": 0}, -1), ({"heads": 3}, -1),
                       ({"heads": 1026}, -1), ({"q_stride": 248}, -1), ({"q_stride": 260}, -1),
                       ({"q_stride": 1 << 31}, -2), ({"table_width": 1 << 25}, -2), ({"seqs": 1 << 24}, -2)]:
        assert attend(c, shape_struct(**more)) == code, more
    s = shape_struct(table_width=900)
    for more in ({"q": None}, {"q": P + 8}, {"table": None}, {"table": P + 2}, {"lengths": None}, {"lengths": P + 2},
                 {"out": None}, {"out": P + 8}, {"lse": P + 2}, {"work": None}, {"work": P + 8}):
        assert attend(c, s, **more) == -1, more
    need = wc._lib.wc_fp4_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(s))
    assert need > 0 and attend(c, s, size=need - 1) == -2
    one = shape_struct(table_width=1)
    assert wc._lib.wc_fp4_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(one)) == 0
    assert wc._lib.wc_fp4_attention(ctypes.byref(c), None, P, P, P, P, None, P, 1 << 40, None) == -5


def test_declared_functions_are_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "wc_attn.h")).read()
    names = re.findall(r"^(?:int|size_t)\s+(wc_\w+)\s*\(", text, re.M)
    assert {"wc_fp4_cache_append", "wc_fp4_cache_read", "wc_fp4_attention_workspace_bytes",
            "wc_fp4_attention"} <= set(names)
    out = subprocess.check_output(["nm", "-D", "--defined-only", wc.LIB_PATH], text=True)
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert set(names) <= exported
    for n in names:
        assert getattr(wc._lib, n).argtypes, n


def test_structs_match_the_header(tmp_path):
    """Sizes and offsets of the structs, by a C program that includes the header."""
    lines = []
    for struct, cls in (("wc_fp4_cache", wc.CacheStruct), ("wc_fp4_attention_shape", wc.AttentionShape)):
        for f, _ in cls._fields_:
            name = "d_data" if f == "data" else f
            lines.append(f'printf("%zu\\n", offsetof({struct}, {name}));')
        lines.append(f'printf("%zu\\n", sizeof({struct}));')
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "wc_attn.h"\nint main(void){\n' +
                   "\n".join(lines) +
                   'printf("%llu\\n", (unsigned long long)WC_FP4_CACHE_BYTES(5, 64, 2, 96));return 0;}\n')
    exe = tmp_path / "s"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                           str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    want = []
    for cls in (wc.CacheStruct, wc.AttentionShape):
        want += [getattr(cls, f).offset for f, _ in cls._fields_] + [ctypes.sizeof(cls)]
    assert got == want + [wc.fp4_cache(5, 64, 2, 96, META).numel()]
