"""The 4-bit tier and the mixture-of-experts layer without a GPU: what the
binding and the C ABI refuse before any device work, the size formulas, and
the 64-bit reference of their GPU tests against hand-written values."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import decode_gemv_sign_amd as wc
from tests import fp4_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
META = torch.device("meta")
P = ctypes.c_void_p


class _StubLib:
    """Stands in for libwc: records calls, returns WC_OK (and a workspace size)."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("wc_"):
            raise AttributeError(name)

        def f(*args):
            if name == "wc_moe_workspace_bytes":
                return 4096
            self.calls.append(name)
            return 0
        return f


class _Stream:
    cuda_stream = 0


@pytest.fixture
def stub(monkeypatch):
    lib = _StubLib()
    monkeypatch.setattr(wc, "_lib", lib)
    monkeypatch.setattr(wc, "_on_device", lambda t: t.device.type == "meta")
    monkeypatch.setattr(wc, "_ptr", lambda t: None)
    monkeypatch.setattr(wc, "_stream", lambda s=None: None)
    monkeypatch.setattr(wc, "_used_on", lambda *a: None)
    return lib


def t(dtype, *shape, device=META):
    return torch.empty(shape, dtype=dtype, device=device)


def b16(*shape, device=META):
    return t(torch.bfloat16, *shape, device=device)


def q4(*shape, device=META):
    g = (shape[-1] + 31) // 32
    return wc.Fp4(t(torch.uint8, *shape[:-1], 16 * g, device=device),
                  t(torch.uint8, *shape[:-1], g, device=device), shape[-1])


# ---- what the binding refuses ------------------------------------------------

def test_valid_fp4_calls_reach_the_library(stub):
    assert tuple(wc.fp4_encode(b16(6, 70)).codes.shape) == (6, 48)
    assert tuple(wc.fp4_encode(b16(2, 6, 70)).scales.shape) == (2, 6, 3)
    assert tuple(wc.fp4_decode(q4(2, 6, 70)).shape) == (2, 6, 70)
    assert tuple(wc.fp4_gemv(q4(6, 70), b16(3, 70)).shape) == (3, 6)
    wc.fp4_gemv(q4(6, 70), b16(70), out=t(torch.float32, 6))
    assert stub.calls == ["wc_fp4_encode"] * 2 + ["wc_fp4_decode"] + ["wc_fp4_gemv"] * 2


@pytest.mark.parametrize("case", ["w_1d", "w_float", "w_host", "w_strided", "out_rows", "out_cols",
                                  "out_dtype", "out_host"])
def test_fp4_encode_rejects(stub, case):
    w, out = b16(6, 70), q4(6, 70)
    if case == "w_1d":
        w = b16(70)
    elif case == "w_float":
        w = t(torch.float32, 6, 70)
    elif case == "w_host":
        w = b16(6, 70, device="cpu")
    elif case == "w_strided":
        w = b16(70, 6).t()
    elif case == "out_rows":
        out = q4(7, 70)
    elif case == "out_cols":
        out = q4(6, 71)
    elif case == "out_dtype":
        out = wc.Fp4(t(torch.int8, 6, 48), out.scales, 70)
    elif case == "out_host":
        out = q4(6, 70, device="cpu")
    with pytest.raises((ValueError, TypeError)):
        wc.fp4_encode(w, out=out)
    assert stub.calls == []


@pytest.mark.parametrize("case", ["scales_short", "codes_short", "cols", "cols_negative", "codes_strided",
                                  "scales_dtype", "out_shape", "out_dtype", "out_strided", "q_1d"])
def test_fp4_decode_rejects(stub, case):
    q, out = q4(6, 70), b16(6, 70)
    if case == "scales_short":
        q = wc.Fp4(q.codes, t(torch.uint8, 6, 2), 70)
    elif case == "codes_short":
        q = wc.Fp4(t(torch.uint8, 6, 35), q.scales, 70)
    elif case == "cols":
        q = wc.Fp4(q.codes, q.scales, 97)
    elif case == "cols_negative":
        q = wc.Fp4(t(torch.uint8, 6, 0), t(torch.uint8, 6, 0), -1)
    elif case == "codes_strided":
        q = wc.Fp4(t(torch.uint8, 48, 6).t(), q.scales, 70)
    elif case == "scales_dtype":
        q = wc.Fp4(q.codes, t(torch.float32, 6, 3), 70)
    elif case == "out_shape":
        out = b16(6, 71)
    elif case == "out_dtype":
        out = t(torch.float32, 6, 70)
    elif case == "out_strided":
        out = b16(70, 6).t()
    elif case == "q_1d":
        q = wc.Fp4(t(torch.uint8, 48), t(torch.uint8, 3), 70)
    with pytest.raises((ValueError, TypeError)):
        wc.fp4_decode(q, out=out)
    assert stub.calls == []


@pytest.mark.parametrize("case", ["stack", "x_cols", "x_3d", "x_dtype", "x_host", "x_strided", "batch_0",
                                  "batch_257", "out_shape", "out_dtype", "codes_host"])
def test_fp4_gemv_rejects(stub, case):
    q, x, out = q4(6, 70), b16(3, 70), t(torch.float32, 3, 6)
    if case == "stack":
        q = q4(1, 6, 70)
    elif case == "x_cols":
        x = b16(3, 69)
    elif case == "x_3d":
        x = b16(1, 3, 70)
    elif case == "x_dtype":
        x = t(torch.float32, 3, 70)
    elif case == "x_host":
        x = b16(3, 70, device="cpu")
    elif case == "x_strided":
        x = b16(3, 140)[:, ::2]
    elif case == "batch_0":
        x, out = b16(0, 70), t(torch.float32, 0, 6)
    elif case == "batch_257":
        x, out = b16(257, 70), t(torch.float32, 257, 6)
    elif case == "out_shape":
        out = t(torch.float32, 3, 7)
    elif case == "out_dtype":
        out = b16(3, 6)
    elif case == "codes_host":
        q = wc.Fp4(t(torch.uint8, 6, 48, device="cpu"), q.scales, 70)
    with pytest.raises((ValueError, TypeError)):
        wc.fp4_gemv(q, x, out=out)
    assert stub.calls == []


def moe_args():
    """tokens 3, hidden 64, inter 40, experts 5."""
    return dict(x=b16(3, 64), router=b16(5, 64), gate_up=b16(5, 80, 64), down=b16(5, 64, 40), top_k=2)


def test_valid_moe_calls_reach_the_library(stub):
    y, ids, weights = wc.moe(**moe_args())
    assert tuple(y.shape) == (3, 64) and tuple(ids.shape) == tuple(weights.shape) == (3, 2)
    wc.moe(**{**moe_args(), "gate_up": q4(5, 80, 64)}, bias=t(torch.float32, 5), scoring=wc.SIGMOID)
    wc.moe(**{**moe_args(), "down": q4(5, 64, 40)}, work=t(torch.uint8, 4096), out=b16(3, 64))
    assert stub.calls == ["wc_moe"] * 3


@pytest.mark.parametrize("case", [
    "x_1d", "x_hidden", "x_dtype", "x_host", "x_strided", "tokens_0", "tokens_65", "router_hidden",
    "router_dtype", "gate_up_rows", "gate_up_2d", "gate_up_experts", "gate_up_strided", "down_rows",
    "down_2d", "down_inter", "fp4_rows", "fp4_codes", "bias_shape", "bias_dtype", "bias_host",
    "work_short", "work_dtype", "out_shape", "out_dtype", "out_host"])
def test_moe_rejects(stub, case):
    a, more = moe_args(), {}
    if case == "x_1d":
        a["x"] = b16(64)
    elif case == "x_hidden":
        a["x"] = b16(3, 63)
    elif case == "x_dtype":
        a["x"] = t(torch.float32, 3, 64)
    elif case == "x_host":
        a["x"] = b16(3, 64, device="cpu")
    elif case == "x_strided":
        a["x"] = b16(3, 128)[:, ::2]
    elif case == "tokens_0":
        a["x"] = b16(0, 64)
    elif case == "tokens_65":
        a["x"] = b16(65, 64)
    elif case == "router_hidden":
        a["router"] = b16(5, 65)
    elif case == "router_dtype":
        a["router"] = t(torch.float32, 5, 64)
    elif case == "gate_up_rows":
        a["gate_up"] = b16(5, 40, 64)
    elif case == "gate_up_2d":
        a["gate_up"] = b16(80, 64)
    elif case == "gate_up_experts":
        a["gate_up"] = b16(4, 80, 64)
    elif case == "gate_up_strided":
        a["gate_up"] = b16(5, 64, 80).transpose(1, 2)
    elif case == "down_rows":
        a["down"] = b16(5, 63, 40)
    elif case == "down_2d":
        a["down"] = b16(64, 40)
    elif case == "down_inter":
        a["down"] = b16(5, 64, 39)
    elif case == "fp4_rows":
        a["gate_up"] = q4(5, 81, 64)
    elif case == "fp4_codes":
        a["down"] = wc.Fp4(t(torch.uint8, 5, 64, 20), t(torch.uint8, 5, 64, 2), 40)
    elif case == "bias_shape":
        more["bias"] = t(torch.float32, 4)
    elif case == "bias_dtype":
        more["bias"] = b16(5)
    elif case == "bias_host":
        more["bias"] = t(torch.float32, 5, device="cpu")
    elif case == "work_short":
        more["work"] = t(torch.uint8, 4095)
    elif case == "work_dtype":
        more["work"] = t(torch.int8, 4096)
    elif case == "out_shape":
        more["out"] = b16(3, 63)
    elif case == "out_dtype":
        more["out"] = t(torch.float32, 3, 64)
    elif case == "out_host":
        more["out"] = b16(3, 64, device="cpu")
    with pytest.raises((ValueError, TypeError)):
        wc.moe(**a, **more)
    assert stub.calls == []


# ---- what the C ABI refuses --------------------------------------------------

def test_fp4_argument_checks_before_device_work():
    lib, ok = wc._lib, P(64)
    for f, rest in ((lib.wc_fp4_encode, (ok, ok)), (lib.wc_fp4_decode, None)):
        call = (lambda a, r, c: f(a, r, c, ok, ok, None)) if rest else \
            (lambda a, r, c: f(ok, a, r, c, ok, None))
        assert call(ok, 1 << 40, 1) == -2
        assert call(ok, 1, (1 << 24) + 1) == -2
        assert call(None, 4, 32) == -1
        assert call(None, 0, 32) == call(None, 4, 0) == 0  # nothing to do
    assert lib.wc_fp4_encode(P(8), 4, 32, ok, ok, None) == -1
    assert lib.wc_fp4_encode(ok, 4, 32, P(8), ok, None) == -1
    assert lib.wc_fp4_decode(P(8), ok, 4, 32, ok, None) == -1
    assert lib.wc_fp4_decode(ok, ok, 4, 32, P(8), None) == -1
    g = lib.wc_fp4_gemv
    assert g(ok, ok, 4, 32, ok, 0, ok, None) == g(ok, ok, 4, 32, ok, 257, ok, None) == -5
    assert g(None, ok, 4, 32, ok, 1, ok, None) == g(ok, None, 4, 32, ok, 1, ok, None) == -1
    assert g(P(8), ok, 4, 32, ok, 1, ok, None) == g(ok, ok, 4, 32, P(8), 1, ok, None) == -1
    assert g(ok, ok, 4, 32, None, 1, ok, None) == g(ok, ok, 4, 32, ok, 1, None, None) == -1
    assert g(ok, ok, 4, 32, ok, 1, P(66), None) == -1
    assert g(ok, ok, 1 << 40, 32, ok, 1, ok, None) == g(ok, ok, 1, (1 << 24) + 1, ok, 1, ok, None) == -2
    assert g(None, None, 0, 32, None, 1, None, None) == 0


def _moe_call(shape=(3, 64, 40, 5, 2, 0, 1, 1.0), x=64, router=64, bias=None, gu=(0, 64, None),
              dn=(1, 64, 7), y=64, ids=None, weights=None, work=64, work_bytes=1 << 30):
    s = None if shape is None else ctypes.byref(wc.MoeShape(*shape))
    e = [None if v is None else ctypes.byref(wc.MoeExperts(*v)) for v in (gu, dn)]
    return wc._lib.wc_moe(s, P(x), P(router), P(bias), *e, P(y), P(ids), P(weights), P(work),
                          work_bytes, None)


@pytest.mark.parametrize("change,code", [
    (dict(shape=None), -1), (dict(gu=None), -1), (dict(dn=None), -1),
    (dict(shape=(0, 64, 40, 5, 2, 0, 1, 1.0)), -5), (dict(shape=(65, 64, 40, 5, 2, 0, 1, 1.0)), -5),
    (dict(shape=(3, 0, 40, 5, 2, 0, 1, 1.0)), -5), (dict(shape=(3, 64, 0, 5, 2, 0, 1, 1.0)), -5),
    (dict(shape=(3, 65537, 40, 5, 2, 0, 1, 1.0)), -5),
    (dict(shape=(3, 64, 40, 0, 0, 0, 1, 1.0)), -5), (dict(shape=(3, 64, 40, 513, 2, 0, 1, 1.0)), -5),
    (dict(shape=(3, 64, 40, 5, 6, 0, 1, 1.0)), -5), (dict(shape=(3, 64, 40, 32, 17, 0, 1, 1.0)), -5),
    (dict(shape=(3, 64, 40, 5, 2, 2, 1, 1.0)), -1), (dict(shape=(3, 64, 40, 5, 2, 0, 2, 1.0)), -1),
    (dict(gu=(2, 64, 7)), -1), (dict(gu=(0, 8, None)), -1), (dict(gu=(0, None, None)), -1),
    (dict(dn=(1, 64, None)), -1), (dict(x=None), -1), (dict(x=8), -1), (dict(router=8), -1),
    (dict(router=None), -1), (dict(bias=66), -1), (dict(y=None), -1), (dict(y=65), -1),
    (dict(ids=2), -1), (dict(weights=2), -1), (dict(work=None), -1), (dict(work=8), -1),
    (dict(work_bytes=100), -2)])
def test_moe_argument_checks_before_device_work(change, code):
    assert _moe_call(**change) == code


def test_moe_workspace_bytes():
    a = wc.moe_workspace_bytes(1, 64, 40, 5, 2)
    assert 0 < a < wc.moe_workspace_bytes(64, 64, 40, 5, 2)
    with pytest.raises(wc.WCError):
        wc.moe_workspace_bytes(65, 64, 40, 5, 2)
    with pytest.raises(wc.WCError):
        wc.moe_workspace_bytes(1, 64, 40, 5, 6)


def test_new_headers_are_c_and_exported(tmp_path):
    names = set()
    for h in ("wc_fp4.h", "wc_moe.h"):
        text = open(os.path.join(ROOT, "include", h)).read()
        names |= set(re.findall(r"^(?:int|size_t)\s+(wc_\w+)\s*\(", text, re.M))
    assert names == {"wc_fp4_encode", "wc_fp4_decode", "wc_fp4_gemv", "wc_moe", "wc_moe_workspace_bytes"}
    for n in names:
        assert hasattr(wc._lib, n)
    src = tmp_path / "h.c"
    src.write_text('#include <stdio.h>\n#include "wc_moe.h"\nint main(void){printf("%zu %zu %llu %llu\\n",'
                   'sizeof(wc_moe_shape), sizeof(wc_moe_experts),'
                   '(unsigned long long)WC_FP4_CODE_BYTES(6, 70),'
                   '(unsigned long long)WC_FP4_SCALE_BYTES(6, 70));return 0;}\n')
    exe = tmp_path / "h"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                           str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [ctypes.sizeof(wc.MoeShape), ctypes.sizeof(wc.MoeExperts), 6 * 48, 6 * 3]


# ---- the reference of the GPU tests ------------------------------------------

def bits(*v):
    return fp4_ref.to_bits(np.array(v, dtype=np.float64)).reshape(1, -1)


def test_reference_rounding_and_scales():
    # max 6: scale 1; ties to the even code; signs, -0 included
    w = bits(6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -5, 0.26, -0.0)
    codes, scales = fp4_ref.encode(w)
    assert scales.tolist() == [[127]]
    assert fp4_ref.values(codes, scales, 12)[0].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.0, -4, 0.5, -0.0]
    # max 7 keeps scale 1 and comes out as 6; just above it the scale doubles
    for top, e, back in ((7.0, 127, 6.0), (7.03125, 128, 8.0), (8.0, 128, 8.0), (3.5, 126, 3.0),
                         (3.515625, 127, 4.0)):
        codes, scales = fp4_ref.encode(bits(top))
        assert (scales[0, 0], fp4_ref.values(codes, scales, 1)[0, 0]) == (e, back), top


def test_reference_limits():
    codes, scales = fp4_ref.encode(bits(0, 0))
    assert scales.tolist() == [[1]] and not codes.any()
    # the largest BF16: 4 * 2^126 would be infinite, so 3 * 2^126
    codes, scales = fp4_ref.encode(np.array([[0x7F7F, 0xFF7F]], dtype=np.uint16))
    assert scales.tolist() == [[253]] and codes[0, 0] == 0xD5
    assert fp4_ref.values(codes, scales, 2)[0].tolist() == [3 * 2.0 ** 126, -3 * 2.0 ** 126]
    for v in (0x7F80, 0xFF80, 0x7FC0):
        codes, scales = fp4_ref.encode(np.array([[v, 0x3F80]], dtype=np.uint16))
        assert scales.tolist() == [[255]] and not codes.any()
        assert np.isnan(fp4_ref.values(codes, scales, 2)).all()
    # no finite weight moves by more than one scale (half of the largest step)
    v = np.arange(1 << 16, dtype=np.uint32)
    v = v[(v >> 7 & 0xFF) != 0xFF].astype(np.uint16)
    v = v[np.random.default_rng(0).permutation(v.size)][: v.size // 32 * 32].reshape(-1, 32)
    codes, scales = fp4_ref.encode(v)
    off = np.abs(fp4_ref.values(codes, scales, 32) - fp4_ref.of_bits(v))
    assert (off <= np.ldexp(1.0, scales.astype(int) - 127)).all()


def test_reference_moe_by_hand():
    x, router = np.array([[1.0, 0.0]]), np.array([[0.0, 1], [2, 0], [2, 0]])
    gu = np.zeros((3, 2, 2))
    gu[1], gu[2] = [[1, 0], [3, 0]], [[2, 0], [1, 0]]
    dn = np.array([[[0.0], [0]], [[1], [0]], [[0], [1]]])
    y, bound, ids, weights, _, _ = fp4_ref.moe(x, router, gu, dn, 2)
    assert ids.tolist() == [[1, 2]] and weights.tolist() == [[0.5, 0.5]]
    silu = lambda a: a / (1 + np.exp(-a))  # noqa: E731
    np.testing.assert_allclose(y, [[0.5 * silu(1) * 3, 0.5 * silu(2)]], rtol=1e-14)
    assert (bound > 2.0 ** -8 * np.abs(y)).all()
