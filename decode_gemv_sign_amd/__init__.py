"""decode_gemv_sign_amd — Python binding of libwc (include/wc.h).

Lossless BF16 sign+exponent coding on AMD MI355X: a per-tensor 15-entry
dictionary of sign+exponent symbols, 4-bit codes, an exact escape stream,
and the raw part kept as stored (byte-split: the low byte; K15: the 7-bit
mantissa) — page "Prueba de GLM-5.2 reduce la memoria BF16 en casi un 25%",
section "Cómo funciona la compresión" — with exact decode and decode fused
into GEMV (page "Compresión de pesos LLM sin pérdida vs 8-bit GGUF: ¿qué está
listo para producción?", section "¿Qué significa “sin pérdida” para los pesos
de un LLM?").

Next to it a 4-bit tier that loses precision, for tensors that 12 bits per
weight leave too large (fp4_encode, fp4_decode, fp4_gemv; include/wc_fp4.h),
a mixture-of-experts layer for a few tokens on BF16 or 4-bit experts
(moe; include/wc_moe.h), a cache of keys and values in the same 4-bit form
with the attention over it (fp4_cache, fp4_cache_append, fp4_cache_read,
fp4_attention), the attention of whole prompts (prompt_attention;
include/wc_attn.h), and the log probabilities of tokens (token_logprobs;
include/wc_logprob.h).

This module only marshals arguments: every step runs in the HIP kernels of
libwc.so, on the caller's current torch stream.  PyTorch provides device
memory and streams.  There is no CPU fallback: importing this package
without a built libwc.so raises ImportError.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

import torch  # loaded first, so libwc binds to the HIP runtime torch already uses

__all__ = [
    "BYTESPLIT", "K15", "RAW", "AUTO", "COMPACT", "FLAG_COMPACT", "Header", "WCError", "workspace_bytes", "build_dict", "encode_into", "encode_into_noalloc",
    "encode", "decode", "decode_gemv", "gemv_bf16", "bits_per_weight", "read_header",
    "crc32", "container_crcs", "artifact_write", "artifact_entries", "artifact_read",
    "artifact_verify", "LIB_PATH",
    "Fp4", "fp4_encode", "fp4_decode", "fp4_gemv", "SOFTMAX", "SIGMOID", "moe", "moe_workspace_bytes",
    "fp4_cache", "fp4_cache_append", "fp4_cache_read", "fp4_attention", "fp4_attention_workspace_bytes",
    "prompt_attention", "token_logprobs", "token_logprobs_workspace_bytes",
]

BYTESPLIT = 0
K15 = 1
RAW = 2   # fallback layout: the BF16 bit patterns as stored
AUTO = 3  # build_dict / encode only: the smallest of the three
COMPACT = 0x10  # OR into a layout: escape symbols only (header flag FLAG_COMPACT)
FLAG_COMPACT = 1
MAX_BATCH = 256
STAGE_SYMBOLS = 256  # WC_STAGE_SYMBOLS
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libwc.so")

_CODES = {0: "WC_OK", -1: "WC_E_ARG", -2: "WC_E_SIZE", -3: "WC_E_CORRUPT", -4: "WC_E_HIP",
          -5: "WC_E_UNSUPPORTED", -6: "WC_E_IO"}


class WCError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {_CODES.get(code, code)}")
        self.code = code


class Header(ctypes.Structure):
    """wc_header: the first 128 bytes of every container."""
    _fields_ = [
        ("magic", ctypes.c_uint32), ("version", ctypes.c_uint16), ("layout", ctypes.c_uint8),
        ("n_dict", ctypes.c_uint8), ("n", ctypes.c_uint64), ("n_esc", ctypes.c_uint64),
        ("dict", ctypes.c_uint16 * 16), ("off_codes", ctypes.c_uint64),
        ("off_raw", ctypes.c_uint64), ("off_esc_pos", ctypes.c_uint64),
        ("off_esc_sym", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64),
        ("off_esc_idx", ctypes.c_uint64), ("flags", ctypes.c_uint8),
        ("reserved", ctypes.c_uint8 * 23),
    ]

    def to_bytes(self) -> bytes:
        return ctypes.string_at(ctypes.addressof(self), ctypes.sizeof(self))

    @classmethod
    def from_bytes(cls, b: bytes) -> "Header":
        if len(b) < 128:
            raise ValueError("a header is 128 bytes")
        return cls.from_buffer_copy(bytes(b[:128]))


assert ctypes.sizeof(Header) == 128


class ArtifactInfo(ctypes.Structure):
    """wc_artifact_info: one entry of a serialized artifact."""
    _fields_ = [
        ("name", ctypes.c_char * 96), ("ndim", ctypes.c_uint32), ("layout", ctypes.c_uint32),
        ("shape", ctypes.c_uint64 * 4), ("offset", ctypes.c_uint64), ("bytes", ctypes.c_uint64),
        ("src_crc", ctypes.c_uint32), ("stream_crc", ctypes.c_uint32 * 6),
        ("reserved", ctypes.c_uint32),
    ]


class MoeShape(ctypes.Structure):
    """wc_moe_shape (include/wc_moe.h)."""
    _fields_ = [(n, ctypes.c_uint32) for n in ("tokens", "hidden", "inter", "experts", "top_k",
                                               "scoring", "flags")] + [("scale", ctypes.c_float)]


class MoeExperts(ctypes.Structure):
    """wc_moe_experts (include/wc_moe.h)."""
    _fields_ = [("kind", ctypes.c_uint32), ("data", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class CacheStruct(ctypes.Structure):
    """wc_fp4_cache (include/wc_attn.h)."""
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_uint64)] + [
        (n, ctypes.c_uint32) for n in ("page_size", "kv_heads", "head_dim")]


class AttentionShape(ctypes.Structure):
    """wc_fp4_attention_shape (include/wc_attn.h)."""
    _fields_ = [("q_stride", ctypes.c_uint64)] + [
        (n, ctypes.c_uint32) for n in ("seqs", "new_tokens", "heads", "table_width", "window")] + [
        ("scale", ctypes.c_float)]


class PromptShape(ctypes.Structure):
    """wc_prompt_shape (include/wc_attn.h)."""
    _fields_ = [(n, ctypes.c_uint64) for n in ("tokens", "q_stride", "k_stride", "v_stride")] + [
        (n, ctypes.c_uint32) for n in ("seqs", "heads", "kv_heads", "head_dim", "window")] + [
        ("scale", ctypes.c_float)]


class LogprobShape(ctypes.Structure):
    """wc_logprob_shape (include/wc_logprob.h)."""
    _fields_ = [("stride", ctypes.c_uint64)] + [(n, ctypes.c_uint32) for n in ("rows", "vocab", "kind", "top")]


def _load(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is not built; run `python -m decode_gemv_sign_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    U64 = ctypes.c_uint64
    HP = ctypes.POINTER(Header)
    lib.wc_build_dict.argtypes = [ctypes.c_int, P, U64, P, ctypes.c_size_t, P, HP]
    lib.wc_encode.argtypes = [HP, P, P, ctypes.c_size_t, P, ctypes.c_size_t, P]
    lib.wc_encode_noalloc.argtypes = [HP, P, P, ctypes.c_size_t, P]
    lib.wc_decode.argtypes = [HP, P, ctypes.c_size_t, P, P]
    lib.wc_decode_gemv.argtypes = [HP, P, ctypes.c_size_t, U64, U64, P, ctypes.c_uint32, P, P]
    lib.wc_gemv_bf16.argtypes = [P, U64, U64, P, ctypes.c_uint32, P, P]
    lib.wc_bits_per_weight.argtypes = [HP, ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_double)]
    lib.wc_crc32.argtypes = [ctypes.c_uint32, P, ctypes.c_size_t]
    lib.wc_crc32.restype = ctypes.c_uint32
    lib.wc_container_crcs.argtypes = [P, ctypes.c_size_t, P]
    lib.wc_artifact_write.argtypes = [ctypes.c_char_p, ctypes.c_uint32,
                                      ctypes.POINTER(ctypes.c_char_p), P, P,
                                      ctypes.POINTER(ctypes.c_void_p), P, P]
    lib.wc_artifact_count.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_uint32)]
    lib.wc_artifact_entry.argtypes = [ctypes.c_char_p, ctypes.c_uint32,
                                      ctypes.POINTER(ArtifactInfo)]
    lib.wc_artifact_read.argtypes = [ctypes.c_char_p, ctypes.c_uint32, P, ctypes.c_size_t]
    lib.wc_fp4_encode.argtypes = [P, U64, U64, P, P, P]
    lib.wc_fp4_decode.argtypes = [P, P, U64, U64, P, P]
    lib.wc_fp4_gemv.argtypes = [P, P, U64, U64, P, ctypes.c_uint32, P, P]
    lib.wc_moe_workspace_bytes.argtypes = [ctypes.POINTER(MoeShape)]
    lib.wc_moe_workspace_bytes.restype = ctypes.c_size_t
    EP = ctypes.POINTER(MoeExperts)
    lib.wc_moe.argtypes = [ctypes.POINTER(MoeShape), P, P, P, EP, EP, P, P, P, P, ctypes.c_size_t, P]
    CP, AP = ctypes.POINTER(CacheStruct), ctypes.POINTER(AttentionShape)
    lib.wc_fp4_cache_append.argtypes = [CP, P, U64, P, U64, P, U64, P]
    lib.wc_fp4_cache_read.argtypes = [CP, P, U64, P, P, P]
    lib.wc_fp4_attention_workspace_bytes.argtypes = [CP, AP]
    lib.wc_fp4_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.wc_fp4_attention.argtypes = [CP, AP, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.wc_prompt_attention.argtypes = [ctypes.POINTER(PromptShape), P, P, P, P, P, P, P]
    LP = ctypes.POINTER(LogprobShape)
    lib.wc_token_logprobs_workspace_bytes.argtypes = [LP]
    lib.wc_token_logprobs_workspace_bytes.restype = ctypes.c_size_t
    lib.wc_token_logprobs.argtypes = [LP, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    for f in (lib.wc_token_logprobs, lib.wc_prompt_attention, lib.wc_fp4_cache_append, lib.wc_fp4_cache_read, lib.wc_fp4_attention, lib.wc_fp4_encode, lib.wc_fp4_decode, lib.wc_fp4_gemv, lib.wc_moe,
              lib.wc_build_dict, lib.wc_encode, lib.wc_encode_noalloc, lib.wc_decode, lib.wc_decode_gemv,
              lib.wc_gemv_bf16, lib.wc_bits_per_weight, lib.wc_container_crcs,
              lib.wc_artifact_write, lib.wc_artifact_count, lib.wc_artifact_entry,
              lib.wc_artifact_read):
        f.restype = ctypes.c_int
    return lib


_lib = _load()


def use_library(path: str):
    """Bind this module to another build of libwc (e.g. a tuning variant)."""
    global _lib
    _lib = _load(path)


def _check(st: int, what: str):
    if st != 0:
        raise WCError(st, what)


def _stream(stream=None) -> int:
    """The hipStream_t to use: the current one's handle, read without building
    a torch Stream (0.2 against 3 us, a fifth of a small call)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _used_on(*tensors):
    """Memory of another stream's pool that the caller reads on the current
    stream is not handed out again before that one is done with it."""
    for t in tensors:
        t.record_stream(torch.cuda.current_stream())


def _empty(shape, dtype, device, stream, returned: bool = True) -> torch.Tensor:
    """Memory for a call on `stream` (None: the current one) to write, and for
    the caller to read if `returned`.  It is taken from that stream's pool: what
    was freed to the current stream's may still be in use by work queued there,
    which `stream` does not wait for."""
    if stream is None or stream.cuda_stream == _stream():
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "device_index"):  # not torch's: an object with the handle alone
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        _used_on(t)
    return t


def _new(like: torch.Tensor, shape, dtype, stream, returned: bool = True) -> torch.Tensor:
    """_empty on the device of `like`, in less time on the current stream."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    return _empty(shape, dtype, like.device, stream, returned)


def _on_device(t: torch.Tensor) -> bool:
    """True for a tensor in GPU memory (the library takes device pointers only)."""
    return t.is_cuda


def _bits16(t: torch.Tensor, what: str) -> torch.Tensor:
    """A contiguous 16-bit device tensor viewed as raw BF16 bit patterns."""
    if not _on_device(t):
        raise ValueError(f"{what} must be a device tensor")
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{what} must hold BF16 bit patterns (bfloat16, int16 or uint16)")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _bytes(t: torch.Tensor, what: str, need: int) -> torch.Tensor:
    """A contiguous uint8 device tensor of at least `need` bytes."""
    if not _on_device(t):
        raise ValueError(f"{what} must be a device tensor")
    if t.dtype != torch.uint8:
        raise TypeError(f"{what} must be a uint8 tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() < need:
        raise ValueError(f"{what} holds {t.numel()} bytes, {need} needed")
    return t


def _same_device(what: str, *ts: torch.Tensor):
    first = ts[0].get_device()
    for t in ts:
        if t.get_device() != first:
            devs = sorted({str(t.device) for t in ts})
            raise ValueError(f"{what}: tensors on different devices {devs}")


def _placed(what: str, stream, *ts: torch.Tensor):
    """The tensors must be on the current device, where the kernels run, and
    so must `stream` (None: the current one)."""
    device = ts[0].get_device()
    for t in ts:
        if t.get_device() != device:
            _same_device(what, *ts)
    if device < 0:  # of no GPU: refused before
        return
    here = torch._C._cuda_getDevice()
    if device != here:
        raise ValueError(f"{what}: tensors on device {device}, the current device is {here}")
    if stream is not None and getattr(stream, "device_index", device) != device:
        raise ValueError(f"{what}: tensors on device {device}, the stream is on {stream.device_index}")


def _batch_of(x: torch.Tensor, cols: int, what: str = "x") -> int:
    """Rows of x, which must be exactly [batch, cols] (or [cols] for batch 1):
    the library reads batch * cols values and cannot check that itself."""
    if x.dim() == 1:
        batch = 1
    elif x.dim() == 2:
        batch = x.shape[0]
    else:
        raise ValueError(f"{what} must be [batch, cols] or [cols], got {tuple(x.shape)}")
    if x.shape[-1] != cols or x.numel() != batch * cols:
        raise ValueError(f"{what} has shape {tuple(x.shape)}, expected ({batch}, {cols})")
    if not 1 <= batch <= MAX_BATCH:
        raise ValueError(f"batch {batch} outside 1..{MAX_BATCH}")
    return batch


def _gemv_out(out: torch.Tensor, batch: int, rows: int, what: str = "out") -> torch.Tensor:
    """y must be fp32 [batch, rows] (or [rows] for batch 1), contiguous, on the device."""
    if not _on_device(out):
        raise ValueError(f"{what} must be a device tensor")
    if out.dtype != torch.float32:
        raise TypeError(f"{what} must be float32")
    if not out.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    ok = tuple(out.shape) == (batch, rows) or (batch == 1 and tuple(out.shape) == (rows,))
    if not ok:
        raise ValueError(f"{what} has shape {tuple(out.shape)}, expected ({batch}, {rows})")
    return out


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def workspace_bytes(n: int) -> int:
    """WC_WORKSPACE_BYTES(n)."""
    return 20528 + (16 + 6 * STAGE_SYMBOLS) * ((n + 8191) // 8192)


def _workspace(n: int, device, stream) -> torch.Tensor:
    return _empty(workspace_bytes(n), torch.uint8, device, stream, returned=False)


def build_dict(w: torch.Tensor, layout: int, work: torch.Tensor | None = None,
               stream=None) -> Header:
    """wc_build_dict: dictionary + complete container header for w (waits)."""
    w = _bits16(w, "w")
    n = w.numel()
    if work is None:
        work = _workspace(n, w.device, stream)
    _bytes(work, "work", workspace_bytes(n))
    _same_device("build_dict", w, work)
    h = Header()
    _check(_lib.wc_build_dict(layout, _ptr(w), n, _ptr(work), work.numel(), _stream(stream),
                              ctypes.byref(h)), "wc_build_dict")
    return h


def encode_into(h: Header, w: torch.Tensor, container: torch.Tensor,
                work: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """wc_encode into a caller-allocated uint8 container (asynchronous)."""
    w = _bits16(w, "w")
    if w.numel() != h.n:
        raise ValueError(f"w has {w.numel()} weights, the header {h.n}")
    _bytes(container, "container", h.total_bytes)
    if work is None:
        work = _workspace(w.numel(), w.device, stream)
    _bytes(work, "work", workspace_bytes(w.numel()))
    _same_device("encode_into", w, container, work)
    _check(_lib.wc_encode(ctypes.byref(h), _ptr(w), _ptr(container), container.numel(),
                          _ptr(work), work.numel(), _stream(stream)), "wc_encode")
    return container


def encode_into_noalloc(h: Header, w: torch.Tensor, container: torch.Tensor,
                        stream=None) -> torch.Tensor:
    """wc_encode_noalloc: as encode_into, with the library's own per-GPU
    scratch instead of a workspace (nothing is allocated; calls that overlap
    on one GPU race)."""
    w = _bits16(w, "w")
    if w.numel() != h.n:
        raise ValueError(f"w has {w.numel()} weights, the header {h.n}")
    _bytes(container, "container", h.total_bytes)
    _same_device("encode_into_noalloc", w, container)
    _check(_lib.wc_encode_noalloc(ctypes.byref(h), _ptr(w), _ptr(container), container.numel(),
                                  _stream(stream)), "wc_encode_noalloc")
    return container


def encode(w: torch.Tensor, layout: int, stream=None):
    """(header, container): dictionary, then the whole container on the device."""
    w = _bits16(w, "w")
    work = _workspace(w.numel(), w.device, stream)
    h = build_dict(w, layout, work, stream)
    c = _empty(h.total_bytes, torch.uint8, w.device, stream)
    encode_into(h, w, c, work, stream)
    return h, c


def read_header(container: torch.Tensor) -> Header:
    """Copy a container's first 128 bytes back to the host (synchronises)."""
    return Header.from_bytes(container[:128].cpu().numpy().tobytes())


def decode(h: Header, container: torch.Tensor, out: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """wc_decode: the n BF16 bit patterns (int16 tensor unless `out` is given)."""
    _bytes(container, "container", h.total_bytes)
    if out is None:
        out = _empty(h.n, torch.int16, container.device, stream)
    out = _bits16(out, "out")
    if out.numel() < h.n:
        raise ValueError(f"out holds {out.numel()} weights, {h.n} needed")
    _same_device("decode", container, out)
    _check(_lib.wc_decode(ctypes.byref(h), _ptr(container), container.numel(), _ptr(out),
                          _stream(stream)), "wc_decode")
    return out


def decode_gemv(h: Header, container: torch.Tensor, rows: int, cols: int, x: torch.Tensor,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """wc_decode_gemv: y [batch, rows] fp32 for x [batch, cols] BF16."""
    _bytes(container, "container", h.total_bytes)
    if rows * cols != h.n:
        raise ValueError(f"rows * cols = {rows * cols}, the header holds {h.n} weights")
    x = _bits16(x, "x")
    batch = _batch_of(x, cols)
    if out is None:
        out = _empty((batch, rows), torch.float32, container.device, stream)
    _gemv_out(out, batch, rows)
    _same_device("decode_gemv", container, x, out)
    _check(_lib.wc_decode_gemv(ctypes.byref(h), _ptr(container), container.numel(), rows, cols,
                               _ptr(x), batch, _ptr(out), _stream(stream)), "wc_decode_gemv")
    return out


def gemv_bf16(w: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """wc_gemv_bf16: plain BF16 GEMV, W [rows, cols], x [batch, cols] -> [batch, rows]."""
    w = _bits16(w, "w")
    if w.dim() != 2:
        raise ValueError(f"w must be [rows, cols], got {tuple(w.shape)}")
    x = _bits16(x, "x")
    rows, cols = w.shape
    batch = _batch_of(x, cols)
    if out is None:
        out = _empty((batch, rows), torch.float32, w.device, stream)
    _gemv_out(out, batch, rows)
    _same_device("gemv_bf16", w, x, out)
    _check(_lib.wc_gemv_bf16(_ptr(w), rows, cols, _ptr(x), batch, _ptr(out), _stream(stream)),
           "wc_gemv_bf16")
    return out


def bits_per_weight(h: Header):
    """(bits/weight with all overhead, payload bits/weight)."""
    b = ctypes.c_double()
    p = ctypes.c_double()
    _check(_lib.wc_bits_per_weight(ctypes.byref(h), ctypes.byref(b), ctypes.byref(p)),
           "wc_bits_per_weight")
    return b.value, p.value


# ---- serialized artifact (host side; include/wc.h) --------------------------

def _host_u8(a):
    import numpy as np
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(a).view(np.uint8).reshape(-1)


def crc32(data, crc: int = 0) -> int:
    """wc_crc32 over a host buffer (numpy array, bytes or CPU/device tensor)."""
    if isinstance(data, (bytes, bytearray)):
        buf = ctypes.create_string_buffer(bytes(data), len(data))
        return _lib.wc_crc32(crc, buf, len(data))
    a = _host_u8(data)
    return _lib.wc_crc32(crc, ctypes.c_void_p(a.ctypes.data), a.size)


def container_crcs(container):
    """The six region CRCs of a container (host copy)."""
    a = _host_u8(container)
    out = (ctypes.c_uint32 * 6)()
    _check(_lib.wc_container_crcs(ctypes.c_void_p(a.ctypes.data), a.size, out), "wc_container_crcs")
    return list(out)


def artifact_write(path: str, items):
    """items: (name, shape, container, src_crc) per tensor; containers are
    copied to the host if they are device tensors."""
    import numpy as np
    items = list(items)
    n = len(items)
    names = (ctypes.c_char_p * max(n, 1))(*[it[0].encode() for it in items])
    ndims = np.zeros(max(n, 1), dtype=np.uint32)
    shapes = np.zeros((max(n, 1), 4), dtype=np.uint64)
    hosts = [_host_u8(it[2]) for it in items]
    ptrs = (ctypes.c_void_p * max(n, 1))(*[h.ctypes.data for h in hosts])
    sizes = np.array([h.size for h in hosts] or [0], dtype=np.uint64)
    crcs = np.array([it[3] for it in items] or [0], dtype=np.uint32)
    for i, it in enumerate(items):
        shp = tuple(int(d) for d in it[1])
        ndims[i] = len(shp)
        shapes[i, :len(shp)] = shp
    _check(_lib.wc_artifact_write(path.encode(), n, names, ctypes.c_void_p(ndims.ctypes.data),
                                  ctypes.c_void_p(shapes.ctypes.data), ptrs,
                                  ctypes.c_void_p(sizes.ctypes.data),
                                  ctypes.c_void_p(crcs.ctypes.data)), "wc_artifact_write")


def artifact_entries(path: str):
    """Every entry's metadata (file header and every entry checked)."""
    cnt = ctypes.c_uint32()
    _check(_lib.wc_artifact_count(path.encode(), ctypes.byref(cnt)), "wc_artifact_count")
    out = []
    for i in range(cnt.value):
        info = ArtifactInfo()
        _check(_lib.wc_artifact_entry(path.encode(), i, ctypes.byref(info)), "wc_artifact_entry")
        out.append({"name": info.name.decode(), "shape": tuple(info.shape[:info.ndim]),
                    "layout": info.layout, "offset": info.offset, "bytes": info.bytes,
                    "src_crc": info.src_crc, "stream_crc": list(info.stream_crc)})
    return out


def artifact_read(path: str, i: int):
    """Container i as a host uint8 array, after every CRC check."""
    import numpy as np
    info = ArtifactInfo()
    _check(_lib.wc_artifact_entry(path.encode(), i, ctypes.byref(info)), "wc_artifact_entry")
    buf = np.empty(info.bytes, dtype=np.uint8)
    _check(_lib.wc_artifact_read(path.encode(), i, ctypes.c_void_p(buf.ctypes.data), buf.size),
           "wc_artifact_read")
    return buf


def artifact_verify(path: str, device="cuda:0"):
    """Streams every tensor of the artifact through the GPU: read (CRCs
    checked), upload, exact decode, and the decoded values' CRC-32 against
    the source's.  Returns (name, matches, bits/weight) per tensor."""
    out = []
    for i, e in enumerate(artifact_entries(path)):
        host = artifact_read(path, i)
        c = torch.from_numpy(host).to(device)
        h = Header.from_bytes(host[:128].tobytes())
        dec = decode(h, c)
        got = crc32(dec)
        bpw = bits_per_weight(h)[0] if h.n else 0.0
        out.append((e["name"], got == e["src_crc"], bpw))
    return out


# ---- 4-bit weights with group scales (include/wc_fp4.h) ----------------------

FP4_GROUP = 32  # columns that share a scale


class Fp4(NamedTuple):
    """A BF16 matrix [rows, cols], or a stack of them [n, rows, cols], as
    4-bit codes: codes uint8 [.., rows, 16 G] and scales uint8 [.., rows, G]
    with G = ceil(cols / 32) groups per row."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int


def _fp4(q: Fp4, what: str):
    """(leading dims, rows, cols) of a checked Fp4."""
    codes, scales, cols = q
    shape, groups = scales.shape, (cols + FP4_GROUP - 1) // FP4_GROUP
    if (len(shape) in (2, 3) and shape[-1] == groups and cols >= 0
            and codes.shape == (*shape[:-1], 16 * groups)
            and codes.dtype is torch.uint8 and scales.dtype is torch.uint8
            and codes.is_contiguous() and scales.is_contiguous()
            and _on_device(codes) and _on_device(scales)):
        return shape[:-2], shape[-2], cols
    for t, name in ((codes, "codes"), (scales, "scales")):
        if not _on_device(t):
            raise ValueError(f"{what}.{name} must be a device tensor")
        if t.dtype != torch.uint8:
            raise TypeError(f"{what}.{name} must be a uint8 tensor")
        if not t.is_contiguous():
            raise ValueError(f"{what}.{name} must be contiguous")
    raise ValueError(f"{what}: codes {tuple(codes.shape)} and scales {tuple(shape)} are not "
                     f"[.., rows, {16 * groups}] and [.., rows, {groups}] of {cols} columns")


def fp4_encode(w: torch.Tensor, out: Fp4 | None = None, stream=None) -> Fp4:
    """wc_fp4_encode: w [rows, cols] or [n, rows, cols], BF16, as 4-bit codes."""
    w = _bits16(w, "w")
    if w.dim() not in (2, 3):
        raise ValueError(f"w must be [rows, cols] or [n, rows, cols], got {tuple(w.shape)}")
    cols = w.shape[-1]
    groups = (cols + FP4_GROUP - 1) // FP4_GROUP
    if out is None:
        _placed("fp4_encode", stream, w)
        out = Fp4(_empty((*w.shape[:-1], 16 * groups), torch.uint8, w.device, stream),
                  _empty((*w.shape[:-1], groups), torch.uint8, w.device, stream), cols)
    else:
        _fp4(out, "out")
        if tuple(out.scales.shape) != (*w.shape[:-1], groups) or out.cols != cols:
            raise ValueError(f"out holds {tuple(out.scales.shape[:-1])} rows of {out.cols} columns, "
                             f"w has shape {tuple(w.shape)}")
        _placed("fp4_encode", stream, w, out.codes, out.scales)
    _check(_lib.wc_fp4_encode(_ptr(w), w.shape[:-1].numel(), cols, _ptr(out.codes),
                              _ptr(out.scales), _stream(stream)), "wc_fp4_encode")
    return out


def fp4_decode(q: Fp4, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """wc_fp4_decode: the BF16 values that q stands for, [.., rows, cols]."""
    lead, rows, cols = _fp4(q, "q")
    shape = (*lead, rows, cols)
    if out is None:
        out = _empty(shape, torch.bfloat16, q.codes.device, stream)
    elif tuple(_bits16(out, "out").shape) != shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {shape}")
    _placed("fp4_decode", stream, q.codes, q.scales, out)
    _check(_lib.wc_fp4_decode(_ptr(q.codes), _ptr(q.scales), out.shape[:-1].numel(), cols,
                              _ptr(out), _stream(stream)), "wc_fp4_decode")
    return out


def fp4_gemv(q: Fp4, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """wc_fp4_gemv: y [batch, rows] fp32 for x [batch, cols] BF16."""
    lead, rows, cols = _fp4(q, "q")
    if lead:
        raise ValueError(f"q must be one matrix, got a stack of {lead[0]}")
    x = _bits16(x, "x")
    batch = _batch_of(x, cols)
    if out is None:
        out = _empty((batch, rows), torch.float32, x.device, stream)
    _gemv_out(out, batch, rows)
    _placed("fp4_gemv", stream, q.codes, q.scales, x, out)
    _check(_lib.wc_fp4_gemv(_ptr(q.codes), _ptr(q.scales), rows, cols, _ptr(x), batch, _ptr(out),
                            _stream(stream)), "wc_fp4_gemv")
    return out


# ---- mixture of experts (include/wc_moe.h) -----------------------------------

SOFTMAX = 0
SIGMOID = 1
MOE_RENORM = 1  # WC_MOE_RENORM
MOE_MAX_TOKENS = 64


def _moe_shape(tokens, hidden, inter, experts, top_k, scoring, renorm, scale) -> MoeShape:
    if (tokens | hidden | inter | experts | top_k | scoring) >> 32:  # ctypes would take it modulo 2^32
        raise ValueError(f"tokens {tokens}, hidden {hidden}, inter {inter}, experts {experts}, top_k {top_k}, "
                         f"scoring {scoring}: one is outside 0..2^32 - 1")
    return MoeShape(tokens, hidden, inter, experts, top_k, scoring, MOE_RENORM if renorm else 0,
                    scale)


@functools.lru_cache(maxsize=256)
def _moe_need(lib, tokens, hidden, inter, experts, top_k) -> int:
    return lib.wc_moe_workspace_bytes(
        ctypes.byref(_moe_shape(tokens, hidden, inter, experts, top_k, SOFTMAX, True, 1.0)))


def moe_workspace_bytes(tokens: int, hidden: int, inter: int, experts: int, top_k: int) -> int:
    """wc_moe_workspace_bytes: device scratch of one moe call of that shape
    (looked up once for each library and shape)."""
    need = _moe_need(_lib, tokens, hidden, inter, experts, top_k)
    if need == 0:
        raise WCError(-5, "wc_moe_workspace_bytes")
    return need


def _moe_experts(w, rows, cols, experts, what):
    """(wc_moe_experts, its tensors) of a stack [experts, rows, cols]."""
    if isinstance(w, Fp4):
        lead, r, c = _fp4(w, what)
        shape, tensors = (*lead, r, c), (w.codes, w.scales)
    else:
        shape, tensors = tuple(_bits16(w, what).shape), (w,)
    if shape != (experts, rows, cols):
        raise ValueError(f"{what} has shape {shape}, expected {(experts, rows, cols)}")
    return MoeExperts(len(tensors) - 1, *(_ptr(t) for t in tensors)), tensors


def moe(x: torch.Tensor, router: torch.Tensor, gate_up, down, top_k: int, *, scoring: int = SOFTMAX,
        bias: torch.Tensor | None = None, renorm: bool = True, scale: float = 1.0,
        work: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """wc_moe: (y [tokens, hidden] BF16, ids [tokens, top_k] int32, weights
    [tokens, top_k] fp32) of a mixture-of-experts layer for up to 64 tokens.

    x [tokens, hidden] and router [experts, hidden] BF16; gate_up
    [experts, 2 * inter, hidden] and down [experts, hidden, inter], each BF16 or
    Fp4; bias fp32 [experts], added to the scores for the choice only (-inf
    takes an expert out).  work: uint8, moe_workspace_bytes(..) of it; a call
    with the same one on another stream must not overlap."""
    x, router = _bits16(x, "x"), _bits16(router, "router")
    if x.dim() != 2 or router.dim() != 2 or x.shape[1] != router.shape[1]:
        raise ValueError(f"x must be [tokens, hidden] and router [experts, hidden], got "
                         f"{tuple(x.shape)} and {tuple(router.shape)}")
    (tokens, hidden), experts = x.shape, router.shape[0]
    if not 1 <= tokens <= MOE_MAX_TOKENS:
        raise ValueError(f"{tokens} tokens outside 1..{MOE_MAX_TOKENS}")
    dshape = down.scales.shape[:-1] + (down.cols,) if isinstance(down, Fp4) else down.shape
    if len(dshape) != 3:
        raise ValueError(f"down must be a stack [experts, hidden, inter], got {tuple(dshape)}")
    inter = int(dshape[-1])
    cgu, tgu = _moe_experts(gate_up, 2 * inter, hidden, experts, "gate_up")
    cdn, tdn = _moe_experts(down, hidden, inter, experts, "down")
    if bias is not None:
        if not _on_device(bias):
            raise ValueError("bias must be a device tensor")
        if bias.dtype != torch.float32:
            raise TypeError("bias must be float32")
        if tuple(bias.shape) != (experts,) or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous [{experts}], got {tuple(bias.shape)}")
    need = moe_workspace_bytes(tokens, hidden, inter, experts, top_k)
    if work is None:
        work = _empty(need, torch.uint8, x.device, stream, returned=False)
    _bytes(work, "work", need)
    if out is None:
        out = _empty((tokens, hidden), torch.bfloat16, x.device, stream)
    if tuple(_bits16(out, "out").shape) != (tokens, hidden):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(tokens, hidden)}")
    ids = _empty((tokens, top_k), torch.int32, x.device, stream)
    weights = _empty((tokens, top_k), torch.float32, x.device, stream)
    _placed("moe", stream, x, router, work, out, *tgu, *tdn, *(() if bias is None else (bias,)))
    shape = _moe_shape(tokens, hidden, inter, experts, top_k, scoring, renorm, scale)
    _check(_lib.wc_moe(ctypes.byref(shape), _ptr(x), _ptr(router), _ptr(bias), ctypes.byref(cgu),
                       ctypes.byref(cdn), _ptr(out), _ptr(ids), _ptr(weights), _ptr(work),
                       work.numel(), _stream(stream)), "wc_moe")
    return out, ids, weights


# ---- 4-bit cache of keys and values, and attention (include/wc_attn.h) -------

ATTN_MAX_DIM = 256
ATTN_MAX_NEW = 16
CACHE_TILE = 32  # tokens; a page is a multiple of it


def fp4_cache(pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda") -> torch.Tensor:
    """An empty 4-bit cache: uint8 [pages, kv_heads, page_size / 32, 34 * head_dim],
    4.25 bits for each number of a key or a value.  head_dim is a multiple of 32
    up to 256, page_size one of 32."""
    if page_size % CACHE_TILE or page_size < CACHE_TILE:
        raise ValueError(f"page_size {page_size} is not a multiple of {CACHE_TILE}")
    if head_dim % 32 or not 32 <= head_dim <= ATTN_MAX_DIM:
        raise ValueError(f"head_dim {head_dim} is not a multiple of 32 up to {ATTN_MAX_DIM}")
    return torch.zeros((pages, kv_heads, page_size // CACHE_TILE, 34 * head_dim), dtype=torch.uint8, device=device)


def _cache(cache: torch.Tensor):
    """(wc_fp4_cache, kv_heads, head_dim) of a checked cache."""
    if not _on_device(cache):
        raise ValueError("cache must be a device tensor")
    if cache.dtype != torch.uint8:
        raise TypeError("cache must be a uint8 tensor")
    shape = cache.shape
    if len(shape) != 4 or shape[3] % (34 * 32) or not 0 < shape[3] <= 34 * ATTN_MAX_DIM or not cache.is_contiguous():
        raise ValueError(f"cache must be a contiguous [pages, kv_heads, page_size / 32, 34 * head_dim], got "
                         f"{tuple(shape)}")
    pages, heads, tiles, width = shape
    if (heads | tiles * CACHE_TILE) >> 32:
        raise ValueError(f"cache has shape {tuple(shape)}: a size does not fit 32 bits")
    return CacheStruct(_ptr(cache), pages, tiles * CACHE_TILE, heads, width // 34), heads, width // 34


def _token_rows(t: torch.Tensor, what: str, heads: int | None, dim: int):
    """(tokens, heads, stride) of BF16 [.., heads, dim] whose leading dimensions
    are tokens one `stride` of numbers apart: whole tensors, or slices by heads of
    wider ones."""
    if not _on_device(t):
        raise ValueError(f"{what} must be a device tensor")
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{what} must hold BF16 bit patterns (bfloat16, int16 or uint16)")
    shape = tuple(t.shape)
    if len(shape) < 3 or shape[-1] != dim or shape[-2] < 1 or (heads is not None and shape[-2] != heads):
        raise ValueError(f"{what} has shape {shape}, expected [.., {'heads' if heads is None else heads}, {dim}]")
    heads = shape[-2]
    stride, step = heads * dim, None
    tokens = t.numel() // stride
    if t.is_contiguous():
        return tokens, heads, stride
    strides = t.stride()
    if len(shape) == 3 and tokens > 1 and strides[1:] == (dim, 1) and strides[0] >= stride and not strides[0] % 8:
        return tokens, heads, strides[0]
    for n, s in zip(reversed(shape[:-2]), reversed(strides[:-2])):  # from the last to the first
        if n > 1 and tokens:
            if step is None:
                stride = step = s
            elif s != step:
                raise ValueError(f"{what}: tokens of strides {strides} are not one step apart")
            step *= n
    if tokens and (strides[-1] != 1 or (heads > 1 and strides[-2] != dim) or stride < heads * dim or stride % 8):
        raise ValueError(f"{what}: strides {strides}; a token's heads must be contiguous and tokens a multiple of 8 "
                         f"numbers apart")
    return tokens, heads, stride


def _whole(t: torch.Tensor, what: str, dtype, shape) -> torch.Tensor:
    """A contiguous device tensor of that type and shape."""
    if not _on_device(t):
        raise ValueError(f"{what} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {tuple(shape)}, got {tuple(t.shape)}")
    return t


def fp4_cache_append(cache: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None):
    """wc_fp4_cache_append: keys and values [tokens, kv_heads, head_dim] BF16 into
    the slots (int64 [tokens]: page * page_size + place) of the cache, each group of
    32 numbers with a scale as by fp4_encode.  A token whose slot is outside the
    cache (-1) is left out; slots of one call must differ.  k and v may be slices
    by heads of a wider tensor, not broadcast over tokens."""
    c, heads, dim = _cache(cache)
    tokens, _, ks = _token_rows(k, "k", heads, dim)
    vt, _, vs = _token_rows(v, "v", heads, dim)
    if vt != tokens:
        raise ValueError(f"k holds {tokens} tokens, v {vt}")
    _whole(slots, "slots", torch.int64, (tokens,))
    _placed("fp4_cache_append", stream, cache, k, v, slots)
    _check(_lib.wc_fp4_cache_append(ctypes.byref(c), _ptr(k), ks, _ptr(v), vs, _ptr(slots), tokens,
                                    _stream(stream)), "wc_fp4_cache_append")
    return cache


def fp4_cache_read(cache: torch.Tensor, slots: torch.Tensor, out=None, stream=None):
    """wc_fp4_cache_read: (k, v), the BF16 values [tokens, kv_heads, head_dim] that
    the cache holds for the slots; NaN for a slot outside it."""
    c, heads, dim = _cache(cache)
    if slots.dim() != 1:
        raise ValueError(f"slots must be [tokens], got {tuple(slots.shape)}")
    _whole(slots, "slots", torch.int64, slots.shape)
    shape = (slots.shape[0], heads, dim)
    if out is None:
        out = _new(cache, shape, torch.bfloat16, stream), _new(cache, shape, torch.bfloat16, stream)
    for t in out:
        if tuple(_bits16(t, "out").shape) != shape:
            raise ValueError(f"out has shape {tuple(t.shape)}, expected {shape}")
    k, v = out
    _placed("fp4_cache_read", stream, cache, slots, k, v)
    _check(_lib.wc_fp4_cache_read(ctypes.byref(c), _ptr(slots), shape[0], _ptr(k), _ptr(v), _stream(stream)),
           "wc_fp4_cache_read")
    return k, v


def _attention_shape(stride, seqs, new, heads, width, window, scale) -> AttentionShape:
    if (seqs | new | heads | width | window) >> 32:  # ctypes would take it modulo 2^32
        raise ValueError(f"seqs {seqs}, new tokens {new}, heads {heads}, table width {width}, window {window}: one "
                         f"is outside 0..2^32 - 1")
    return AttentionShape(stride, seqs, new, heads, width, window, scale)


@functools.lru_cache(maxsize=1024)
def _attention_need(lib, device, pages, page_size, kv_heads, dim, seqs, new, heads, width, window) -> int:
    return lib.wc_fp4_attention_workspace_bytes(
        ctypes.byref(CacheStruct(16, pages, page_size, kv_heads, dim)),
        ctypes.byref(_attention_shape(heads * dim, seqs, new, heads, width, window, 1.0)))


def fp4_attention_workspace_bytes(cache: torch.Tensor, seqs: int, new_tokens: int, heads: int, table_width: int,
                                  window: int = 0) -> int:
    """wc_fp4_attention_workspace_bytes: device scratch of one fp4_attention call
    of that shape on the current device (looked up once for each)."""
    c, _, _ = _cache(cache)
    return _attention_need(_lib, torch._C._cuda_getDevice(), c.pages, c.page_size, c.kv_heads, c.head_dim, seqs,
                           new_tokens, heads, table_width, window)


def fp4_attention(q: torch.Tensor, cache: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor, *,
                  scale: float | None = None, window: int = 0, work: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, stream=None):
    """wc_fp4_attention: (out, lse) of the newest tokens of every sequence over the
    4-bit cache.  q BF16 [seqs, heads, head_dim], or [seqs, new, heads, head_dim] with
    up to 16 new tokens each, which are in the cache already; table int32
    [seqs, width], the pages of each sequence in order; lengths int32 [seqs], tokens
    of each in the cache.  Query i of a sequence of length n is at position
    n - new + i and attends to the positions up to its own, the last `window` of them
    (0: all).  heads is a multiple of the cache's; scale: head_dim ** -0.5.

    out BF16 like q, lse fp32 [.., heads]: the logarithm of the sum of the scores'
    exponentials.  A query without any position gets 0 and -inf.  q may be a slice by
    heads of a wider tensor, not one that is broadcast over tokens.  Limits of sizes (WCError)
    go by the table's width, not by the lengths: include/wc_attn.h.  work: uint8,
    fp4_attention_workspace_bytes(..) of it; a call with the same one on another
    stream must not overlap."""
    c, kv_heads, dim = _cache(cache)
    tokens, heads, stride = _token_rows(q, "q", None, dim)
    if q.dim() not in (3, 4):
        raise ValueError(f"q must be [seqs, heads, head_dim] or [seqs, new, heads, head_dim], got {tuple(q.shape)}")
    seqs, new = q.shape[0], (q.shape[1] if q.dim() == 4 else 1)
    if heads % kv_heads:
        raise ValueError(f"{heads} heads are no multiple of the cache's {kv_heads}")
    if not 1 <= new <= ATTN_MAX_NEW:
        raise ValueError(f"{new} new tokens outside 1..{ATTN_MAX_NEW}")
    if table.dim() != 2:
        raise ValueError(f"table must be [seqs, width], got {tuple(table.shape)}")
    width = table.shape[1]
    _whole(table, "table", torch.int32, (seqs, width))
    _whole(lengths, "lengths", torch.int32, (seqs,))
    need = _attention_need(_lib, q.get_device(), c.pages, c.page_size, kv_heads, dim, seqs, new, heads, width, window)
    shape = _attention_shape(stride, seqs, new, heads, width, window, dim ** -0.5 if scale is None else scale)
    rows = (seqs, new, heads) if q.dim() == 4 else (seqs, heads)
    if out is None:
        out = _new(q, (*rows, dim), torch.bfloat16, stream)
    elif tuple(_bits16(out, "out").shape) != (*rows, dim):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(*rows, dim)}")
    lse = _new(q, rows, torch.float32, stream)
    if need:
        if work is None:
            work = _new(q, (need,), torch.uint8, stream, returned=False)
        _bytes(work, "work", need)
        _placed("fp4_attention", stream, q, cache, table, lengths, out, work)
    else:
        _placed("fp4_attention", stream, q, cache, table, lengths, out)
    _check(_lib.wc_fp4_attention(ctypes.byref(c), ctypes.byref(shape), _ptr(q), _ptr(table), _ptr(lengths),
                                 _ptr(out), _ptr(lse), _ptr(work) if need else None, need, _stream(stream)),
           "wc_fp4_attention")
    return out, lse


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor, *,
                     scale: float | None = None, window: int = 0, out: torch.Tensor | None = None, stream=None):
    """wc_prompt_attention: (out, lse) of causal attention over whole prompts,
    packed one after the other.  q BF16 [tokens, heads, head_dim], k and v [tokens,
    kv_heads, head_dim], each possibly a slice by heads of a wider tensor; starts
    int32 [seqs + 1], not falling: sequence i is the tokens starts[i] ..
    starts[i + 1] - 1.  head_dim is a multiple of 32 up to 256, heads one of
    kv_heads; a token attends to its sequence up to itself, the last `window` tokens
    of it (0: all); scale: head_dim ** -0.5.

    out BF16 [tokens, heads, head_dim], lse fp32 [tokens, heads]; rows of tokens of no
    sequence are not written."""
    dim = q.shape[-1] if q.dim() else 0
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q, k and v must be [tokens, heads, head_dim], got {tuple(q.shape)}, {tuple(k.shape)} and "
                         f"{tuple(v.shape)}")
    if dim % 32 or not 32 <= dim <= ATTN_MAX_DIM:
        raise ValueError(f"head_dim {dim} is not a multiple of 32 up to {ATTN_MAX_DIM}")
    tokens, heads, qs = _token_rows(q, "q", None, dim)
    kt, kv_heads, ks = _token_rows(k, "k", None, dim)
    vt, _, vs = _token_rows(v, "v", kv_heads, dim)
    if kt != tokens or vt != tokens:
        raise ValueError(f"q holds {tokens} tokens, k {kt}, v {vt}")
    if heads % kv_heads:
        raise ValueError(f"{heads} heads are no multiple of {kv_heads}")
    if starts.dim() != 1 or starts.shape[0] < 1:
        raise ValueError(f"starts must be [seqs + 1], got {tuple(starts.shape)}")
    seqs = starts.shape[0] - 1
    _whole(starts, "starts", torch.int32, (seqs + 1,))
    if window >> 32:
        raise ValueError(f"window {window} is outside 0..2^32 - 1")
    shape = (tokens, heads, dim)
    if out is None:
        out = _new(q, shape, torch.bfloat16, stream)
    elif tuple(_bits16(out, "out").shape) != shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {shape}")
    lse = _new(q, (tokens, heads), torch.float32, stream)
    _placed("prompt_attention", stream, q, k, v, starts, out)
    c = PromptShape(tokens, qs, ks, vs, seqs, heads, kv_heads, dim, window, dim ** -0.5 if scale is None else scale)
    _check(_lib.wc_prompt_attention(ctypes.byref(c), _ptr(q), _ptr(k), _ptr(v), _ptr(starts), _ptr(out), _ptr(lse),
                                    _stream(stream)), "wc_prompt_attention")
    return out, lse


# ---- log probabilities of tokens (include/wc_logprob.h) ----------------------

LOGPROB_MAX_TOP = 32


@functools.lru_cache(maxsize=1024)
def _logprob_need(lib, device, rows, vocab, f32, top) -> int:
    return lib.wc_token_logprobs_workspace_bytes(ctypes.byref(LogprobShape(vocab, rows, vocab, f32, top)))


def _logprob_sizes(rows, vocab, top, dtype) -> bool:
    """True for fp32 logits; what the library cannot take is refused."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be float32 or bfloat16")
    if (rows | vocab) >> 31 or vocab < 1:
        raise ValueError(f"rows {rows} or vocab {vocab} outside 0..2^31 - 1 (vocab from 1)")
    if not 0 <= top <= LOGPROB_MAX_TOP:
        raise ValueError(f"top {top} outside 0..{LOGPROB_MAX_TOP}")
    return dtype == torch.float32


def token_logprobs_workspace_bytes(rows: int, vocab: int, top: int = 0, dtype=torch.float32) -> int:
    """wc_token_logprobs_workspace_bytes: device scratch of one token_logprobs call
    of that shape on the current device (looked up once for each)."""
    f32 = _logprob_sizes(rows, vocab, top, dtype)
    return _logprob_need(_lib, torch._C._cuda_getDevice(), rows, vocab, f32, top)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, *, work: torch.Tensor | None = None,
                   stream=None):
    """wc_token_logprobs: (logprobs [rows], entropy [rows], top_ids [rows, top] int32,
    top_logprobs [rows, top]) of logits [rows, vocab], fp32 (as fp4_gemv and
    decode_gemv give them) or BF16, whose rows may be further apart than vocab.
    tokens int64 [rows]: the log probability of each under its row's softmax; the
    entropy in nats; the `top` (0..32) most likely tokens, ties to the lower index.
    Logits of -inf are no alternatives (id -1 and -inf where too few others are
    left); a token outside the vocabulary gets NaN.  work: uint8,
    token_logprobs_workspace_bytes(..) of it; a call with the same one on another
    stream must not overlap."""
    if not _on_device(logits):
        raise ValueError("logits must be a device tensor")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [rows, vocab], got {tuple(logits.shape)}")
    rows, vocab = logits.shape
    f32 = _logprob_sizes(rows, vocab, top, logits.dtype)
    stride = logits.stride(0) if rows > 1 else vocab
    if (vocab > 1 and logits.stride(1) != 1) or stride < vocab:
        raise ValueError(f"logits of strides {logits.stride()}: a row must be contiguous and rows must not overlap")
    _whole(tokens, "tokens", torch.int64, (rows,))
    need = _logprob_need(_lib, logits.get_device(), rows, vocab, f32, top)
    logprobs, entropy = _new(logits, (rows,), torch.float32, stream), _new(logits, (rows,), torch.float32, stream)
    ids, best = _new(logits, (rows, top), torch.int32, stream), _new(logits, (rows, top), torch.float32, stream)
    if need:
        if work is None:
            work = _new(logits, (need,), torch.uint8, stream, returned=False)
        _bytes(work, "work", need)
        _placed("token_logprobs", stream, logits, tokens, work)
    else:
        _placed("token_logprobs", stream, logits, tokens)
    c = LogprobShape(stride, rows, vocab, f32, top)
    _check(_lib.wc_token_logprobs(ctypes.byref(c), _ptr(logits), _ptr(tokens), _ptr(logprobs), _ptr(entropy),
                                  _ptr(ids), _ptr(best), _ptr(work) if need else None, need, _stream(stream)),
           "wc_token_logprobs")
    return logprobs, entropy, ids, best
