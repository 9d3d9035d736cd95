"""The GEMV entry points refuse more rows than a grid of fewer than 2^32 threads
takes, on the host, before any device work."""
import ctypes

import numpy as np
import pytest

import decode_gemv_sign_amd as wc
import oracle

OK = ctypes.c_void_p(64)
TOO_MANY = [(1 << 26, 5, 1), ((1 << 26) - 15, 7, 1), ((1 << 28) - 15, 8, 3), ((1 << 32) - 255, 0, 1), (1 << 26, 63, 16), ((1 << 28) + 3, 9, 4), (1 << 28, 8, 1), (1 << 29, 8, 256),
            (1 << 32, 0, 1), (1 << 31, 0, 2), (1 << 40, 0, 1)]


def raw_header(n):
    """The header of n weights kept as they are (everything after them is empty)."""
    h = wc.Header.from_bytes(oracle.encode(wc.RAW, np.zeros(0, dtype=np.uint16)).tobytes())
    h.n = n
    h.off_esc_pos = h.off_esc_sym = h.off_esc_idx = h.total_bytes = (128 + 2 * n + 15) // 16 * 16
    return h


@pytest.mark.parametrize("rows,cols,batch", TOO_MANY)
def test_plain_gemv(rows, cols, batch):
    assert wc._lib.wc_gemv_bf16(OK, rows, cols, OK, batch, OK, None) == -2


@pytest.mark.parametrize("rows,cols,batch", [c for c in TOO_MANY if c[0] * c[1] < 1 << 32])
def test_decode_gemv(rows, cols, batch):
    h = raw_header(rows * cols)
    if h.n:
        assert 16 <= wc.bits_per_weight(h)[0] < 16.01  # a header that the library takes
    room = h.total_bytes
    assert wc._lib.wc_decode_gemv(ctypes.byref(h), OK, room, rows, cols, OK, batch, OK, None) == -2
    if h.n:  # by the rows, not by the buffer
        assert wc._lib.wc_decode_gemv(ctypes.byref(h), OK, room, 1, rows * cols + 1, OK, batch, OK, None) == -1
