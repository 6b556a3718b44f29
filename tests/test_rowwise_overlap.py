"""Host-side refusals of the row-wise entry points (no GPU): outputs over the
arrays that a call reads, and sizes past the counters."""

import ctypes

import pytest

from mask_free_b200 import build as B_
from mask_free_b200 import ops
from tests.test_rowwise_checks import at

INVALID, UNSUPPORTED = 1, 2


def off(n, d):
    return ctypes.c_void_p(at(n).value + d)


@pytest.fixture(scope="module")
def lib():
    B_.build()
    return ops.lib()


def test_norm_outputs_over_w_or_S(lib):
    def call(x=at(0), full=0, res=at(1), S=None, k=0, w=at(2), h=at(3), h_full=0, y=at(4), q=None, qs=None, B=2, N=16, D=64):
        return lib.safe_rms_norm(x, full, res, S, k, w, 1e-6, h, h_full, y, q, qs, 4, B, N, D, None)

    rows, e = dict(S=at(5), k=4), 2 * 64
    assert call(y=at(2)) == INVALID and call(h=at(2)) == INVALID      # w: 256 bytes
    assert call(y=off(2, 240)) == INVALID and call(w=off(4, 2 * 16 * e - 16)) == INVALID
    assert call(w=off(3, 16)) == INVALID
    assert call(**rows, y=at(5)) == INVALID and call(**rows, h=at(5)) == INVALID  # S: 32 bytes
    assert call(**rows, y=off(5, 16)) == INVALID and call(S=off(3, 2 * 4 * e - 4), k=4) == INVALID
    assert call(**rows, h=at(1), h_full=1, w=off(1, 2 * 16 * e - 16)) == INVALID  # w, S inside the stream
    assert call(S=off(1, 64), k=4, h=at(1), h_full=1) == INVALID
    quant = dict(q=at(6), qs=at(7))
    assert call(**rows, q=at(5), qs=at(7), y=None) == INVALID and call(**rows, q=at(6), qs=at(5), y=None) == INVALID
    assert call(**quant, y=None, w=off(6, 16)) == INVALID


def test_layer_output_over_bias(lib):
    def call(Y=at(4), bias=at(5), rows=16, o=64, fmt=0):
        return lib.safe_mx_linear(at(0), at(1), at(2), at(3), fmt, 1.0, bias, 0, Y, rows, 64, o, None, 0, None)

    for fmt in (0, 1, 2):
        assert call(bias=at(4), fmt=fmt) == INVALID and call(Y=off(5, 240), fmt=fmt) == INVALID
        assert call(bias=off(4, 16 * 64 * 2 - 4), fmt=fmt) == INVALID


def test_quantised_rows_over_S(lib):
    def call(S=at(3), k=4, data=at(1), sc=at(2), fmt=0, B=2):
        return lib.safe_mx_quantize(at(0), 4, S, k, fmt, 1.0, data, sc, B, 16, 64, None)

    for fmt in (0, 1, 2):
        assert call(data=at(3), fmt=fmt) == INVALID and call(sc=at(3), fmt=fmt) == INVALID
        assert call(data=off(3, 16), fmt=fmt) == INVALID and call(S=off(2, 508), fmt=fmt) == INVALID
        assert call(S=off(1, 2 * 4 * (64 if fmt == 0 else 32) - 4), fmt=fmt) == INVALID
