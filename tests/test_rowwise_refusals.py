"""Host-side refusals of the row-wise entry points (no GPU): outputs over the
arrays that a call reads, sizes past the counters, and what a refused call
leaves behind."""

import ctypes

import pytest
import torch

from mask_free_b200 import build as B_
from mask_free_b200 import ops
from tests.test_binding_checks import rec, t  # noqa: F401
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


def test_rope_outputs_over_freq_pos_or_S(lib):
    i3, fused = ctypes.c_int64 * 3, (16 * 640, 640, 64)

    def call(q=at(0), qs=None, oq=at(1), oqs=None, ok=at(3), freq=at(4), pos=None, batched=0, S=None, sec=(32,), R=16):
        i3n = lambda v: None if v is None else i3(*v)
        return lib.safe_rope(q, i3n(qs), oq, i3n(oqs), 4, at(2), None, ok, None, 2, 4, ctypes.cast(freq, ops._i64p),
                             (ctypes.c_int32 * len(sec))(*sec), len(sec), pos, batched, S, 2, 16, R, 64, 64, 0, 1.0, None)

    qb, kb = 2 * 16 * 4 * 64 * 2, 2 * 16 * 2 * 64 * 2
    assert call(freq=at(1)) == INVALID and call(freq=off(1, qb - 8)) == INVALID and call(freq=off(3, kb - 8)) == INVALID
    assert call(oq=off(4, 240)) == INVALID  # freq: 256 bytes
    assert call(pos=at(3)) == INVALID and call(pos=off(1, qb - 4)) == INVALID and call(ok=off(6, 48), pos=at(6)) == INVALID
    two = dict(sec=(16, 16), pos=at(6))     # 128 bytes shared, 256 batched
    assert call(ok=off(6, 112), **two) == INVALID and call(ok=off(6, 240), batched=1, **two) == INVALID
    rows = dict(pos=at(6), S=at(5))         # 128 bytes
    assert call(ok=at(5), **rows) == INVALID and call(oq=off(5, 112), **rows) == INVALID
    assert call(q=at(0), qs=fused, oq=at(0), oqs=fused, freq=off(0, 2 * 16 * 640 * 2 - 6 * 64 * 2 - 8)) == INVALID


def test_a_refused_call_leaves_out_as_it_was(rec, monkeypatch):
    x, out = t(2, 8, 64), ops.MxTensor(torch.zeros((2, 8, 32), dtype=torch.uint8),
                                       torch.zeros(ops.mx_scale_bytes(16, 64, "nvfp4"), dtype=torch.uint8), "nvfp4", 0.5)

    def refuse(name, *args):
        raise ops.SafeError(name, INVALID)

    with monkeypatch.context() as m:
        m.setattr(ops, "_run", refuse)
        with pytest.raises(ops.SafeError):
            ops.mx_quantize(x, "nvfp4", scale=0.25, out=out)
    assert out.scale == 0.5  # the old elements keep their factor
    assert ops.mx_quantize(x, "nvfp4", scale=0.25, out=out) is out and out.scale == 0.25


def test_layers_of_rows_past_the_counters(lib):
    far = [ctypes.c_void_p((i + 1) << 44) for i in range(6)]

    def call(fmt, d_in, ws=None, wb=0):
        return lib.safe_mx_linear(far[0], far[1], far[2], far[3], fmt, 1.0, None, 0, far[4], 16, d_in, 64, ws, wb, None)

    for fmt in (0, 1, 2):
        for d_in in (2 ** 31 - 32, 2 ** 31 - 128, 2 ** 30, 2 ** 20 + 32):  # the rows that quantising takes end at 2^20
            assert call(fmt, d_in) == UNSUPPORTED and call(fmt, d_in, far[5], 1 << 40) == UNSUPPORTED
            assert lib.safe_mx_linear_workspace_bytes(16, d_in, 64, fmt) == 0


def test_sizes_that_an_int_cannot_hold_are_refused(rec):
    # the entry points' sizes are ints: 2^32 + 5 rows must not run as 5
    big = 2 ** 32 + 5

    def m(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")

    i32, u8 = torch.int32, torch.uint8
    for shape in ((1, big, 1), (big, 1, 1), (1, 1, big)):
        with pytest.raises(ValueError):
            ops.rms_norm(m(*shape))
    with pytest.raises(ValueError):
        ops.rms_norm(m(1, 3, 1), residual=m(1, big, 1), S=m(1, 3, dtype=i32), x_compact=True)
    tab = ops.RopeTable(torch.zeros(1, dtype=torch.int64, device="meta"), [1])
    for q, k in ((m(1, big, 1, 2), None), (m(big, 1, 1, 2), None), (m(1, 1, big, 2), None), (m(1, 1, 1, 2), m(1, 1, big, 2)),
                 (m(1, 1, 1, big + 1), None)):
        with pytest.raises(ValueError):
            ops.rope(q, k, tab)
    with pytest.raises(ValueError):
        ops.rope(m(1, 3, 1, 2), None, tab, pos=m(big, 1, dtype=i32), S=m(1, 3, dtype=i32))
    wide = 2 ** 32 + 64
    for fmt in ("mxfp8", "mxfp4", "nvfp4"):
        for shape in ((1, big, 64), (big, 1, 64), (1, 1, wide), (big, 64)):
            with pytest.raises(ValueError):
                ops.mx_quantize(m(*shape), fmt)

        def mx(rows, D):
            data = m(rows, D, dtype=torch.float8_e4m3fn) if fmt == "mxfp8" else m(rows, D // 2, dtype=u8)
            return ops.MxTensor(data, m(ops.mx_scale_bytes(rows, D, fmt), dtype=u8), fmt)

        with pytest.raises(ValueError):
            ops.mx_dequantize(mx(1, wide))
        for X, W in ((mx(1, wide), mx(8, wide)), (mx(1, 64), mx(2 ** 32 + 8, 64))):
            with pytest.raises(ValueError):
                ops.mx_linear(X, W, ws=False)
        for sizes in ((1, wide, 8), (1, 64, 2 ** 32 + 8)):
            with pytest.raises(ValueError):
                ops.mx_linear_workspace_bytes(*sizes, fmt)
    assert rec.calls == []
