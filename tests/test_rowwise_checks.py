"""CPU checks of the row-wise operators (norm, rotary positions, microscaled
layers): pins of their fp64 oracle, the binding's refusals and the library's
own host-side validation."""

import ctypes
import math

import numpy as np
import pytest
import torch

from mask_free_b200 import build as B_
from mask_free_b200 import ops
from oracle import rowwise as O
from tests.test_binding_checks import _last, _refused, rec, t  # noqa: F401

bf16, f16, f32, i32, u8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8
e4m3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    B_.build()
    return ops.lib()


# ---------------------------------------------------------------- pins of the oracle
def test_norm_pins():
    # one row of 3, 4: mean square 12.5; with eps 3.5 the divisor is 4
    h, y = O.rms_norm([[[1.0, 1.0]]], w=[2.0, 1.0], res=[[[2.0, 3.0]]], eps=3.5)
    assert h.tolist() == [[[3.0, 4.0]]] and y.tolist() == [[[1.5, 1.0]]]
    # rows S: res at the tokens, x at the rows unless it is full
    res = np.arange(12.0).reshape(1, 6, 2)
    h, _ = O.rms_norm(np.zeros((1, 2, 2)), res=res, S=np.array([[5, 1]]))
    assert h.tolist() == [[[10.0, 11.0], [2.0, 3.0]]]
    h, _ = O.rms_norm(res, S=np.array([[5, 1]]), x_full=True)
    assert h.tolist() == [[[10.0, 11.0], [2.0, 3.0]]]
    # unit mean square after the norm
    _, y = O.rms_norm(np.random.default_rng(0).normal(size=(1, 1, 64)), eps=0.0)
    assert abs((y * y).mean() - 1) < 1e-14


def test_rope_pins():
    # a quarter turn takes (a, b) to (-b, a); the tail passes through
    x = np.arange(1.0, 7.0).reshape(1, 1, 1, 6)
    half = O.rope(x, [math.pi / 2, math.pi / 2], [2], [[[1]]])
    np.testing.assert_allclose(half[0, 0, 0], [-3, -4, 1, 2, 5, 6], atol=1e-15)
    pairs = O.rope(x, [math.pi / 2, math.pi / 2], [2], [[[1]]], interleaved=True, m=2.0)
    np.testing.assert_allclose(pairs[0, 0, 0], [-4, 2, -8, 6, 5, 6], atol=1e-14)
    # scores depend on position differences only (relative positions)
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 1, 1, 1, 16))
    f, _ = ops.rope_frequencies(16)
    s = [float((O.rope(q, f, [8], [[[p]]]) * O.rope(k, f, [8], [[[p - 3]]])).sum()) for p in (3, 500)]
    assert abs(s[0] - s[1]) < 1e-12
    # two axes: each section turns by its own position
    two = O.rope(x[..., :4], [math.pi / 2, math.pi / 2], [1, 1], [[[0, 1]]])
    np.testing.assert_allclose(two[0, 0, 0], [1, -4, 3, 2], atol=1e-15)


def test_frequencies():
    f, m = ops.rope_frequencies(8, base=100.0)
    np.testing.assert_allclose(f, [1, 100 ** -0.25, 100 ** -0.5, 100 ** -0.75], rtol=1e-15)
    assert m == 1.0
    g, _ = ops.rope_frequencies(8, base=100.0, kind="linear", factor=4.0)
    np.testing.assert_allclose(g, np.array(f) / 4, rtol=1e-15)
    g, _ = ops.rope_frequencies(8, base=100.0, kind="ntk", factor=4.0)
    assert g[0] == 1.0 and abs(g[-1] - f[-1] / 4) < 1e-15  # the fastest kept, the slowest divided by the factor
    g, m = ops.rope_frequencies(64, kind="yarn", factor=4.0, original_len=1024)
    f, _ = ops.rope_frequencies(64)
    turns = 1024 * np.array(f) / (2 * math.pi)
    ratio = np.array(g) / np.array(f)
    assert np.all(ratio[turns > 64] == 1.0) and np.allclose(ratio[turns < 0.5], 0.25) and np.all(np.diff(ratio) <= 0)
    assert abs(m - (0.1 * math.log(4.0) + 1.0)) < 1e-15
    assert ops.rope_frequencies(64, kind="yarn", factor=4.0, original_len=1024, attn_factor=1.0)[1] == 1.0
    # sections: each axis has a series of its own
    g, _ = ops.rope_frequencies(12, sections=[2, 4])
    assert g == ops.rope_frequencies(4)[0] + ops.rope_frequencies(8)[0]
    for bad in (dict(r=7), dict(r=0), dict(r=8, sections=[1, 2]), dict(r=8, sections=[1, 1, 1, 1]), dict(r=8, kind="x"),
                dict(r=8, base=1.0), dict(r=8, factor=0.5), dict(r=8, kind="yarn", factor=2.0),
                dict(r=8, sections=[5, -1])):
        _refused(ops.rope_frequencies, **bad)


def test_rope_table_is_the_frequencies_in_turns(rec):
    f, m = ops.rope_frequencies(64, kind="yarn", factor=4.0, original_len=1024)
    tab = ops.rope_table(64, device="cpu", kind="yarn", factor=4.0, original_len=1024)
    got = [int(v) % 2 ** 64 / 2.0 ** 64 for v in tab.freq]
    # half a unit of the fixed point, and fp64's roundings
    np.testing.assert_allclose(got, np.array(f) / (2 * math.pi), rtol=2.0 ** -50, atol=2.0 ** -65)
    assert tab.m == m and tab.sections == (32,) and tab.r == 64


def test_microscaled_pins():
    # e4m3 table: largest 448, one 56; torch's own conversion agrees on every code
    assert len(O.E4M3) == 127 and O.E4M3[126] == 448.0 and O.E4M3[56] == 1.0
    want = torch.arange(127, dtype=u8).view(e4m3).double().numpy()
    assert np.array_equal(O.E4M3, want)
    # mxfp4: a = 7 -> scale 2^0; 7 saturates at 6; ties go to the even code (2.5 -> 2, 3.5 -> 4, 0.25 -> 0, 0.75 -> 1)
    x = np.zeros((1, 32))
    x[0, :6] = [7, 2.5, 3.5, 0.25, -0.75, 5.0]
    code, byte = O.mx_encode(x, "mxfp4")
    assert byte.tolist() == [[127]] and code[0, :6].tolist() == [7, 4, 6, 0, 10, 6]
    assert O.mx_decode(code, byte, "mxfp4")[0, :6].tolist() == [6, 2, 4, 0, -1, 4]
    # mxfp8: a = 500 lies below 512 -> 2^(8 - 8); 500 saturates
    x[0, :3] = [500, 17.0, 19.0]
    code, byte = O.mx_encode(x, "mxfp8")
    assert byte[0, 0] == 127 and O.mx_decode(code, byte, "mxfp8")[0, :3].tolist() == [448, 16, 20]
    # nvfp4: a / (6 g) to e4m3, elements by scale * g
    x = np.zeros((1, 16))
    x[0, :2] = [12.0, -3.0]
    code, byte = O.mx_encode(x, "nvfp4", 0.5)
    assert O.E4M3[byte[0, 0]] == 4.0 and O.mx_decode(code, byte, "nvfp4", 0.5)[0, :2].tolist() == [12.0, -3.0]
    # zeros
    for fmt in O.MX_BLOCK:
        code, byte = O.mx_encode(np.zeros((1, 32)), fmt)
        assert not code.any() and not byte.any()
    # tiles: row 33, scale 5 of 128 x 8
    b = np.zeros((130, 6), dtype=np.uint8)
    b[33, 5], b[129, 0] = 9, 8
    flat = O.mx_tile(b)
    assert flat[512 + 16 + 4 + 1] == 9 and flat[1024 + 16] == 8 and flat.sum() == 17
    back, rest = O.mx_untile(flat, 130, 6)
    assert np.array_equal(back, b) and not rest.any() and len(rest) == 2048 - 780
    assert np.array_equal(O.mx_unpack(O.mx_pack(np.arange(16, dtype=np.uint8)[None], "nvfp4"), "nvfp4")[0], np.arange(16))


# ---------------------------------------------------------------- the binding
B, N, D, k = 2, 40, 64, 7


def table(r=32, sections=None, **kw):
    return ops.rope_table(r, sections=sections, device="cpu", **kw)


def mx(*lead, D=64, fmt="mxfp8", scale=1.0):
    w = D if fmt == "mxfp8" else D // 2
    data = torch.zeros((*lead, w), dtype=e4m3 if fmt == "mxfp8" else u8)
    return ops.MxTensor(data, torch.zeros(ops.mx_scale_bytes(math.prod(lead), D, fmt), dtype=u8), fmt, scale)


def test_valid_calls_reach_the_abi_with_their_sizes(rec):
    x, S, w = t(B, N, D), t(B, k, dtype=i32), t(D, dtype=f32)
    y = ops.rms_norm(x, w)
    assert y.shape == x.shape and _last(rec, "safe_rms_norm")[12:16] == (4, B, N, D)
    y, h = ops.rms_norm(t(B, k, D), w, residual=x, S=S, x_compact=True)
    a = _last(rec, "safe_rms_norm")
    assert y.shape == h.shape == (B, k, D) and a[1] == 0 and a[4] == k and a[8] == 0
    y, h = ops.rms_norm(x, w, residual=x.clone(), S=S, quant="mxfp8", update=True)
    a = _last(rec, "safe_rms_norm")
    assert a[1] == 1 and a[8] == 1 and a[9] is None and a[7] == a[2] and y.shape == (B, k, D) and h.shape == (B, N, D)
    tab = table(32)
    q, kk = t(B, N, 6, 64, dtype=f16), t(B, N, 2, 64, dtype=f16)
    oq, ok = ops.rope(q, kk, tab)
    a = _last(rec, "safe_rope")
    assert oq.shape == q.shape and ok.shape == kk.shape and a[4] == 6 and a[9] == 2 and a[10] == 3
    assert a[17:22] == (B, N, N, 64, 32)
    qkv = t(B, k, 10, 64)
    oq, ok = ops.rope(qkv[:, :, :6], qkv[:, :, 6:8], table(64, [16, 16]), pos=t(N, 2, dtype=i32), S=S, inplace=True)
    a = _last(rec, "safe_rope")
    assert oq.data_ptr() == qkv.data_ptr() and list(a[1]) == [k * 640, 640, 64] and a[13] == 2 and a[15] == 0
    assert a[17:22] == (B, N, k, 64, 64)
    oq, ok = ops.rope(q, None, tab, pos=t(B, N, 1, dtype=i32), interleaved=True)
    a = _last(rec, "safe_rope")
    assert ok is None and a[5] is None and a[15] == 1 and a[22] == 1
    for fmt, width in (("mxfp8", 64), ("mxfp4", 32), ("nvfp4", 32)):
        m = ops.mx_quantize(x, fmt, S=S)
        a = _last(rec, "safe_mx_quantize")
        assert m.data.shape == (B, k, width) and m.shape == (B, k, D) and a[1] == 4 and a[3] == k and a[8:11] == (B, N, D)
        assert ops.mx_dequantize(m, f16).shape == (B, k, D)
        assert _last(rec, "safe_mx_dequantize")[5:8] == (3, B * k, D)
        y = ops.mx_linear(m, mx(40, fmt=fmt), bias=t(40, dtype=f32), act="gelu_tanh")
        a = _last(rec, "safe_mx_linear")
        assert y.shape == (B, k, 40) and a[7] == 1 and a[9:12] == (B * k, D, 40)
    assert ops.mx_quantize(t(40, 64), "nvfp4", scale=0.25).data.shape == (40, 32)
    assert ops.mx_linear(mx(B, k, fmt="nvfp4", scale=0.5), mx(40, fmt="nvfp4", scale=0.25)).shape == (B, k, 40)
    assert _last(rec, "safe_mx_linear")[5] == 0.125


def test_mismatched_arguments_are_refused_before_any_launch(rec):
    x, S, w = t(B, N, D), t(B, k, dtype=i32), t(D, dtype=f32)
    _refused(ops.rms_norm, x.to(torch.float64))
    _refused(ops.rms_norm, x[:, ::2])
    _refused(ops.rms_norm, x, t(D + 1, dtype=f32))
    _refused(ops.rms_norm, x, t(D))
    _refused(ops.rms_norm, x, residual=t(B, N + 1, D))
    _refused(ops.rms_norm, x, residual=t(B, N, D, dtype=f32))
    _refused(ops.rms_norm, x, residual=x.clone(), S=S, x_compact=True)
    _refused(ops.rms_norm, t(B, k, D), residual=x, S=S)
    _refused(ops.rms_norm, t(B, k, D), S=S, x_compact=True)
    _refused(ops.rms_norm, x, S=t(B, N + 1, dtype=i32))
    _refused(ops.rms_norm, x, S=t(B + 1, k, dtype=i32))
    _refused(ops.rms_norm, x, S=t(B, 0, dtype=i32))
    _refused(ops.rms_norm, x, update=True)
    _refused(ops.rms_norm, x, residual=x.clone(), update=True, h=x.clone())
    _refused(ops.rms_norm, x, quant="mxfp4")
    _refused(ops.rms_norm, t(B, N, 40), quant="mxfp8")
    _refused(ops.rms_norm, x, out=t(B, N, D, dtype=f32))
    _refused(ops.rms_norm, x, quant="mxfp8", out=mx(B, N + 1))
    q, kk, tab = t(B, N, 6, 64), t(B, N, 2, 64), table(32)
    pos = t(N, 1, dtype=i32)
    _refused(ops.rope, q, t(B, N + 1, 2, 64), tab)
    _refused(ops.rope, q, t(B, N, 2, 32), tab)
    _refused(ops.rope, q, t(B, N, 2, 64, dtype=f32), tab)
    _refused(ops.rope, q, kk, table(96))
    _refused(ops.rope, q, kk, table(32, [8, 8]))
    _refused(ops.rope, q, kk, table(32, [8, 8]), pos=pos)
    _refused(ops.rope, q, kk, tab, pos=t(N + 1, 1, dtype=i32))
    _refused(ops.rope, q, kk, tab, pos=t(N, 1))
    _refused(ops.rope, q, kk, tab, pos=t(B + 1, N, 1, dtype=i32))
    _refused(ops.rope, q, kk, tab, S=t(B, N, dtype=i32))
    _refused(ops.rope, q, kk, tab, pos=pos, S=t(B, k, dtype=i32))
    _refused(ops.rope, q, kk, tab, pos=t(N - 1, 1, dtype=i32), S=t(B, N, dtype=i32))
    _refused(ops.rope, q.transpose(2, 3), None, tab)
    _refused(ops.rope, q, kk, tab, inplace=True, out=(q, kk))
    _refused(ops.rope, q, kk, tab, out=(kk, q))
    _refused(ops.rope, q, None, tab, out=(None, kk))
    _refused(ops.rope, q, kk, tab.freq)
    _refused(ops.RopeTable, tab.freq, [8, 9])
    _refused(ops.RopeTable, tab.freq, [16], float("nan"))
    _refused(ops.mx_quantize, x, "mxfp6")
    _refused(ops.mx_quantize, t(B, N, 48), "mxfp8")
    _refused(ops.mx_quantize, x, "mxfp8", scale=2.0)
    _refused(ops.mx_quantize, x, "nvfp4", scale=0.0)
    _refused(ops.mx_quantize, x, "nvfp4", scale=float("nan"))
    _refused(ops.mx_quantize, x, "nvfp4", scale=2.0 ** 101)
    _refused(ops.mx_quantize, x[0], "nvfp4", S=S)
    _refused(ops.mx_quantize, x, "nvfp4", out=mx(B, N, fmt="mxfp4"))
    _refused(ops.mx_dequantize, x)
    _refused(ops.mx_dequantize, mx(B, N), torch.float64)
    _refused(ops.mx_linear, mx(B, N), mx(40, fmt="mxfp4"))
    _refused(ops.mx_linear, mx(B, N), mx(40, D=96))
    _refused(ops.mx_linear, mx(B, N), mx(2, 40))
    _refused(ops.mx_linear, mx(B, N), mx(40), bias=t(41, dtype=f32))
    _refused(ops.mx_linear, mx(B, N), mx(40), act="relu")
    _refused(ops.mx_linear, mx(B, N), mx(40), out=t(B, N, 41))
    _refused(ops.mx_linear, mx(B, N), mx(40), ws=t(64))
    _refused(ops.mx_linear, mx(B, N, fmt="nvfp4", scale=2.0 ** -80), mx(40, fmt="nvfp4", scale=2.0 ** -80))
    _refused(ops.MxTensor, torch.zeros((4, 64), dtype=u8), torch.zeros(512, dtype=u8), "mxfp8")
    _refused(ops.MxTensor, torch.zeros((4, 64), dtype=u8), torch.zeros(512, dtype=u8), "nvfp4")  # two tiles along a row
    _refused(ops.MxTensor, torch.zeros((4, 24), dtype=u8), torch.zeros(512, dtype=u8), "mxfp4")
    _refused(ops.MxTensor, torch.zeros((4, 64), dtype=u8), torch.zeros(512, dtype=u8), "mxfp4", 2.0)
    assert rec.calls == []


def test_binding_refuses_cpu_tensors():
    x = t(B, N, D)
    _refused(ops.rms_norm, x)
    _refused(ops.rope, t(B, N, 2, 64), None, object())
    _refused(ops.mx_quantize, x, "mxfp8")


def test_calls_run_on_the_tensors_device(rec, monkeypatch):
    # tensors of another device than the current one: the call runs there, on
    # that device's current stream
    entered = []

    class Device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            entered.append(self.i)

        def __exit__(self, *a):
            entered.append(-1)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(ops, "_raw_stream", lambda i: 100 + i)
    ops._run("safe_mx_dequantize", torch.device("cuda", 0), 1)
    assert entered == [] and rec.calls[-1][1] == (1, 100)
    ops._run("safe_mx_dequantize", torch.device("cuda", 1), 1)
    assert entered == [1, -1] and rec.calls[-1][1] == (1, 101)
    assert ops._on(torch.device("cuda", 2), lambda v: v, 5) == 5 and entered[2:] == [2, -1]


def test_checked_operands_cannot_be_exchanged(rec):
    m, tab = mx(4, 64), table(32)
    for obj, name in ((m, "data"), (m, "scales"), (m, "scale"), (tab, "freq"), (tab, "sections")):
        with pytest.raises(AttributeError):
            setattr(obj, name, getattr(obj, name))


# ---------------------------------------------------------------- the library


def at(n):
    return ctypes.c_void_p(0x100000 + n * 0x1000000)


def test_scale_bytes(lib):
    for fmt, code in (("mxfp8", 0), ("mxfp4", 1), ("nvfp4", 2)):
        for rows in (1, 127, 128, 129, 51200):
            for D_ in (32, 64, 96, 128, 160, 2304):
                n = -(-rows // 128) * -(-(D_ // O.MX_BLOCK[fmt]) // 4) * 512
                assert lib.safe_mx_scale_bytes(rows, D_, code) == n == ops.mx_scale_bytes(rows, D_, fmt)
    assert lib.safe_mx_scale_bytes(0, 32, 0) == 0 and lib.safe_mx_scale_bytes(4, 33, 0) == 0
    assert lib.safe_mx_scale_bytes(4, 32, 3) == 0 and ops.mx_scale_bytes(0, 32, "mxfp8") == 0


def test_rms_norm_validates_on_host(lib):
    def call(x=at(0), full=0, res=at(1), S=None, k=0, w=at(2), eps=1e-6, h=at(3), h_full=0, y=at(4), q=None, qs=None,
             dtype=4, B=1, N=16, D=64):
        return lib.safe_rms_norm(x, full, res, S, k, w, eps, h, h_full, y, q, qs, dtype, B, N, D, None)

    assert call(x=None) == 1 and call(y=None) == 1 and call(dtype=1) == 2 and call(N=0) == 1 and call(D=0) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(full=1) == 1 and call(h_full=1) == 1
    assert call(S=at(5), k=17) == 1 and call(S=at(5), k=0) == 1
    assert call(S=at(5), k=4, h_full=1) == 1                          # in place, but h is not res
    assert call(q=at(6)) == 1 and call(qs=at(6)) == 1
    assert call(q=at(6), qs=at(7), D=40) == 1                         # 8 bits: multiples of 32
    assert call(q=at(6), qs=at(7), x=ctypes.c_void_p(0x100002)) == 1  # and 16-byte alignment
    assert call(q=at(6), qs=at(7), D=40992) == 2
    assert call(N=1, D=2 ** 31 - 1, x=ctypes.c_void_p(1 << 40), res=None, w=None, h=None) == 2  # counters would wrap
    assert call(x=ctypes.c_void_p(0x100001)) == 1 and call(S=ctypes.c_void_p(0x9000002), k=4) == 1
    assert call(y=ctypes.c_void_p(0x100000 + 64)) == 1                # output overlaps an input in part
    assert call(y=at(3)) == 1                                         # outputs overlap
    assert call(S=at(5), k=4, y=at(1)) == 1                           # rows S: not over the stream
    assert call(q=at(3), qs=at(7)) == 1 and call(q=at(6), qs=at(6)) == 1


def test_rope_validates_on_host(lib):
    i3 = ctypes.c_int64 * 3

    def call(q=at(0), qs=(4096, 256, 64), oq=at(1), oqs=(4096, 256, 64), Hq=4, k=at(2), ks=(2048, 128, 64), ok=at(3),
             oks=(2048, 128, 64), Hk=2, dtype=4, freq=at(4), sec=(32,), pos=None, batched=0, S=None, B=2, N=16, R=16,
             d=64, r=64, il=0, m=1.0):
        return lib.safe_rope(q, i3(*qs), oq, i3(*oqs), Hq, k, None if ks is None else i3(*ks), ok,
                             None if oks is None else i3(*oks), Hk, dtype, ctypes.cast(freq, ops._i64p),
                             (ctypes.c_int32 * len(sec))(*sec), len(sec), pos, batched, S, B, N, R, d, r, il, m, None)

    assert call(q=None) == 1 and call(oq=None) == 1 and call(Hq=0) == 1 and call(dtype=0) == 2
    assert call(k=None) == 1 and call(k=None, ok=None, Hk=1) == 1 and call(ok=None) == 1 and call(Hk=0) == 1
    assert call(R=15) == 1 and call(R=17, S=at(5)) == 1 and call(N=0, R=0) == 1
    assert call(r=63) == 1 and call(r=66) == 1 and call(r=0, sec=(0,)) == 1 and call(m=float("inf")) == 1
    assert call(sec=(31,)) == 1 and call(sec=(16, 16)) == 1 and call(sec=(8, 8, 8, 8), pos=at(6)) == 1
    assert call(sec=(33, -1), pos=at(6)) == 1
    assert call(d=1026, r=64) == 2
    assert call(qs=(4096, -256, 64)) == 1
    assert call(oqs=(4096, 256, 63)) == 1 and call(oqs=(4096, 255, 64)) == 1 and call(oqs=(4095, 256, 64)) == 1
    assert call(oqs=(4096, 0, 64)) == 1
    assert call(oq=at(3)) == 1 and call(oq=at(2)) == 1 and call(oq=ctypes.c_void_p(0x100000 + 128)) == 1
    assert call(oq=at(0), oqs=(8192, 512, 64)) == 1                   # the input's memory, other strides
    fused, one = (16384, 1024, 64), lambda h: ctypes.c_void_p(0x100000 + h * 128)
    # in place, heads 3.. of the fused tensor overlap heads ..3 of the queries
    assert call(q=one(0), qs=fused, oq=one(0), oqs=fused, k=one(3), ks=fused, ok=one(3), oks=fused) == 1
    # a key view past the end of the row reaches the next row's queries
    assert call(q=one(0), qs=fused, oq=one(0), oqs=fused, k=one(15), ks=fused, ok=one(15), oks=fused) == 1
    assert call(freq=ctypes.c_void_p(0x100004)) == 1 and call(pos=ctypes.c_void_p(0x100002)) == 1


def test_microscaled_entry_points_validate_on_host(lib):
    def quant(X=at(0), dtype=4, S=None, k=0, fmt=2, g=1.0, data=at(1), sc=at(2), B=1, N=16, D=64):
        return lib.safe_mx_quantize(X, dtype, S, k, fmt, g, data, sc, B, N, D, None)

    assert quant(X=None) == 1 and quant(data=None) == 1 and quant(sc=None) == 1 and quant(dtype=0) == 2
    assert quant(D=48) == 1 and quant(D=0) == 1 and quant(N=0) == 1 and quant(fmt=3) == 1 and quant(fmt=-1) == 1
    assert quant(g=0.0) == 1 and quant(g=-1.0) == 1 and quant(g=float("inf")) == 1 and quant(g=2.0 ** -101) == 1
    assert quant(fmt=0, g=2.0) == 1 and quant(S=at(3), k=0) == 1 and quant(S=at(3), k=17) == 1
    assert quant(data=at(0)) == 1 and quant(sc=at(0)) == 1 and quant(sc=at(1)) == 1
    assert quant(X=ctypes.c_void_p(0x100008)) == 1 and quant(data=ctypes.c_void_p(0x1100008)) == 1

    def deq(data=at(0), sc=at(1), fmt=1, g=1.0, Y=at(2), dtype=4, rows=16, D=64):
        return lib.safe_mx_dequantize(data, sc, fmt, g, Y, dtype, rows, D, None)

    assert deq(data=None) == 1 and deq(sc=None) == 1 and deq(Y=None) == 1 and deq(dtype=1) == 2 and deq(rows=0) == 1
    assert deq(D=40) == 1 and deq(g=2.0) == 1 and deq(Y=at(0)) == 1 and deq(Y=at(1)) == 1 and deq(rows=2 ** 31) == 1

    def lin(X=at(0), Xs=at(1), W=at(2), Ws=at(3), fmt=2, a=1.0, bias=None, act=0, Y=at(4), rows=16, i=64, o=64, ws=None, wb=0):
        return lib.safe_mx_linear(X, Xs, W, Ws, fmt, a, bias, act, Y, rows, i, o, ws, wb, None)

    assert lin(X=None) == 1 and lin(Xs=None) == 1 and lin(W=None) == 1 and lin(Ws=None) == 1 and lin(Y=None) == 1
    assert lin(fmt=3) == 1 and lin(a=float("nan")) == 1 and lin(a=0.0) == 1 and lin(act=2) == 1
    assert lin(rows=0) == 1 and lin(rows=2 ** 31) == 1 and lin(i=32) == 1 and lin(i=80) == 1 and lin(o=12) == 1 and lin(o=0) == 1
    assert lin(bias=ctypes.c_void_p(0x100002)) == 1 and lin(Y=at(0)) == 1 and lin(Y=at(3)) == 1
    far = [ctypes.c_void_p((i + 1) << 44) for i in range(5)]
    huge = dict(X=far[0], Xs=far[1], W=far[2], Ws=far[3], Y=far[4])
    assert lin(**huge, rows=2 ** 31 - 8) == 2 and lin(**huge, o=2 ** 31 - 8) == 2 and lin(**huge, rows=2 ** 31 - 8, o=2 ** 31 - 8) == 2
    # the split of the last wave's tiles (9 of 74 pairs, 72 stages): its workspace, apart from the rest
    big = dict(fmt=0, rows=200, i=9216, o=2304)
    n = lib.safe_mx_linear_workspace_bytes(200, 9216, 2304, 0)
    assert n == 9 * 8 * 256 * 256 * 4
    assert lin(**big, ws=ctypes.c_void_p(0x10000010), wb=n) == 1 and lin(**big, ws=at(4), wb=n) == 1
    assert lin(**big, ws=at(2), wb=n) == 1
    assert lib.safe_mx_linear_workspace_bytes(200, 2304, 2304, 2) == 0     # 9 stages: not worth it
    assert lib.safe_mx_linear_workspace_bytes(18944, 9216, 2304, 0) == 0   # whole waves
    assert lib.safe_mx_linear_workspace_bytes(0, 64, 64, 0) == 0 and lib.safe_mx_linear_workspace_bytes(4, 80, 64, 0) == 0
    assert lib.safe_mx_linear_workspace_bytes(4, 64, 12, 0) == 0 and lib.safe_mx_linear_workspace_bytes(4, 64, 64, 3) == 0
