"""GPU parity of the row-wise operators around the block's attention (norm with
the residual, rotary positions, microscaled quantisation and layers) against
their fp64 oracle. Every tolerance is an arithmetic bound: half a step of the
output type plus the fp32 roundings of the kernel's own sums and products.
Outputs lie inside larger buffers whose other bytes must not change."""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from mask_free_b200 import ops
from oracle import rowwise as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24  # half a step of fp32
FLAG = 1 << ops.SAFE_ERR_DEVICE_CHECK


@pytest.fixture(autouse=True)
def _status_clean():
    ops.device_status()
    yield


def to64(x):
    return x.detach().double().cpu().numpy()


def half_step(dtype, v):
    """Half a step of dtype at |v|, its subnormals included."""
    fi = torch.finfo(dtype)
    return np.abs(v) * (fi.eps / 2) + fi.tiny * (fi.eps / 2)


def randn(shape, seed, dtype=f32):
    return torch.from_numpy(np.random.default_rng(seed).normal(size=shape)).to(dtype)


def rows(B, N, k, seed):
    rng = np.random.default_rng(seed)
    return np.stack([np.sort(rng.choice(N, k, replace=False)) for _ in range(B)]).astype(np.int32)


def guarded(shape, dtype, pad=256):
    """(buffer, a contiguous view of `shape` inside it): the pads hold a pattern."""
    n = math.prod(shape)
    e = torch.empty((), dtype=dtype).element_size()
    buf = torch.full((n * e + 2 * pad,), 0x5A, dtype=torch.uint8, device=DEV)
    return buf, buf[pad:pad + n * e].view(dtype).view(shape)


def untouched(buf, pad=256):
    return bool((buf[:pad] == 0x5A).all()) and bool((buf[-pad:] == 0x5A).all())


def dev(x):
    return None if x is None else (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).to(DEV)


# ---------------------------------------------------------------- norm
def norm_tol(y, D):
    """Relative roundings of y before the last: the sum h, its squares and their
    sum (D terms of one sign, halved by the square root), the division, eps,
    the square root, the reciprocal and two products."""
    return np.abs(y) * (D / 2 + 8) * U


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("B,N,D,k", [
    (1, 1, 1, 0), (2, 5, 3, 0), (1, 7, 33, 4), (3, 50, 128, 17), (2, 33, 500, 0), (1, 9, 1283, 0), (2, 20, 2304, 11),
    (1, 130, 2560, 0), (1, 3, 2563, 2), (1, 5, 4096, 0), (1, 4, 7168, 0), (1, 3, 10240, 0), (1, 2, 20480, 0),
    (1, 2, 40960, 0), (1, 3, 41000, 2), (1, 2, 514, 0), (1, 2, 1036, 1), (2, 3, 320, 0), (2, 3, 640, 0), (1, 3, 1800, 0)])
def test_norm_parity(dtype, B, N, D, k):
    S = rows(B, N, k, D) if k else None
    R = k or N
    w = 1 + 0.2 * randn((D,), 1)
    for res in (False, True):
        for full in ((True,) if not k else (False, True) if res else (True,)):
            x = randn((B, N if full else R, D), 2, dtype)
            r = randn((B, N, D), 3, dtype) * 2 if res else None
            href, yref = O.rms_norm(to64(x), to64(w), None if r is None else to64(r), S, 1e-6, full)
            buf, out = guarded((B, R, D), dtype)
            hbuf, h = guarded((B, R, D), dtype)
            got = ops.rms_norm(dev(x), dev(w), dev(r), dev(S), 1e-6, x_compact=not full, out=out, h=h if res else None)
            y = got[0] if res else got
            assert np.all(np.abs(to64(y) - yref) <= half_step(dtype, yref) * (1 + 1e-6) + norm_tol(yref, D))
            if res:  # one rounding to fp32, one to the type
                assert np.all(np.abs(to64(got[1]) - href) <= half_step(dtype, href) * (1 + 1e-6) + np.abs(href) * U)
            assert untouched(buf) and untouched(hbuf)
    assert ops.device_status() == 0


@pytest.mark.parametrize("offset", [1, 2, 4])
def test_norm_of_unaligned_tensors(offset):
    # rows that begin at 2, 4 and 8 bytes: the same values as aligned ones
    B, N, D = 2, 9, 256
    x, r, w = randn((B, N, D), 1, bf16).to(DEV), randn((B, N, D), 2, bf16).to(DEV), randn((D,), 3).to(DEV)
    want = ops.rms_norm(x, w, r)

    def shifted(t):
        buf = torch.empty(t.numel() + 16, dtype=t.dtype, device=DEV)
        v = buf[offset:offset + t.numel()].view(t.shape)
        return v.copy_(t)

    got = ops.rms_norm(shifted(x), shifted(w) if offset != 2 else w, shifted(r), out=shifted(x), h=shifted(x))
    assert torch.equal(got[1], want[1])
    yref = O.rms_norm(to64(x), to64(w), to64(r))[1]
    for y in (got[0], want[0]):
        assert np.all(np.abs(to64(y) - yref) <= half_step(bf16, yref) * (1 + 1e-6) + norm_tol(yref, D))


def check_mxfp8(m, y, delta):
    """Codes and scales of an mxfp8 matrix whose values before quantisation lie within
    y (1 +- delta): a scale is right for some value in that range, and every
    element is within half a step (or saturated) of it."""
    D = y.shape[-1]
    n, flat = y.reshape(-1, D).shape[0], y.reshape(-1, D)
    byte, rest = O.mx_untile(m.scales.cpu().numpy(), n, D // 32)
    assert not rest.any()
    top = np.abs(flat).reshape(n, -1, 32).max(-1)
    lo, hi = O.mx_encode(flat * (1 - delta), "mxfp8")[1], O.mx_encode(flat * (1 + delta), "mxfp8")[1]
    assert np.all((byte >= lo) & (byte <= hi)), (top[(byte < lo) | (byte > hi)])
    s = np.repeat(O.mx_scale_values(byte, "mxfp8"), 32, axis=-1)
    v = O.mx_decode(m.data.view(torch.uint8).cpu().numpy().reshape(n, D), byte, "mxfp8")
    want = np.minimum(np.abs(flat), 448 * s)
    # half a step: 2^-4 of the value, 2^-10 of the scale below e4m3's smallest normal number
    assert np.all(np.abs(np.abs(v) - want) <= np.maximum(want * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-6) + np.abs(flat) * delta)
    big = np.abs(flat) > s * 2.0 ** -9
    assert np.all(np.sign(v[big]) == np.sign(flat[big]))


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("B,N,D,k", [(1, 1, 32, 0), (2, 70, 96, 9), (1, 129, 160, 0), (2, 20, 2304, 11), (1, 257, 512, 0),
                                     (1, 3, 4096, 0), (1, 2, 8192, 0), (1, 2, 11296, 0), (1, 2, 40960, 0), (1, 128, 64, 0)])
def test_norm_in_8_bits(dtype, B, N, D, k):
    S = rows(B, N, k, D) if k else None
    R = k or N
    x, r, w = randn((B, R, D), 4, dtype), randn((B, N, D), 5, dtype), 1 + 0.2 * randn((D,), 6)
    x[..., ::17] *= 8
    y, h = ops.rms_norm(dev(x), dev(w), dev(r), dev(S), x_compact=True, quant="mxfp8")
    href, yref = O.rms_norm(to64(x), to64(w), to64(r), S)
    assert np.all(np.abs(to64(h) - href) <= half_step(dtype, href) * (1 + 1e-6) + np.abs(href) * U)
    check_mxfp8(y, yref, (D / 2 + 8) * U)
    v = ops.mx_dequantize(y, f32)
    byte, _ = O.mx_untile(y.scales.cpu().numpy(), B * R, D // 32)
    assert np.array_equal(to64(v).reshape(-1, D),
                          O.mx_decode(y.data.view(torch.uint8).cpu().numpy().reshape(-1, D), byte, "mxfp8"))
    assert ops.device_status() == 0


def test_norm_updates_the_stream_in_place():
    B, N, D, k = 2, 60, 2304, 13
    S = rows(B, N, k, 1)
    x, r, w = randn((B, k, D), 1, bf16).to(DEV), randn((B, N, D), 2, bf16).to(DEV), randn((D,), 3).to(DEV)
    y0, h0 = ops.rms_norm(x, w, r, dev(S), x_compact=True)
    stream = r.clone()
    y1, h1 = ops.rms_norm(x, w, stream, dev(S), x_compact=True, update=True)
    assert h1 is stream and torch.equal(y0, y1)
    want = r.clone()
    for b in range(B):
        want[b, torch.from_numpy(S[b]).long().to(DEV)] = h0[b]
    assert torch.equal(stream, want)
    # every row: the stream, and y over x
    x = randn((B, N, D), 4, bf16).to(DEV)
    y0, h0 = ops.rms_norm(x, w, r)
    stream, xc = r.clone(), x.clone()
    y1, h1 = ops.rms_norm(xc, w, stream, update=True, out=xc)
    assert torch.equal(stream, h0) and torch.equal(xc, y0) and y1 is xc
    # long rows, which the kernel reads twice
    x, r = randn((1, 3, 41000), 5, bf16).to(DEV), randn((1, 3, 41000), 6, bf16).to(DEV)
    y0, h0 = ops.rms_norm(x, None, r)
    stream = r.clone()
    assert torch.equal(ops.rms_norm(x, None, stream, update=True)[0], y0) and torch.equal(stream, h0)
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("D", [65, 131, 1021, 2303, 4100])
def test_norm_of_odd_widths_in_place_and_beside_nan(dtype, D):
    # rows that share 16-byte units with their neighbours: in place the same
    # bits as apart, and a NaN or an infinity stays in its row
    x, r, w = randn((2, 37, D), 1, dtype).to(DEV), randn((2, 37, D), 2, dtype).to(DEV), randn((D,), 3).to(DEV)
    y0, h0 = ops.rms_norm(x, w, r)
    xs, rs = x.clone(), r.clone()
    y1, h1 = ops.rms_norm(xs, w, rs, update=True, out=xs)
    assert y1 is xs and h1 is rs and torch.equal(y1, y0) and torch.equal(h1, h0)
    x[0, 5, D - 1], x[1, 0, 0], x[1, 36, D - 1] = float("nan"), float("inf"), float("nan")
    y2, h2 = ops.rms_norm(x, w, r)
    clean = torch.ones((2, 37), dtype=torch.bool, device=DEV)
    clean[0, 5] = clean[1, 0] = clean[1, 36] = False
    assert torch.equal(y2[clean], y0[clean]) and torch.equal(h2[clean], h0[clean])
    assert y2[0, 5].isnan().all() and y2[1, 36].isnan().all() and ops.device_status() == 0


@pytest.mark.parametrize("D", [64, 2304])
def test_norm_with_both_outputs(D):
    # the C entry point writes y and its 8-bit form in one call
    x, w = randn((1, 130, D), 1, bf16).to(DEV), randn((D,), 2).to(DEV)
    y, m = torch.empty_like(x), ops.rms_norm(x, w, quant="mxfp8")
    q, sc = torch.zeros_like(m.data.view(torch.uint8)), torch.zeros_like(m.scales)
    st = ops.lib().safe_rms_norm(x.data_ptr(), 0, None, None, 0, w.data_ptr(), 1e-6, None, 0, y.data_ptr(), q.data_ptr(),
                                 sc.data_ptr(), 4, 1, 130, D, torch.cuda.current_stream().cuda_stream)
    assert st == ops.SAFE_OK and torch.equal(y, ops.rms_norm(x, w))
    assert torch.equal(q, m.data.view(torch.uint8)) and torch.equal(sc, m.scales)


@pytest.mark.parametrize("D", [64, 63, 41000])
def test_norm_bad_rows_are_flagged_and_zero(D):
    x, r = randn((1, 5, D), 1, bf16).to(DEV), randn((1, 9, D), 2, bf16).to(DEV)
    S = torch.tensor([[3, 9, -1, 8, 2 ** 31 - 1]], dtype=torch.int32, device=DEV)
    y, h = ops.rms_norm(x, None, r, S, x_compact=True)
    assert ops.device_status() == FLAG
    good = ops.rms_norm(x[:, [0, 3]].contiguous(), None, r, S[:, [0, 3]].contiguous(), x_compact=True)
    assert torch.equal(y[:, [0, 3]], good[0]) and torch.equal(h[:, [0, 3]], good[1])
    assert not y[:, [1, 2, 4]].any() and not h[:, [1, 2, 4]].any()
    # in place: bad rows and rows out of order leave the stream as it is
    S = torch.tensor([[3, 3, 2, 9, 8]], dtype=torch.int32, device=DEV)
    stream = r.clone()
    ops.rms_norm(x, None, stream, S, x_compact=True, update=True)
    assert ops.device_status() == FLAG
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(stream[:, keep], r[:, keep]) and not torch.equal(stream[:, 3], r[:, 3])
    if D % 32 == 0:
        y, _ = ops.rms_norm(x, None, r, torch.tensor([[3, 9, -1, 8, 1]], dtype=torch.int32, device=DEV), x_compact=True,
                            quant="mxfp8")
        assert ops.device_status() == FLAG
        v = ops.mx_dequantize(y)
        assert not v[:, 1:3].any() and v[:, 0].any()


def test_norm_of_zeros_infinities_and_nan():
    x = torch.zeros((1, 4, 64), dtype=f32, device=DEV)
    x[0, 1, 5], x[0, 2, 5], x[0, 3] = float("inf"), float("nan"), 2.0
    y = ops.rms_norm(x, None, eps=0.25)
    assert not y[0, 0].any() and y[0, 1, 5].isnan() and not y[0, 1, :5].any() and y[0, 2].isnan().all()
    assert torch.allclose(y[0, 3], torch.full((64,), 2 / math.sqrt(4.25), device=DEV), rtol=1e-6)
    m = ops.rms_norm(x, None, eps=0.25, quant="mxfp8")
    v = ops.mx_dequantize(m)
    assert not v[0, 0].any() and v[0, 1, :32].isnan().all() and not v[0, 1, 32:].any() and v[0, 2].isnan().all()
    assert (m.scales.cpu().numpy() == 255).sum() == 3


# ---------------------------------------------------------------- rotary positions
SCALINGS = [dict(), dict(kind="linear", factor=4.0), dict(kind="ntk", factor=8.0),
            dict(kind="yarn", factor=4.0, original_len=1024)]


def rope_check(got, x, ref, dtype, r, m):
    """A turned element: the angle in turns is rounded to 2^-25 of half a turn
    (pi 2^-25 radians, below 2^-23), cos and sin to 2^-23, their products with
    m and with the elements to 2^-24 each: less than 2^-21 of |a| + |b| times m."""
    x, g = np.abs(to64(x)), to64(got)
    tol = half_step(dtype, ref) * (1 + 1e-6) + 2 * x.max(axis=-1, keepdims=True) * m * 2.0 ** -21
    assert np.all(np.abs(g - ref)[..., :r] <= tol[..., :r]), np.abs(g - ref)[..., :r].max()
    assert np.array_equal(g[..., r:], ref[..., r:])


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("B,N,k,H,Hk,d,r,axes,far", [
    (1, 1, 0, 2, 1, 64, 64, 1, 1000003), (2, 37, 0, 3, 3, 96, 96, 2, 0), (2, 50, 13, 24, 24, 96, 64, 1, 7),
    (3, 20, 0, 5, 1, 128, 128, 2, 2 ** 31 - 30), (1, 33, 9, 4, 2, 80, 20, 1, 0), (2, 9, 0, 1, 1, 10, 6, 1, -2 ** 31),
    (1, 12, 5, 2, 2, 128, 48, 3, 100), (1, 6, 0, 2, 1, 2, 2, 1, 5), (1, 3, 0, 2, 2, 1024, 1024, 1, 0),
    (2, 129, 0, 8, 2, 64, 32, 1, 31), (1, 40, 0, 1, 4, 72, 8, 1, 0)])
def test_rope_parity(dtype, B, N, k, H, Hk, d, r, axes, far):
    n = r // 2
    sec = [n] if axes == 1 else [n - n // 2, n // 2] if axes == 2 else [n - 2 * (n // 3), n // 3, n // 3]
    S = rows(B, N, k, d) if k else None
    R = k or N
    rng = np.random.default_rng(d + r)
    for i, sc in enumerate(SCALINGS):
        interleaved, fused = bool(i & 1), i >= 2
        tab = ops.rope_table(r, 10000.0, sec, **sc)
        f, m = ops.rope_frequencies(r, 10000.0, sec, **sc)
        if fused:  # views of one projection
            qkv = randn((B, R, H + 2 * Hk, d), 3, dtype)
            q, kk = qkv[:, :, :H], qkv[:, :, H:H + Hk]
            dq = qkv.to(DEV)
            gq, gk = dq[:, :, :H], dq[:, :, H:H + Hk]
        else:
            q, kk = randn((B, R, H, d), 1, dtype), randn((B, R, Hk, d), 2, dtype)
            gq, gk = q.to(DEV), kk.to(DEV)
        batched = i == 3
        span = min(N, 2 ** 31 - 1 - max(far, 0))
        pos = (rng.integers(0, span, size=(B, N, axes) if batched else (N, axes)) + far).astype(np.int32)
        at = pos if batched else np.broadcast_to(pos, (B, N, axes))
        if S is not None:
            at = np.stack([at[b, S[b]] for b in range(B)])
        bufs, outs = zip(*[guarded((B, R, h, d), dtype) for h in (H, Hk)])
        oq, ok = ops.rope(gq, gk, tab, pos=dev(pos), S=dev(S), interleaved=interleaved, out=outs)
        rope_check(oq, q, O.rope(to64(q), f, sec, at, interleaved, m), dtype, r, m)
        rope_check(ok, kk, O.rope(to64(kk), f, sec, at, interleaved, m), dtype, r, m)
        assert all(map(untouched, bufs))
        # new tensors, and in place: the same bits
        nq, nk = ops.rope(gq, gk, tab, pos=dev(pos), S=dev(S), interleaved=interleaved)
        assert torch.equal(nq, oq) and torch.equal(nk, ok) and nq.is_contiguous()
        q1, _ = ops.rope(gq, None, tab, pos=dev(pos), S=dev(S), interleaved=interleaved)
        assert torch.equal(q1, oq)
        iq, _ = ops.rope(gq, gk, tab, pos=dev(pos), S=dev(S), interleaved=interleaved, inplace=True)
        assert iq is gq and torch.equal(gq, oq) and torch.equal(gk, ok)
        if fused:
            assert torch.equal(dq[:, :, H + Hk:].cpu(), qkv[:, :, H + Hk:])
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype,H,Hk,d,r,interleaved", [
    (bf16, 24, 8, 96, 96, False), (bf16, 24, 24, 96, 64, True), (f16, 12, 6, 128, 128, False), (bf16, 36, 0, 64, 64, True),
    (f16, 3, 2, 512, 512, False), (bf16, 1, 1, 1024, 1024, True), (f32, 9, 3, 96, 96, True)])
def test_rope_of_many_tokens(dtype, H, Hk, d, r, interleaved):
    # enough tokens for the ring of bulk copies: rows S, positions of each
    # sample, fused views, in place; sampled rows against the oracle
    B, N, k = 2, 3000, 2700
    sec = [r // 2 - r // 8, r // 8]
    tab, (f, m) = ops.rope_table(r, sections=sec), ops.rope_frequencies(r, sections=sec)
    S, rng = rows(B, N, k, 1), np.random.default_rng(2)
    pos = rng.integers(-1000, 1000000, size=(B, N, 2)).astype(np.int32)
    pick = np.unique(np.r_[0, 1, k - 2, k - 1, rng.choice(k, 60, replace=False)])
    at = np.stack([pos[b, S[b, pick]] for b in range(B)])
    gen = torch.Generator(device=DEV).manual_seed(3)
    qkv = torch.randn((B, k, H + 2 * max(Hk, 1), d), generator=gen, device=DEV).to(dtype)
    before = qkv.clone()
    q, kk = qkv[:, :, :H], qkv[:, :, H:H + Hk] if Hk else None
    pk = torch.from_numpy(pick).to(DEV)
    want = [O.rope(to64(t[:, pk]), f, sec, at, interleaved, m) for t in (q, kk) if t is not None]
    new = ops.rope(q, kk, tab, pos=dev(pos), S=dev(S), interleaved=interleaved)
    for t, got, ref in zip((q, kk), new, want):
        rope_check(got[:, pk], t[:, pk], ref, dtype, r, m)
    buf, o = guarded((B, k, H, d), dtype)
    ops.rope(q, kk, tab, pos=dev(pos), S=dev(S), interleaved=interleaved, out=(o, None))
    assert torch.equal(o, new[0]) and untouched(buf) and torch.equal(qkv, before)
    ops.rope(q, kk, tab, pos=dev(pos), S=dev(S), interleaved=interleaved, inplace=True)
    assert torch.equal(q, new[0]) and (kk is None or torch.equal(kk, new[1]))
    assert torch.equal(qkv[:, :, H + Hk:], before[:, :, H + Hk:])
    bad = dev(S).clone()
    bad[1, 17] = N
    got, _ = ops.rope(before[:, :, :H], None, tab, pos=dev(pos), S=bad, interleaved=interleaved)
    assert ops.device_status() == FLAG
    bad[1, 17] = 0
    assert torch.equal(got, ops.rope(before[:, :, :H], None, tab, pos=dev(pos), S=bad, interleaved=interleaved)[0])
    assert ops.device_status() == 0


def test_rope_layouts():
    # token index as position, head-major inputs and outputs, unaligned views, a broadcast input
    B, N, H, d = 2, 21, 4, 64
    tab = ops.rope_table(d)
    f, _ = ops.rope_frequencies(d)
    at = np.broadcast_to(np.arange(N)[None, :, None], (B, N, 1))
    x = randn((B, H, N, d), 1, bf16)
    want = O.rope(to64(x.transpose(1, 2)), f, [d // 2], at)
    xt = x.to(DEV).transpose(1, 2)
    o = torch.empty((B, H, N, d), dtype=bf16, device=DEV).transpose(1, 2)
    got, _ = ops.rope(xt, None, tab, out=(o, None))
    rope_check(got, x.transpose(1, 2), want, bf16, d, 1.0)
    one, _ = ops.rope(xt.contiguous(), None, tab, pos=torch.arange(N, dtype=torch.int32, device=DEV))
    assert torch.equal(one, got)
    buf = torch.empty(xt.numel() + 8, dtype=bf16, device=DEV)
    shifted = buf[3:3 + xt.numel()].view(B, N, H, d).copy_(xt)
    assert torch.equal(ops.rope(shifted, None, tab)[0], got)
    assert torch.equal(ops.rope(shifted, None, tab, inplace=True)[0], got)
    wide = xt[:, :, :1].expand(B, N, 3, d)  # heads of stride 0: read, never written
    got, _ = ops.rope(wide, None, tab)
    assert all(torch.equal(got[:, :, h], one[:, :, 0]) for h in range(3))
    with pytest.raises(ops.SafeError):
        ops.rope(wide, None, tab, inplace=True)
    # both outputs in one fused tensor
    q, k = randn((B, N, H, d), 2, bf16).to(DEV), randn((B, N, 2, d), 3, bf16).to(DEV)
    fused = torch.zeros((B, N, H + 2, d), dtype=bf16, device=DEV)
    ops.rope(q, k, tab, out=(fused[:, :, :H], fused[:, :, H:]))
    a, b = ops.rope(q, k, tab)
    assert torch.equal(fused, torch.cat([a, b], dim=2))
    assert ops.device_status() == 0


def test_rope_far_positions_and_bad_rows():
    # phases are exact at any position: a whole number of turns changes nothing
    d, N = 64, 8
    x = randn((1, N, 2, d), 1, f32).to(DEV)
    tab = ops.RopeTable((torch.arange(1, d // 2 + 1, dtype=torch.int64, device=DEV) << 40), [d // 2])  # n 2^-24 turns
    p = torch.arange(N, dtype=torch.int32, device=DEV)
    near, _ = ops.rope(x, None, tab, pos=p)
    far, _ = ops.rope(x, None, tab, pos=p + 2 ** 24 * 100)
    assert torch.equal(near, far)
    S = torch.tensor([[2, N, -1, 7]], dtype=torch.int32, device=DEV)
    got, _ = ops.rope(x[:, :4], None, tab, pos=p, S=S)
    assert ops.device_status() == FLAG
    want, _ = ops.rope(x[:, :4], None, tab, pos=p, S=torch.tensor([[2, 0, 0, 7]], dtype=torch.int32, device=DEV))
    assert torch.equal(got, want)  # replaced by token 0


# ---------------------------------------------------------------- microscaled rows
def spread(shape, seed):
    """Rows with blocks of zeros, large and small scales, exact ties and their neighbours."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=shape) * np.exp2(rng.integers(-12, 10, size=(*shape[:-1], 1)))
    x = x.reshape(-1, 16)
    x[::7] = 0.0
    x[1::5, 3] *= 40
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 4.5, 5.5, -0.25, -2.5, -5.0, 6.0])
    x[3::11] = ties * np.exp2(rng.integers(-5, 5, size=(len(x[3::11]), 1)))
    x[4::11] = ties * 1.0078125 * np.exp2(rng.integers(-5, 5, size=(len(x[4::11]), 1)))
    return x.reshape(shape)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("B,N,D,k", [(1, 1, 32, 0), (2, 70, 96, 9), (1, 129, 160, 0), (2, 37, 2304, 11), (1, 300, 64, 0),
                                     (3, 128, 128, 0), (1, 5, 8192, 3)])
def test_quantise_parity(fmt, dtype, B, N, D, k):
    S = rows(B, N, k, D) if k else None
    R = k or N
    x = torch.from_numpy(spread((B, N, D), D)).to(dtype)
    for g in ([1.0] if fmt != "nvfp4" else [1.0, 0.0029761905, 0.1, 1e-6, 300.0]):
        g = float(np.float32(g))
        buf, data = guarded((B, R, D) if fmt == "mxfp8" else (B, R, D // 2), torch.uint8)
        if fmt == "mxfp8":
            data = data.view(torch.float8_e4m3fn)
        sbuf, sc = guarded((ops.mx_scale_bytes(B * R, D, fmt),), torch.uint8)
        out = ops.MxTensor(data, sc, fmt, g)
        m = ops.mx_quantize(dev(x), fmt, S=dev(S), scale=g, out=out)
        sel = to64(x) if S is None else np.stack([to64(x)[b, S[b]] for b in range(B)])
        code, byte = O.mx_encode(sel.reshape(-1, D), fmt, g)
        gb, rest = O.mx_untile(m.scales.cpu().numpy(), B * R, D // O.MX_BLOCK[fmt])
        assert np.array_equal(gb, byte) and not rest.any()
        # a block whose input overflowed fp16 has any codes
        got = O.mx_unpack(m.data.view(torch.uint8).cpu().numpy().reshape(B * R, -1), fmt)
        known = np.repeat(np.isfinite(O.mx_scale_values(byte, fmt)), O.MX_BLOCK[fmt], axis=-1)
        assert np.array_equal(got[known], code[known])
        assert untouched(buf) and untouched(sbuf)
        want = O.mx_decode(code, byte, fmt, g).reshape(B, R, D)
        for dt in (f32, bf16, f16):
            # the product with g rounds to fp32 once (exact without g), then to the type
            v = to64(ops.mx_dequantize(m, dt))
            assert np.array_equal(np.isnan(v), ~known.reshape(v.shape))
            ok = np.abs(want) <= torch.finfo(dt).max
            assert np.all((np.abs(v - want) <= half_step(dt, want) * (1 + 1e-6) + np.abs(want) * U)[ok])
    if D == 64 and dtype == bf16:  # a weight of two dims
        w = ops.mx_quantize(dev(x)[0], fmt)
        assert w.shape == (N, D) and torch.equal(w.data.view(torch.uint8), ops.mx_quantize(dev(x), fmt).data.view(torch.uint8)[0])
    assert ops.device_status() == 0


@pytest.mark.parametrize("g", [1.0, 0.1, 0.0029761905, 7.3e-4])
def test_nvfp4_borders(g):
    # fp32 inputs at every border of scales and elements, and one step to either side
    g = float(np.float32(g))
    s = O.E4M3[1:127]
    blocks = []
    for up in (0, 1, -1):
        a = (6.0 * g * (s[:-1] + s[1:]) / 2).astype(np.float32)  # between two scales
        a = np.nextafter(a, np.float32(np.inf) if up > 0 else np.float32(0)) if up else a
        x = np.zeros((len(a), 16), dtype=np.float32)
        x[:, 0] = a
        mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float64)
        e = (mid[None, :] * s[:-1, None] * g).astype(np.float32)
        x[:, 1:8] = np.nextafter(e, np.float32(np.inf) if up > 0 else np.float32(0)) if up else e
        x[:, 8:15] = -x[:, 1:8]
        x[:, 15] = 6 * s[:-1] * g
        blocks.append(x)
        y = x.copy()
        y[:, 0] = 0
        blocks.append(y)
    x = np.concatenate(blocks).reshape(1, -1, 1)
    n = x.size // 64 * 64
    x = x.reshape(-1)[:n].reshape(1, -1, 64).astype(np.float32)
    m = ops.mx_quantize(torch.from_numpy(x).to(DEV), "nvfp4", scale=g)
    code, byte = O.mx_encode(x[0].astype(np.float64), "nvfp4", g)
    gb, _ = O.mx_untile(m.scales.cpu().numpy(), x.shape[1], 4)
    assert np.array_equal(gb, byte) and np.array_equal(m.data.cpu().numpy()[0], O.mx_pack(code, "nvfp4"))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_quantise_extremes(fmt):
    x = torch.zeros((1, 8, 64), dtype=f32, device=DEV)
    x[0, 0, 3], x[0, 1, 40], x[0, 2, 0] = float("inf"), float("nan"), -float("inf")
    x[0, 3], x[0, 4], x[0, 5], x[0, 6, ::2] = 2.0 ** -149, torch.finfo(f32).max, -torch.finfo(f32).max, -0.0
    x[0, 7, 0] = 1.0
    m = ops.mx_quantize(x, fmt)
    blk = O.MX_BLOCK[fmt]
    gb, rest = O.mx_untile(m.scales.cpu().numpy(), 8, 64 // blk)
    nan = 127 if fmt == "nvfp4" else 255
    bad = {(0, 3 // blk), (1, 40 // blk), (2, 0)}
    assert {(int(i), int(j)) for i, j in np.argwhere(gb == nan)} == bad and not rest.any()
    keep = [3, 4, 5, 6, 7]
    code, byte = O.mx_encode(to64(x)[0, keep], fmt)
    assert np.array_equal(gb[keep], byte)
    assert np.array_equal(m.data.view(torch.uint8).cpu().numpy()[0, keep], O.mx_pack(code, fmt))
    v = ops.mx_dequantize(m, f32)
    assert v[0, 0, 3 // blk * blk:(3 // blk + 1) * blk].isnan().all() and v[0, 3:].isfinite().all()
    # an index out of range is flagged and replaced by row 0
    y = randn((1, 5, 64), 1, bf16).to(DEV)
    a = ops.mx_quantize(y, fmt, S=torch.tensor([[4, 5, -1, 4]], dtype=torch.int32, device=DEV))
    assert ops.device_status() == FLAG
    b = ops.mx_quantize(y, fmt, S=torch.tensor([[4, 0, 0, 4]], dtype=torch.int32, device=DEV))
    assert ops.device_status() == 0
    assert torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8)) and torch.equal(a.scales, b.scales)


# ---------------------------------------------------------------- microscaled layers
def operand(rows_, D, fmt, seed, g=1.0):
    """A microscaled matrix of random codes and scales (host arrays and MxTensor)."""
    rng = np.random.default_rng(seed)
    blk = O.MX_BLOCK[fmt]
    if fmt == "mxfp8":
        code = rng.integers(0, 127, size=(rows_, D)).astype(np.uint8) | (rng.integers(0, 2, size=(rows_, D)) << 7).astype(np.uint8)
    else:
        code = rng.integers(0, 16, size=(rows_, D)).astype(np.uint8)
    if fmt == "nvfp4":
        byte = rng.integers(24, 80, size=(rows_, D // blk)).astype(np.uint8)
    else:
        byte = rng.integers(118, 130, size=(rows_, D // blk)).astype(np.uint8)
    data = torch.from_numpy(O.mx_pack(code, fmt)).to(DEV)
    if fmt == "mxfp8":
        data = data.view(torch.float8_e4m3fn)
    m = ops.MxTensor(data, torch.from_numpy(O.mx_tile(byte)).to(DEV), fmt, g)
    return O.mx_decode(code, byte, fmt, m.scale), m


def linear_check(y, X, W, bias, act):
    """The products of elements and scales are exact; d_in of them are added in
    fp32 (d_in 2^-24 of the sum of their magnitudes; GELU's largest slope is
    1.13), then alpha, the bias and tanh (1e-6 of the value and absolute),
    then bf16's half step."""
    pre = X @ W.T + (0 if bias is None else bias)
    mag = np.abs(X) @ np.abs(W).T
    ref = oracle.gelu_tanh(pre) if act == "gelu_tanh" else pre
    tol = half_step(bf16, ref) * (1 + 1e-6) + 1.13 * (X.shape[1] * U * mag + 2 * U * np.abs(pre)) + 1e-6 * (1 + np.abs(ref))
    g = to64(y).reshape(ref.shape)
    assert np.all(np.isfinite(g))
    assert np.all(np.abs(g - ref) <= tol), float((np.abs(g - ref) - tol).max())


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,d_in,d_out,act,with_bias", [
    (1, 64, 8, "none", False), (2, 96, 40, "gelu_tanh", True), (5, 256, 192, "none", True), (130, 160, 200, "none", False),
    (257, 288, 392, "gelu_tanh", True), (300, 512, 576, "none", True), (700, 1312, 1000, "none", True),
    (64, 2304, 4000, "none", True), (1, 2304, 13824, "none", True), (3, 1184, 6912, "gelu_tanh", True),
    (513, 64, 3000, "none", False), (33, 4608, 328, "none", False), (16, 320, 264, "none", True), (17, 320, 264, "none", True)])
def test_mx_linear_parity(fmt, M, d_in, d_out, act, with_bias):
    gx, gw = (0.03, 0.2) if fmt == "nvfp4" else (1.0, 1.0)
    X, mX = operand(M, d_in, fmt, 1, gx)
    W, mW = operand(d_out, d_in, fmt, 2, gw)
    bias = None
    if with_bias:
        bias = np.random.default_rng(3).normal(size=d_out).astype(np.float32) * float(np.abs(X @ W[:8].T).mean())
    buf, out = guarded((M, d_out), bf16)
    y = ops.mx_linear(mX, mW, dev(bias), act, out=out)
    linear_check(y, X, W, bias, act)
    assert untouched(buf) and ops.device_status() == 0
    assert torch.equal(ops.mx_linear(mX, mW, dev(bias), act), y)  # the same bits again


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("d_in", [64, 96, 192, 288, 512])
def test_mx_linear_short_rows_many_tiles(fmt, d_in):
    # one to four stages of K a tile, several tiles to a CTA pair; Y aligned to
    # 16 bytes only
    M, d_out = 6000, 2304
    X, mX = operand(M, d_in, fmt, 11)
    W, mW = operand(d_out, d_in, fmt, 12)
    bias = np.random.default_rng(3).normal(size=d_out).astype(np.float32) * 100
    pick = np.random.default_rng(0).choice(M, 300, replace=False)
    buf, out = guarded((M, d_out), bf16, pad=272)
    y = ops.mx_linear(mX, mW, dev(bias), out=out)
    linear_check(y[torch.from_numpy(pick).to(DEV)], X[pick], W, bias, "none")
    assert untouched(buf, pad=272) and torch.equal(ops.mx_linear(mX, mW, dev(bias)), y) and ops.device_status() == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_mx_linear_many_tiles_and_nan_rows(fmt):
    # several tiles to a CTA pair; a NaN row stays in its row
    M, d_in, d_out = 2500, 256, 4608
    X, mX = operand(M, d_in, fmt, 5)
    W, mW = operand(d_out, d_in, fmt, 6)
    pick = np.random.default_rng(0).choice(M, 200, replace=False)
    y = ops.mx_linear(mX, mW)
    linear_check(y[torch.from_numpy(pick).to(DEV)], X[pick], W, None, "none")
    byte, _ = O.mx_untile(mX.scales.cpu().numpy(), M, d_in // O.MX_BLOCK[fmt])
    byte[1000, 2] = 127 if fmt == "nvfp4" else 255
    bad = ops.mx_linear(ops.MxTensor(mX.data, torch.from_numpy(O.mx_tile(byte)).to(DEV), fmt), mW)
    assert bad[1000].isnan().all()
    rest = torch.arange(M, device=DEV) != 1000
    assert torch.equal(bad[rest], y[rest]) and ops.device_status() == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,d_in,d_out,act", [(1, 9216, 264, "none"), (300, 9216, 520, "gelu_tanh"),
                                              (2458, 9216, 2304, "none"), (700, 20000, 1000, "gelu_tanh")])
def test_mx_linear_split_along_d_in(fmt, M, d_in, d_out, act):
    # the last wave's tiles in pieces: against the oracle on some rows, and
    # against whole tiles, which add in another order
    gx, gw = (0.03, 0.2) if fmt == "nvfp4" else (1.0, 1.0)
    X, mX = operand(M, d_in, fmt, 7, gx)
    W, mW = operand(d_out, d_in, fmt, 8, gw)
    pick = np.unique(np.r_[0, M - 1, np.random.default_rng(1).choice(M, min(M, 60), replace=False)])
    bias = np.random.default_rng(3).normal(size=d_out).astype(np.float32) * float(np.abs(X[pick] @ W[:8].T).mean())
    n = ops.mx_linear_workspace_bytes(M, d_in, d_out, fmt)
    assert (n > 0) == (M != 2458 or fmt == "mxfp8")  # 36 stages of 4 bits: not worth it
    buf, ws = guarded((n,), torch.uint8)
    obuf, out = guarded((M, d_out), bf16)
    y = ops.mx_linear(mX, mW, dev(bias), act, out=out, ws=ws)
    at = torch.from_numpy(pick).to(DEV)
    linear_check(y[at], X[pick], W, bias, act)
    assert untouched(buf) and untouched(obuf)
    assert torch.equal(ops.mx_linear(mX, mW, dev(bias), act), y)
    whole = ops.mx_linear(mX, mW, dev(bias), act, ws=False)
    linear_check(whole[at], X[pick], W, bias, act)
    # a workspace that is too small: whole tiles
    assert torch.equal(ops.mx_linear(mX, mW, dev(bias), act, ws=ws[:max(n - 32, 0)]), whole)
    assert ops.device_status() == 0


def test_mx_linear_gelu_over_its_range():
    X, mX = operand(20, 64, "mxfp8", 1)
    W, mW = operand(512, 64, "mxfp8", 2)
    X, W = X * 0, W
    zero = ops.MxTensor(torch.zeros_like(mX.data.view(torch.uint8)).view(torch.float8_e4m3fn), mX.scales, "mxfp8")
    bias = np.linspace(-12, 12, 512).astype(np.float32)
    linear_check(ops.mx_linear(zero, mW, dev(bias), "gelu_tanh"), X, W, bias, "gelu_tanh")
    # far values: x or (nearly) nothing, a NaN stays a NaN beside them
    far = np.array([1e4, -1e4, 1e20, -1e20, np.inf, -np.inf, np.nan, 1.0] * 64, dtype=np.float32)
    y = to64(ops.mx_linear(zero, mW, dev(far), "gelu_tanh"))[:, :8]
    assert np.allclose(y[:, [0, 2, 7]], [1e4, 1e20, 0.8411920], rtol=2.0 ** -8) and np.all(y[:, 4] == np.inf)
    # -inf gives -inf * 0, a NaN, as the formula in fp32 does
    assert np.all(np.abs(y[:, [1, 3]]) < 1e-16) and np.all(np.isnan(y[:, 5:7]))


# ---------------------------------------------------------------- together
def test_row_selective_block_in_low_precision():
    """norm in 8 bits -> q, k, v -> rotary positions in place -> assembled SRSU ->
    quantised rows -> projection -> the stream's rows and the next norm -> MLP,
    each step against its oracle on the GPU's own inputs."""
    B, N, H, d, k = 2, 300, 3, 64, 70
    D = H * d
    S = rows(B, N, k, 1)
    Sd = dev(S)
    stream = randn((B, N, D), 2, bf16).to(DEV)
    w = (1 + 0.2 * randn((D,), 3)).to(DEV)
    wq, wo, wu, wd = (ops.mx_quantize((randn((o, i), 4 + o) / math.sqrt(i)).to(DEV), f)
                      for o, i, f in ((3 * D, D, "mxfp8"), (D, D, "mxfp8"), (4 * D, D, "mxfp8"), (D, 4 * D, "mxfp8")))

    def values(m):
        return to64(ops.mx_dequantize(m, f32)).reshape(-1, m.shape[-1])

    sel = np.stack([to64(stream)[b, S[b]] for b in range(B)])
    x = ops.rms_norm(stream, w, S=Sd, quant="mxfp8")
    check_mxfp8(x, O.rms_norm(sel, to64(w))[1], (D / 2 + 8) * U)
    qkv = ops.mx_linear(x, wq)
    linear_check(qkv, values(x), values(wq), None, "none")
    qkv = qkv.view(B, k, 3 * H, d)
    q, kk, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:].contiguous()
    at = np.stack(np.meshgrid(np.arange(15), np.arange(20), indexing="ij"), -1).reshape(-1, 2).astype(np.int32)
    f, m = ops.rope_frequencies(d, sections=[16, 16])
    before = q.clone().cpu(), kk.clone().cpu()
    ops.rope(q, kk, ops.rope_table(d, sections=[16, 16]), pos=dev(at), S=Sd, inplace=True)
    ps = np.stack([at[S[b]] for b in range(B)])
    rope_check(q, before[0], O.rope(to64(before[0]), f, [16, 16], ps), bf16, d, m)
    rope_check(kk, before[1], O.rope(to64(before[1]), f, [16, 16], ps), bf16, d, m)
    Kc, Vc = randn((B, N, H, d), 8, bf16).to(DEV), randn((B, N, H, d), 9, bf16).to(DEV)
    o = ops.srsu_attn_assembled(q.contiguous(), Sd, kk.contiguous(), v, Kc, Vc, q_compact=True, cur_compact=True)
    Ka, Va = Kc.clone(), Vc.clone()
    for b in range(B):
        Ka[b, Sd[b].long()], Va[b, Sd[b].long()] = kk[b], v[b]
    from tests.helpers import assert_attn_close
    s = np.einsum("brhd,bnhd->bhrn", to64(q), to64(Ka)) / math.sqrt(d)
    p = np.exp(s - s.max(-1, keepdims=True))
    assert_attn_close(o, np.einsum("bhrn,bnhd->brhd", p / p.sum(-1, keepdims=True), to64(Va)), "srsu")
    oq = ops.mx_quantize(o.view(B, k, D), "mxfp8")
    y = ops.mx_linear(oq, wo)
    linear_check(y, values(oq), values(wo), None, "none")
    old = stream.clone()
    x, h = ops.rms_norm(y, w, stream, Sd, x_compact=True, quant="mxfp8", update=True)
    href, yref = O.rms_norm(to64(y), to64(w), to64(old), S)
    hs = np.stack([to64(h)[b, S[b]] for b in range(B)])
    assert h is stream and np.all(np.abs(hs - href) <= half_step(bf16, href) * (1 + 1e-6) + np.abs(href) * U)
    check_mxfp8(x, yref, (D / 2 + 8) * U)
    u = ops.mx_linear(x, wu, act="gelu_tanh")
    linear_check(u, values(x), values(wu), None, "gelu_tanh")
    uq = ops.mx_quantize(u, "mxfp8")
    linear_check(ops.mx_linear(uq, wd), values(uq), values(wd), None, "none")
    assert ops.device_status() == 0


def chain(x, r, w, S, tab, pos, W):
    y, h = ops.rms_norm(x, w, r, S, x_compact=True)
    m = ops.mx_quantize(y, W.fmt, scale=1.0)
    z = ops.mx_linear(m, W, act="gelu_tanh")
    q, _ = ops.rope(z.view(*z.shape[:2], -1, 64), None, tab, pos=pos, S=S)
    return h, q


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("k", [6, 90])
def test_streams_and_graphs(fmt, k):
    B, N, D = 2, 200, 256
    S, w, pos = dev(rows(B, N, k, 1)), randn((D,), 2).to(DEV), torch.arange(N, dtype=torch.int32, device=DEV)
    W = ops.mx_quantize((randn((192, D), 3) / 16).to(DEV), fmt)
    tab = ops.rope_table(64)
    xs = [(randn((B, k, D), 10 + i, bf16).to(DEV), randn((B, N, D), 20 + i, bf16).to(DEV)) for i in range(3)]
    want = [chain(x, r, w, S, tab, pos, W) for x, r in xs]
    torch.cuda.synchronize()
    # two streams at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            got.append([chain(*xs[i], w, S, tab, pos, W) for _ in range(4)][-1])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    # captured, replayed on other inputs; a second graph of the same leaves beside it
    x, r = xs[0][0].clone(), xs[0][1].clone()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(chain(x, r, w, S, tab, pos, W))
        graphs.append(g)
    for i in (1, 2, 0):
        x.copy_(xs[i][0])
        r.copy_(xs[i][1])
        for g, o in zip(graphs, outs):
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want[i]))
    assert ops.device_status() == 0


@pytest.mark.parametrize("rows_,d,hidden", [(16, 256, 512), (700, 512, 2304), (4096, 2304, 6912)])
def test_layers_that_write_what_the_one_before_reads(rows_, d, hidden):
    # one set of buffers, taken in turn by launches that overlap at their ends; the
    # last size splits its last wave. Against the same calls one at a time.
    up = ops.mx_quantize((randn((hidden, d), 1) / math.sqrt(d)).to(DEV), "mxfp8")
    down = ops.mx_quantize((randn((d, hidden), 2) / math.sqrt(hidden)).to(DEV), "mxfp8")
    first = randn((rows_, d), 3, bf16).to(DEV)
    x, h, bias = torch.empty_like(first), torch.empty((rows_, hidden), dtype=bf16, device=DEV), torch.empty(d, device=DEV)
    nbytes = ops.mx_linear_workspace_bytes(rows_, hidden, d, "mxfp8")
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=DEV)
    X = ops.mx_quantize(first, "mxfp8")
    H = ops.mx_quantize(torch.zeros_like(h), "mxfp8")

    def run(wait):
        x.copy_(first)
        bias.zero_()
        for i in range(4):
            ops.mx_quantize(x, "mxfp8", out=X)
            wait()
            ops.mx_linear(X, up, act="gelu_tanh", out=h)
            wait()
            ops.mx_quantize(h, "mxfp8", out=H)
            wait()
            bias.add_(0.25)
            ops.mx_linear(H, down, bias, out=x, ws=ws)
            wait()
            ops.mx_linear(H, down, bias, out=x, ws=ws)  # the same again, behind its own kernels
            wait()
        return x.clone()

    want = run(torch.cuda.synchronize)
    assert want.isfinite().all()
    for _ in range(5):
        assert torch.equal(run(lambda: None), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = run(lambda: None)
    for _ in range(3):
        y.zero_()
        g.replay()
        assert torch.equal(y, want)
    assert ops.device_status() == 0


def test_first_calls_inside_a_capture():
    # a process whose first calls are captured: nothing in them needs a stream
    code = """
import torch
from mask_free_b200 import ops
x = torch.randn((1, 300, 256), device="cuda").to(torch.bfloat16)
w = torch.randn((192, 256), device="cuda").to(torch.bfloat16)
tab = ops.rope_table(64)
ops.lib()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = ops.rms_norm(x, quant="mxfp8")
    z = ops.mx_linear(y, ops.mx_quantize(w, "mxfp8"), act="gelu_tanh")
    q, _ = ops.rope(z.view(1, 300, 3, 64), None, tab)
g.replay()
torch.cuda.synchronize()
z = ops.mx_linear(ops.rms_norm(x, quant="mxfp8"), ops.mx_quantize(w, "mxfp8"), act="gelu_tanh")
assert torch.equal(q, ops.rope(z.view(1, 300, 3, 64), None, tab)[0]) and ops.device_status() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_long_tensors():
    # more than 2^31 elements: offsets of rows, elements and scales
    N, D = 2 ** 31 // 2304 + 300, 2304
    x = torch.zeros((1, N, D), dtype=bf16, device=DEV)
    tail = randn((1, 200, D), 1, bf16).to(DEV)
    x[:, -200:] = tail
    w = (1 + 0.1 * randn((D,), 2)).to(DEV)
    y = ops.rms_norm(x, w)
    assert torch.equal(y[:, -200:], ops.rms_norm(tail, w)) and not y[:, :1000].any()
    del y
    for fmt in ("mxfp8", "nvfp4"):
        m = ops.mx_quantize(x, fmt)
        ref = ops.mx_quantize(tail, fmt)
        assert torch.equal(m.data[:, -200:].view(torch.uint8), ref.data.view(torch.uint8))
        assert torch.equal(ops.mx_dequantize(m)[:, -200:], ops.mx_dequantize(ref))
        if fmt == "nvfp4":  # its last rows as a layer's input, with a small weight
            W = ops.mx_quantize((randn((8, D), 3) / 48).to(DEV), fmt)
            assert torch.equal(ops.mx_linear(m, W)[:, -200:], ops.mx_linear(ref, W))
        del m
    S = torch.tensor([[N - 1, N - 200, 0]], dtype=torch.int32, device=DEV)
    assert torch.equal(ops.rms_norm(x, w, S=S)[:, :2], ops.rms_norm(tail[:, [199, 0]].contiguous(), w))
    q, _ = ops.rope(x.view(1, N, 36, 64), None, ops.rope_table(64), inplace=True)
    pos = torch.arange(N - 200, N, dtype=torch.int32, device=DEV)
    assert torch.equal(q[:, -200:], ops.rope(tail.view(1, 200, 36, 64), None, ops.rope_table(64), pos=pos)[0])
    assert ops.device_status() == 0
