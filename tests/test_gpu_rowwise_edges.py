"""GPU tests of the row-wise operators at calls off their usual path: lists of
rows out of order, and the widths at which the norm's launch changes its form.
Bounds and helpers: test_gpu_rowwise.py."""

import numpy as np
import pytest
import torch

from mask_free_b200 import ops
from oracle import rowwise as O
from tests.test_gpu_rowwise import DEV, FLAG, U, bf16, check_mxfp8, dev, f16, f32, half_step, norm_tol, randn, rows, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean():
    ops.device_status()
    yield


# ---------------------------------------------------------------- rows out of order, in place
def counted(S, N):
    """Rows that an update in place takes: inside [0, N), above every earlier index."""
    S = np.asarray(S, dtype=np.int64)
    before = np.maximum.accumulate(np.concatenate([np.full((len(S), 1), -1), S], axis=1), axis=1)[:, :-1]
    return (S > before) & (S < N)


def update_check(S, N, D, dtype, quant, seed):
    B, k = S.shape
    x, r, w = randn((B, k, D), seed, dtype), randn((B, N, D), seed + 1, dtype), 1 + 0.2 * randn((D,), seed + 2)
    ok = counted(S, N)
    stream = r.to(DEV)
    y, h = ops.rms_norm(x.to(DEV), w.to(DEV), stream, dev(S), x_compact=True, quant=quant, update=True)
    assert h is stream and ops.device_status() == (0 if ok.all() else FLAG)
    want, keep = to64(r), np.ones((B, N), dtype=bool)
    yref = np.zeros((B, k, D))
    for b, i in np.argwhere(ok):
        hb, yref[b, i] = O.rms_norm(to64(x)[None, b, i:i + 1], to64(w), want[None, b, S[b, i]:S[b, i] + 1])
        want[b, S[b, i]], keep[b, S[b, i]] = hb[0, 0], False
    got = to64(h)
    assert np.array_equal(got[keep], want[keep])  # every other row of the stream as it was
    assert np.all(np.abs(got - want) <= half_step(dtype, want) * (1 + 1e-6) + np.abs(want) * U)
    if quant is None:
        assert np.all(np.abs(to64(y) - yref) <= half_step(dtype, yref) * (1 + 1e-6) + norm_tol(yref, D))
        assert not to64(y)[~ok].any()
    else:
        check_mxfp8(y, yref, (D / 2 + 8) * U)
        assert not ops.mx_dequantize(y, f32)[torch.from_numpy(~ok).to(DEV)].any()


@pytest.mark.parametrize("dtype,D,quant", [(bf16, 1, None), (f16, 63, None), (f32, 64, None), (bf16, 2304, None),
                                           (bf16, 41000, None), (bf16, 96, "mxfp8"), (f32, 2304, "mxfp8")])
@pytest.mark.parametrize("S", [[[5, 3, 5]], [[8, 1, 2, 8]], [[5, 3, 4, 5]], [[3, -1, 3]], [[2, 9, 3]], [[0, 0]], [[7]], [[-1]],
                               [[1, 2, 3, 4], [4, 3, 2, 1], [6, 6, 7, 6], [0, 2 ** 31 - 1, 5, -2 ** 31]]])
def test_update_in_place_takes_an_index_once(S, dtype, D, quant):
    update_check(np.array(S, dtype=np.int32), 9, D, dtype, quant, 7)


@pytest.mark.parametrize("k", [1023, 1024, 1025, 2500])
def test_update_in_place_of_long_lists(k):
    # equal and smaller indices far behind the first, in the same and in other runs of 1024
    N = 3000
    S = rows(3, N, k, k)
    S[1, k - 1] = S[1, 3]
    S[2, 700] = N - 1  # every row behind it is out of order
    assert counted(S, N)[0].all() and not counted(S, N)[1, k - 1] and not counted(S, N)[2, 701:].any()
    for dtype, D, quant in ((bf16, 32, "mxfp8"), (f32, 40, None)):
        update_check(S, N, D, dtype, quant, 11)


# ---------------------------------------------------------------- every form of the norm, at both ends of its widths
def norm_check(dtype, N, D, S, seed):
    w = 1 + 0.2 * randn((D,), seed)
    x, r = randn((1, len(S[0]) if S is not None else N, D), seed + 1, dtype), 2 * randn((1, N, D), seed + 2, dtype)
    href, yref = O.rms_norm(to64(x), to64(w), to64(r), S)
    y, h = ops.rms_norm(dev(x), dev(w), dev(r), dev(S), x_compact=S is not None)
    assert np.all(np.abs(to64(y) - yref) <= half_step(dtype, yref) * (1 + 1e-6) + norm_tol(yref, D))
    assert np.all(np.abs(to64(h) - href) <= half_step(dtype, href) * (1 + 1e-6) + np.abs(href) * U)
    if S is None:  # without the residual and the weight
        _, yref = O.rms_norm(to64(x))
        y = ops.rms_norm(dev(x))
        assert np.all(np.abs(to64(y) - yref) <= half_step(dtype, yref) * (1 + 1e-6) + norm_tol(yref, D))
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("D", [8, 64, 72, 256, 264, 512, 520, 1024, 1032, 1536, 1544, 2048, 2056, 2304, 2312, 3064, 3080, 4096,
                               4104, 7168, 7176, 10240, 10248, 20480, 20488, 40960, 40968])
def test_norm_of_widths_in_units_of_8(dtype, D):
    for N in (5, 37) if D < 4096 else (5,):
        norm_check(dtype, N, D, None, D)
    norm_check(dtype, 9, D, np.array([[0, 3, 4, 8]], dtype=np.int32), D)


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("D", [1, 7, 9, 63, 65, 249, 250, 319, 321, 505, 507, 1009, 1019, 1279, 1281, 1521, 1531, 2001, 2033, 2043,
                               2289, 2299, 2303, 2559, 2561, 3057, 3059, 4081, 4083, 7153, 7155, 10225, 10227, 20465, 20467])
def test_norm_of_other_widths(dtype, D):
    # without S by shifted units, with S one by one; rows that share units with both neighbours
    norm_check(dtype, 11, D, None, D)
    norm_check(dtype, 9, D, np.array([[0, 3, 4, 8]], dtype=np.int32), D)


@pytest.mark.parametrize("dtype", [bf16, f16, f32])
@pytest.mark.parametrize("D", [32, 64, 256, 288, 512, 544, 1024, 1056, 1536, 1568, 2048, 2080, 2304, 2336, 3040, 3104, 4096, 4128,
                               7168, 7200, 10240, 10272, 20480, 20512, 40960])
def test_norm_in_8_bits_of_every_width(dtype, D):
    N = 133 if D < 4096 else 5  # more than one tile of scales
    x, r, w = randn((1, N, D), D, dtype), randn((1, N, D), D + 1, dtype), 1 + 0.2 * randn((D,), D + 2)
    x[..., ::17] *= 8
    for S in (None, np.arange(1, N, 2, dtype=np.int32)[None]):
        xs = x if S is None else x[:, :S.shape[1]].contiguous()
        href, yref = O.rms_norm(to64(xs), to64(w), to64(r), S)
        y, h = ops.rms_norm(dev(xs), dev(w), dev(r), dev(S), x_compact=S is not None, quant="mxfp8")
        assert np.all(np.abs(to64(h) - href) <= half_step(dtype, href) * (1 + 1e-6) + np.abs(href) * U)
        check_mxfp8(y, yref, (D / 2 + 8) * U)
    assert ops.device_status() == 0


@pytest.mark.parametrize("dtype,D,quant", [(bf16, 8, None), (bf16, 2304, None), (f32, 63, None), (bf16, 41000, None),
                                           (bf16, 32, "mxfp8"), (f16, 2304, "mxfp8")])
def test_update_in_place_of_bad_rows_only(dtype, D, quant):
    # rows of no token: their y is zeros, whichever of the call's two kernels comes to it last
    B, N, k = (2, 30000, 25000) if D < 64 else (2, 3000, 2600) if D < 4096 else (2, 400, 300)
    S = torch.full((B, k), -1, dtype=torch.int32, device=DEV)
    S[1, ::3] = N
    x, stream = (torch.ones((B, n, D), dtype=dtype, device=DEV) for n in (k, N))
    for _ in range(10):
        y, _ = ops.rms_norm(x, None, stream, S, x_compact=True, quant=quant, update=True)
        v = y if quant is None else ops.mx_dequantize(y, f32)
        assert not v.any() and ops.device_status() == FLAG
        if quant is not None:
            assert not y.data.view(torch.uint8).any() and not y.scales.any()
    assert bool((stream == 1).all())


@pytest.mark.parametrize("k", [128 * 1024, 128 * 1024 + 1, 300007])
def test_update_in_place_of_very_long_lists(k):
    # more than 1024 rows to a CTA of the marks; an index again from other runs, rows behind a large one
    N, D = 300500, 8
    S = rows(2, N, k, k)
    again = [(1023, 5), (1024, 1023), (3000, 3000 - 1), (k - 1, k // 2), (k // 2 + 7, 0)]
    for at, of in again:
        S[0, at] = S[0, of]
    S[1, k - 3000] = N - 1
    ok = counted(S, N)
    assert not any(ok[0, at] for at, _ in again) and not ok[1, k - 2999:].any() and ok[1, :k - 2999].all()
    x, r = randn((2, k, D), 1, bf16).to(DEV), randn((2, N, D), 2, bf16).to(DEV)
    stream = r.clone()
    y, _ = ops.rms_norm(x, None, stream, dev(S), x_compact=True, update=True)
    assert ops.device_status() == FLAG
    y0, h0 = ops.rms_norm(x, None, r, dev(S), x_compact=True)  # apart, an index may come again
    okd = torch.from_numpy(ok).to(DEV)
    want = r.clone()
    for b in range(2):
        want[b, torch.from_numpy(S[b][ok[b]]).long().to(DEV)] = h0[b][okd[b]]
    assert torch.equal(stream, want) and torch.equal(y, torch.where(okd[..., None], y0, torch.zeros_like(y0)))


def test_norm_past_the_range_of_its_squares():
    # finite rows whose sum of squares is infinite in fp32: zeros, and their sums h as they are
    x = torch.full((1, 3, 64), 1e19, dtype=f32, device=DEV)
    x[0, 1] = 3.0
    y, h = ops.rms_norm(x, None, torch.zeros_like(x))
    assert not y[0, 0].any() and not y[0, 2].any() and torch.equal(h, x)
    assert torch.allclose(y[0, 1], torch.ones(64, device=DEV), rtol=1e-6)


@pytest.mark.parametrize("quant", [None, "mxfp8"])
@pytest.mark.parametrize("D,k", [(64, 90), (2304, 1500)])
def test_update_in_place_captured_and_on_two_streams(D, k, quant):
    # the marks and the norm behind them: replayed on other lists and inputs, full x, two calls at once
    B, N = 2, 1600
    w = (1 + 0.2 * randn((D,), 1)).to(DEV)
    lists = [rows(B, N, k, i) for i in range(3)]
    lists[1][0, k // 2] = lists[1][0, 1]  # an index again
    lists[2][1, 3], lists[2][1, 7] = -1, N
    cases = [(dev(S), randn((B, N, D), 10 + i, bf16).to(DEV), randn((B, N, D), 20 + i, bf16).to(DEV)) for i, S in enumerate(lists)]

    def call(S, x, stream):
        y, _ = ops.rms_norm(x, w, stream, S, quant=quant, update=True)
        return y if quant is None else ops.mx_dequantize(y)

    want = []
    for (S, x, r), host in zip(cases, lists):
        stream, ok = r.clone(), torch.from_numpy(counted(host, N)).to(DEV)
        want.append((call(S, x, stream), stream))
        y0, h0 = ops.rms_norm(x, w, r, S, quant=quant)  # apart
        y0 = y0 if quant is None else ops.mx_dequantize(y0)
        assert torch.equal(want[-1][0], torch.where(ok[..., None], y0, torch.zeros_like(y0)))
        full = r.clone()
        for b in range(B):
            full[b, S[b][ok[b]].long()] = h0[b][ok[b]]
        assert torch.equal(stream, full)
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(3):
        for (S, x, r), st in zip(cases, streams):
            with torch.cuda.stream(st):
                stream = r.clone()
                got.append((call(S, x, stream), stream))
    torch.cuda.synchronize()
    for i, (y, stream) in enumerate(got):
        assert torch.equal(y, want[i % 2][0]) and torch.equal(stream, want[i % 2][1])
    S, x, r = (t.clone() for t in cases[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = call(S, x, r)
    for i in (1, 2, 0, 1):
        for a, b in zip((S, x, r), cases[i]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i][0]) and torch.equal(r, want[i][1])
    assert ops.device_status() == FLAG
