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
