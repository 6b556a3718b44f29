"""fp64 definitions of the row-wise operators around the block's attention:
root-mean-square norm with the residual, rotary positions, microscaled
quantisation (test infrastructure only; numpy, nothing shared with the CUDA
library). Arguments and results are float64 arrays, and codes and scale bytes
uint8."""

from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

# ---------------------------------------------------------------- norm


def rms_norm(x, w=None, res=None, S=None, eps: float = 1e-6, x_full: bool = False):
    """(h, y): h = x + res, y = h / sqrt(mean(h^2) + eps) * w. With S [B, k] the
    rows S of res, and of x when x_full (else x holds them already)."""
    x = np.asarray(x, dtype=np.float64)
    pick = (lambda t: t) if S is None else (lambda t: np.stack([t[b, S[b]] for b in range(t.shape[0])]))
    h = pick(x) if x_full or S is None else x
    if res is not None:
        h = h + pick(np.asarray(res, dtype=np.float64))
    y = h / np.sqrt((h * h).mean(axis=-1, keepdims=True) + eps)
    return h, y if w is None else y * np.asarray(w, dtype=np.float64)


# ---------------------------------------------------------------- rotary positions


def rope(x, freqs: Sequence[float], sections: Sequence[int], pos, interleaved: bool = False, m: float = 1.0):
    """Pair i of every head of x [B, R, H, d] times the complex number m e^(i angle),
    angle = position * freqs[i]; pos [B, R, axes], pair i takes the axis its
    section names."""
    x = np.array(x, dtype=np.float64)
    n = len(freqs)
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = np.asarray(pos, dtype=np.float64)[:, :, axis] * np.asarray(freqs)          # [B, R, n]
    turn = (m * np.exp(1j * angle))[:, :, None, :]
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    z = (x[..., a] + 1j * x[..., b]) * turn
    x[..., a], x[..., b] = z.real, z.imag
    return x


# ---------------------------------------------------------------- microscaled formats

MX_BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3 magnitudes by code: subnormals m 2^-9, then (8 + m) 2^(e - 10); code 127 is NaN
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119])


def nearest_code(v, table):
    """Index of the entry of an ascending table nearest to v >= 0; ties to the
    even index, values past the end to the last entry."""
    v = np.asarray(v, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    up, down = table[hi] - v, v - table[lo]
    return np.where(up < down, hi, np.where(down < up, lo, np.where(lo % 2 == 0, lo, hi))).astype(np.uint8)


def mx_encode(x, fmt: str, g: float = 1.0):
    """(codes [..., D], scale bytes [..., D / block]) of x: the element codes with
    the sign in the top bit, the scales as e8m0 or e4m3 bytes. A block with an
    infinity or a NaN has the NaN scale, and any codes (zeros here)."""
    x = np.asarray(x, dtype=np.float64)
    blk = MX_BLOCK[fmt]
    xb = x.reshape(*x.shape[:-1], -1, blk)
    finite = np.isfinite(xb).all(axis=-1)
    xb = np.where(finite[..., None], xb, 0.0)
    top = np.abs(xb).max(axis=-1)
    if fmt == "nvfp4":
        byte = nearest_code(top / (6.0 * g), E4M3)
        unit = E4M3[byte] * g
    else:
        e = np.frexp(top)[1] - 1 - (8 if fmt == "mxfp8" else 2)
        e = np.where(top > 0, np.clip(e, -127, 127), -127)
        byte = (e + 127).astype(np.uint8)
        unit = np.ldexp(1.0, e)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(unit[..., None] > 0, np.abs(xb) / unit[..., None], 0.0)
    code = nearest_code(r, E4M3 if fmt == "mxfp8" else E2M1)
    code |= np.signbit(xb).astype(np.uint8) << (7 if fmt == "mxfp8" else 3)
    return code.reshape(x.shape), np.where(finite, byte, 127 if fmt == "nvfp4" else 255).astype(np.uint8)


def mx_scale_values(byte, fmt: str):
    byte = np.asarray(byte)
    if fmt == "nvfp4":
        return np.append(E4M3, np.nan)[byte & 127]
    return np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))


def mx_decode(code, byte, fmt: str, g: float = 1.0):
    """The values that codes and scale bytes stand for."""
    code = np.asarray(code)
    if fmt == "mxfp8":
        v = np.append(E4M3, np.nan)[code & 127] * np.where(code & 128, -1.0, 1.0)
    else:
        v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.repeat(mx_scale_values(byte, fmt), MX_BLOCK[fmt], axis=-1)
    return v * s * g


def mx_pack(code, fmt: str):
    """Codes to bytes: two of 4 bits to a byte, the even element in the low half."""
    return code if fmt == "mxfp8" else (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def mx_unpack(data, fmt: str):
    if fmt == "mxfp8":
        return data
    return np.stack([data & 15, data >> 4], axis=-1).reshape(*data.shape[:-1], -1)


def mx_tile(byte, fill: int = 0):
    """Scale bytes [rows, n] in tiles of 128 rows x 4 scales: row i and scale j of
    a tile at byte (i % 32) 16 + (i // 32) 4 + j."""
    rows, n = byte.shape
    rt, ct = -(-rows // 128), -(-n // 4)
    out = np.full((rt, ct, 512), fill, dtype=np.uint8)
    for i in range(rows):
        for j in range(n):
            out[i // 128, j // 4, (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4] = byte[i, j]
    return out.reshape(-1)


def mx_untile(flat, rows: int, n: int):
    """(scale bytes [rows, n], the bytes that only fill tiles up)."""
    rt, ct = -(-rows // 128), -(-n // 4)
    i, j = np.meshgrid(np.arange(rows), np.arange(n), indexing="ij")
    at = ((i // 128) * ct + j // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4
    rest = np.ones(rt * ct * 512, dtype=bool)
    rest[at.reshape(-1)] = False
    return flat[at], flat[rest]
