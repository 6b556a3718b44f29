"""Thin Python binding over libsafe_attn.so (argument marshalling only).

Every function takes CUDA torch tensors, checks their dtype / shape /
contiguity, passes raw pointers and the current torch stream to the C ABI of
``include/safe_attn.h`` and raises ``SafeError`` on a non-OK status. All
computation runs in the library's CUDA kernels; there is no CPU fallback: if
the library is missing or fails to load, every call raises.
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsafe_attn.so")
_lib = None

SAFE_OK, SAFE_ERR_INVALID_ARG, SAFE_ERR_UNSUPPORTED, SAFE_ERR_CUDA, SAFE_ERR_TIMEOUT, SAFE_ERR_DEVICE_CHECK = range(6)
_MASK_DTYPES = {torch.bool: 0, torch.uint8: 1, torch.float32: 2, torch.float16: 3, torch.bfloat16: 4}

_vp, _i, _f, _i64p, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.POINTER(ctypes.c_int64), ctypes.c_size_t
_i64, _i32p = ctypes.c_int64, ctypes.POINTER(ctypes.c_int32)

# name -> argtypes (restype is int for every entry point except the ones listed)
_SIGS = {
    "safe_abi_version": [],
    "safe_mask_classify": [_vp, _i, _i64p, _i64p, _vp, _vp],
    "safe_mask_classify_sync": [_vp, _i, _i64p, _i64p, _vp, _i64p, _vp],
    "safe_attn_workspace_bytes": [_i, _i, _i, _i, _i],
    "safe_attn_self": [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _sz, _vp],
    "safe_attn_cross": [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp],
    "safe_pcsp_workspace_bytes": [_i, _i, _i],
    "safe_pcsp_topk": [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _i, _i, _vp, _vp, _vp, _sz, _vp],
    "safe_topk_partition": [_vp, _i, _i, _i, _vp, _vp, _vp],
    "safe_srsu_workspace_bytes": [_i, _i, _i, _i, _i],
    "safe_srsu_attn": [_vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _sz, _vp],
    "safe_srsu_attn_assembled": [_vp, _i, _vp, _i, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _vp, _sz,
                                 _vp],
    "safe_ctx_cache_scatter": [_vp, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _vp],
    "safe_get_device_status": [ctypes.POINTER(ctypes.c_int), _vp],
    "safe_status_string": [_i],
    "safe_selftest_wait_timeout": [ctypes.c_uint64, _vp],
    "safe_pcsp_topk_noalloc": [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _i, _i, _vp, _vp, _vp],
    "safe_attn_cross_pcsp": [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _i, _i, _vp, _vp, _vp,
                             _sz, _vp],
    "safe_sensitivity_workspace_bytes": [_i, _i],
    "safe_sensitivity_field": [_vp, _vp, _i, _i, _i, _f, _f, _vp, _sz, _vp],
    "safe_partition_indicator": [_vp, _i, _vp, _i, _i, _vp],
    "safe_sw_cfg": [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _f, _vp],
    "safe_gather_linear_workspace_bytes": [_i, _i, _i],
    "safe_gather_linear": [_vp, _vp, _i, _vp, _vp, _i, _vp, _i, _i, _i, _i, _vp, _sz, _vp],
    "safe_rms_norm": [_vp, _i, _vp, _vp, _i, _vp, _f, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _vp],
    "safe_rope": [_vp, _i64p, _vp, _i64p, _i, _vp, _i64p, _vp, _i64p, _i, _i, _vp, _i32p, _i, _vp, _i, _vp, _i, _i, _i,
                  _i, _i, _i, _f, _vp],
    "safe_mx_scale_bytes": [_i64, _i, _i],
    "safe_mx_quantize": [_vp, _i, _vp, _i, _i, _f, _vp, _vp, _i, _i, _i, _vp],
    "safe_mx_dequantize": [_vp, _vp, _i, _f, _vp, _i, _i64, _i, _vp],
    "safe_mx_linear_workspace_bytes": [_i64, _i, _i, _i],
    "safe_mx_linear": [_vp, _vp, _vp, _vp, _i, _f, _vp, _i, _vp, _i64, _i, _i, _vp, _sz, _vp],
}
_RESTYPES = {"safe_pcsp_workspace_bytes": _sz, "safe_attn_workspace_bytes": _sz, "safe_sensitivity_workspace_bytes": _sz,
             "safe_gather_linear_workspace_bytes": _sz, "safe_srsu_workspace_bytes": _sz,
             "safe_mx_scale_bytes": _sz,
             "safe_mx_linear_workspace_bytes": _sz, "safe_status_string": ctypes.c_char_p}


class SafeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({_status_string(status)})")


def lib():
    """Load libsafe_attn.so (once). Raises if it is missing: no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with `python -m mask_free_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = _RESTYPES.get(name, ctypes.c_int)
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


def _status_string(st: int) -> str:
    try:
        return lib().safe_status_string(st).decode()
    except Exception:  # pragma: no cover
        return "?"


def _check(fn: str, st: int):
    if st != SAFE_OK:
        raise SafeError(fn, st)


def _stream() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on_device(t: torch.Tensor) -> bool:
    return t.is_cuda


def _need(t: torch.Tensor, name: str, dtype, ndim: int, shape=None, device=None):
    """Check a tensor argument: a contiguous CUDA tensor of `dtype` and `ndim`
    dims; with `shape` exactly that shape, with `device` on that device. The
    library trusts the sizes it is given, so every tensor whose extent follows
    from another argument is checked here before any launch."""
    if not isinstance(t, torch.Tensor) or not _on_device(t):
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _out(t, name: str, dtype, shape, device):
    """An output buffer: a new one, or the given one checked like an input."""
    if t is None:
        return torch.empty(tuple(shape), dtype=dtype, device=device)
    _need(t, name, dtype, len(shape), shape, device)
    return t


def _text_kv(Ky, Vy, B, H, d, device):
    """Check the text keys / values [B, M, H, d]; returns M."""
    _need(Ky, "Ky", torch.bfloat16, 4, device=device)
    M = Ky.shape[1]
    _need(Ky, "Ky", torch.bfloat16, 4, (B, M, H, d), device)
    if Vy is not None:
        _need(Vy, "Vy", torch.bfloat16, 4, (B, M, H, d), device)
    return M


def _split_bufs(S, C, B, N, k, device, with_c=True):
    """S [B, k] and C [B, N - k] int32 buffers of the top-k split."""
    if k > N:
        raise ValueError(f"k = {k} exceeds N = {N}")
    S = _out(S, "S", torch.int32, (B, k), device)
    if with_c:
        C = _out(C, "C", torch.int32, (B, N - k), device)
    return S, C


def abi_version() -> int:
    return lib().safe_abi_version()


def mask_classify(mask: torch.Tensor, sync: bool = True, result: Optional[torch.Tensor] = None):
    """Row-constant mask classification (Eq. (6)) of a 4-D [B, H, n_q, n_k]
    mask view (any strides; stride 0 = broadcast). Returns (verdict, nfail,
    first_fail) as Python ints when sync, else the device int64[3] tensor."""
    if not isinstance(mask, torch.Tensor) or mask.dim() != 4 or not _on_device(mask) or mask.dtype not in _MASK_DTYPES:
        raise ValueError("mask must be a 4-D CUDA tensor of dtype bool/uint8/float32/float16/bfloat16")
    sizes = (ctypes.c_int64 * 4)(*mask.shape)
    strides = (ctypes.c_int64 * 4)(*mask.stride())
    result = _out(result, "result", torch.int64, (3,), mask.device)
    if sync:
        h = (ctypes.c_int64 * 3)()
        _check("safe_mask_classify_sync",
               lib().safe_mask_classify_sync(_p(mask), _MASK_DTYPES[mask.dtype], sizes, strides, _p(result), h,
                                             _stream()))
        return int(h[0]), int(h[1]), int(h[2])
    _check("safe_mask_classify",
           lib().safe_mask_classify(_p(mask), _MASK_DTYPES[mask.dtype], sizes, strides, _p(result), _stream()))
    return result


def _scale(d: int, scale: Optional[float]) -> float:
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def attn_workspace_bytes(B: int, n_q: int, N: int, H: int, d: int) -> int:
    return int(lib().safe_attn_workspace_bytes(B, n_q, N, H, d))


def _attn_ws(ws, B, n_q, N, H, d, device):
    """Workspace for the wave-balancing key split: the given tensor, a fresh
    one (ws=None), or no split at all (ws=False)."""
    if ws is False:
        return None, 0
    if ws is None:
        nbytes = attn_workspace_bytes(B, n_q, N, H, d)
        if nbytes == 0:
            return None, 0
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def attn_self(Q, K, V, scale=None, return_lse=False, out=None, lse=None, ws=None):
    """Mask-free image self-attention (Eq. (3) with the mask elided)."""
    _need(Q, "Q", torch.bfloat16, 4)
    B, N, H, d = Q.shape
    dev = Q.device
    _need(K, "K", torch.bfloat16, 4, Q.shape, dev)
    _need(V, "V", torch.bfloat16, 4, Q.shape, dev)
    out = _out(out, "out", torch.bfloat16, (B, N, H, d), dev)
    if return_lse:
        lse = _out(lse, "lse", torch.float32, (B, H, N), dev)
    w, wb = _attn_ws(ws, B, N, N, H, d, Q.device)
    _check("safe_attn_self", lib().safe_attn_self(_p(Q), _p(K), _p(V), _p(out), _p(lse if return_lse else None),
                                                  B, N, H, d, _scale(d, scale), _p(w), wb, _stream()))
    return (out, lse) if return_lse else out


def attn_cross(Q, Ky, Vy, valid_len, q_idx=None, scale=None, out=None):
    """Image->text cross-attention with the padding kept as valid lengths
    (Eq. (4)); with q_idx = S the row-selective form (Eq. (17))."""
    _need(Q, "Q", torch.bfloat16, 4)
    B, N, H, d = Q.shape
    dev = Q.device
    M = _text_kv(Ky, Vy, B, H, d, dev)
    _need(valid_len, "valid_len", torch.int32, 1, (B,), dev)
    nq = N
    if q_idx is not None:
        _need(q_idx, "q_idx", torch.int32, 2, device=dev)
        nq = q_idx.shape[1]
        _need(q_idx, "q_idx", torch.int32, 2, (B, nq), dev)
    out = _out(out, "out", torch.bfloat16, (B, nq, H, d), dev)
    _check("safe_attn_cross", lib().safe_attn_cross(_p(Q), _p(q_idx), nq, _p(Ky), _p(Vy), _p(valid_len), _p(out),
                                                    B, N, M, H, d, _scale(d, scale), _stream()))
    return out


def pcsp_workspace_bytes(B: int, N: int, H: int) -> int:
    return int(lib().safe_pcsp_workspace_bytes(B, N, H))


def pcsp_topk(Q, Ky, valid_len, w=None, scores=None, accumulate=False, k=0, scale=None, S=None, C=None, ws=None):
    """PCSP scores (Eq. (10)) for one step / layer and, if k > 0, the top-k
    partition (Eq. (12)). Returns (scores, S, C)."""
    if Q is not None:
        _need(Q, "Q", torch.bfloat16, 4)
        B, N, H, d = Q.shape
        dev = Q.device
        M = _text_kv(Ky, None, B, H, d, dev)
        _need(valid_len, "valid_len", torch.int32, 1, (B,), dev)
        if w is not None:
            _need(w, "w", torch.float32, 2, (B, M), dev)
    else:
        _need(scores, "scores", torch.float32, 2)
        B, N = scores.shape
        H, d, M = 1, 64, 1
        dev = scores.device
    if scores is None:
        scores = torch.zeros((B, N), dtype=torch.float32, device=dev)
    else:
        _need(scores, "scores", torch.float32, 2, (B, N), dev)
    if k > 0:
        S, C = _split_bufs(S, C, B, N, k, dev)
    nbytes = pcsp_workspace_bytes(B, N, H) if Q is not None else 0
    if Q is not None and ws is None:
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    _check("safe_pcsp_topk", lib().safe_pcsp_topk(
        _p(Q), _p(Ky), _p(valid_len), _p(w), B, N, M, H, d, _scale(d, scale), _p(scores), 1 if accumulate else 0, k,
        _p(S), _p(C), _p(ws), ws.numel() if ws is not None else 0, _stream()))
    return scores, S, C


def attn_cross_pcsp(Q, Ky, Vy, valid_len, w=None, out=None, scores=None, accumulate=False, k=0, scale=None, S=None,
                    C=None, ws=None):
    """Cross-attention (Eq. (4)) and the PCSP scores of Eq. (10) from the same
    probabilities, in one pass over Q; with k > 0 also the top-k split
    (Eq. (12)). Returns (O, scores, S, C)."""
    _need(Q, "Q", torch.bfloat16, 4)
    B, N, H, d = Q.shape
    dev = Q.device
    M = _text_kv(Ky, Vy, B, H, d, dev)
    _need(valid_len, "valid_len", torch.int32, 1, (B,), dev)
    if w is not None:
        _need(w, "w", torch.float32, 2, (B, M), dev)
    out = _out(out, "out", torch.bfloat16, (B, N, H, d), dev)
    if scores is None:
        scores = torch.zeros((B, N), dtype=torch.float32, device=dev)
    else:
        _need(scores, "scores", torch.float32, 2, (B, N), dev)
    if k > 0:
        S, C = _split_bufs(S, C, B, N, k, dev)
    if ws is None:
        ws = torch.empty(max(pcsp_workspace_bytes(B, N, H), 256), dtype=torch.uint8, device=Q.device)
    _check("safe_attn_cross_pcsp", lib().safe_attn_cross_pcsp(
        _p(Q), _p(Ky), _p(Vy), _p(valid_len), _p(w), _p(out), B, N, M, H, d, _scale(d, scale), _p(scores),
        1 if accumulate else 0, k, _p(S), _p(C), _p(ws), ws.numel(), _stream()))
    return out, scores, S, C


def topk_partition(scores, k, S=None, C=None, with_c=True):
    """Exact tie-stable top-k split of Eq. (12) on given scores."""
    _need(scores, "scores", torch.float32, 2)
    B, N = scores.shape
    S, C = _split_bufs(S, C, B, N, k, scores.device, with_c)
    _check("safe_topk_partition", lib().safe_topk_partition(_p(scores), B, N, k, _p(S), _p(C if with_c else None),
                                                            _stream()))
    return S, C


def srsu_workspace_bytes(B: int, k: int, N: int, H: int, d: int) -> int:
    return int(lib().safe_srsu_workspace_bytes(B, k, N, H, d))


def _srsu_ws(ws, B, k, N, H, d, device):
    """Workspace of an SRSU call: the given tensor, a fresh one of
    srsu_workspace_bytes (ws=None: room for the compact query rows and the
    key split), or none (ws=False)."""
    if ws is False:
        return None, 0
    if ws is None:
        nbytes = srsu_workspace_bytes(B, k, N, H, d)
        if nbytes == 0:
            return None, 0
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def _srsu_args(Q, S, Kc, Vc, q_compact):
    """Check the SRSU inputs: cache K/V [B, N, H, d], S [B, k], Q [B, k, H, d]
    (compact) or [B, N, H, d]; returns B, N, H, d, k, device."""
    _need(Kc, "Kc", torch.bfloat16, 4)
    B, N, H, d = Kc.shape
    dev = Kc.device
    _need(Vc, "Vc", torch.bfloat16, 4, Kc.shape, dev)
    _need(S, "S", torch.int32, 2, device=dev)
    k = S.shape[1]
    _need(S, "S", torch.int32, 2, (B, k), dev)
    _need(Q, "Q", torch.bfloat16, 4, (B, k if q_compact else N, H, d), dev)
    return B, N, H, d, k, dev


def srsu_attn(Q, S, Kc, Vc, q_compact=False, scale=None, return_lse=False, out=None, lse=None, ws=None):
    """SRSU selective self-attention (Eq. (16)): rows S of Q against all N
    keys of the assembled global K/V."""
    B, N, H, d, k, dev = _srsu_args(Q, S, Kc, Vc, q_compact)
    out = _out(out, "out", torch.bfloat16, (B, k, H, d), dev)
    if return_lse:
        lse = _out(lse, "lse", torch.float32, (B, H, k), dev)
    w, wb = _srsu_ws(ws, B, k, N, H, d, dev)
    _check("safe_srsu_attn", lib().safe_srsu_attn(_p(Q), 1 if q_compact else 0, _p(S), k, _p(Kc), _p(Vc), _p(out),
                                                  _p(lse if return_lse else None), B, N, H, d, _scale(d, scale),
                                                  _p(w), wb, _stream()))
    return (out, lse) if return_lse else out


def srsu_attn_assembled(Q, S, Kcur, Vcur, Kc, Vc, q_compact=False, cur_compact=False, scale=None, return_lse=False,
                        out=None, lse=None, ws=None):
    """SRSU (Eq. (16)) with K/V of S u C assembled in the kernel (Eq. (14)):
    rows of S from the current Kcur/Vcur ([B, k, H, d] when cur_compact, else
    [B, N, H, d]), the other rows from the cache Kc/Vc, which is not written.
    S must be strictly ascending."""
    B, N, H, d, k, dev = _srsu_args(Q, S, Kc, Vc, q_compact)
    cur_shape = (B, k if cur_compact else N, H, d)
    _need(Kcur, "Kcur", torch.bfloat16, 4, cur_shape, dev)
    _need(Vcur, "Vcur", torch.bfloat16, 4, cur_shape, dev)
    out = _out(out, "out", torch.bfloat16, (B, k, H, d), dev)
    if return_lse:
        lse = _out(lse, "lse", torch.float32, (B, H, k), dev)
    w, wb = _srsu_ws(ws, B, k, N, H, d, dev)
    _check("safe_srsu_attn_assembled", lib().safe_srsu_attn_assembled(
        _p(Q), 1 if q_compact else 0, _p(S), k, _p(Kcur), _p(Vcur), 1 if cur_compact else 0, _p(Kc), _p(Vc), _p(out),
        _p(lse if return_lse else None), B, N, H, d, _scale(d, scale), _p(w), wb, _stream()))
    return (out, lse) if return_lse else out


def ctx_cache_scatter(Ksrc, Vsrc, S, Kc, Vc, src_compact=True):
    """In-place cache update (Eq. (14)/(16)); S=None is the anchor refresh
    (Eq. (19))."""
    _need(Kc, "Kc", torch.bfloat16, 4)
    B, N, H, d = Kc.shape
    dev = Kc.device
    _need(Vc, "Vc", torch.bfloat16, 4, Kc.shape, dev)
    k = 0
    if S is not None:
        _need(S, "S", torch.int32, 2, device=dev)
        k = S.shape[1]
        _need(S, "S", torch.int32, 2, (B, k), dev)
    src_shape = (B, k, H, d) if (src_compact and S is not None) else (B, N, H, d)
    _need(Ksrc, "Ksrc", torch.bfloat16, 4, src_shape, dev)
    _need(Vsrc, "Vsrc", torch.bfloat16, 4, src_shape, dev)
    _check("safe_ctx_cache_scatter", lib().safe_ctx_cache_scatter(
        _p(Ksrc), _p(Vsrc), 1 if (src_compact and S is not None) else 0, _p(S), k, _p(Kc), _p(Vc), B, N, H, d,
        _stream()))
    return Kc, Vc


def device_status() -> int:
    """Read and clear the library's device status word (synchronises)."""
    v = ctypes.c_int(0)
    _check("safe_get_device_status", lib().safe_get_device_status(ctypes.byref(v), _stream()))
    return v.value


def selftest_wait_timeout(limit_ns: int = 1_000_000) -> None:
    """Launch the bounded-wait self-test (see safe_selftest_wait_timeout)."""
    _check("safe_selftest_wait_timeout", lib().safe_selftest_wait_timeout(int(limit_ns), _stream()))


def shared_partition(scores, k, sample: int = 0, B: int = None):
    """One partition for a whole CFG pair (or batch): the top-k split of
    Eq. (12) of one sample's scores (by default the conditional one,
    sample 0), repeated for every sample, so that all of them update the
    same sensitive rows. Returns S [B, k], C [B, N - k] (int32, device)."""
    _need(scores, "scores", torch.float32, 2)
    B = scores.shape[0] if B is None else B
    S1, C1 = topk_partition(scores[sample:sample + 1], k)
    return S1.expand(B, -1).contiguous(), C1.expand(B, -1).contiguous()


def sensitivity_workspace_bytes(B: int, N: int) -> int:
    return int(lib().safe_sensitivity_workspace_bytes(B, N))


def sensitivity_field(scores, grid_h: int, grid_w: int, sigma: float, truncate: float = 4.0, out=None, ws=None):
    """s = Norm(G_sigma * s~) of Eq. (11) on the grid_h x grid_w latent grid
    (row-major tokens), per sample: [B, N] fp32 -> [B, N] fp32 in [0, 1]."""
    _need(scores, "scores", torch.float32, 2)
    B, N = scores.shape
    if N != grid_h * grid_w:
        raise ValueError(f"scores hold {N} tokens per sample, the grid {grid_h} x {grid_w} has {grid_h * grid_w}")
    out = _out(out, "out", torch.float32, (B, N), scores.device)
    nbytes = sensitivity_workspace_bytes(B, N)
    if ws is None:
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=scores.device)
    _check("safe_sensitivity_field", lib().safe_sensitivity_field(
        _p(scores), _p(out), B, grid_h, grid_w, float(sigma), float(truncate), _p(ws), ws.numel(), _stream()))
    return out


def partition_indicator(S, N: int, out=None):
    """Binary field of the SW-CFG binary variant: 1 on S, 0 on C ([B, N] fp32)."""
    _need(S, "S", torch.int32, 2)
    B, k = S.shape
    out = _out(out, "out", torch.float32, (B, N), S.device)
    _check("safe_partition_indicator", lib().safe_partition_indicator(_p(S), k, _p(out), B, N, _stream()))
    return out


_CFG_DTYPES = {torch.float32: 2, torch.bfloat16: 4}


def sw_cfg(f_c, f_u, s, gamma_ctx: float, gamma_sens: float, out=None):
    """Sensitivity-weighted CFG, Eq. (20), (21): f_u + gamma_i (f_c - f_u),
    gamma_i = gamma_ctx + (gamma_sens - gamma_ctx) s_i. f_c, f_u [B, N, C]
    (fp32 or bf16), s [B, N] fp32; out may be f_c or f_u (in place)."""
    if f_c.dtype not in _CFG_DTYPES or f_u.dtype != f_c.dtype:
        raise ValueError("f_c and f_u must both be float32 or both bfloat16")
    _need(f_c, "f_c", f_c.dtype, 3)
    B, N, C = f_c.shape
    dev = f_c.device
    _need(f_u, "f_u", f_c.dtype, 3, f_c.shape, dev)
    _need(s, "s", torch.float32, 2, (B, N), dev)
    out = _out(out, "out", f_c.dtype, (B, N, C), dev)
    _check("safe_sw_cfg", lib().safe_sw_cfg(_p(f_c), _p(f_u), _p(s), _p(out), _CFG_DTYPES[f_c.dtype], B, N, C,
                                            float(gamma_ctx), float(gamma_sens), _stream()))
    return out



_ACTS = {"none": 0, "gelu_tanh": 1}


def gather_linear_workspace_bytes(B: int, k: int, d_in: int) -> int:
    return int(lib().safe_gather_linear_workspace_bytes(B, k, d_in))


def gather_linear(X, Wt, S=None, bias=None, act="none", out=None, ws=None):
    """A row-wise layer of the row-selective block (Eq. (13), (15)):
    Y[b, r, :] = act(X[b, S[b, r], :] W^T + bias); S = None: every row (the
    dense block). X [B, N, d_in] bf16, Wt [d_out, d_in] bf16, S [B, k] int32,
    bias [d_out] fp32, act "none" or "gelu_tanh". Returns [B, k or N, d_out].
    ws: the workspace for the compact copy of the rows of S (a fresh one when
    None; False: the GEMM gathers the rows itself)."""
    _need(X, "X", torch.bfloat16, 3)
    B, N, d_in = X.shape
    dev = X.device
    _need(Wt, "Wt", torch.bfloat16, 2, device=dev)
    d_out = Wt.shape[0]
    _need(Wt, "Wt", torch.bfloat16, 2, (d_out, d_in), dev)
    k, R = 0, N
    if S is not None:
        _need(S, "S", torch.int32, 2, device=dev)
        k = R = S.shape[1]
        _need(S, "S", torch.int32, 2, (B, k), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, 1, (d_out,), dev)
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    out = _out(out, "out", torch.bfloat16, (B, R, d_out), dev)
    w, wb = None, 0
    if S is not None and ws is not False:
        if ws is None:
            ws = torch.empty(gather_linear_workspace_bytes(B, k, d_in), dtype=torch.uint8, device=dev)
        _need(ws, "ws", torch.uint8, 1, device=dev)
        w, wb = ws, ws.numel()
    _check("safe_gather_linear", lib().safe_gather_linear(_p(X), _p(S), k, _p(Wt), _p(bias), _ACTS[act], _p(out), B,
                                                          N, d_in, d_out, _p(w), wb, _stream()))
    return out


# ---------------------------------------------------------------- norm, positions, microscaled layers
_FLOATS = {torch.float32: 2, torch.float16: 3, torch.bfloat16: 4}
_FORMATS = {"mxfp8": 0, "mxfp4": 1, "nvfp4": 2}
_i64x3 = ctypes.c_int64 * 3


def _on(dev: torch.device, fn, *args):
    """fn(*args) with `dev` as the current device."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(dev.index):
        return fn(*args)


def _run(name: str, dev: torch.device, *args):
    """Call entry point `name` on `dev` (which need not be the current device)
    with that device's current stream as the last argument."""
    fn, idx = getattr(lib(), name), dev.index
    if idx is None:
        st = fn(*args, _stream())
    elif idx == torch.cuda.current_device():
        st = fn(*args, _raw_stream(idx))
    else:
        st = _on(dev, fn, *args, _raw_stream(idx))
    if st != SAFE_OK:
        raise SafeError(name, st)


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same number without a Stream object around it (3 us of a small call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check_tensor(t, name: str, dtype, shape, dev):
    """_need for a known shape on a known device, quick when all is well."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _need(t, name, dtype, len(shape), shape, dev)


def _out_like(t, name: str, like, dtype, shape):
    """An output buffer on the device of `like`: new, or the given one checked."""
    if t is not None:
        _check_tensor(t, name, dtype, shape, like.device)
        return t
    if dtype is like.dtype and like.shape == shape and like.is_contiguous():
        return torch.empty_like(like)
    return _new(shape, dtype, like.device)


def _new(shape, dtype, dev) -> torch.Tensor:
    """A contiguous tensor of undefined contents (torch.empty takes 1 us more of
    the host's time than its strided form)."""
    if len(shape) == 3:
        return torch.empty_strided(shape, (shape[1] * shape[2], shape[2], 1), dtype=dtype, device=dev)
    if len(shape) == 1:
        return torch.empty_strided(shape, (1,), dtype=dtype, device=dev)
    return torch.empty(shape, dtype=dtype, device=dev)


def _check_ints(*sizes):
    """Sizes that go to the library as ints (ctypes would drop their upper bits)."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"sizes above 2^31 - 1 are not supported, got {sizes}")


def _float_code(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in _FLOATS:
        raise ValueError(f"{name} must be a float32, float16 or bfloat16 tensor")
    return _FLOATS[t.dtype]


def _rows_of(S, B: int, N: int, dev) -> int:
    """Rows of each sample: N, or k of S [B, k] (checked)."""
    if S is None:
        return N
    if not (isinstance(S, torch.Tensor) and S.dtype is torch.int32 and S.device == dev and S.is_contiguous()):
        _need(S, "S", torch.int32, 2, device=dev)
    if S.dim() != 2 or S.shape[0] != B or not 1 <= S.shape[1] <= N:
        raise ValueError(f"S must have shape ({B}, 1..{N}), got {tuple(S.shape)}")
    return S.shape[1]


class MxTensor:
    """A microscaled matrix: `data` [..., D] e4m3 (mxfp8) or [..., D / 2] uint8
    (mxfp4, nvfp4: two e2m1 to a byte, the even element in the low half),
    `scales` the scale bytes in tiles of 128 rows x 4 (flat uint8, the rows of
    data's leading dims one after another; layout: safe_mx_quantize in
    include/safe_attn.h), `fmt` "mxfp8", "mxfp4" or "nvfp4", and `scale` the
    factor of the whole matrix (nvfp4; 1 otherwise). Checked once, here: its
    parts cannot be exchanged afterwards; a call that takes it as `out` fills
    it anew, with its factor."""

    __slots__ = ("_data", "_scales", "_fmt", "_scale", "_rows", "_D")

    def __init__(self, data: torch.Tensor, scales: torch.Tensor, fmt: str, scale: float = 1.0):
        if fmt not in _FORMATS:
            raise ValueError(f"fmt must be one of {sorted(_FORMATS)}, got {fmt!r}")
        want = torch.float8_e4m3fn if fmt == "mxfp8" else torch.uint8
        if not isinstance(data, torch.Tensor) or data.dim() < 2:
            raise ValueError("data must be a tensor of at least 2 dims")
        if not (_on_device(data) and data.dtype is want and data.is_contiguous()):
            _need(data, "data", want, data.dim())
        w, n = data.shape[-1], data.numel()
        D = w if fmt == "mxfp8" else 2 * w
        if D < 32 or D % 32 or n == 0:
            raise ValueError(f"rows of a microscaled matrix have a multiple of 32 elements, got {tuple(data.shape)}")
        rows = n // w
        _check_tensor(scales, "scales", torch.uint8, (mx_scale_bytes(rows, D, fmt),), data.device)
        self._data, self._scales, self._fmt, self._scale = data, scales, fmt, _factor(fmt, scale)
        self._rows, self._D = rows, D

    data = property(lambda self: self._data)
    scales = property(lambda self: self._scales)
    fmt = property(lambda self: self._fmt)
    scale = property(lambda self: self._scale)

    @property
    def shape(self) -> Tuple[int, ...]:
        """The shape of the values that the matrix stands for."""
        return (*self._data.shape[:-1], self._D)

    @property
    def device(self) -> torch.device:
        return self._data.device


def mx_scale_bytes(rows: int, D: int, fmt: str) -> int:
    """Bytes of the scales of a microscaled [rows, D] matrix (0: no such form)."""
    if fmt not in _FORMATS:
        raise ValueError(f"fmt must be one of {sorted(_FORMATS)}, got {fmt!r}")
    if rows < 1 or D < 1 or D % 32:
        return 0
    return -(-rows // 128) * -(-D // (64 if fmt == "nvfp4" else 128)) * 512


def _mx_out(out, lead, D: int, fmt: str, scale: float, like) -> MxTensor:
    """A microscaled matrix [*lead, D] on the device of `like`: one of undefined
    contents, or the given one checked (its factor is set behind the call that
    fills it: a refused one leaves it as it was)."""
    if out is None:
        m = MxTensor.__new__(MxTensor)  # made to fit: nothing to check
        rows = math.prod(lead)
        if fmt == "mxfp8":
            m._data = _new((*lead, D), torch.float8_e4m3fn, like.device)
        else:
            m._data = _new((*lead, D // 2), torch.uint8, like.device)
        m._scales = _new((mx_scale_bytes(rows, D, fmt),), torch.uint8, like.device)
        m._fmt, m._scale, m._rows, m._D = fmt, scale, rows, D
        return m
    if not isinstance(out, MxTensor) or out.fmt != fmt or out.shape != (*lead, D) or out.device != like.device:
        raise ValueError(f"out must be an MxTensor {fmt} of shape {(*lead, D)} on {like.device}")
    return out


def rms_norm(x, w=None, residual=None, S=None, eps=1e-6, x_compact=False, quant=None, update=False, out=None, h=None):
    """Root-mean-square norm of rows with the residual's addition: h = x +
    residual, y = h / sqrt(mean(h^2) + eps) * w; returns y, or (y, h) with a
    residual. x [B, N, D] (fp32, fp16 or bf16), residual [B, N, D] of the same
    type, w [D] fp32 or None.
    S [B, k] int32: only the rows S of the stream (Eq. (13)); x then is
    [B, k, D] with x_compact (a row-selective branch's output), else [B, N, D],
    and y, h are [B, k, D].
    quant "mxfp8": y is an MxTensor (8 bits with a scale for each 32
    elements), as mx_linear takes it; D is then a multiple of 32.
    update: h is the residual itself, its rows (of S, strictly ascending, or
    all) updated in place. out, h: buffers for the results."""
    dt = _float_code(x, "x")
    if not _on_device(x) or x.dim() != 3:
        _need(x, "x", x.dtype, 3)
    dev, dtype = x.device, x.dtype
    if residual is not None and (not isinstance(residual, torch.Tensor) or residual.dim() != 3):
        _need(residual, "residual", dtype, 3, device=dev)
    B, N, D = x.shape if residual is None else residual.shape
    _check_ints(B, N, D)
    k, full = 0, False
    if S is None:
        R = N
    else:
        if residual is None and x_compact:
            raise ValueError("x_compact needs a residual: the rows of S are already gathered in x")
        R = k = _rows_of(S, B, N, dev)
        full = not x_compact
    _check_tensor(x, "x", dtype, (B, N if full else R, D), dev)
    if w is not None:
        _check_tensor(w, "w", torch.float32, (D,), dev)
    shape = (B, R, D)
    if residual is None:
        if update or h is not None:
            raise ValueError("update and h need a residual")
    else:
        _check_tensor(residual, "residual", dtype, (B, N, D), dev)
        if not update:
            h = _out_like(h, "h", x, dtype, shape)
        elif h is not None:
            raise ValueError("update writes the sums to the residual: h must be None")
        else:
            h = residual
    if quant is None:
        y = _out_like(out, "out", x, dtype, shape)
        yp, qp, sp = y.data_ptr(), None, None
    else:
        if quant != "mxfp8":
            raise ValueError(f"quant must be None or 'mxfp8', got {quant!r}")
        if D % 32:
            raise ValueError(f"an 8-bit output needs D a multiple of 32, got {D}")
        y = _mx_out(out, (B, R), D, quant, 1.0, x)
        yp, qp, sp = None, y._data.data_ptr(), y._scales.data_ptr()
    _run("safe_rms_norm", dev, x.data_ptr(), 1 if full else 0, _ptr(residual), _ptr(S), k, _ptr(w), eps, _ptr(h),
         1 if update and k else 0, yp, qp, sp, dt, B, N, D)
    return y if residual is None else (y, h)


class RopeTable:
    """The frequencies of rotary positions (made by rope_table): `freq` [r / 2]
    int64 in 2^-64 turns, `sections` the pairs of each position axis, `m` the
    factor on the rotated elements. Checked once, here: its parts cannot be
    exchanged afterwards."""

    __slots__ = ("_freq", "_sections", "_m", "_r", "_counts", "_freq_ptr")

    def __init__(self, freq: torch.Tensor, sections: Sequence[int], m: float = 1.0):
        _need(freq, "freq", torch.int64, 1)
        self._sections = tuple(int(n) for n in sections)
        self._r = 2 * freq.shape[0]
        n = self._sections
        if not 1 <= len(n) <= 3 or min(n) < 0 or 2 * sum(n) != self._r or self._r < 2:
            raise ValueError(f"sections must be 1 to 3 counts that share out {self._r // 2} pairs, got {self._sections}")
        if not math.isfinite(m):
            raise ValueError(f"m must be finite, got {m}")
        self._freq, self._m = freq, float(m)
        self._counts = (ctypes.c_int32 * len(self._sections))(*self._sections)
        self._freq_ptr = ctypes.cast(freq.data_ptr(), _i64p)

    freq = property(lambda self: self._freq)
    sections = property(lambda self: self._sections)
    m = property(lambda self: self._m)
    r = property(lambda self: self._r)


def rope_frequencies(r: int, base: float = 10000.0, sections: Optional[Sequence[int]] = None, kind: str = "none",
                     factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     attn_factor: Optional[float] = None):
    """(frequencies in radians for each position of the r / 2 pairs, factor m on
    the rotated elements). An axis with n pairs has r' = 2 n and the
    frequencies base^(-2 i / r'), stretched for contexts `factor` times longer:
      linear  divided by factor
      ntk     base * factor^(r' / (r' - 2)): the last is divided by factor, the first kept
      yarn    pairs that turn more than beta_fast times over original_len are
              kept, those below beta_slow turns divided by factor, a ramp over
              the pairs in between; m = 0.1 ln(factor) + 1 (or attn_factor)."""
    if r < 2 or r % 2:
        raise ValueError(f"r must be even and at least 2, got {r}")
    sections = [r // 2] if sections is None else [int(n) for n in sections]
    if not 1 <= len(sections) <= 3 or min(sections) < 0 or 2 * sum(sections) != r:
        raise ValueError(f"sections must be 1 to 3 counts that share out {r // 2} pairs, got {sections}")
    if kind not in ("none", "linear", "ntk", "yarn"):
        raise ValueError(f"kind must be none, linear, ntk or yarn, got {kind!r}")
    if not base > 1 or not math.isfinite(base) or not factor >= 1 or not math.isfinite(factor):
        raise ValueError(f"base must be above 1 and factor at least 1, got {base} and {factor}")
    if kind == "yarn" and (original_len < 1 or not 0 < beta_slow < beta_fast):
        raise ValueError("yarn needs original_len and 0 < beta_slow < beta_fast")
    f = []
    for n in sections:
        b = base * factor ** (n / (n - 1)) if kind == "ntk" and n > 1 else base
        w = [b ** (-i / n) for i in range(n)]
        if kind == "linear":
            w = [v / factor for v in w]
        elif kind == "yarn" and n:
            # the pair that turns `t` times over the original length
            lo, hi = (n * math.log(original_len / (2 * math.pi * t)) / math.log(base) for t in (beta_fast, beta_slow))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), 2 * n - 1)
            ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(n)]
            w = [v / factor * t + v * (1 - t) for v, t in zip(w, ramp)]
        f += w
    m = 1.0
    if kind == "yarn":
        m = 0.1 * math.log(factor) + 1.0
    return f, m if attn_factor is None else float(attn_factor)


def rope_table(r: int, base: float = 10000.0, sections: Optional[Sequence[int]] = None, device="cuda", **scaling):
    """The table of rotary positions that rope takes; arguments:
    rope_frequencies. sections share the r / 2 pairs out over up to three
    position axes (e.g. rows and columns of the latent grid)."""
    f, m = rope_frequencies(r, base, sections, **scaling)
    turns = np.array(f) / (2 * math.pi)
    fixed = np.rint(np.ldexp(turns - np.floor(turns), 64)).astype(np.uint64).view(np.int64)  # at most 2^64 - 2^11
    return RopeTable(torch.from_numpy(fixed).to(device), [r // 2] if sections is None else sections, m)


def _heads(t, name: str, dtype, B, R, d, dev):
    """Check a [B, R, H, d] tensor or view (contiguous in d); returns H, strides."""
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}")
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 4 or shape[0] != B or shape[1] != R or shape[2] < 1 or shape[3] != d:
        raise ValueError(f"{name} must be {dtype} of shape ({B}, {R}, heads, {d}), got {t.dtype} {tuple(shape)}")
    if t.is_contiguous():
        return shape[2], None
    b, n, h, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} must be contiguous in its last dim")
    return shape[2], _i64x3(b, n, h)


def rope(q, k, table: RopeTable, pos=None, S=None, interleaved=False, inplace=False, out=None):
    """Rotary positions: every pair of the first table.r elements of a head
    turns by position * frequency. q [B, R, H, d], k [B, R, Hk, d] or None
    (fp32, fp16 or bf16; views of a fused projection too, contiguous in the
    last dim). pos: int32 [N, axes] shared by the samples (one axis: [N] will
    do) or [B, N, axes]; None: the token index. S [B, R] int32: row r is token
    S[b, r], else token r. interleaved: pairs (2i, 2i + 1) instead of
    (i, i + r / 2). Returns (q, k) turned: new contiguous tensors, those of
    out=(q, k), or with inplace q and k themselves."""
    dt = _float_code(q, "q")
    if not isinstance(table, RopeTable):
        raise ValueError("table must be a RopeTable")
    if not _on_device(q) or q.dim() != 4:
        raise ValueError(f"q must be a CUDA tensor of 4 dims, got {tuple(q.shape)} on {q.device}")
    B, R, H, d = q.shape
    dev, dtype, axes, r = q.device, q.dtype, len(table._sections), table._r
    qs = None if q.is_contiguous() else _heads(q, "q", dtype, B, R, d, dev)[1]
    Hk, ks, kp = 0, None, None
    if k is not None:
        Hk, ks = _heads(k, "k", dtype, B, R, d, dev)
        kp = k.data_ptr()
    if table._freq.device != dev:
        raise ValueError(f"table must be on {dev}")
    if r > d:
        raise ValueError(f"the table turns {r} elements, heads have {d}")
    N, batched, pp, sp = R, 0, None, None
    if pos is None:
        if axes != 1:
            raise ValueError(f"a table of {axes} axes needs pos")
        if S is not None:
            raise ValueError("S needs pos (the positions of all tokens)")
    else:
        if not isinstance(pos, torch.Tensor) or not 1 <= pos.dim() <= 3 or (pos.dim() == 1 and axes != 1):
            raise ValueError(f"pos must be a tensor [tokens, {axes}] or [{B}, tokens, {axes}]")
        shape = pos.shape
        if len(shape) == 1:
            N = shape[0]
        else:
            batched, N = len(shape) - 2, shape[-2]
            shape = (B, N, axes) if batched else (N, axes)
        _check_tensor(pos, "pos", torch.int32, shape, dev)
        pp = pos.data_ptr()
    if S is not None:
        _check_tensor(S, "S", torch.int32, (B, R), dev)
        if R > N:
            raise ValueError(f"S names {R} rows of {N} tokens")
        sp = S.data_ptr()
    elif N != R:
        raise ValueError(f"pos has {N} tokens, q {R} rows")
    _check_ints(B, N, H, Hk, d)
    if inplace:
        if out is not None:
            raise ValueError("inplace writes to q and k: out must be None")
        oq, ok, oqs, oks = q, k, qs, ks
    else:
        oq, ok = (None, None) if out is None else out
        oqs = oks = None
        if oq is None:
            oq = torch.empty_like(q) if qs is None else torch.empty((B, R, H, d), dtype=dtype, device=dev)
        else:
            n, oqs = _heads(oq, "out[0]", dtype, B, R, d, dev)
            if n != H:
                raise ValueError(f"out[0] must have {H} heads, got {n}")
        if k is None:
            if ok is not None:
                raise ValueError("out[1] needs k")
        elif ok is None:
            ok = torch.empty_like(k) if ks is None else torch.empty((B, R, Hk, d), dtype=dtype, device=dev)
        else:
            n, oks = _heads(ok, "out[1]", dtype, B, R, d, dev)
            if n != Hk:
                raise ValueError(f"out[1] must have {Hk} heads, got {n}")
    _run("safe_rope", dev, q.data_ptr(), qs, oq.data_ptr(), oqs, H, kp, ks, None if k is None else ok.data_ptr(), oks, Hk,
         dt, table._freq_ptr, table._counts, axes, pp, batched, sp, B, N, R, d, r, 1 if interleaved else 0, table._m)
    return oq, ok


def _factor(fmt: str, scale: float) -> float:
    """The factor of a microscaled matrix as the fp32 number that is kept."""
    if scale == 1.0:
        return 1.0
    s = ctypes.c_float(scale).value
    if fmt == "nvfp4" and not 2.0 ** -100 <= s <= 2.0 ** 100:
        raise ValueError(f"scale must lie in [2^-100, 2^100], got {scale}")
    if fmt != "nvfp4" and s != 1.0:
        raise ValueError(f"{fmt} has no factor of the whole matrix: scale must be 1, got {scale}")
    return s


def mx_quantize(x, fmt: str, S=None, scale: float = 1.0, out=None) -> MxTensor:
    """The rows of x [B, N, D] (or [N, D]: a weight; fp32, fp16 or bf16), or its
    rows S [B, k], in microscaled 8 or 4 bits: fmt "mxfp8", "mxfp4" or "nvfp4".
    scale: the factor of an nvfp4 matrix (largest magnitude / 2688 lets every
    block scale be represented). Returns an MxTensor [B, k or N, D]."""
    dt = _float_code(x, "x")
    code = _FORMATS.get(fmt)
    if code is None:
        raise ValueError(f"fmt must be one of {sorted(_FORMATS)}, got {fmt!r}")
    nd = x.dim()
    if nd not in (2, 3):
        raise ValueError(f"x must have 2 or 3 dims, got {tuple(x.shape)}")
    if not (_on_device(x) and x.is_contiguous()):
        _need(x, "x", x.dtype, nd)
    B, N, D = x.shape if nd == 3 else (1, *x.shape)
    if D < 32 or D % 32:
        raise ValueError(f"rows must have a multiple of 32 elements, got {D}")
    _check_ints(B, N, D)
    dev, g, k = x.device, _factor(fmt, scale), 0
    R = N
    if S is not None:
        if nd == 2:
            raise ValueError("S needs x of 3 dims")
        R = k = _rows_of(S, B, N, dev)
    m = _mx_out(out, (B, R) if nd == 3 else (N,), D, fmt, g, x)
    _run("safe_mx_quantize", dev, x.data_ptr(), dt, _ptr(S), k, code, g, m._data.data_ptr(), m._scales.data_ptr(), B, N,
         D)
    m._scale = g
    return m


def mx_dequantize(m: MxTensor, dtype=torch.bfloat16, out=None):
    """The values that a microscaled matrix stands for, rounded to dtype."""
    if not isinstance(m, MxTensor):
        raise ValueError("m must be an MxTensor")
    if dtype not in _FLOATS:
        raise ValueError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    data, D = m._data, m._D
    _check_ints(D)
    out = _out_like(out, "out", m._scales, dtype, (*data.shape[:-1], D))
    _run("safe_mx_dequantize", data.device, data.data_ptr(), m._scales.data_ptr(), _FORMATS[m._fmt], m._scale,
         out.data_ptr(), _FLOATS[dtype], m._rows, D)
    return out


def mx_linear_workspace_bytes(rows: int, d_in: int, d_out: int, fmt: str) -> int:
    if fmt not in _FORMATS:
        raise ValueError(f"fmt must be one of {sorted(_FORMATS)}, got {fmt!r}")
    _check_ints(d_in, d_out)
    return int(lib().safe_mx_linear_workspace_bytes(rows, d_in, d_out, _FORMATS[fmt]))


def mx_linear(X: MxTensor, W: MxTensor, bias=None, act="none", out=None, ws=None):
    """A row-wise layer with microscaled operands, Y = act(X W^T + bias): X
    [..., d_in] (mx_quantize, rms_norm with quant; the rows of S for the
    row-selective block), W [d_out, d_in], both of one format; bias [d_out]
    fp32, act "none" or "gelu_tanh". Returns bf16 [..., d_out].
    ws: the workspace for splitting the last wave's tiles along d_in (a fresh
    one when None; False: every tile whole; not shared by calls that may run at
    the same time)."""
    if not isinstance(X, MxTensor) or not isinstance(W, MxTensor):
        raise ValueError("X and W must be MxTensors")
    fmt, x, w = X._fmt, X._data, W._data
    if fmt != W._fmt:
        raise ValueError(f"X is {fmt}, W is {W._fmt}: both operands must have one format")
    rows, d_in, d_out, dev = X._rows, X._D, W._rows, x.device
    if w.dim() != 2 or W._D != d_in or w.device != dev:
        raise ValueError(f"W must be [d_out, {d_in}] on {dev}, got {W.shape} on {W.device}")
    _check_ints(d_in, d_out)
    if bias is not None:
        _check_tensor(bias, "bias", torch.float32, (d_out,), dev)
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    alpha = X._scale * W._scale
    if not 2.0 ** -126 <= abs(alpha) < 2.0 ** 128:
        raise ValueError(f"the product of the operands' factors is out of range: {alpha}")
    out = _out_like(out, "out", X._scales, torch.bfloat16, (*x.shape[:-1], d_out))
    code, wp, wb = _FORMATS[fmt], None, 0
    if ws is None:
        if x.shape[-1] > 1536:  # up to 12 stages of 128 bytes a split saves less than it costs
            wb = _on(dev, lib().safe_mx_linear_workspace_bytes, rows, d_in, d_out, code)
            if wb:
                ws = _new((wb,), torch.uint8, dev)
                wp = ws.data_ptr()
    elif ws is not False:
        _need(ws, "ws", torch.uint8, 1, device=dev)
        wp, wb = ws.data_ptr(), ws.numel()
    _run("safe_mx_linear", dev, x.data_ptr(), X._scales.data_ptr(), w.data_ptr(), W._scales.data_ptr(), code, alpha,
         _ptr(bias), _ACTS[act], out.data_ptr(), rows, d_in, d_out, wp, wb)
    return out
