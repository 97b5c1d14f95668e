"""The dense 4-bit linear, written out in float64.

w[n][k] = scale * (code - zero) for INT4 (one scale and zero per group of K,
zero 8 if none are given), E2M1 * E8M0 for MXFP4, E2M1 * E4M3 * tensor scale
for NVFP4; y = x W^T; SwiGLU: silu of the first half of the rows times the
second half.
"""
from __future__ import annotations

import numpy as np

from . import formats
from .moe import silu


def unpack_codes(codes) -> np.ndarray:
    """[N, K/2] bytes -> [N, K] codes, element 2i in the low nibble."""
    c = np.asarray(codes, dtype=np.uint8)
    return np.stack([c & 15, c >> 4], axis=2).reshape(c.shape[0], -1)


def dequant_int4(codes, scales, group: int, zeros=None) -> np.ndarray:
    q = unpack_codes(codes).astype(np.float64)
    K = q.shape[1]
    s = np.repeat(np.asarray(scales, dtype=np.float64), group, axis=1)[:, :K]
    z = 8.0 if zeros is None else np.repeat((np.asarray(zeros) & 15).astype(np.float64), group, axis=1)[:, :K]
    return (q - z) * s


def weights(fmt: str, codes, scales, group: int, zeros=None, tensor_scale: float = 1.0) -> np.ndarray:
    if fmt == "int4":
        return dequant_int4(codes, scales, group, zeros)
    if fmt == "mxfp4":
        return formats.dequant_mxfp4(codes, scales)
    return formats.dequant_nvfp4(codes, scales, tensor_scale)


def linear(x, w, swiglu: bool = False, y0=None) -> np.ndarray:
    y = np.asarray(x, dtype=np.float64) @ w.T
    if swiglu:
        half = w.shape[0] // 2
        y = silu(y[:, :half]) * y[:, half:]
    return y if y0 is None else y + np.asarray(y0, dtype=np.float64)
