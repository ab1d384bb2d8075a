"""Float64 definitions of the operators around the expert FFN: the residual addition
with root-mean-square norm and quantisation into an activation format, and the
router's logits.

TEST INFRASTRUCTURE ONLY, like the rest of this package; written from the
definitions in include/moe_ffn.h and shared with nothing on the GPU path.
"""
from __future__ import annotations

import numpy as np

from .codecs import round_e2m1_sat, round_e4m3_sat
from .moe import BF16, FP8_BLOCK128, NVFP4, NVFP4_W4A16, W4A8_MX, mx_exponent

FP32_MIN_NORMAL = 2.0 ** -126


def add_rmsnorm(x: np.ndarray, residual, weight: np.ndarray, eps: float):
    """(z, n): z = x + residual, n = z / sqrt(mean(z^2) + eps) * weight, per row."""
    z = np.asarray(x, np.float64)
    if residual is not None:
        z = z + np.asarray(residual, np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        r = 1.0 / np.sqrt((z * z).mean(axis=1, keepdims=True) + eps)
        return z, z * r * np.asarray(weight, np.float64)[None, :]


def act_scales(fmt: str, n: np.ndarray, x_gs: float = 1.0) -> np.ndarray:
    """The block scales of n in an activation format [T, H / block]: FP8 fp32(amax / 448)
    (here unrounded; 1 for a zero block, at least 2^-126), MX 2**e, NVFP4 the E4M3 value."""
    block = {FP8_BLOCK128: 128, W4A8_MX: 32, NVFP4: 16}[fmt]
    amax = np.abs(n.reshape(n.shape[0], -1, block)).max(axis=2)
    if fmt == FP8_BLOCK128:
        return np.where(amax == 0, 1.0, np.maximum(amax / 448.0, FP32_MIN_NORMAL))
    if fmt == W4A8_MX:
        return np.ldexp(1.0, mx_exponent(amax).astype(np.int32))
    return round_e4m3_sat(amax / (6.0 * x_gs))


def act_codes(fmt: str, n: np.ndarray, scales: np.ndarray, x_gs: float = 1.0) -> np.ndarray:
    """The code values of n for given block scales [T, H]."""
    block = n.shape[1] // scales.shape[1]
    s = np.repeat(np.asarray(scales, np.float64), block, axis=1) * (x_gs if fmt == NVFP4 else 1.0)
    q = np.where(s > 0, n / np.where(s > 0, s, 1.0), 0.0)
    return round_e2m1_sat(q) if fmt == NVFP4 else round_e4m3_sat(q)


def router_logits(x: np.ndarray, w: np.ndarray) -> np.ndarray:
    return np.asarray(x, np.float64) @ np.asarray(w, np.float64).T


__all__ = ["add_rmsnorm", "act_scales", "act_codes", "router_logits", "BF16", "NVFP4_W4A16"]
