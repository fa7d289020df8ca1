"""The operators between a layer's residual stream and its attention, in plain fp64 numpy: RMSNorm with the
residual's addition and its gradient, quantisation to e4m3, the block-scaled product, rotary positions.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_TOP = 448.0
LEAST_SCALE = 2.0 ** -126
BLOCK = 128


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """The e4m3 value nearest to v (ties to even, magnitudes held to 448, NaN kept)."""
    v = np.asarray(v, dtype=np.float64)
    mag = np.minimum(np.abs(v), E4M3_TOP)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(mag > 0, mag, 1.0))), -6.0)
    step = np.exp2(np.where(np.isnan(e), 0.0, e) - 3.0)
    return np.copysign(np.minimum(np.round(mag / step) * step, E4M3_TOP), v)


def block_scales(v: np.ndarray, up: int, across: int = BLOCK) -> np.ndarray:
    rows, cols = v.shape
    out = np.empty((-(-rows // up), -(-cols // across)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = np.max(np.abs(v[i * up:(i + 1) * up, j * across:(j + 1) * across]))
    return np.maximum(out / E4M3_TOP, LEAST_SCALE)


def spread(scale: np.ndarray, shape, up: int, across: int = BLOCK) -> np.ndarray:
    """The scale that each value of a matrix of `shape` stands under."""
    return np.repeat(np.repeat(scale, up, axis=0), across, axis=1)[:shape[0], :shape[1]]


def rmsnorm(x, residual, weight, eps, w_offset=0.0):
    """(s, n, rstd) of the header's formulas, before any rounding."""
    s = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s, s * rstd[:, None] * (weight + w_offset), rstd


def rmsnorm_bwd(dy, dh, h, weight, rstd, w_offset=0.0):
    u = dy * (weight + w_offset)
    dx = rstd[:, None] * u - h * (rstd ** 3 * np.mean(u * h, axis=1))[:, None]
    return (dx if dh is None else dx + dh), np.sum(dy * h * rstd[:, None], axis=0)


def gemm_fp8(A, sA, W, sW):
    """A [M, K], W [N, K]: the values that the 8 bits stand for, unscaled."""
    return (A * spread(sA, A.shape, 1)) @ (W * spread(sW, W.shape, BLOCK)).T


def rope_frequencies(rot, base, scaling="none", stretch=1.0, trained=0.0, slow=0.0, fast=0.0):
    """Radians a position of each pair, and the factor on the rotated values."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "none":
        return np.array(f), 1.0
    if scaling == "linear":
        return np.array(f) / stretch, 1.0
    keep = []
    if scaling == "wavelength":
        for v in f:
            turns = trained * v / (2 * math.pi)
            keep.append(0.0 if turns <= slow else 1.0 if turns >= fast else (turns - slow) / (fast - slow))
        factor = 1.0
    else:
        def index_at(turns):   # where base^(-2i/rot) * trained = 2 pi turns
            return rot / 2 * math.log(trained / (2 * math.pi * turns), base)
        lo, hi = max(math.floor(index_at(fast)), 0), min(math.ceil(index_at(slow)), rot - 1)
        keep = [min(max(1 - (i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(rot // 2)]
        factor = 0.1 * math.log(stretch) + 1.0
    return np.array([k * v + (1 - k) * v / stretch for k, v in zip(keep, f)]), factor


def rope(x, positions, f, factor, head_dim, layout, inverse=False):
    """x [rows, heads * head_dim], every head turned."""
    rows, pairs = x.shape[0], len(f)
    v = x.reshape(rows, -1, head_dim)
    out = v.copy()
    angle = np.outer(positions, f)[:, None, :] * (-1 if inverse else 1)
    c, s = factor * np.cos(angle), factor * np.sin(angle)
    ia = np.arange(pairs) if layout == "half" else 2 * np.arange(pairs)
    ib = ia + pairs if layout == "half" else ia + 1
    a, b = v[:, :, ia], v[:, :, ib]
    out[:, :, ia], out[:, :, ib] = a * c - b * s, b * c + a * s
    return out.reshape(rows, -1)
