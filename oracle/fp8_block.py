"""FP8 with one fp32 scale per block of 128, and the norm before an expert layer, in fp64 (test infrastructure).

Format: E4M3 codes; a block's scale is m / 448 with m = max(amax, 2^-100), its codes are those of v * (448 / m), both
quotients and the product rounded to fp32 (the definition's own roundings, so that codes can be compared bit by bit),
to the nearest E4M3 value, ties to even.  Blocks are 1 x 128 along the last axis or 128 x 128; the last one of an axis
may be shorter.  A block with an infinity or NaN has the scale NaN.
"""
from __future__ import annotations

import numpy as np

from . import mx

BLOCK = 128


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def spread(s, R: int, C: int, tile: bool):
    """The scale of every value of [R, C]."""
    s = np.repeat(s, BLOCK, axis=-1)[..., :C]
    return np.repeat(s, BLOCK, axis=-2)[..., :R, :] if tile else s


def quantize(x, tile: bool = False):
    """x [R, C] -> (codes uint8 [R, C], scales fp32 [R, ceil(C/128)] or [ceil(R/128), ceil(C/128)])."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    br = blocks(R) if tile else R
    p = np.zeros((br * (BLOCK if tile else 1), blocks(C) * BLOCK), np.float32)
    p[:R, :C] = np.abs(x)
    amax = p.reshape(br, -1, blocks(C), BLOCK).max((1, 3))
    m = np.maximum(amax, np.float32(2.0 ** -100)).astype(np.float32)
    bad = ~np.isfinite(amax)
    s = np.where(bad, np.float32(np.nan), m / np.float32(448)).astype(np.float32)
    inv = np.where(bad, np.float32(0), np.float32(448) / np.where(bad, np.float32(1), m)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        v = (x * spread(inv, R, C, tile)).astype(np.float32)
    return mx.e4m3_encode(np.nan_to_num(v).astype(np.float64)), s


def quantize_cols(x, tile: bool = False):
    """The row form of the transpose, the rows padded with zeros to a multiple of 32."""
    R, C = x.shape
    p = np.zeros(((R + 31) // 32 * 32, C), np.float32)
    p[:R] = x
    q, s = quantize(np.ascontiguousarray(p.T), tile)
    return q, s


def decode(codes, scales, tile: bool = False):
    R, C = codes.shape[-2:]
    return mx.e4m3_decode(codes) * spread(np.asarray(scales, np.float64), R, C, tile)


def rmsnorm(r, w, eps):
    """(y, rstd) of the rows of r, in fp64."""
    r = np.asarray(r, np.float64)
    rstd = 1 / np.sqrt((r * r).mean(-1) + eps)
    return r * rstd[..., None] * np.asarray(w, np.float64), rstd


def rmsnorm_bwd(dy, r, w, rstd):
    """(dx, dw) for a given rstd, in fp64."""
    dy, r, w, rstd = (np.asarray(t, np.float64) for t in (dy, r, w, rstd))
    xhat = r * rstd[:, None]
    g = dy * w
    return rstd[:, None] * (g - xhat * (g * xhat).mean(-1, keepdims=True)), (dy * xhat).sum(0)


def swiglu(gu, p):
    """p silu(G) U of [G U] rows."""
    F = gu.shape[1] // 2
    G, U = gu[:, :F], gu[:, F:]
    return p[:, None] * (G / (1 + np.exp(-G))) * U
