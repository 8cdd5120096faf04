"""4-bit matrices in float64 (test infrastructure): quantising, reading back, products.

NVFP4 holds E2M1 codes, one E4M3 scale per 16 elements and one fp32 scale of the
matrix; MXFP4 one E8M0 scale per 32 elements (OCP Microscaling Formats v1.0).
Every rounding is to nearest, ties to even, of the exact quotient.
"""
import numpy as np

from .formats import E2M1_TABLE, E4M3_TABLE

GROUP = {"nvfp4": 16, "mxfp4": 32}


def _nearest(v, grid):
    """Index of the grid value nearest to each v >= 0 (grid ascending from 0), ties to the even index."""
    mid = 0.5 * (grid[1:] + grid[:-1])
    lo = np.searchsorted(mid, v, side="left")      # a tie goes down
    hi = np.searchsorted(mid, v, side="right")     # a tie goes up
    return np.where(lo % 2 == 0, lo, hi)


def quantize(w, fmt, gs=None):
    """w [R, K] -> (codes [R, K] of 0..15, scale bytes [R, K/g], gs float32 or None)."""
    w = np.asarray(w, dtype=np.float64)
    R, K = w.shape
    g = GROUP[fmt]
    b = w.reshape(R, K // g, g)
    finite = np.isfinite(b)
    bad = ~finite.all(-1)
    a = np.where(finite, np.abs(b), 0.0)
    top = a.max(-1) if K else np.zeros((R, 0))
    if fmt == "nvfp4":
        if gs is None:
            gs = np.float32(a.max() / 2688.0) if a.size else np.float32(1)
            gs = gs if gs > 0 else np.float32(1)
        grid = E4M3_TABLE[:127]
        sb = _nearest(top / (6.0 * float(gs)), grid).astype(np.uint8)
        d = grid[sb] * float(gs)
        sb = np.where(bad, 0x7F, sb).astype(np.uint8)
    else:
        _, e = np.frexp(top)
        e = np.where(top > 0, np.clip(e - 3, -127, 127), -127)
        d = np.ldexp(1.0, e)
        sb = np.where(bad, 0xFF, e + 127).astype(np.uint8)
    # the borders times the scale are exact in float64; so is the comparison
    mid = 0.5 * (E2M1_TABLE[1:8] + E2M1_TABLE[:7])
    cut = d[..., None, None] * mid
    up = (a[..., None] > cut).sum(-1)
    tie = (a[..., None] == cut).any(-1) & (up % 2 == 1)
    c = np.where((d > 0)[..., None] & ~bad[..., None], up + tie, 0)
    sign = np.where((d > 0)[..., None] & ~bad[..., None], np.signbit(b), False)
    return (c + 8 * sign).astype(np.uint8).reshape(R, K), sb, gs


def scale_values(sb, fmt):
    sb = np.asarray(sb, dtype=np.uint8)
    if fmt == "nvfp4":
        return E4M3_TABLE[sb]
    return np.where(sb == 255, np.nan, np.ldexp(1.0, sb.astype(np.int64) - 127))


def values(codes, sb, fmt, gs=None):
    """The float64 matrix that codes [R, K] stand for."""
    v = E2M1_TABLE[codes] * np.repeat(scale_values(sb, fmt), GROUP[fmt], axis=1)
    return v if gs is None else v * float(np.float32(gs))


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    packed = np.asarray(packed, np.uint8)
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out
