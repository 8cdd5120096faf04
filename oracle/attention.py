"""Attention over prompts and over a 4-bit key/value cache, and eviction from it,
in float64 (test infrastructure).

Each result comes with a bound of its error for sums in fp32 and a P rounded by
at most `p_eps` of its value, derived next to it."""
import numpy as np

from . import fp4


def quantized(x, fmt, gs=None):
    """The values that rows x [tokens, heads, dim] have in the cache."""
    t, h, d = x.shape
    codes, sb, _ = fp4.quantize(np.asarray(x, np.float64).reshape(t * h, d), fmt, 1.0 if gs is None and fmt == "nvfp4" else gs)
    return fp4.values(codes, sb, fmt, gs).reshape(t, h, d)


def attend(q, k, v, scale, p_eps, p_abs=0.0):
    """q [rows, heads, dim] are the last rows of k, v [keys, kv_heads, dim].  Returns out, lse, the
    probabilities' sums [keys, kv_heads], and bounds of the absolute errors of the three before out is rounded.

    A score is a sum of dim exact products times a factor: its error is at most e_s = (dim + 4) 2^-24 scale sum|q k|
    (any order of summation).  A probability is off by a factor of exp(+-2 e_s) for the score and the maximum, by p_eps, and by
    the 2^-22 of exp2 and of its argument's rounding (|argument| < 64 there or the probability is below 2^-64); sums of n
    terms add n 2^-24.  Where P is fp16 with the largest at 2^14, subnormal steps of 2^-24 round it by up to 2^-25,
    which is p_abs = 2^-39 of the largest probability."""
    R, H, D = q.shape
    n, hk = k.shape[0], k.shape[1]
    G = H // hk
    out, lse = np.zeros((R, H, D)), np.full((R, H), -np.inf)
    w, e_out, e_lse, e_w = np.zeros((n, hk)), np.zeros((R, H, D)), np.zeros((R, H)), np.zeros((n, hk))
    for r in range(R):
        top = max(0, min(n, n - R + r + 1))
        if top == 0:
            continue
        for h in range(H):
            kk, vv = k[:top, h // G], v[:top, h // G]
            with np.errstate(invalid="ignore"):
                s = kk @ q[r, h] * scale
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
            p = p / l
            e_s = (D + 4) * 2.0 ** -24 * scale * (np.abs(kk) @ np.abs(q[r, h])).max() + 2.0 ** -22 * (1 + np.abs(m))
            rel = 2 * e_s + 2.0 ** -22 * 64 + top * 2.0 ** -24
            out[r, h], lse[r, h] = p @ vv, m + np.log(l)
            e_out[r, h] = (2 * rel + p_eps) * (p @ np.abs(vv)) + p_abs * p.max() * np.abs(vv).sum(0) + 1e-30
            e_lse[r, h] = rel + 2.0 ** -22 * (1 + np.abs(lse[r, h]))
            w[:top, h // G] += p
            e_w[:top, h // G] += p * 2 * rel
    return out, lse, w, e_out, e_lse, e_w + w * 2.0 ** -22 * R * G


def evict(weights, positions, keep, recent, sinks):
    """weights, positions [n] of one head's places.  Returns the places whose tokens are at places 0 .. min(n, keep)
    - 1 afterwards."""
    n = len(weights)
    if n <= keep:
        return np.arange(n)
    last = int(positions.max()) - recent

    def key(i):
        if positions[i] < sinks or positions[i] > last:
            return (0, 0.0, i)
        if np.isnan(weights[i]):
            return (1, 0.0, i)
        return (2, -float(weights[i]), i)

    stays = sorted(sorted(range(n), key=key)[:keep])
    behind = [i for i in stays if i >= keep]
    here = set(stays)
    return np.array([i if i in here else behind.pop(0) for i in range(keep)])
