"""A whole mixture-of-experts layer in float64 (test infrastructure).

logits = x R^T; the k largest scores per row (ties to the lower id, NaN lowest);
"softmax": scores are the logits, weights the softmax over the chosen ones;
"sigmoid": chosen by sigmoid(logit) + bias, weights the chosen sigmoids over
their sum (equal shares when it is 0).  y = scale * sum_j w_j D_j(silu(G_j x) *
(U_j x)) + the shared expert's output.
"""
import numpy as np

from .blob import dequant_expert
from .expert import expert_apply
from .routing import _order_key, route


def route_layer(x, router, k, score="softmax", bias=None, scale=1.0):
    """x [M, H], router [E, H] -> (ids [M, k], weights [M, k], gap [M]): gap is the distance between the
    last chosen and the first unchosen score (inf without one), what a rounded score must not bridge."""
    with np.errstate(invalid="ignore", over="ignore"):
        z = x @ router.T
        p = z if score == "softmax" else 1.0 / (1.0 + np.exp(-z))
    by = p if bias is None else p + bias
    M, E = z.shape
    ids = np.empty((M, k), np.int64)
    gap = np.full(M, np.inf)
    for m in range(M):
        order = sorted(range(E), key=lambda e: _order_key(float(by[m, e]), e))
        ids[m] = order[:k]
        seq = by[m, order[:k + 1]]
        d = np.abs(np.diff(seq))
        if d.size and np.isfinite(d).any():
            gap[m] = d[np.isfinite(d)].min()
    if score == "softmax":
        w = np.empty((M, k))
        for m in range(M):
            _, wm = route(p[m:m + 1, ids[m]].astype(np.float32), k)
            v = p[m, ids[m]]
            if np.isfinite(v).all():
                v = np.exp(v - v.max())
                w[m] = v / v.sum()
            else:
                w[m] = wm[0]
    else:
        w = np.take_along_axis(p, ids, 1)
        w = np.where(np.isnan(w), 0.0, w)
        s = w.sum(1, keepdims=True)
        w = np.where(s > 0, w / np.where(s > 0, s, 1.0), 1.0 / k)
    return ids, w * scale, gap


def moe_layer(x, ids, w, fetch, gs, H, I, shared=None, shared_gs=None, shared_inter=0):
    """y [M, H] float64; also the sum of magnitudes that rounding is measured against."""
    M, k = ids.shape
    y, mag = np.zeros((M, H)), np.zeros((M, H))
    mats = {int(e): dequant_expert(fetch(int(e)), H, I, gs[e][0], gs[e][1]) for e in np.unique(ids)}
    if shared is not None:
        sh = dequant_expert(shared, H, shared_inter, shared_gs[0], shared_gs[1])

    def add(m, mat, coef):
        G, U, D = mat
        out, h = expert_apply(G, U, D, x[m])
        y[m] += coef * out
        # h moves by its own rounding and by that of the gate and up sums
        g, u = np.abs(G) @ np.abs(x[m]), np.abs(U) @ np.abs(x[m])
        gate, upv = G @ x[m], U @ x[m]
        dh = np.abs(h) + 1.1 * g * np.abs(upv) + np.abs(gate) * u
        mag[m] += abs(coef) * (np.abs(D) @ dh)

    for m in range(M):
        for j in range(k):
            add(m, mats[int(ids[m, j])], w[m, j])
        if shared is not None:
            add(m, sh, 1.0)
    return y, mag
