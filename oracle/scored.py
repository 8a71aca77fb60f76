"""fp64 attention over the packed mask with changed scores, and its gradients, written from the
definition:

    s = scale q.k,   s <- cap tanh(s / cap) (cap > 0),   s <- s - slope_h |pos_q - pos_k|,
    P = softmax of s over the legal keys,   O = P V,   LSE = ln sum exp s.

Gradients: dV = P^T dO, dP = dO V^T, dS = P (dP - rowsum(dO O)) ds/dx with
ds/dx = 1 - tanh^2 of the scaled product x, dQ = scale dS K, dK = scale dS^T Q.

Beside every result stands a bound on what rounding P and dS to bf16 (relative error h each) and O
to bf16 before delta = rowsum(dO O) can do to it:
    O:   h P |V|                       delta: rowsum |dO| (h P |V| + h |O|)
    dV:  h P^T |dO|                    dS:    h |dS| + P ds/dx |delta's|
    dQ:  scale (dS's) |K|              dK:    scale (dS's)^T |Q|
These hold for any roundings.  "noise" holds the variances of the gradients' errors for
independent roundings of the same sizes (each error's variance is at most its bound squared): the
terms' squares are summed, but delta's error, one for a row of dS, acts on the row as a whole.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import _f64


def distance(pos):
    """|pos_q - pos_k| of all pairs of tokens."""
    p = np.asarray(pos, np.int64)
    return np.abs(p[:, None] - p[None, :]).astype(np.float64)


def attention(q, k, v, mask, cap=0.0, slopes=None, pos=None, scale=None, do=None, h=0.0):
    """q [N, Hq, d], k / v [N, Hkv, d], mask [N, N] -> dict with O, LSE and, with do, dq, dk, dv;
    under "bound" the same names with the bounds above."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    n, hq, d = q.shape
    group = hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    far = distance(np.arange(n) if pos is None else pos) if slopes is not None else None
    out = {"O": np.zeros_like(q), "LSE": np.full((hq, n), -np.inf)}
    names = ["O"]
    if do is not None:
        do = _f64(do)
        out.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
        names += ["dq", "dk", "dv"]
    bound = {x: np.zeros_like(out[x]) for x in names}
    noise = {x: np.zeros_like(out[x]) for x in names[1:]}
    for i in range(hq):
        j = i // group
        Q, K, V = q[:, i], k[:, j], v[:, j]
        x = Q @ K.T * scale
        slope = np.ones_like(x)
        if cap:
            t = np.tanh(x / cap)
            x, slope = cap * t, 1 - t * t
        if far is not None:
            x = x - float(slopes[i]) * far
        x = np.where(mask, x, -np.inf)
        top = x.max(1)
        live = np.isfinite(top)
        e = np.where(mask, np.exp(x - np.where(live, top, 0)[:, None]), 0.0)
        total = e.sum(1)
        out["LSE"][i] = np.where(live, np.where(live, top, 0) + np.log(np.where(live, total, 1)),
                                 -np.inf)
        P = e / np.where(live, total, 1)[:, None]
        O = P @ V
        out["O"][:, i] = O
        ob = h * (P @ np.abs(V))
        bound["O"][:, i] = ob
        if do is None:
            continue
        g = do[:, i]
        out["dv"][:, j] += P.T @ g
        bound["dv"][:, j] += h * (P.T @ np.abs(g))
        dS = P * (g @ V.T - (g * O).sum(1)[:, None]) * slope
        off = (np.abs(g) * (ob + h * np.abs(O))).sum(1)
        sb = h * np.abs(dS) + P * slope * off[:, None]
        out["dq"][:, i] = scale * (dS @ K)
        out["dk"][:, j] += scale * (dS.T @ Q)
        bound["dq"][:, i] = scale * (sb @ np.abs(K))
        bound["dk"][:, j] += scale * (sb.T @ np.abs(Q))
        w = P * slope
        v2 = (g * g * h * h * ((P * P) @ (V * V) + O * O)).sum(1)[:, None]  # delta's variance
        noise["dv"][:, j] += h * h * ((P * P).T @ (g * g))
        noise["dq"][:, i] = scale ** 2 * (h * h * (dS * dS) @ (K * K) + v2 * (w @ K) ** 2)
        noise["dk"][:, j] += scale ** 2 * ((h * h * dS * dS + v2 * w * w).T @ (Q * Q))
    out["bound"], out["noise"] = bound, noise
    return out
