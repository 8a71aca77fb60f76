"""fp64 rotary positions with several axes, the heads' RMS norm before them and the gradient of
both, written from the definition.

Pair i of a head, channels (a, b), is turned by angle_i = pos[axis_i] * freq_i:
    a' = a cos - b sin,  b' = a sin + b cos.
The pair is (i, i + rot / 2) ("halves") or (2 i, 2 i + 1) ("adjacent"); channels from rot on are
kept.  With a weight w a head is first normalised: x * w / sqrt(mean(x^2) + eps).
"""
from __future__ import annotations

import numpy as np


def pair_channels(rot, pairing):
    i = np.arange(rot // 2)
    if pairing == "halves":
        return i, i + rot // 2
    return 2 * i, 2 * i + 1


def angles(pos, freq, axis):
    """pos [axes, n] -> angles [n, pairs] in [-pi, pi]: the product and its whole turns in
    extended precision (64 bits of mantissa or more), so that far positions keep theirs."""
    a = np.asarray(pos, np.int64)[np.asarray(axis)].T.astype(np.longdouble) * \
        np.asarray(freq, np.longdouble)
    two_pi = np.longdouble("6.28318530717958647692528676655900576839")
    return (a - two_pi * np.rint(a / two_pi)).astype(np.float64)


def normed(x, w, eps):
    if w is None:
        return x
    return x * np.asarray(w, np.float64) / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def turn(x, ang, pairing, back=False):
    """x [n, heads, d] turned by ang [n, pairs] (back: by -ang)."""
    a, b = pair_channels(2 * ang.shape[1], pairing)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1 if back else 1)
    y = np.array(x, np.float64)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def forward(x, pos, freq, axis, pairing, w=None, eps=1e-6):
    x = np.asarray(x, np.float64)
    return turn(normed(x, w, eps), angles(pos, freq, axis), pairing)


def backward(g, x, pos, freq, axis, pairing, w=None, eps=1e-6):
    """g: gradient of forward()'s result -> (dx, dw or None); x is read only with a weight."""
    g = turn(np.asarray(g, np.float64), angles(pos, freq, axis), pairing, back=True)
    if w is None:
        return g, None
    x = np.asarray(x, np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1))
    gw = g * np.asarray(w, np.float64)
    return r * gw - x * r ** 3 * (gw * x).mean(-1, keepdims=True), dw
