"""CPU oracle of what include/mqconv_train.h computes, in plain fp64 numpy from
the definitions. Tensors are [H][W][N][C], weights [Cout][Kh][Kw][Cin].

TEST INFRASTRUCTURE: shares no code with the GPU library.
"""
from __future__ import annotations

import numpy as np


def layer_norm(s, gamma, beta, eps):
    """(y, mean, rstd) of rows s [..., C]."""
    s = np.asarray(s, np.float64)
    mean = s.mean(axis=-1)
    d = s - mean[..., None]
    rstd = 1 / np.sqrt((d * d).mean(axis=-1) + eps)
    return gamma * d * rstd[..., None] + beta, mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd, dskip=0.0):
    """(dx, dgamma, dbeta, parts) from the forward's mean and rstd; parts are what a bound on dx's error is made of."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    m, r = np.asarray(mean, np.float64)[..., None], np.asarray(rstd, np.float64)[..., None]
    xh = (x - m) * r
    g = gamma * dy
    k1, k2 = g.mean(axis=-1, keepdims=True), (g * xh).mean(axis=-1, keepdims=True)
    dx = r * (g - k1 - xh * k2) + dskip
    rows = tuple(range(dy.ndim - 1))
    return dx, (dy * xh).sum(axis=rows), dy.sum(axis=rows), {"xh": xh, "g": g, "k1": k1, "k2": k2, "r": r}


def round_bits(v, bits):
    """v to the nearest value of `bits` significant bits (None: as it is)."""
    if bits is None:
        return v
    mant, e = np.frexp(v)
    return np.ldexp(np.round(np.ldexp(mant, bits)), e - bits)


def newton(u, steps, a, b, c, eps, bits=None):
    """The Newton-Schulz steps on u [rows][cols]; bits: what every stored matrix is rounded to."""
    x = np.asarray(u, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = round_bits(x / (np.sqrt((x * x).sum()) + eps), bits)
    for _ in range(steps):
        s = round_bits(x @ x.T, bits)
        f = round_bits(a * np.eye(len(s)) + b * s + c * (s @ s), bits)
        x = round_bits(f @ x, bits)
    return x.T if tall else x


def muon(g, m, w, lr, momentum, decay, nesterov, scale, newton_args, bits=None):
    """(m, w) after one step."""
    m = momentum * np.asarray(m, np.float64) + g
    u = g + momentum * m if nesterov else m
    rows, cols = np.shape(g)
    s = (1.0, np.sqrt(max(1.0, rows / cols)), 0.2 * np.sqrt(max(rows, cols)))[scale]
    return m, (1 - lr * decay) * np.asarray(w, np.float64) - lr * s * newton(u, *newton_args, bits=bits)
