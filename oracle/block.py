"""CPU oracle of the operators around the convolutions, in plain fp64 numpy
from their definitions: group normalization with an activation and its
gradient, dropout from a counter-based generator, and the replay cache's
lines. Tensors are [H][W][N][C].

TEST INFRASTRUCTURE: shares no code with the GPU library.
"""
from __future__ import annotations

import math

import numpy as np

import oracle

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3
_MASK = 0xFFFFFFFF


def philox_words(rows: int, octets: int, seed: int) -> np.ndarray:
    """Philox4x32-10 at counters (row, octet, 1, 0): uint32 [rows][octets][4]."""
    c = [np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, octets)).copy(),
         np.broadcast_to(np.arange(octets, dtype=np.uint64)[None, :], (rows, octets)).copy(),
         np.ones((rows, octets), np.uint64), np.zeros((rows, octets), np.uint64)]
    k0, k1 = seed & _MASK, (seed >> 32) & _MASK
    low, s32 = np.uint64(_MASK), np.uint64(32)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> s32) ^ c[1] ^ np.uint64(k0), q & low, (p >> s32) ^ c[3] ^ np.uint64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) & _MASK, (k1 + 0xBB67AE85) & _MASK
    return np.stack(c, axis=-1).astype(np.uint32)


def drop_threshold(p: float) -> int:
    return int(math.floor(float(np.float32(p)) * 65536 + 0.5))


def drop_factor(shape, p: float, seed: int) -> np.ndarray:
    """0 or 65536 / (65536 - q), rounded to fp32, for every element."""
    c = shape[-1]
    rows = int(np.prod(shape[:-1]))
    q = drop_threshold(p)
    if q == 0:
        return np.ones(shape)
    w = philox_words(rows, (c + 7) // 8, seed & ((1 << 64) - 1))
    half = np.stack([w & 0xFFFF, w >> 16], axis=-1).reshape(rows, -1)[:, :c]
    scale = float(np.float32(65536.0 / (65536 - q))) if q < 65536 else 0.0
    return np.where(half >= q, scale, 0.0).reshape(shape)


_erf = np.frompyfunc(math.erf, 1, 1)


def _cdf(u):
    return 0.5 * (1 + _erf(u * math.sqrt(0.5)).astype(np.float64))


def _sigmoid(u):
    return 1 / (1 + np.exp(-u))


def act(kind: int, u: np.ndarray) -> np.ndarray:
    if kind == ACT_RELU:
        return np.where(u < 0, 0.0, u)
    if kind == ACT_SILU:
        return u * _sigmoid(u)
    if kind == ACT_GELU:
        return u * _cdf(u)
    return u


def act_slope(kind: int, u: np.ndarray) -> np.ndarray:
    if kind == ACT_RELU:
        return (u > 0).astype(np.float64)
    if kind == ACT_SILU:
        s = _sigmoid(u)
        return s + u * s * (1 - s)
    if kind == ACT_GELU:
        return _cdf(u) + u * np.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    return np.ones_like(u)


def _groups(v, g):  # [H][W][N][C] -> [H*W][N][G][D]
    h, w, n, c = v.shape
    return v.reshape(h * w, n, g, c // g)


def stats(x, groups: int, eps: float):
    """mean, rstd [N][groups]."""
    xg = _groups(np.asarray(x, np.float64), groups)
    mean = xg.mean(axis=(0, 3))
    var = ((xg - mean[None, :, :, None]) ** 2).mean(axis=(0, 3))
    return mean, 1 / np.sqrt(var + eps)


def _spread(v, d):  # [N][G] -> [N][C]
    return np.repeat(v, d, axis=1)


def group_norm(x, gamma, beta, groups, kind, eps, factor=1.0):
    """(y, mean, rstd, u)."""
    x = np.asarray(x, np.float64)
    mean, rstd = stats(x, groups, eps)
    d = x.shape[3] // groups
    u = (x - _spread(mean, d)) * _spread(rstd, d) * gamma + beta
    return act(kind, u) * factor, mean, rstd, u


def group_norm_backward(dy, x, gamma, beta, mean, rstd, groups, kind, factor=1.0):
    """(dx, dgamma, dbeta, parts) from the forward's mean and rstd; parts are
    the quantities that a bound on the error of dx is made of."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    d = x.shape[3] // groups
    m, r = _spread(np.asarray(mean, np.float64), d), _spread(np.asarray(rstd, np.float64), d)
    xh = (x - m) * r
    u = xh * gamma + beta
    g = dy * factor * act_slope(kind, u)
    gg = g * gamma
    fold = lambda v: _spread(_groups(v, groups).mean(axis=(0, 3)), d)  # noqa: E731
    dx = r * (gg - fold(gg) - xh * fold(gg * xh))
    return dx, (g * xh).sum(axis=(0, 1, 2)), g.sum(axis=(0, 1, 2)), {"u": u, "g": g, "xh": xh, "r": r, "fold": fold}


def cache_lines(x, fmt: int):
    """Codes (packed) [N][H*W*row_bytes] and scales [N][H*W*ncb] of every
    sample of x [H][W][N][C], each quantized by itself in lines."""
    codes, scales = [], []
    for n in range(x.shape[2]):
        c, s, _ = oracle.quantize(oracle.ROLE_ACT, fmt, 1, np.ascontiguousarray(x[:, :, n:n + 1]))
        codes.append(oracle.pack(fmt, c).reshape(-1))
        scales.append(s.reshape(-1))
    return np.stack(codes), np.stack(scales)


def cache_values(codes, scales, fmt: int, h: int, w: int, c: int):
    """Values [H][W][N][C] of packed lines [N][...]."""
    out = []
    for q, s in zip(codes, scales):
        logical = oracle.unpack(fmt, q.reshape(h, w, 1, -1), c)
        out.append(oracle.dequantize(oracle.ROLE_ACT, fmt, 1, logical, s.reshape(h, w, 1, -1)))
    return np.concatenate(out, axis=2)
