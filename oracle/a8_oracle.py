"""Plain fp64 definitions of the 8-bit activation path, for tests only: RMS norm with the residual's
addition, gated activation, 8-bit rows with a scale each, and the product with the packed weight."""
import math

import numpy as np

from oracle import awq_oracle as o

FLOOR = 2.0 ** -100
QMAX = {"int8": 127.0, "e4m3": 448.0}


def rmsnorm(x, r, gamma, eps):
    """(h, y) in fp64; r may be None."""
    h = x.astype(np.float64) + (0.0 if r is None else r.astype(np.float64))
    ms = np.mean(h * h, axis=1, keepdims=True)
    return h, h / np.sqrt(ms + eps) * gamma.astype(np.float64)[None, :]


_erfc = np.vectorize(math.erfc)


def act_mul(g, u, s, act):
    y = g.astype(np.float64)
    if act == "silu":
        with np.errstate(over="ignore"):
            y = y / (1.0 + np.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * _erfc(-y / math.sqrt(2.0))
    if u is not None:
        y = y * u.astype(np.float64)
    return y if s is None else y / s.astype(np.float64)[None, :]


def round_e4m3(v):
    """Nearest e4m3 value (ties to even), saturating at 448."""
    a = np.minimum(np.abs(v), 448.0)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -40))), -6.0)
    step = 2.0 ** (e - 3)
    return np.sign(v) * np.minimum(np.rint(a / step) * step, 448.0)


def round_code(v, kind):
    return np.clip(np.rint(v), -127, 127) if kind == "int8" else round_e4m3(v)


def row_scale(y, kind):
    return np.maximum(np.max(np.abs(y), axis=1), FLOOR) / QMAX[kind]


def w4a8(codes, scale, art):
    """Y and the magnitude sum_g D (|sum x q| + z |sum x|) that its roundings scale with, and the
    larger one with the absolute values inside the sums."""
    q = o.unpack_words(art["qweight"]).astype(np.float64)
    d, z = art["scales"].astype(np.float64), art["zeros"].astype(np.float64)
    N, G = d.shape
    M = codes.shape[0]
    x = codes.astype(np.float64)
    Y, mag, absmag = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    for g in range(G):
        xg, qg = x[:, 128 * g:128 * g + 128], q[:, 128 * g:128 * g + 128]
        a, b = xg @ qg.T, xg.sum(1)[:, None] * z[None, :, g]
        Y += d[None, :, g] * (a - b)
        mag += d[None, :, g] * (np.abs(a) + np.abs(b))
        absmag += d[None, :, g] * (np.abs(xg) @ qg.T + np.abs(xg).sum(1)[:, None] * z[None, :, g])
    s = scale.astype(np.float64)[:, None]
    return Y * s, mag * s, absmag * s
