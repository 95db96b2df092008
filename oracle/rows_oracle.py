"""Plain fp64 definitions of the operators whose rows choose their weights, for tests only: the router, a mixture of
experts over packed 4-bit weights, low-rank adapters; each with a bound on what a kernel's roundings may add."""
import math

import numpy as np

from oracle import awq_oracle as o
from oracle.a8_oracle import act_mul

U = 2.0 ** -24


def route(logits, k, score, renormalize):
    """(ids, weights) of finite or -Inf logits: the first of the largest, k times."""
    v = logits.astype(np.float64)
    M, E = v.shape
    ids, w = np.full((M, k), -1, dtype=np.int32), np.zeros((M, k))
    for m in range(M):
        order = sorted((e for e in range(E) if v[m, e] > -math.inf), key=lambda e: (-v[m, e], e))[:k]
        if not order:
            continue
        c = v[m, order[0]]
        if score == "softmax":
            p = np.exp(v[m] - c)
            p = p[order] / (p[order].sum() if renormalize else p.sum())
        else:
            if renormalize and c < 0:  # the ratios of scores that underflow
                p = np.exp(v[m, order] - c) / (1.0 + np.exp(v[m, order]))
            else:
                p = np.array([1.0 / (1.0 + math.exp(-x)) if x > -700 else 0.0 for x in v[m, order]])
            p = p / p.sum() if renormalize else p
        ids[m, :len(order)], w[m, :len(order)] = order, p
    return ids, w


def linear(x, art):
    """x [rows, K] times one packed weight: Y, sum |x| D |q - z|, and sum |x| D (32 + q + z), which the kernel's two sums
    (codes and zero points, each moved up by sixteen, and halved) are bounded by."""
    q = o.unpack_words(art["qweight"]).astype(np.float64)
    d, z = art["scales"].astype(np.float64), art["zeros"].astype(np.float64)
    dk, zk = np.repeat(d, 128, axis=1), np.repeat(z, 128, axis=1)
    W = dk * (q - zk)
    a = np.abs(x)
    return x @ W.T, a @ np.abs(W).T, a @ (dk * (32.0 + q + zk)).T


def moe(x, ids, weights, gate_up, down, act, terms_x, terms_h):
    """(Y, bound): gate_up and down are lists of artefacts, one per expert.  terms_x: bf16 terms of an element of x;
    terms_h: of act(gate) * up.  The bound, without the last rounding:
    - a product's sums add 128 terms (per bf16 term) in fp32, G groups with two roundings each, and eight waves, then the
      channel's power of two (exact) and the row's scale: (136 terms + 2 G + 18) u of the sum of the magnitudes;
    - the activation's slope is at most 1.13; its own roundings are (20 + |g|) u (SiLU), (28 + 2 g^2) u (GELU);
    - h in two terms is off by 2^-17, in three by nothing."""
    M, H = x.shape
    E = len(gate_up)
    Y, B = np.zeros((M, H)), np.zeros((M, H))
    for m in range(M):
        total, mag = np.zeros(H), np.zeros(H)
        for j in range(ids.shape[1]):
            e = int(ids[m, j])
            if not 0 <= e < E:
                continue
            y, _, big = linear(x[m:m + 1], gate_up[e])
            I = y.shape[1] // 2
            dy = (136 * terms_x + 2 * (H // 128) + 18) * U * big
            g, u, dg, du = y[:, :I], y[:, I:], dy[:, :I], dy[:, I:]
            a = act_mul(g, None, None, act)
            h = a * u
            own = (20 + np.abs(g) if act == "silu" else 28 + 2 * g * g) * U
            dh = 1.13 * dg * (np.abs(u) + du) + np.abs(a) * du + own * np.abs(h) + 2e-38
            if terms_h == 2:
                dh = dh + 2.0 ** -17 * (np.abs(h) + dh)
            r, _, big = linear(h, down[e])
            s = linear(dh, down[e])[1] + (136 * terms_h + 2 * (I // 128) + 18) * U * linear(np.abs(h) + dh, down[e])[2]
            w = float(weights[m, j])
            total += w * r[0]
            mag += abs(w) * np.abs(r[0])
            B[m] += abs(w) * s[0]
        Y[m] = total
        B[m] += (ids.shape[1] + 3) * U * (mag + B[m])
    return Y, B


def lora(x, A, B, ids, base, scale, ranks, terms_x, terms_t, waves):
    """(Y, bound).  A row's sum over K is shared by ``waves`` waves: K terms_x / waves + waves fp32 additions, rounded up by
    two steps of 32 channels each; scale and the row's scale 3 u; the sum over the splits with it; t in two terms 2^-17, in
    three nothing; the sum over the ranks R terms_t additions; the base's addition u of the result (added by the caller's
    half step)."""
    M, N = base.shape
    Y, D = base.astype(np.float64).copy(), np.zeros((M, N))
    K, R = A.shape[2], A.shape[1]
    for m in range(M):
        a = int(ids[m])
        if not 0 <= a < A.shape[0]:
            continue
        r = R if ranks is None else min(max(int(ranks[a]), 0), R)
        s = 1.0 if scale is None else float(scale[a])
        Aa, Ba = A[a, :r], B[a, :, :r]
        t, mag = Aa @ x[m], np.abs(Aa) @ np.abs(x[m])
        dt = abs(s) * ((K * terms_x / waves + 64 * terms_x + waves + 3) * U * mag)
        t = s * t
        if terms_t == 2:
            dt = dt + 2.0 ** -17 * (np.abs(t) + dt)
        Y[m] += Ba @ t
        D[m] = np.abs(Ba) @ dt + (r + 32) * terms_t * U * (np.abs(Ba) @ (np.abs(t) + dt)) + U * np.abs(Y[m])
    return Y, D
