"""Inputs of the experts and the adapters on which every fp32 sum that the kernels state is exact, so that their fp32 results
can be held to the bits: a kernel that hands act(gate) * up or A x on in two bf16 terms, reads an fp32 X in two, or lets a sum
grow past 32 products before the zero point leaves it, gives others.

Experts.  Per token: channel ``a`` is 1, channel ``c`` of the same group a number of 18 bits, channel ``b``, alone in a group
of its own, one of 24 bits and 2^12 times as large.  A gate's row has q - z = 8 at ``a`` and step 4, so the gate is 32, whose
SiLU is 32 in fp32 (exp(-32) is below 2^-24).  Up's rows have q - z = 8 at ``c`` in one row a group and q = z elsewhere, so h
has one value of 18 bits a group.  Down's rows have q - z = 0 or +-1, 2, 4, 8 there.  Multiplied as 8 + q / 2 (five bits) an
18-bit number's terms stay within 2^5 .. 2^-18 of it: 24 bits, exact.  ``b``'s terms of eight bits cancel one by one (13 bits
each) where the zero point leaves after 32 products; summed before, they need up to 29 bits.
A code's row scale has nine bits, so that its square, the factor of h, has 18."""
import numpy as np

from oracle import awq_oracle as o


def words(q):
    """Codes [N, K] to the artefact's int32 words, eight per word."""
    s = np.arange(0, 32, 4, dtype=np.uint32)
    w = np.bitwise_or.reduce(q.reshape(q.shape[0], -1, 8).astype(np.uint32) << s, axis=-1).astype(np.uint32).view(np.int32)
    assert np.array_equal(o.unpack_words(w), q)
    return w


def odd(rng, n, bits):
    """n numbers in [1, 2) that need exactly ``bits`` bits."""
    return 1.0 + (2 * rng.integers(0, 2 ** (bits - 2), n) + 1) / 2.0 ** (bits - 1)


def weight(rng, N, K, step):
    """Codes equal to their zero points (0 .. 7, one a row and group) and steps that are powers of two."""
    z = rng.integers(0, 8, (N, K // 128))
    return np.repeat(z, 128, axis=1), z, step * np.ones((N, K // 128))


def artefact(q, z, d):
    return {"qweight": words(q), "scales": d.astype(np.float16), "zeros": z.astype(np.float16)}


def experts(rng, M, E, H, I, codes):
    """(x [M, H] in fp64: for codes, the codes; row scales or None; gate_up, down; the function of one expert that gives Y)."""
    ga, gb = rng.permutation(H // 128)[:2]
    a, c = 128 * ga + rng.permutation(128)[:2]
    b = 128 * gb + rng.integers(0, 128)
    x, s = np.zeros((M, H)), None
    x[:, a] = 1.0
    if codes:
        x[:, c], x[:, b], s = 64.0, 32.0, odd(rng, M, 9)
    else:
        x[:, c], x[:, b] = odd(rng, M, 18), 4096.0 * odd(rng, M, 24)
    gate_up, down, used = [], [], []
    for _ in range(E):
        q, z, d = weight(rng, 2 * I, H, 4.0)
        z[:I], q[:I] = 7, 7
        q[:I, a] = 15
        d[I:] = 2.0 ** -rng.integers(0, 8, (I, 1))
        one = 128 * np.arange(I // 128) + rng.integers(0, 128, I // 128)  # h's values that are not 0
        q[I + one, c] += 8
        gate_up.append(artefact(q, z, d))
        q, z, d = weight(rng, H, I, 1.0)
        d[:] = 2.0 ** -rng.integers(0, 8, (H, 1))
        at = one[rng.integers(0, len(one), H)]  # of which a row of down reads one
        zero = q[np.arange(H), at]
        off = rng.choice([0, 1, 2, 4, 8, -1, -2, -4], H)
        q[np.arange(H), at] += np.where(zero + off >= 0, off, 8)
        down.append(artefact(q, z, d))
        used.append(one)
    xs = x if s is None else x * s[:, None]

    def dense(art):
        d, z = art["scales"].astype(np.float64), art["zeros"].astype(np.float64)
        return np.repeat(d, 128, 1) * (o.unpack_words(art["qweight"]) - np.repeat(z, 128, 1))

    def result(e, hand_on=lambda h: h):
        y = xs @ dense(gate_up[e]).T
        assert np.all(y[:, :I] == 32.0 * (1.0 if s is None else s[:, None]))  # its SiLU in fp32 is itself
        return hand_on(y[:, :I] * y[:, I:]) @ dense(down[e]).T

    return x, s, gate_up, down, result


def adapters(rng, M, n, K, N, R):
    """(x [M, K] with one number of 24 bits a row, A, B, ids, Y): every row of A reads one channel, every row of B one rank, so
    that a row of Y holds that number, or 0."""
    x, A, B = np.zeros((M, K)), np.zeros((n, R, K)), np.zeros((n, N, R))
    ch, rank = rng.integers(0, K, n), rng.integers(0, R, n)
    ids = (np.arange(M) % n).astype(np.int32)
    x[np.arange(M), ch[ids]] = odd(rng, M, 24) * rng.choice([-1.0, 1.0], M)
    A[np.arange(n), rank, ch] = 1.0
    B[np.arange(n), :, rank] = rng.choice([0.0, 1.0, -2.0], (n, N))
    Y = np.stack([B[i] @ (A[i] @ v) for i, v in zip(ids, x)])
    return x, A, B, ids, Y
