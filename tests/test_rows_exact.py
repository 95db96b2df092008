"""CPU tests of the inputs in tests/rows_exact.py: what the kernels state gives exact results on them, what they must not do
gives others."""
import numpy as np
import pytest

from tests import rows_exact as rx

F = np.float32


def cut(v):
    return (v.astype(F).view(np.uint32) & np.uint32(0xffff0000)).view(F)


def rounded(v):
    u = v.astype(F).view(np.uint32).astype(np.uint64)
    return ((u + 0x7fff + (u >> 16 & 1)) & 0xffff0000).astype(np.uint32).view(F)


def terms(v, n):
    """n bf16 terms of fp32 values: all but the last cut, the last rounded."""
    out, v = [], v.astype(F)
    for _ in range(n - 1):
        out.append(cut(v))
        v = v - out[-1]
    return out + [rounded(v)]


def group(x, q, z, inner):
    """sum x (q - z) / 2 of one group in fp32, 32 products a step (each step exact, then rounded): with the zero point after each
    32, or after the group."""
    r = F(0)
    for t in terms(x, 3)[::-1]:
        for s in range(4):
            k = slice(32 * s, 32 * s + 32)
            r = F(np.float64(r) + np.dot(t[k].astype(np.float64), 8.0 + q[k] / 2))
            if inner:
                r = F(np.float64(r) - t[k].astype(np.float64).sum() * (8.0 + z / 2))
    if not inner:
        r = F(np.float64(r) - (8.0 + z / 2) * np.float64(F(x.astype(np.float64).sum())))
    return r


@pytest.mark.parametrize("codes", [False, True])
def test_two_terms_of_the_intermediate_give_other_bits(codes):
    x, s, gu, down, result = rx.experts(np.random.default_rng(1), 9, 2, 256, 256, codes)
    for e in range(2):
        Y = result(e)
        assert np.array_equal(Y, Y.astype(F).astype(np.float64)) and np.any(Y != 0)
        for n in (2, 3):
            same = result(e, lambda h: np.sum([t.astype(np.float64) for t in terms(h, n)], axis=0)) == Y
            assert np.all(same) if n == 3 else np.mean(same[Y != 0]) < 0.5  # (two hold what has zeros behind eight bits)


def test_zero_points_after_the_group_give_other_bits():
    x, s, gu, down, result = rx.experts(np.random.default_rng(2), 20, 1, 256, 128, False)
    q, d, z = rx.o.unpack_words(gu[0]["qweight"]), gu[0]["scales"].astype(F), gu[0]["zeros"].astype(np.float64)
    differ = 0
    for row in (0, 1, 128, 129):
        W = d[row].astype(np.float64).repeat(128) * (q[row] - z[row].repeat(128))
        for v in x:
            for inner in (True, False):
                parts = (slice(0, 128), slice(128, 256))
                got = sum(2 * d[row, g] * group(v[k], q[row, k].astype(np.float64), z[row, g], inner)
                          for g, k in enumerate(parts))
                assert got == W @ v or not inner
                differ += got != W @ v
    assert differ > 20


def test_two_terms_of_the_adapters_give_other_bits():
    x, A, B, ids, Y = rx.adapters(np.random.default_rng(3), 7, 3, 64, 40, 16)
    assert np.array_equal(Y, Y.astype(F).astype(np.float64)) and np.any(Y != 0)
    v = x[x != 0]
    assert np.array_equal(np.sum([t.astype(np.float64) for t in terms(v, 3)], axis=0), v)
    assert np.mean(np.sum([t.astype(np.float64) for t in terms(v, 2)], axis=0) == v) < 0.5
