"""CPU tests of the definitions in oracle/rows_oracle.py against the plain torch forms of perf/more_operators.py."""
import numpy as np
import pytest
import torch

from oracle import awq_oracle as o
from oracle import rows_oracle as ro
from perf import more_operators as plain


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(score, renorm):
    v = torch.randn(9, 30, generator=torch.Generator().manual_seed(1))
    v[3] = v[3].round()  # ties
    ids, w = ro.route(v.double().numpy(), 7, score, renorm)
    pids, pw = plain._route(v, 7, score, renorm)
    assert np.array_equal(ids, pids.numpy()) and np.allclose(w, pw.numpy(), rtol=1e-5)


def test_route_masked():
    v = np.full((2, 4), -np.inf)
    v[0, 2] = 1.0
    ids, w = ro.route(v, 3, "softmax", True)
    assert ids.tolist() == [[2, -1, -1], [-1, -1, -1]] and w.tolist() == [[1, 0, 0], [0, 0, 0]]


def artefacts(rng, E, N, K):
    q = rng.integers(0, 2 ** 32, (E, N, K // 8), dtype=np.uint32).view(np.int32)
    s = (rng.uniform(0.5, 1.5, (E, N, K // 128)) / 50).astype(np.float16)
    z = rng.integers(0, 16, (E, N, K // 128)).astype(np.float16)
    return [dict(qweight=q[e], scales=s[e], zeros=z[e]) for e in range(E)], tuple(torch.from_numpy(t) for t in (q, s, z))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_moe(act):
    rng = np.random.default_rng(2)
    M, E, k, H, I = 6, 5, 3, 256, 128
    gu, tgu = artefacts(rng, E, 2 * I, H)
    down, td = artefacts(rng, E, H, I)
    assert np.array_equal(ro.linear(np.eye(H), gu[0])[0].T.astype(np.float32),
                          (o.unpack_words(gu[0]["qweight"]).astype(np.float32) - np.repeat(gu[0]["zeros"], 128, 1).astype(np.float32))
                          * np.repeat(gu[0]["scales"], 128, 1).astype(np.float32))
    x = rng.standard_normal((M, H)).astype(np.float32)
    ids = rng.integers(-1, E + 1, (M, k)).astype(np.int32)
    ids[0] = 2  # an expert three times
    w = rng.uniform(0, 1, (M, k)).astype(np.float32)
    Y, B = ro.moe(x.astype(np.float64), ids, w, gu, down, act, 3, 3)
    y = plain._moe(torch.from_numpy(x), torch.from_numpy(ids), torch.from_numpy(w), tgu, td, act, "f32").numpy()
    assert np.allclose(Y, y, rtol=1e-4, atol=1e-4 * np.abs(Y).max()) and np.all(B >= 0) and np.all(np.abs(Y - y) <= B + 1e-30)


def test_lora():
    rng = np.random.default_rng(3)
    M, K, N, R, n = 7, 40, 24, 16, 3
    x = rng.standard_normal((M, K)).astype(np.float32)
    A = torch.from_numpy(rng.standard_normal((n, R, K))).bfloat16()
    B = torch.from_numpy(rng.standard_normal((n, N, R))).bfloat16()
    ids = np.array([0, 1, 2, -1, 3, 1, 0], dtype=np.int32)
    base, scale = rng.standard_normal((M, N)).astype(np.float32), rng.uniform(0, 2, n).astype(np.float32)
    ranks = np.array([16, 5, 0], dtype=np.int32)
    Y, D = ro.lora(x.astype(np.float64), A.double().numpy(), B.double().numpy(), ids, base.astype(np.float64), scale, ranks, 3, 3, 8)
    y = plain._lora(torch.from_numpy(x), A, B, torch.from_numpy(ids), torch.from_numpy(base), torch.from_numpy(scale),
                    torch.from_numpy(ranks)).numpy()
    assert np.allclose(Y, y, rtol=1e-4, atol=1e-4) and np.array_equal(y[3], base[3]) and np.array_equal(Y[2], base[2].astype(np.float64))
