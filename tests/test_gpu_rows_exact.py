"""GPU tests of the experts and the adapters with fp32 results where every sum is exact (tests/rows_exact.py): equal to the
bits, on every kernel."""
import numpy as np
import pytest
import torch

from tests import rows_exact as rx
from tests.test_gpu_moe import DEV, E4M3, F32, BF16, I8, awq, banner, f64, handle, rng_of  # noqa: F401 (awq is a fixture)

pytestmark = pytest.mark.gpu


def operand(awq, x, s, kind):
    t = torch.from_numpy(x).to(kind).to(DEV)
    assert np.array_equal(f64(t.float()), x)
    return t if s is None else awq.Act8(t, torch.from_numpy(s).float().to(DEV))


# fewer pairs than experts, more, tiles, one expert with all tokens of several tiles (a block takes more than one in turn);
# groups of one wave each, of eight waves twice, of sixteen waves once and twice, pairs of channel tiles
@pytest.mark.parametrize("M,E,k,crowd", [(1, 4, 2, False), (7, 4, 2, False), (25, 4, 2, False), (150, 4, 1, True),
                                         (130, 8, 2, True)])
@pytest.mark.parametrize("H,I", [(256, 128), (1152, 256), (256, 1280), (2304, 256), (256, 2304)])
@pytest.mark.parametrize("kind", [F32, I8, E4M3])
def test_moe(awq, M, E, k, crowd, H, I, kind):
    banner(f"exact moe M={M} E={E} k={k} H={H} I={I} {kind} crowd={crowd}")
    rng = rng_of(M + H + I)
    x, s, gu, down, result = rx.experts(rng, M, E, H, I, kind != F32)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(M)]).astype(np.int32)
    if crowd:
        ids[:, 0] = 1
        ids[:, 1:] = np.where(rng.random((M, k - 1)) < 0.9, -1, ids[:, 1:])
    w = 2.0 ** rng.integers(-2, 3, (M, k))
    routing = awq.Routing(torch.from_numpy(ids).to(DEV), torch.from_numpy(w).float().to(DEV))
    y = awq.moe(operand(awq, x, s, kind), routing, handle(awq, gu), handle(awq, down), dtype=F32)
    each = np.stack([result(e) for e in range(E)])
    Y = np.zeros((M, H), dtype=np.float32)
    for j in range(k):  # of two experts the sum is rounded, once
        there = ids[:, j] >= 0
        Y[there] += (w[there, j, None] * each[ids[there, j], np.nonzero(there)[0]]).astype(np.float32)
    assert np.array_equal(y.cpu().numpy(), Y)


@pytest.mark.parametrize("M,n,K,N,R", [(1, 1, 64, 40, 8), (20, 3, 1032, 300, 24), (250, 30, 2048, 129, 64),
                                       (300, 4, 512, 512, 16), (300, 2, 4096, 260, 72)])
@pytest.mark.parametrize("codes", [False, True])
def test_lora(awq, M, n, K, N, R, codes):
    """The one number of a row reaches Y, whether X holds it or a code's row scale does."""
    banner(f"exact lora M={M} n={n} K={K} N={N} R={R} codes={codes}")
    x, A, B, ids, Y = rx.adapters(rng_of(M + K), M, n, K, N, R)
    if codes:
        s = np.abs(x).sum(1)
        X = operand(awq, np.sign(x), s, I8)
    else:
        X = operand(awq, x, None, F32)
    y = awq.lora(X, torch.from_numpy(A).to(BF16).to(DEV), torch.from_numpy(B).to(BF16).to(DEV), torch.from_numpy(ids).to(DEV),
                 torch.zeros(M, N, device=DEV))
    assert np.array_equal(f64(y), Y)
