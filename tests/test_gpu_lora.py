"""GPU tests of the low-rank adapters against their fp64 definition (oracle/rows_oracle.py, which holds the bounds).
Beside the worst case the error's 2-norm is held to what roundings of either sign give: at most 14336 products a sum in
steps of 32, about sqrt(450) u = 1.3e-6 for A x, less for B t, so 4e-6 of the result's norm; a bf16 result adds at most
2^-8 / sqrt(3)."""
import numpy as np
import pytest
import torch

from oracle import rows_oracle as ro
from tests.test_gpu_moe import BF16, DEV, E4M3, F32, HALF, I8, activations, artefact, banner, f64, rng_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_mean_amd import awq as _awq
    _awq.lib()
    return _awq


def adapters(rng, n, K, N, R):
    A = torch.from_numpy(rng.standard_normal((n, R, K)) / np.sqrt(K)).to(BF16)
    B = torch.from_numpy(rng.standard_normal((n, N, R)) / np.sqrt(R)).to(BF16)
    return A, B


def check_lora(awq, x, x64, A, B, ids, base, scale=None, ranks=None, **kw):
    kind = x[0].dtype if isinstance(x, tuple) else x.dtype
    before = f64(base)
    dev = {n: None if t is None else torch.from_numpy(t).to(DEV) for n, t in (("scale", scale), ("ranks", ranks))}
    y = awq.lora(awq.Act8(*x) if isinstance(x, tuple) else x, A.to(DEV), B.to(DEV), torch.from_numpy(ids).to(DEV), base, **dev,
                 **kw)
    assert y.dtype == base.dtype and y.shape == base.shape
    Y, D = ro.lora(x64, f64(A), f64(B), ids, before, scale, ranks, 3 if kind == F32 else 1, 2 if base.dtype == BF16 else 3, 8)
    err, lim = np.abs(f64(y) - Y), D + HALF[base.dtype] * (np.abs(Y) + D) + 1e-36
    assert np.all(err <= lim), (np.argwhere(err > lim)[:4].tolist(), float(np.max(err / lim)))
    # a single bf16 rounding is off by up to 2^-8 (0.57649 is stored as 0.578125: 2.8e-3); 256 of them by 2^-8 / sqrt(3)
    half = 0.0 if base.dtype == F32 else 2.0 ** -8 if Y.size < 256 else 2.0 ** -8 / 3 ** 0.5
    assert np.linalg.norm(err) <= (4e-6 + half) * np.linalg.norm(Y)
    untouched = [m for m in range(len(ids)) if not 0 <= ids[m] < A.shape[0]]
    assert np.array_equal(f64(y)[untouched], before[untouched])
    return y


# M, K, N, R, adapters: one token, less than a tile, tiles with a rest, more than 256 tokens (a block takes a tile's
# adapters in turn); K off 32 and off 128, N odd, off 64 and off 256, R of one and of several tiles of 16 and 32
SHAPES = [(1, 8, 1, 8, 1), (1, 4096, 512, 16, 3), (2, 136, 65, 8, 2), (15, 512, 300, 24, 20), (16, 1000, 64, 40, 4),
          (17, 264, 257, 64, 40), (50, 2048, 777, 16, 7), (130, 96, 128, 256, 5), (257, 256, 320, 16, 3),
          (300, 520, 131, 48, 6), (400, 128, 96, 72, 9), (513, 64, 70, 32, 1), (260, 64, 2104, 16, 3), (257, 72, 1160, 40, 2)]


@pytest.mark.parametrize("M,K,N,R,n", SHAPES)
@pytest.mark.parametrize("kind,out", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16), (I8, BF16), (E4M3, F32)])
def test_lora(awq, M, K, N, R, n, kind, out):
    banner(f"lora M={M} K={K} N={N} R={R} n={n} {kind} {out}")
    rng = rng_of(M + K)
    A, B = adapters(rng, n, K, N, R)
    x, x64 = activations(rng, M, K, kind)
    ids = rng.integers(-1, n, M).astype(np.int32)
    ids[0] = n - 1
    base = torch.from_numpy(rng.standard_normal((M, N)) * 2).to(out).to(DEV)
    scale = rng.uniform(-2, 2, n).astype(np.float32)
    ranks = rng.integers(0, R + 1, n).astype(np.int32)
    ranks[n - 1] = R
    check_lora(awq, x, x64, A, B, ids, base, scale, ranks)
    check_lora(awq, x, x64, A, B, ids, base)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_lora_ranks_cut_what_is_stored_beyond(awq, M):
    """NaN beyond an adapter's rank is not read; ranks outside 0 .. R count as the nearer end; a rank of 0 adds nothing."""
    rng = rng_of(2)
    K, N, R, n = 256, 192, 40, 6
    A, B = adapters(rng, n, K, N, R)
    ranks = np.array([1, 5, 16, 33, 0, 39], dtype=np.int32)
    for a, r in enumerate(ranks):
        A[a, r:], B[a, :, r:] = float("nan"), float("nan")
    x, x64 = activations(rng, M, K, BF16)
    base = torch.from_numpy(rng.standard_normal((M, N))).to(BF16).to(DEV)
    for first in range(n):
        ids = ((np.arange(M) + first) % n).astype(np.int32)
        An, Bn = torch.nan_to_num(A), torch.nan_to_num(B)
        y = check_lora(awq, x, x64, An, Bn, ids, base, None, ranks)
        z = awq.lora(x, A.to(DEV), B.to(DEV), torch.from_numpy(ids).to(DEV), base, ranks=torch.from_numpy(ranks).to(DEV))
        assert torch.equal(y, z)
    An, Bn = torch.nan_to_num(A), torch.nan_to_num(B)
    ids = (np.arange(M) % n).astype(np.int32)
    check_lora(awq, x, x64, An, Bn, ids, base, None, np.array([-1, -2 ** 31, 41, 2 ** 31 - 1, 40, 0], dtype=np.int32))


@pytest.mark.parametrize("M", [5, 40, 270])
def test_lora_ids(awq, M):
    """All rows of one adapter, none of any, every row its own, ids far outside; the base's bits stay where no adapter is."""
    rng = rng_of(3)
    K, N, R, n = 128, 96, 16, 300
    A, B = adapters(rng, n, K, N, R)
    x, x64 = activations(rng, M, K, BF16)
    base = torch.from_numpy(rng.standard_normal((M, N))).to(BF16).to(DEV)
    base[0, 3] = float("nan")
    base[0, 4] = -0.0
    for ids in (np.full(M, 7), np.arange(M), np.arange(M)[::-1], np.where(np.arange(M) % 2, 3, n)):
        ids = ids.astype(np.int32).copy()
        ids[0] = -5
        y = awq.lora(x, A.to(DEV), B.to(DEV), torch.from_numpy(ids).to(DEV), base)
        assert torch.equal(y[0].view(torch.int16), base[0].view(torch.int16))
        clean = base.clone()
        clean[0] = 1.0
        check_lora(awq, x, x64, A, B, ids, clean)
    for v in (-1, n, 2 ** 31 - 1, -2 ** 31):
        ids = torch.full((M,), v, dtype=torch.int32, device=DEV)
        assert torch.equal(awq.lora(x, A.to(DEV), B.to(DEV), ids, base).view(torch.int16), base.view(torch.int16))


@pytest.mark.parametrize("M", [1, 33, 280])
@pytest.mark.parametrize("kind,out", [(BF16, BF16), (F32, F32), (I8, BF16)])
def test_lora_in_place_strides_and_guards(awq, M, kind, out):
    """Row strides of X, base and Y; in place; rows that start anywhere; nothing beside Y or behind the workspace written."""
    rng = rng_of(4)
    K, N, R, n = 256, 200, 16, 4
    A, B = adapters(rng, n, K, N, R)
    x, x64 = activations(rng, M, K, kind, ld=K + 16)
    ids = rng.integers(-1, n, M).astype(np.int32)
    need = awq.lora_workspace_bytes(M, K, N, R)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    v = torch.from_numpy(rng.standard_normal((M + 2, N + 24)) * 2).to(out).to(DEV)
    want = check_lora(awq, x, x64, A, B, ids, v[1:M + 1, 8:N + 8].contiguous())
    for off in (8, 3):
        big, base = v.clone(), v.clone()
        base[1:M + 1, off:N + off] = v[1:M + 1, 8:N + 8]
        view = big[1:M + 1, off:N + off]
        y = awq.lora(awq.Act8(*x) if isinstance(x, tuple) else x, A.to(DEV), B.to(DEV), torch.from_numpy(ids).to(DEV),
                     base[1:M + 1, off:N + off], out=view, workspace=ws[:need])
        assert y is view and torch.equal(view, want)
        big[1:M + 1, off:N + off] = v[1:M + 1, off:N + off]
        assert torch.equal(big, v) and torch.all(ws[need:] == 0xA5)
        y = awq.lora(awq.Act8(*x) if isinstance(x, tuple) else x, A.to(DEV), B.to(DEV), torch.from_numpy(ids).to(DEV),
                     base[1:M + 1, off:N + off], out=base[1:M + 1, off:N + off])
        assert torch.equal(y, want)
        base[1:M + 1, off:N + off] = v[1:M + 1, off:N + off]
        assert torch.equal(base, v)


@pytest.mark.parametrize("M", [6, 300])
def test_lora_not_finite(awq, M):
    """NaN and Inf of a row, of a row's scale, of an adapter stay with that row, or that adapter's rows."""
    rng = rng_of(5)
    K, N, R, n = 128, 64, 16, 3
    A, B = adapters(rng, n, K, N, R)
    ids = (np.arange(M) % n).astype(np.int32)
    base = torch.from_numpy(rng.standard_normal((M, N))).float().to(DEV)
    for kind in (F32, BF16, E4M3):
        x, _ = activations(rng, M, K, kind)
        X = awq.Act8(*x) if isinstance(x, tuple) else x
        args = (A.to(DEV), B.to(DEV), torch.from_numpy(ids).to(DEV), base)
        clean = awq.lora(X, *args)
        if isinstance(x, tuple):
            x[1][1] = float("nan")
        else:
            x[1, 3] = float("inf")
        y = awq.lora(X, *args)
        assert not torch.isfinite(y[1]).any()
        y[1] = clean[1]
        assert torch.equal(y, clean)
    x, _ = activations(rng, M, K, BF16)
    clean = awq.lora(x, A.to(DEV), B.to(DEV), torch.from_numpy(ids).to(DEV), base)
    A[2, 0, 0] = float("nan")
    y = awq.lora(x, A.to(DEV), B.to(DEV), torch.from_numpy(ids).to(DEV), base).cpu()
    own = torch.from_numpy(ids == 2)
    assert not torch.isfinite(y[own]).any() and torch.equal(y[~own], clean.cpu()[~own])


def test_lora_far_adapter(awq):
    """An adapter whose weights start beyond 2^31 elements of the stack."""
    K, R, N, n = 8192, 256, 64, 1100
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    rng = rng_of(6)
    A = torch.zeros(n, R, K, dtype=BF16, device=DEV)
    B = torch.zeros(n, N, R, dtype=BF16, device=DEV)
    a, b = adapters(rng, 1, K, N, R)
    A[n - 1], B[n - 1] = a[0].to(DEV), b[0].to(DEV)
    x, x64 = activations(rng, 2, K, BF16)
    base = torch.zeros(2, N, device=DEV)
    y = awq.lora(x, A, B, torch.tensor([n - 1, 5], dtype=torch.int32, device=DEV), base)
    Y, D = ro.lora(x64, f64(a), f64(b), np.array([0, -1]), f64(base), None, None, 1, 3, 8)
    assert np.all(np.abs(f64(y) - Y) <= D + HALF[F32] * np.abs(Y)) and torch.all(y[1] == 0)


def test_lora_beside_the_packed_projection(awq):
    """As it is used: norm to 8 bits, the shared product on the packed weight, the adapters in place; eagerly, captured and
    replayed, on two streams."""
    rng = rng_of(7)
    M, K, N, R, n = 12, 512, 640, 16, 5
    art = artefact(rng, 1, N, K)[0]
    wt = awq.w4a8_weight(*(torch.from_numpy(art[k]).to(DEV) for k in ("qweight", "scales", "zeros")))
    A, B = (t.to(DEV) for t in adapters(rng, n, K, N, R))
    gamma = torch.ones(K, device=DEV)

    def layer(x, ids):
        a = awq.rmsnorm(x, gamma, dtype=I8)
        y = awq.w4a8(a, wt, dtype=BF16)
        return awq.lora(a, A, B, ids, y, out=y)

    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        return torch.randn(M, K, generator=g).to(BF16).to(DEV), torch.randint(-1, n, (M,), generator=g).to(torch.int32).to(DEV)

    x, ids = inputs(1)
    layer(x, ids)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer(x, ids)
    for seed in range(2, 7):
        nx, nids = inputs(seed)
        want = layer(nx, nids)
        x.copy_(nx), ids.copy_(nids)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        a = awq.rmsnorm(nx, gamma, dtype=I8)
        base = awq.w4a8(a, wt, dtype=BF16)
        x64 = f64(a.q.float()) * f64(a.scale)[:, None]
        Y, D = ro.lora(x64, f64(A), f64(B), nids.cpu().numpy(), f64(base), None, None, 1, 2, 8)
        assert np.all(np.abs(f64(want) - Y) <= D + HALF[BF16] * (np.abs(Y) + D))
    s = [torch.cuda.Stream() for _ in range(2)]
    data = [inputs(30 + i) for i in range(2)]
    want = [layer(*d) for d in data]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(s[i]):
                got[i] = layer(*data[i])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_lora_workspace_of_the_largest_batch_serves_all(awq):
    """One workspace, laid out for the largest batch, for batches of every split of K; its guard stays as it was."""
    rng = rng_of(7177)
    K, N, R, n, most = 4096, 512, 48, 3, 700
    A, B = adapters(rng, n, K, N, R)
    need = awq.lora_workspace_bytes(most, K, N, R)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    for M in (1, 15, 64, 65, 256, 257, most):
        x, x64 = activations(rng, M, K, BF16)
        ids = rng.integers(-1, n, M).astype(np.int32)
        base = torch.from_numpy(rng.standard_normal((M, N))).to(BF16).to(DEV)
        check_lora(awq, x, x64, A, B, ids, base, workspace=ws[:need])
        assert (ws[need:] == 0xA5).all()
