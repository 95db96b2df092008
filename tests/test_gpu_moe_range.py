"""GPU tests of the experts at the upper end of fp32: finite activations whose result is finite give it, as the definition
does, although a code is multiplied as 8 + q / 2.  The tokens are built so that the fp64 result fits fp32 and no sum has small
terms beside a large one that cancels; so each token's result is held to the error's norm of ordinary tokens."""
import numpy as np
import pytest
import torch

from oracle import awq_oracle as o
from oracle import rows_oracle as ro
from tests.test_gpu_moe import BF16, DEV, E4M3, F32, I8, NORM, activations, artefact, awq, banner, f64, handle, rng_of, \
    routing_of  # noqa: F401 (awq is a fixture)
from tests.rows_exact import words

pytestmark = pytest.mark.gpu
FAR = 3 * 2.0 ** 123  # 3.2e37: 10.7 of them leave fp32, and eight bits hold it


def check_rows(awq, X, x64, ids, w, gu, down, out):
    r = awq.Routing(torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV))
    y = f64(awq.moe(X, r, handle(awq, gu), handle(awq, down), dtype=out))
    Y, _ = ro.moe(x64, ids, w, gu, down, "silu", 1, 3)
    assert np.abs(Y).max() < torch.finfo(F32).max / 4 and np.all(np.isfinite(y))
    err, norm = np.linalg.norm(y - Y, axis=1), np.linalg.norm(Y, axis=1)
    assert np.all(err <= NORM[out] * norm), (err / norm).tolist()


# a slot per pair, a slot per expert, tiles
SIZES = [(1, 4, 2), (5, 4, 2), (40, 4, 2)]


@pytest.mark.parametrize("M,E,k", SIZES)
@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("out", [BF16, F32])
def test_an_activation_at_the_upper_end(awq, M, E, k, kind, out):
    """One channel of 3e37, alone in its group, that the gate does not read (q = z) and up does."""
    banner(f"moe far activation M={M} E={E} k={k} {kind} {out}")
    rng = rng_of(31)
    H, I, at = 256, 128, 37
    gu, down = artefact(rng, E, 2 * I, H), artefact(rng, E, H, I)
    for art in gu:
        q = o.unpack_words(art["qweight"])
        q[:I, at] = art["zeros"][:I, 0]
        art["qweight"] = words(q)
    x, _ = activations(rng, M, H, kind)
    x[:, :128] = 0.0
    x[:, at] = torch.tensor([FAR, -FAR], device=DEV).repeat(M)[:M].to(kind)
    ids, w = routing_of(rng, M, E, k)
    check_rows(awq, x, f64(x), ids, w, gu, down, out)


@pytest.mark.parametrize("M,E,k", SIZES)
@pytest.mark.parametrize("kind", [BF16, F32, I8, E4M3])
@pytest.mark.parametrize("out", [BF16, F32])
def test_an_intermediate_at_the_upper_end(awq, M, E, k, kind, out):
    """act(gate) * up of 1e37 and more, whose products with down's weights stay inside fp32."""
    banner(f"moe far intermediate M={M} E={E} k={k} {kind} {out}")
    rng = rng_of(32)
    H, I, far = 256, 256, 2.0 ** 60
    gu, down = artefact(rng, E, 2 * I, H), artefact(rng, E, H, I)
    x, x64 = activations(rng, M, H, kind)
    X = awq.Act8(x[0], x[1] * far) if isinstance(x, tuple) else x * far
    ids, w = routing_of(rng, M, E, k)
    check_rows(awq, X, x64 * far, ids, w, gu, down, out)
