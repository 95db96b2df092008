"""Which kernel the W4A8 product takes by size (CPU): the GPU tests' shapes together reach every one, each kind of sum and
each shape of block, so that a change of the plan's costs cannot leave one untested unseen."""
import itertools
import os
import subprocess

import pytest
import torch

from tests import test_gpu_a8 as gpu
from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "post_weight_quantization_mean_amd", "csrc")
STREAM, SPLIT, TILE = 0, 1, 2
PROGRAM = """
#include <cstdio>

#include "rows8_plan.h"
#include "w4a8_plan.h"

int main(int argc, char**) {
  long long m, k, n;
  while (std::scanf("%lld %lld %lld", &m, &k, &n) == 3) {
    if (argc > 1) {  // rows: the third number says whether they are aligned
      const awq::RowLayout l = awq::row_layout(m, k, n != 0);
      std::printf("%d %d\\n", l.waves, l.units);
      continue;
    }
    const awq::Plan p = awq::w4a8_plan(m, k, n);
    std::printf("%d %d %d %d %d %d %d\\n", p.path, p.tm, p.splits, p.per_split, p.ct, p.waves,
                (int)awq::matrix_sums(awq::kSumsDefault, true, m));
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")],
                   check=True, timeout=120)

    def ask(shapes, *mode):
        text = "\n".join("%d %d %d" % s for s in shapes)
        out = subprocess.run([str(d / "plan"), *mode], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return ask


def parameters(test):
    """(values of one parametrize mark by name) of a test function."""
    marks = [m for m in test.pytestmark if m.name == "parametrize"]
    return {m.args[0]: list(m.args[1]) for m in marks}


def cases():
    """((M, K, N), codes, result, kind of sum asked for) of every product that a GPU test compares with the definition."""
    for test in (gpu.test_w4a8, gpu.test_w4a8_tiles, gpu.test_w4a8_some_tokens, gpu.test_w4a8_wide_and_split):
        p = parameters(test)
        for shape, (xt, yt) in itertools.product(p["M,K,N"], p["xt,yt"]):
            yield shape, xt, yt, None
    p = parameters(gpu.test_w4a8_matrix_sums_on_request)
    for shape, yt in itertools.product(p["M,K,N"], p["yt"]):
        yield shape, torch.float8_e4m3fn, yt, "matrix"


def test_every_kernel_is_reached(plan):
    got = list(cases())
    seen = set()
    for (shape, xt, yt, asked), (path, tm, splits, per, ct, waves, matrix) in zip(got, plan([c[0] for c in got])):
        G = shape[1] // 128
        kind = "int8" if xt == torch.int8 else "fast" if asked or (matrix and yt == torch.bfloat16) else "wide"
        if path == STREAM:
            seen.add((kind, STREAM, tm, ct, waves))
        elif path == SPLIT:
            seen.add((kind, SPLIT, tm, "parts" if splits > 1 else "whole"))
            seen.add((kind, SPLIT, tm, "odd" if per % 2 else "even"))
            if G % per:
                seen.add((kind, SPLIT, tm, "fewer in the last"))
        else:
            tm = 4 if kind == "wide" else tm  # the fp32 sums of e4m3 codes have 64-token tiles only
            seen.add((kind, TILE, tm, G % 4))
    want = set()
    for kind in ("int8", "fast", "wide"):
        want |= {(kind, STREAM, 1, 1, 16), (kind, STREAM, 1, 2, 8)}
        want |= {(kind, STREAM, 2, *b) for b in ((2, 8), (3, 8), (4, 8), (3, 4), (4, 4))}
        want |= {(kind, SPLIT, tm, x) for tm in (2, 4) for x in ("parts", "odd", "even", "fewer in the last")}
        want.add((kind, SPLIT, 2, "whole"))
        want |= {(kind, TILE, 4, r) for r in range(4)}
        if kind != "wide":
            want |= {(kind, TILE, 8, r) for r in (0, 1, 2, 3)}
    assert want <= seen, sorted(map(str, want - seen))


def test_plan_is_sound(plan):
    """Over a grid of sizes: every block of a split has a group, splits cover the groups once, blocks have their limits."""
    shapes = [(m, 128 * g, n) for m in (1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 100, 128, 129, 256, 257, 511, 1000, 4096, 100000)
              for g in (1, 2, 3, 7, 8, 9, 31, 32, 86, 112, 500) for n in (1, 16, 17, 255, 256, 257, 4096, 5104, 5105, 28672, 200001)]
    for (m, k, n), (path, tm, splits, per, ct, waves, matrix) in zip(shapes, plan(shapes)):
        G = k // 128
        assert path in (STREAM, SPLIT, TILE) and matrix == (m > 256)
        if path == STREAM:
            assert m <= 256 and (tm, ct, waves) in {(1, 1, 16), (1, 2, 8), (2, 2, 8), (2, 3, 8), (2, 4, 8), (2, 3, 4), (2, 4, 4)}
            assert (m <= 16) == (tm == 1)
        elif path == SPLIT:
            assert m > 16 and tm in (2, 4) and splits * per >= G > (splits - 1) * per
        else:
            assert m > 16 and tm in (4, 8)


def test_every_row_layout_is_reached(plan):
    """Both operators, rows that start at multiples of 16 bytes and others, over the GPU tests' shapes (whose rows are
    contiguous: they are aligned where K is a multiple of 8)."""
    sizes = [(m, k, int(k % 8 == 0)) for m in (1, 256, 257, 5000) for k in range(1, 33100, 67)]
    sizes += [(m, 8 * u, 1) for m in (1, 257) for u in range(1, 4200)]
    every = {(a, *l) for (_, _, a), l in zip(sizes, plan(sizes, "rows"))}
    assert len(every) == 11 + 8
    for tests in ((gpu.test_rmsnorm, gpu.test_long_rows, gpu.test_rmsnorm_row_layouts),
                  (gpu.test_act_mul, gpu.test_long_rows, gpu.test_act_mul_row_layouts)):
        shapes = [(m, k, int(k % 8 == 0)) for t in tests for m, k in parameters(t)["M,K"]]
        seen = {(a, *l) for (_, _, a), l in zip(shapes, plan(shapes, "rows"))}
        assert every <= seen, sorted(every - seen)
