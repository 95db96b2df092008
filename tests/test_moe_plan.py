"""How the experts' products run by size (CPU)."""
import os
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "post_weight_quantization_mean_amd", "csrc")
PROGRAM = """
#include <cstdio>

#include "moe_plan.h"

int main() {
  int slots, units, waves, per_simd;
  while (std::scanf("%d %d %d %d", &slots, &units, &waves, &per_simd) == 4)
    std::printf("%d\\n", awq::units_per_block(slots, units, waves, per_simd));
}
"""


@pytest.fixture(scope="module")
def units_per_block(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")],
                   check=True, timeout=120)

    def ask(rows):
        text = "\n".join("%d %d %d %d" % r for r in rows)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True, timeout=60).stdout
        return [int(line) for line in out.splitlines()]
    return ask


@pytest.mark.parametrize("waves,per_simd", [(8, 4), (8, 2), (16, 4), (16, 2)])
def test_a_round_of_blocks_reaches_every_cu(units_per_block, waves, per_simd):
    """Blocks for one round: all that fit the 256 CUs together, or one unit each where there are fewer units; a block of
    sixteen waves is a CU's whether a SIMD takes four of its waves or the kernel was built for two."""
    fit = 256 * max(1, 4 * per_simd // waves)
    rows = [(s, u, waves, per_simd) for s in (1, 2, 8, 64, 256, 1024) for u in (1, 8, 16, 64, 128, 256, 896, 4096)]
    for (s, u, *_), per in zip(rows, units_per_block(rows)):
        blocks = s * -(-u // per)
        assert blocks <= max(fit, s) and (per == 1 or 2 * blocks > fit), (s, u, per, blocks)
        if s <= fit and fit % s == 0 and u * s % fit == 0:
            assert blocks == fit, (s, u, per, blocks)
