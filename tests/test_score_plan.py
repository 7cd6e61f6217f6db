"""Workspace layout of the accumulated weights (csrc/compact_plan.h) on the CPU: its parts follow one another without
overlap, whatever the base's alignment, and fit what the size function asks for."""
import json
import os
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "causal_head_latent_b200", "csrc")
CASES = [(1, 1, 1, 64), (3, 777, 7, 192), (5, 4000, 64, 512), (5, 4000, 65, 512), (23, 65536, 96, 64), (32, 131072, 96, 512)]

PROGRAM = r"""
#include <cstdio>
#include "compact_plan.h"
using namespace gmla;
int main() {
  const long long cases[][4] = {%s};
  bool first = true;
  std::printf("[");
  for (auto &c : cases)
    for (int k = 0; k < 16; ++k) {
      const unsigned long long base = 0x7f0000000000ull + 16 * k;
      const long long n = score_group(c[0], c[1], c[2]);
      const ScoreLayout o = score_layout(base, c[0], c[1], c[2], c[3]);
      std::printf("%%s{\"base\":%%llu,\"case\":[%%lld,%%lld,%%lld,%%lld],\"n\":%%lld,\"R\":%%lld,\"at\":[%%zu,%%zu,%%zu,%%zu,%%zu,%%zu,%%zu,%%zu]}",
                  first ? "" : ",", base, c[0], c[1], c[2], c[3], n, share_records(n, c[1], kScoreTileKeys, kScorePieceTiles),
                  o.hi, o.lo, o.third, o.pm, o.pl, o.lse, o.s, o.end);
      first = false;
    }
  std::printf("]\n");
}
"""


@pytest.fixture(scope="module")
def layouts(tmp_path_factory):
    d = tmp_path_factory.mktemp("score_plan")
    (d / "c.cpp").write_text(PROGRAM % ",".join("{%d,%d,%d,%d}" % c for c in CASES))
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, str(d / "c.cpp"), "-o", str(d / "c")], check=True)
    return json.loads(subprocess.run([str(d / "c")], capture_output=True, text=True, check=True).stdout)


def test_score_workspace(layouts):
    import causal_head_latent_b200 as g
    for c in layouts:
        (B, L, H, dc), n, R, at = c["case"], c["n"], c["R"], c["at"]
        part = 2 * B * H * dc
        scores = n * -(-L // 128) * 128 * (-(-H // 32) * 32) * 4
        sizes = [part, part, part if H <= 64 else 0, 4 * R * H, 4 * R * H, 4 * n * H, scores]
        assert 1 <= n <= B and (c["base"] + at[0]) % 256 == 0
        for k, size in enumerate(sizes):
            assert at[k] % 256 == at[0] % 256 and at[k] + size <= at[k + 1]
        assert at[-1] <= g.gmla_cache_score_workspace_size(B, L, H, dc)
