"""Launch plans and workspace layouts of the compact-cache operators, on the CPU.

The plans are pure integer arithmetic (csrc/compact_plan.h); a small C++ program
compiled here walks every share of ragged batches the way the kernels do."""
import ctypes  # noqa: F401  (the library is loaded through the package)
import json
import os
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "causal_head_latent_b200", "csrc")

CHECKER = r"""
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>
#include "compact_plan.h"
using namespace gmla;
static int bad(const char *what, long long a, long long b) { std::printf("BAD %s %lld %lld\n", what, a, b); return 1; }
// Every tile in exactly one piece, records distinct and inside the workspace, share_of() the inverse of
// share_begin(), every share between a sequence's first and last holding a piece of it, as the kernels use them.
static int shares(const std::vector<long long> &lens, long long L, int tile, int extra) {
  const long long B = (long long)lens.size(), Gmax = share_count(B, L, tile, extra), R = share_records(B, L, tile, extra);
  std::vector<long long> tiles(B), before(B + 1, 0), seen(B, 0);
  for (long long b = 0; b < B; ++b) {
    tiles[b] = (lens[b] + tile - 1) / tile;
    before[b + 1] = before[b] + share_places(tiles[b], extra);
  }
  const long long total = before[B], G = Gmax < total ? Gmax : total;
  if (Gmax < 1 || Gmax > kShares) return bad("share count", Gmax, 0);
  std::set<long long> used;
  long long at = 0, most = 0, least = 1ll << 60;
  for (long long i = 0; i < G; ++i) {
    const long long t0 = share_begin(i, total, G), t1 = share_begin(i + 1, total, G);
    if (t0 != at || t1 <= t0) return bad("share range", t0, t1);
    if (t1 - t0 > most) most = t1 - t0;
    if (t1 - t0 < least) least = t1 - t0;
    for (long long t = t0; t < t1; ++t)
      if (share_of(t, total, G) != i) return bad("share_of", t, i);
    for (long long b = 0; b < B; ++b) {
      if (tiles[b] == 0) continue;
      const long long first = before[b] + extra;
      const long long lo = t0 > first ? t0 : first, hi = t1 < before[b + 1] ? t1 : before[b + 1];
      const bool inside = i >= share_of(first, total, G) && i <= share_of(first + tiles[b] - 1, total, G);
      if ((lo < hi) != inside) return bad("share without a piece", i, b);
      if (lo >= hi) continue;
      if (lo - first != seen[b]) return bad("tiles out of order", lo - first, seen[b]);
      seen[b] += hi - lo;
      if (!used.insert(i + b).second) return bad("record used twice", i, b);
      if (i + b >= R) return bad("record outside", i + b, R);
    }
    at = t1;
  }
  if (at != total) return bad("places left over", at, total);
  for (long long b = 0; b < B; ++b)
    if (seen[b] != tiles[b]) return bad("tiles left over", b, seen[b]);
  if (G > 0 && most - least > 1) return bad("uneven shares", most, least);
  return 0;
}
int main() {
  std::srand(1);
  for (int tile : {48, 128}) {
    for (long long B : {1, 2, 3, 32, 147, 148, 149, 500})
      for (long long L : {1, 63, 64, 65, 1000, 5000})
        for (int kind = 0; kind < 4; ++kind) {
          std::vector<long long> lens(B, L);
          for (auto &x : lens)
            if (kind == 1) x = std::rand() % (L + 1);
            else if (kind == 2) x = std::rand() % 3 ? 0 : 1 + std::rand() % L;
            else if (kind == 3) x = 0;
          if (shares(lens, L, tile, 0) || shares(lens, L, tile, tile == 48 ? kFp4PieceTiles : kScorePieceTiles)) return 1;
        }
  }
  std::printf("[");
  const long long cases[][4] = {{1, 1, 1, 64}, {3, 777, 7, 192}, {32, 131072, 96, 512}, {200, 5000, 96, 512}};
  bool first = true;
  for (auto &c : cases)
    for (int k = 0; k < 16; ++k) {
      const unsigned long long base = 0x7f0000000000ull + 16 * k;
      const Fp4DecodeLayout o = fp4_decode_layout(base, c[0], c[1], c[2], c[3]);
      std::printf("%s{\"base\":%llu,\"B\":%lld,\"L\":%lld,\"H\":%lld,\"dc\":%lld,\"R\":%lld,\"at\":[%zu,%zu,%zu,%zu,%zu],"
                  "\"need\":%zu}", first ? "" : ",", base, c[0], c[1], c[2], c[3],
                  share_records(c[0], c[1], kFp4TileKeys, kFp4PieceTiles), o.qt, o.pm, o.pl, o.pacc, o.end,
                  fp4_decode_layout_bytes(c[0], c[1], c[2], c[3]));
      first = false;
    }
  std::printf("]\n");
  return 0;
}
"""


@pytest.fixture(scope="module")
def checked(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "c.cpp").write_text(CHECKER)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, str(d / "c.cpp"), "-o", str(d / "c")], check=True)
    r = subprocess.run([str(d / "c")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    return json.loads(r.stdout)


def test_shares_cover_every_tile_once(checked):
    assert checked  # the program walked the shares and found nothing wrong


def test_fp4_decode_workspace(checked):
    import causal_head_latent_b200 as g
    for c in checked:
        B, H, dc, R, at = c["B"], c["H"], c["dc"], c["R"], c["at"]
        sizes = [2 * B * H * dc, 4 * R * H, 4 * R * H, 4 * R * H * dc]
        assert (c["base"] + at[0]) % 256 == 0
        for k, n in enumerate(sizes):
            assert at[k] % 256 == at[0] % 256 and at[k] + n <= at[k + 1]
        assert at[-1] <= c["need"] == g.gmla_attend_decode_fp4_workspace_size(B, c["L"], H, dc)
