"""The tree attention's schedule (csrc/tree_schedule.h), compiled for the host: every tile of every
block of query rows is taken once, in order, and no CTA takes more segments than it can list, whatever
the rows' lengths."""

import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HARNESS = r"""
#include <stdio.h>
#include <vector>
#include "tree_schedule.h"
using namespace fade;
#define MUST(x) if (!(x)) return printf("line %d: %s\n", __LINE__, #x), 1
// Per case B H G rows and the CTAs wanted, then n, held16, n_mid of every row; prints the CTAs, the
// charge, the tiles in all, and the most segments and tiles of a CTA.
int main() {
  int B, H, G, rows, wanted;
  while (scanf("%d %d %d %d %d", &B, &H, &G, &rows, &wanted) == 5) {
    std::vector<RowTiles> r(B);
    std::vector<int> tiles(B + 1, 0), blocks(B + 1, 0);
    for (int b = 0; b < B; ++b) {
      int n, held, mid;
      if (scanf("%d %d %d", &n, &held, &mid) != 3) return 2;
      r[b] = make_row_tiles(n, G, rows, held, mid);
      tiles[b + 1] = tiles[b] + H * r[b].blocks * r[b].tiles;
      blocks[b + 1] = blocks[b] + H * r[b].blocks;
    }
    const int N = tiles[B], P = tree_ctas(blocks[B], wanted);
    const Rows all{tiles.data(), blocks.data(), B, tree_charge(N, blocks[B], P)};
    int most = 0, longest = 0, b = 0, blk = 0, t = 0;   // the tile that has to come next
    auto skip = [&]() { while (b < B && blk == H * r[b].blocks) ++b, blk = 0; };
    MUST(cta_start(all, P, 0) == 0 && cta_start(all, P, P) == N);
    for (int c = 0; c < P; ++c) {
      const int g_first = cta_start(all, P, c), g_end = cta_start(all, P, c + 1);
      MUST(g_first <= g_end);
      if (g_first == g_end) continue;
      if (g_end - g_first > longest) longest = g_end - g_first;
      for (int k = 0;; ++k) {
        const Place at = block_from([&](int i) { return r[i]; }, all, H, g_first, k, g_end);
        if (at.g0 >= g_end) break;
        if (k + 1 > most) most = k + 1;
        const int begin = g_first > at.g0 ? g_first - at.g0 : 0;
        const int end = at.rt.tiles < g_end - at.g0 ? at.rt.tiles : g_end - at.g0;
        skip();
        MUST(at.b == b && at.blk == blk && begin == t && end > begin);
        for (int i = begin; i < end; ++i) MUST(cta_of(all, P, b, at.g0, at.rt.tiles, i) == c);
        t = end;
        if (t == r[b].tiles) t = 0, ++blk;
      }
    }
    skip();
    MUST(b == B && t == 0 && most <= kMaxSeg);
    printf("%d %d %d %d %d\n", P, all.charge, N, most, longest);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("schedule")
    (d / "replay.cpp").write_text(HARNESS)
    csrc = os.path.join(ROOT, "tiered_mixed_precision_gb300", "csrc")
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", csrc, str(d / "replay.cpp"), "-o",
                    str(d / "replay")], check=True)

    def run(cases):
        text = "\n".join(" ".join(str(int(x)) for x in (*head, *np.asarray(rows).ravel()))
                         for head, rows in cases)
        r = subprocess.run([str(d / "replay")], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout[-200:]
        return [tuple(int(x) for x in line.split()) for line in r.stdout.splitlines()]

    return run


def test_every_tile_is_taken_once(replay):
    rng = np.random.default_rng(0)
    cases = []
    for _ in range(400):
        B = int(np.exp(rng.uniform(0, np.log(257))))
        H, G = int(rng.choice([1, 2, 8])), int(rng.choice([1, 2, 4, 8]))
        T = int(rng.integers(1, 65))
        n = rng.integers(0, T + 1, B)
        held = rng.integers(0, 69, B)
        mid = np.where(rng.random(B) < rng.random(), 0,
                       np.exp(rng.uniform(0, np.log(131072), B)).astype(int))
        rows = 64 if T * G <= 64 else 128
        cases.append(((B, H, G, rows, int(rng.choice([1, 7, 152, 160]))),
                      np.stack([n, held, mid], 1)))
    got = replay(cases)
    assert len(got) == len(cases)
    assert any(charge for _, charge, *_ in got) and any(not charge for _, charge, *_ in got)


@pytest.mark.parametrize("B,n_long,length", [(64, 32, 16384), (128, 64, 8192), (256, 20, 32768),
                                             (256, 3, 131072)])
@pytest.mark.parametrize("blocks", [1, 4])
def test_short_rows_beside_long_ones(replay, B, n_long, length, blocks):
    """One-tile blocks beside long rows, where equal tiles would give a CTA hundreds of them; no CTA
    takes more than twice an equal share of tiles."""
    G, n = (4, 16) if blocks == 1 else (8, 64)
    rows = [(n, 67, length - 67)] * n_long + [(n, 60, 0)] * (B - n_long)
    (P, charge, N, most, longest), = replay([((B, 8, G, 64 if blocks == 1 else 128, 152), rows)])
    assert charge > 0 and most <= 128 and longest <= 2 * (N / P + 1)
