"""The prompt attention's schedule (csrc/prompt_schedule.h), compiled for the host: every tile of every
block of queries is taken once, items that CTAs share are joined from the partials that they leave, and no
CTA has much more than its share, whatever the rows' lengths."""

import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HARNESS = r"""
#include <stdio.h>
#include <map>
#include <set>
#include <vector>
#include "prompt_schedule.h"
using namespace fade;
#define MUST(x) if (!(x)) return printf("line %d: %s\n", __LINE__, #x), 1
// Per case B H log_g sink window sms, then q_len, kv_len of every row; prints the CTAs, the joins, the
// whole items, the mean and the largest cost of a CTA, and the largest item's.
int main() {
  PromptShape s{};
  int sms;
  while (scanf("%d %d %d %d %d %d", &s.B, &s.H, &s.log_g, &s.sight.sink, &s.sight.window, &sms) == 6) {
    s.G = 1 << s.log_g;
    s.Hq = s.H * s.G;
    static PromptRows rows;
    int blocks = 0;
    for (int b = 0; b < s.B; ++b) {
      if (scanf("%d %d", &rows.q_len[b], &rows.kv_len[b]) != 2) return 2;
      rows.order[b] = (uint8_t)b;
      blocks = std::max(blocks, (rows.q_len[b] * s.G + 255) / 256);
    }
    if (s.sight.window == 0) s.sight.sink = 0;
    std::stable_sort(rows.order, rows.order + s.B,
                     [&](uint8_t x, uint8_t y) { return rows.kv_len[x] > rows.kv_len[y]; });
    static PromptSchedule a;
    a = PromptSchedule{};
    int P = 0;
    const int joins = prompt_schedule(s, rows, blocks, sms, a, &P);
    MUST(P >= 1 && P <= sms && joins <= P);
    // what the CTAs do: per item the ranges of tiles, by CTA
    struct Range { int c, begin, n, slot; };
    std::map<std::pair<int, std::pair<int, int>>, std::vector<Range>> got;   // (b, h, tok0)
    double most = 0, total = 0, largest = 0;
    auto each = [](const PromptItem& it) { return it.active == 2 ? kCostTwo : kCostOne; };
    for (int c = 0; c < P; ++c) {
      PromptWalk<PromptItem> walk;
      PromptItem it;
      std::set<int> slots;
      double cost = 0;
      auto at = [&](int index) { return prompt_item(s, rows, index); };
      while (walk.next(a, P, c, at, it)) {
        MUST(it.n > 0 && it.begin >= 0 && it.begin + it.n <= it.all);
        MUST(it.b >= 0 && it.b < s.B && it.h >= 0 && it.h < s.H);
        const int slot = it.n == it.all ? -1 : 2 * c + (it.begin == 0 ? 1 : 0);
        if (slot >= 0) MUST(slots.insert(slot).second);   // a partial of its own
        got[{it.b, {it.h, it.tok0}}].push_back({c, it.begin, it.n, slot});
        // the tiles of the item, and which may hide something from a query
        int before = -1, masked = 0;
        for (int j = 0; j < it.n; ++j) {
          const int kt = it.tile(j);
          MUST(kt > before && kt * kPromptTile <= it.p1);
          before = kt;
          const int t0 = kt * kPromptTile, t1 = t0 + kPromptTile - 1;
          masked += t1 > it.p0 || (s.sight.window && t0 < it.p1 - s.sight.window + 1 &&
                                   t1 >= s.sight.sink);
        }
        MUST(masked <= 7);
        cost += it.n * each(it);
        largest = std::max<double>(largest, kCostStart + it.all * each(it));
      }
      most = std::max(most, cost);
      total += cost;
    }
    int shared = 0, taken = 0;
    for (int b = 0; b < s.B; ++b)
      for (int rank = 0; rank < blocks; ++rank) {
        const PromptItem it = prompt_block(s, b, rows.q_len[b], rows.kv_len[b], rank);
        // the tiles of the block: those that some query sees a token of
        if (it.all) {
          std::set<int> need;
          for (int p = it.p0; p <= it.p1; ++p) {
            const int w = s.sight.window;
            need.insert(p / kPromptTile);
            const int lo = w ? std::max(0, p - w + 1) : 0;
            for (int t = lo / kPromptTile; t <= p / kPromptTile; ++t) need.insert(t);
            for (int j = 0; j < std::min(s.sight.sink, p + 1); ++j) need.insert(j / kPromptTile);
          }
          std::set<int> have;
          for (int j = 0; j < it.all; ++j) have.insert(it.tile(j));
          MUST((int)have.size() == it.all);
          for (int t : need) MUST(have.count(t));
        }
        for (int h = 0; it.all && h < s.H; ++h) {
          auto& r = got[{b, {h, it.tok0}}];
          std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.begin < y.begin; });
          int at = 0;
          for (auto& x : r) {
            MUST(x.begin == at);
            at += x.n;
          }
          MUST(at == it.all);
          ++taken;
          if (r.size() > 1) {   // joined, from the right partials
            int found = 0;
            for (int j = 0; j < joins; ++j) {
              const PromptItem x = prompt_item(s, rows, a.join[j].item);
              if (x.b != b || x.h != h || x.tok0 != it.tok0) continue;
              ++found;
              size_t i = 0;
              for (int c = a.join[j].first; c <= a.join[j].last; ++c) {
                if (a.start[c].item == a.start[c + 1].item && a.start[c].tile == a.start[c + 1].tile)
                  continue;   // no share
                MUST(i < r.size() && r[i].c == c && r[i].slot == 2 * c + (c == a.join[j].first ? 1 : 0));
                ++i;
              }
              MUST(i == r.size());
            }
            MUST(found == 1);
            ++shared;
          }
        }
      }
    MUST(taken == (int)got.size() && shared == joins);
    // ---- the column sums: every query tile that sees a key of a pair meets it once
    s.n_kv = 1;
    for (int b = 0; b < s.B; ++b) s.n_kv = std::max(s.n_kv, rows.kv_len[b]);
    const int pairs = (s.n_kv + 255) / 256, per = kPromptTile >> s.log_g;
    static PromptSchedule m;
    m = PromptSchedule{};
    int Pm = 0, sharedm = 0;
    const int joinsm = mass_schedule(s, rows, sms, m, &Pm);
    MUST(Pm >= 1 && Pm <= sms && joinsm <= Pm && m.whole == 0);
    std::map<std::pair<int, std::pair<int, int>>, std::vector<Range>> met;   // (b, h, k0)
    double mostm = 0, totalm = 0;
    for (int c = 0; c < Pm; ++c) {
      PromptWalk<MassItem> walk;
      MassItem it;
      std::set<int> slots;
      int tiles = 0;
      auto at = [&](int index) { return mass_item(s, rows, index); };
      while (walk.next(m, Pm, c, at, it)) {
        MUST(it.n > 0 && it.begin >= 0 && it.begin + it.n <= it.all);
        const int slot = it.n == it.all ? -1 : 2 * c + (it.begin == 0 ? 1 : 0);
        if (slot >= 0) MUST(slots.insert(slot).second);
        met[{it.b, {it.h, it.k0}}].push_back({c, it.begin, it.n, slot});
        tiles += it.n;
        totalm += it.n + (it.begin == 0 ? 2 + s.G : 0);
      }
      mostm = std::max<double>(mostm, tiles);
    }
    for (int i = 0; i < pairs * s.B * s.H; ++i) {
      const MassItem it = mass_item(s, rows, i);
      const int kv = rows.kv_len[it.b], q = rows.q_len[it.b], w = s.sight.window;
      for (int tok = 0; tok < q; ++tok) {   // a query that sees one of the keys is in a tile
        const int p = kv - q + tok, hi = std::min(std::min(it.k0 + 255, kv - 1), p);
        const bool sees = it.k0 <= hi && (!w || hi > p - w || it.k0 < s.sight.sink);
        if (sees) MUST(tok / per >= it.first && tok / per < it.first + it.all);
      }
      MUST(it.all == 0 || it.first + it.all <= (q + per - 1) / per);
      auto& r = met[{it.b, {it.h, it.k0}}];
      std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.begin < y.begin; });
      int at = 0;
      for (auto& x : r) {
        MUST(x.begin == at);
        at += x.n;
      }
      MUST(at == it.all);
      if (r.size() > 1) {
        int found = 0;
        for (int j = 0; j < joinsm; ++j) found += m.join[j].item == i && m.join[j].first == r[0].c &&
                                                  m.join[j].last == r.back().c;
        MUST(found == 1);
        ++sharedm;
      }
    }
    MUST(sharedm == joinsm && mostm <= 1.3 * totalm / Pm + 2 + s.G);
    printf("%d %d %d %g %g %g\n", P, joins, a.whole, (total + kCostStart * taken) / P, most, largest);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("schedule")
    (d / "main.cpp").write_text(HARNESS)
    subprocess.run([gxx, "-O1", "-std=c++17", "-Wall", "-Werror",
                    f"-I{ROOT}/tiered_mixed_precision_gb300/csrc", f"-I{ROOT}/include",
                    str(d / "main.cpp"), "-o", str(d / "main")], check=True)

    def go(B, H, log_g, sink, window, q_len, kv_len, sms=152):
        text = f"{B} {H} {log_g} {sink} {window} {sms}\n" + "\n".join(
            f"{int(a)} {int(b)}" for a, b in zip(q_len, kv_len))
        r = subprocess.run([str(d / "main")], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout[-500:]
        return [float(x) for x in r.stdout.split()]

    return go


def test_random_calls(run):
    rng = np.random.default_rng(1)
    for _ in range(150):
        B, H = int(rng.integers(1, 20)), int(rng.choice([1, 2, 3, 8]))
        top = int(np.exp(rng.uniform(0, np.log(6000))))
        kv = rng.integers(0, top + 1, B)
        q = np.minimum(kv, rng.integers(0, max(1, min(top, 700)) + 1, B)) if rng.random() < 0.5 else kv
        if not q.any():
            continue
        window = int(rng.choice([0, rng.integers(1, top + 1)]))
        run(B, H, int(rng.integers(0, 4)), int(rng.integers(0, 300)), window, q, kv,
            int(rng.choice([1, 2, 132, 152, 160])))


@pytest.mark.parametrize("name,args,slack", [
    ("one token", (1, 2, 3, 0, 0, [1], [4096]), 1.0),
    ("a batch of tokens", (64, 8, 2, 4, 4160, [1] * 64, [8191] * 64), 1.1),
    ("short prompts", (8, 8, 2, 0, 0, [2048, 1940, 1888, 1299, 1295, 1199, 1826, 1206],
                       [2048, 1940, 1888, 1299, 1295, 1199, 1826, 1206]), 1.1),
    ("a long prompt", (1, 8, 2, 0, 0, [16383], [16383]), 1.05),
    ("windows", (2, 8, 2, 4, 4160, [32768] * 2, [32768] * 2), 1.05),
    ("chunks", (4, 8, 2, 0, 0, [509] * 4, [65536, 51200, 40000, 36000]), 1.05),
    ("one long row among short ones", (256, 1, 2, 0, 0, [4096] + [16] * 255, [4096] + [16] * 255), 1.2),
])
def test_balance(run, name, args, slack):
    """The largest share of tiles is near the mean of tiles and items' starts."""
    P, joins, whole, mean, most, largest = run(*args)
    assert most <= slack * mean + 16, (name, P, joins, whole, mean, most, largest)


def test_divisor(tmp_path):
    """Divisions by multiplication, at multiples, their neighbours and the ends of the range."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    (tmp_path / "main.cpp").write_text(r"""
#include <stdio.h>
#include "prompt_schedule.h"
int main() {
  const int last = 0x7fffffff;
  for (int d = 1; d <= 65536; d += d < 2100 ? 1 : 61) {
    fade::PromptDivisor by;
    by.set(d);
    unsigned seed = d;
    for (int i = 0; i < 600; ++i) {
      seed = seed * 1664525u + 1013904223u;
      const int q = (int)(seed >> 1) / d, x = q * d;
      for (int y : {x, x - 1, (int)(seed >> 1), i, last - i})
        if (y >= 0 && by.of(y) != y / d) return printf("%d / %d\n", y, d), 1;
    }
  }
  return 0;
}
""")
    subprocess.run([gxx, "-O1", "-std=c++17", "-Wall", "-Werror",
                    f"-I{ROOT}/tiered_mixed_precision_gb300/csrc", f"-I{ROOT}/include",
                    str(tmp_path / "main.cpp"), "-o", str(tmp_path / "main")], check=True)
    r = subprocess.run([str(tmp_path / "main")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
