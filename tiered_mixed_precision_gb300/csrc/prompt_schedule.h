// Schedule of the prompt attention: how blocks of queries, and tiles of the tokens that they see, are
// dealt to the CTAs. Made on the host (and checked there by its test), followed on the device.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "fade.h"

#ifndef FADE_SCHED
#ifdef __CUDACC__
#define FADE_SCHED __host__ __device__ __forceinline__
#else
#define FADE_SCHED inline
#endif
#endif

namespace fade {

constexpr int kPromptTile = 128;   // tokens of a tile, and query rows of one
constexpr int kPromptSMs = 160;    // CTAs at most

// The rows of a call. Queries are the last q_len of a row's kv_len tokens.
struct PromptRows {
  int32_t q_len[FADE_MAX_BATCH], kv_len[FADE_MAX_BATCH];
  uint8_t order[FADE_MAX_BATCH];   // rows, the most tokens first
};

// What queries see: token j of position i's past if window is 0, j > i - window or j < sink.
struct Sight {
  int sink, window;   // window 0: sink 0, too
};

struct PromptShape {
  int B, H, G, log_g, Hq, n_q, n_kv;
  Sight sight;
  // 0 where a stride is 0 (a broadcast dimension): the tensor map's extent is 1 there
  int q_row, kv_row[2], kv_head[2];
};

struct PromptSchedule {
  int whole;   // items [0, whole) are taken whole, the others are the tail
  struct {
    int32_t item, tile;
  } start[kPromptSMs + 1];   // CTA c's share of the tail, up to that of CTA c + 1
  struct {
    int32_t item;
    int16_t first, last;   // the CTAs that share the item
  } join[kPromptSMs];
};

// A block of two query tiles of a unit, and the part of its tiles [begin, begin + n) at hand.
struct PromptItem {
  int b, h, tok0, active;   // first query token, query tiles with queries
  int off;                  // position of query token 0
  int p0, p1;               // positions of the block's first and last query
  int sinks, lo;            // tiles: 0 .. sinks - 1, then lo, lo + 1, ..
  int begin, n, all;
  FADE_SCHED int tile(int j) const {
    const int t = begin + j;
    return t < sinks ? t : lo + t - sinks;
  }
};
// The block of rank `rank` (0: a row's last queries) of row b, whole.
FADE_SCHED PromptItem prompt_block(const PromptShape& s, int b, int q_len, int kv_len, int rank) {
  const int per = kPromptTile >> s.log_g, blocks = (q_len + 2 * per - 1) >> (8 - s.log_g);
  PromptItem it;
  it.b = b;
  it.h = 0;
  it.begin = it.n = it.all = 0;
  if (rank >= blocks) return it;
  it.tok0 = (blocks - 1 - rank) * 2 * per;
  const int left = q_len - it.tok0;
  it.active = left > per ? 2 : 1;
  it.off = kv_len - q_len;
  it.p0 = it.off + it.tok0;
  it.p1 = it.p0 + (left < 2 * per ? left : 2 * per) - 1;
  const int first = it.p0 - s.sight.window + 1;
  it.lo = s.sight.window && first > 0 ? first / kPromptTile : 0;
  const int sinks = (s.sight.sink + kPromptTile - 1) / kPromptTile;
  it.sinks = sinks < it.lo ? sinks : it.lo;
  it.n = it.all = it.sinks + it.p1 / kPromptTile - it.lo + 1;
  return it;
}
// Items by rank, then row (in their order by length), then head.
FADE_SCHED PromptItem prompt_item(const PromptShape& s, const PromptRows& rows, int index) {
  const int units = s.B * s.H, rank = index / units, u = index - rank * units;
  const int row = u / s.H, b = rows.order[row];
  PromptItem it = prompt_block(s, b, rows.q_len[b], rows.kv_len[b], rank);
  it.h = u - row * s.H;
  return it;
}
// A CTA's items one after another: whole ones, forth and back over the CTAs so that the order by length
// evens out; then its share of the tail.
struct PromptWalk {
  int k = 0, item = -1, tile = 0;
  FADE_SCHED bool next(const PromptShape& s, const PromptRows& rows, const PromptSchedule& a, int P,
                       int c, PromptItem& it) {
    while (k * P < a.whole) {
      const int index = k * P + ((k & 1) ? P - 1 - c : c);
      ++k;
      if (index >= a.whole) continue;
      it = prompt_item(s, rows, index);
      if (it.n > 0) return true;
    }
    if (item < 0) {
      item = a.start[c].item;
      tile = a.start[c].tile;
    }
    const int last = a.start[c + 1].item, end = a.start[c + 1].tile;
    while (item < last || (item == last && tile < end)) {
      it = prompt_item(s, rows, item);
      it.begin = tile;
      it.n = (item == last ? end : it.all) - tile;
      ++item;
      tile = 0;
      if (it.n > 0) return true;
    }
    return false;
  }
};

constexpr int kShareTiles = 2;     // tiles of a share of an item at least
// What an item costs, in quarters of a tile of two query tiles: its tiles, and its start and end.
constexpr int kCostStart = 8, kCostTwo = 4, kCostOne = 3;

inline int prompt_tile_cost(const PromptItem& it) { return it.active == 2 ? kCostTwo : kCostOne; }
inline int prompt_cost(const PromptItem& it) {
  return it.all ? kCostStart + it.all * prompt_tile_cost(it) : 0;
}

// The schedule: `whole` items first, as many rounds over the CTAs as leave no CTA above the mean; the
// tail's tiles then fill every CTA up to the mean. Sets the CTAs that have work; returns the number of
// items that CTAs share.
inline int prompt_schedule(const PromptShape& s, const PromptRows& rows, int blocks, int sms,
                           PromptSchedule& a, int* ctas) {
  const int units = s.B * s.H, items = blocks * units;
  auto item = [&](int index) {
    const int b = rows.order[index % units / s.H];
    return prompt_block(s, b, rows.q_len[b], rows.kv_len[b], index / units);
  };
  long long total = 0, tiles = 0, load[kPromptSMs] = {}, then[kPromptSMs];
  for (int index = 0; index < items; index += s.H) {   // (the heads of a row cost the same)
    const PromptItem it = item(index);
    total += (long long)s.H * prompt_cost(it);
    tiles += (long long)s.H * it.all;
  }
  const int P = *ctas = (int)std::min<long long>(sms, std::max(tiles / kShareTiles, 1LL));
  const double mean = (double)total / P;
  long long placed = 0, work = 0;   // cost of the whole items; of the tail's tiles alone
  a.whole = 0;
  for (int k = 0, row = -1, cost = 0; (long long)k * P < items; ++k) {
    long long most = 0, sum = placed;
    std::copy(load, load + P, then);
    for (int c = 0; c < P && k * P + c < items; ++c) {
      const int index = k * P + c;
      if (index / s.H != row) {
        row = index / s.H;
        cost = prompt_cost(item(index));
      }
      long long& l = then[(k & 1) ? P - 1 - c : c];
      l += cost;
      sum += cost;
      most = std::max(most, l);
    }
    if ((double)most > mean) break;
    std::copy(then, then + P, load);
    placed = sum;
    a.whole = std::min((k + 1) * P, items);
  }
  for (int index = a.whole; index < items; ++index) {
    const PromptItem it = item(index);
    if (it.all) work += (long long)it.all * prompt_tile_cost(it);
  }
  // the tail: CTA c takes tiles worth mean - load[c], the items' starts spread over their tiles
  const double price = work ? (double)(total - placed) / work : 1.0;
  int at = a.whole, tile = 0, joins = 0, open = -1;
  double owed = 0;   // what the CTAs so far should have taken beyond what they took
  PromptItem it = at < items ? item(at) : PromptItem{};
  for (int c = 0; c < P; ++c) {
    a.start[c].item = at;
    a.start[c].tile = tile;
    owed += mean - (double)load[c];
    while (at < items) {
      if (it.all == 0) {
        if (++at < items) it = item(at);
        continue;
      }
      const double each = price * prompt_tile_cost(it);
      const int left = it.all - tile;
      int take = c + 1 == P ? left : (int)std::min<double>(left, owed / each + 0.5);
      if (take + kShareTiles > left) take = left;
      if (take < std::min(kShareTiles, left)) break;
      owed -= each * take;
      if (take < left || tile > 0) {   // shared with other CTAs
        if (open != at) {
          open = at;
          a.join[joins].item = at;
          a.join[joins].first = (int16_t)c;
          ++joins;
        }
        a.join[joins - 1].last = (int16_t)c;
      }
      if (take < left) {
        tile += take;
        break;
      }
      tile = 0;
      if (++at < items) it = item(at);
    }
  }
  a.start[P].item = at;
  a.start[P].tile = tile;
  return joins;
}

}  // namespace fade
