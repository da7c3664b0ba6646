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
// x / d for 0 <= x < 2^31 by a multiplication (Granlund and Montgomery): a division by what only the
// host knows takes longer than the rest of an item, and a CTA's next item is waited for (8 short prompts
// of d = 64: attention 145 -> 136 us, mass 95.5 -> 94).
struct PromptDivisor {
  int d, shift;
  uint32_t mul;
  void set(int by) {
    d = by;
    for (shift = 0; (1LL << shift) < by; ++shift) {
    }
    mul = (uint32_t)((((1ULL << shift) - by) << 32) / by + 1);
  }
  FADE_SCHED int of(int x) const {
#ifdef __CUDA_ARCH__
    const uint32_t high = __umulhi((uint32_t)x, mul);
#else
    const uint32_t high = (uint32_t)(((uint64_t)(uint32_t)x * mul) >> 32);
#endif
    return (int)((high + (uint32_t)x) >> shift);
  }
};
struct PromptUnits {
  PromptDivisor all, heads;   // by B H, by H
  void set(const PromptShape& s) {
    all.set(s.B * s.H);
    heads.set(s.H);
  }
};
// Items by rank, then row (in their order by length), then head.
FADE_SCHED PromptItem prompt_item(const PromptShape& s, const PromptRows& rows, const PromptUnits& n,
                                  int index) {
  const int rank = n.all.of(index), u = index - rank * n.all.d;
  const int row = n.heads.of(u), b = rows.order[row];
  PromptItem it = prompt_block(s, b, rows.q_len[b], rows.kv_len[b], rank);
  it.h = u - row * s.H;
  return it;
}
inline PromptItem prompt_item(const PromptShape& s, const PromptRows& rows, int index) {
  PromptUnits n;
  n.set(s);
  return prompt_item(s, rows, n, index);
}
// Two tiles of 128 keys of a unit, and the query tiles [begin, begin + n) that meet them; `all` of them
// do, from the first-th on.
struct MassItem {
  int b, h, k0;     // first key
  int off, q_len;   // position of query token 0; the row's queries
  int first, begin, n, all;
};
// Items by pair of key tiles, then row (in their order by length), then head.
FADE_SCHED MassItem mass_item(const PromptShape& s, const PromptRows& rows, const PromptUnits& n,
                              int index) {
  const int pair = n.all.of(index), u = index - pair * n.all.d, row = n.heads.of(u);
  const int per = kPromptTile >> s.log_g;
  MassItem it;
  it.b = rows.order[row];
  it.h = u - row * s.H;
  it.k0 = pair * 2 * kPromptTile;
  it.q_len = rows.q_len[it.b];
  const int kv_len = rows.kv_len[it.b];
  it.off = kv_len - it.q_len;
  const int from = it.k0 > it.off ? it.k0 - it.off : 0;   // queries before their keys see none
  int to = it.q_len - 1;
  if (s.sight.window && it.k0 >= s.sight.sink) {
    const int last = it.k0 + 2 * kPromptTile - 1 + s.sight.window - 1 - it.off;
    if (last < to) to = last;
  }
  it.begin = 0;
  it.first = from / per;
  it.n = it.all = it.k0 < kv_len && from <= to ? to / per - it.first + 1 : 0;
  return it;
}

inline MassItem mass_item(const PromptShape& s, const PromptRows& rows, int index) {
  PromptUnits n;
  n.set(s);
  return mass_item(s, rows, n, index);
}

// A CTA's items one after another: whole ones, forth and back over the CTAs so that the order by length
// evens out; then its share of the tail. item_at: the whole item of an index.
template <class Item>
struct PromptWalk {
  int k = 0, item = -1, tile = 0;
  template <class F>
  FADE_SCHED bool next(const PromptSchedule& a, int P, int c, const F& item_at, Item& it) {
    while (k * P < a.whole) {
      const int index = k * P + ((k & 1) ? P - 1 - c : c);
      ++k;
      if (index >= a.whole) continue;
      it = item_at(index);
      if (it.n > 0) return true;
    }
    if (item < 0) {
      item = a.start[c].item;
      tile = a.start[c].tile;
    }
    const int last = a.start[c + 1].item, end = a.start[c + 1].tile;
    while (item < last || (item == last && tile < end)) {
      it = item_at(item);
      it.begin = tile;
      it.n = (item == last ? end : it.all) - tile;
      ++item;
      tile = 0;
      if (it.n > 0) return true;
    }
    return false;
  }
};

constexpr int kShareTiles = 2;   // tiles of a share of an item at least

// An item's tiles, what one costs, and what the item's start costs.
struct PromptWork {
  int tiles, each, start;
};
// Deals items 0 .. items - 1 (work: of an index; `group` consecutive ones cost the same) to at most sms
// CTAs. rounds: whole items first, as many rounds over the CTAs as leave no CTA above the mean. The
// others' tiles then fill every CTA up to the mean, an item's start charged to who takes its first tile.
// Sets the CTAs that have work; returns the number of items that CTAs share.
template <class F>
int prompt_deal(int items, int group, int sms, bool rounds, const F& work, PromptSchedule& a,
                int* ctas) {
  long long alone = 0, tiles = 0, load[kPromptSMs] = {}, then[kPromptSMs];
  for (int index = 0; index < items; index += group) {
    const PromptWork w = work(index);
    alone += (long long)group * w.tiles * w.each;
    tiles += (long long)group * w.tiles;
  }
  const int P = *ctas = (int)std::min<long long>(sms, std::max(tiles / kShareTiles, 1LL));
  // (shares of a few tiles all have their start: only beside long ones does it count)
  auto start_of = [&](const PromptWork& w) { return (int)std::min<long long>(w.start, alone / P / 4); };
  auto cost_of = [&](const PromptWork& w) {
    return w.tiles ? start_of(w) + (long long)w.tiles * w.each : 0;
  };
  long long total = 0;
  for (int index = 0; index < items; index += group) total += group * cost_of(work(index));
  const double mean = (double)total / P;
  long long cost = 0;
  a.whole = 0;
  for (int k = 0, last = -1; rounds && (long long)k * P < items; ++k) {
    long long most = 0;
    std::copy(load, load + P, then);
    for (int c = 0; c < P && k * P + c < items; ++c) {
      const int index = k * P + c;
      if (index / group != last) {
        last = index / group;
        cost = cost_of(work(index));
      }
      long long& l = then[(k & 1) ? P - 1 - c : c];
      l += cost;
      most = std::max(most, l);
    }
    if ((double)most > mean) break;
    std::copy(then, then + P, load);
    a.whole = std::min((k + 1) * P, items);
  }
  // the tail: CTA c takes tiles worth mean - load[c]
  int at = a.whole, tile = 0, joins = 0, open = -1;
  double owed = 0;   // what the CTAs so far should have taken beyond what they took
  PromptWork w = at < items ? work(at) : PromptWork{};
  for (int c = 0; c < P; ++c) {
    a.start[c].item = at;
    a.start[c].tile = tile;
    owed += mean - (double)load[c];
    while (at < items) {
      if (w.tiles == 0) {
        if (++at < items) w = work(at);
        continue;
      }
      const int left = w.tiles - tile, start = tile == 0 ? start_of(w) : 0;
      int take = c + 1 == P ? left : (int)std::min<double>(left, (owed - start) / w.each + 0.5);
      if (take + kShareTiles > left) take = left;
      if (take < std::min(kShareTiles, left)) break;
      owed -= start + (double)w.each * take;
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
      if (++at < items) w = work(at);
    }
  }
  a.start[P].item = at;
  a.start[P].tile = tile;
  return joins;
}

// What an item of the attention costs, in quarters of a tile of two query tiles: its tiles, and its
// start and end.
constexpr int kCostStart = 12, kCostTwo = 4, kCostOne = 3;

inline int prompt_schedule(const PromptShape& s, const PromptRows& rows, int blocks, int sms,
                           PromptSchedule& a, int* ctas) {
  PromptUnits n;
  n.set(s);
  auto work = [&](int index) {
    const PromptItem it = prompt_item(s, rows, n, index);
    return PromptWork{it.all, it.all == 0 || it.active == 2 ? kCostTwo : kCostOne, kCostStart};
  };
  return prompt_deal(blocks * s.B * s.H, s.H, sms, true, work, a, ctas);
}
inline int mass_schedule(const PromptShape& s, const PromptRows& rows, int sms, PromptSchedule& a,
                         int* ctas) {
  const int pairs = (s.n_kv + 2 * kPromptTile - 1) / (2 * kPromptTile);
  // a pair's first 2 G tiles hide some keys from some queries, which costs half as much again; so do
  // all of a pair with sinks and other tokens (one of its two key tiles, mostly)
  PromptUnits n;
  n.set(s);
  auto work = [&](int index) {
    const MassItem it = mass_item(s, rows, n, index);
    return PromptWork{it.all, s.sight.window && it.k0 < s.sight.sink ? 10 : 8, 16 + 8 * s.G};
  };
  return prompt_deal(pairs * s.B * s.H, s.H, sms, false, work, a, ctas);
}

}  // namespace fade
