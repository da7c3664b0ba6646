// Schedule of the tree attention. Tiles are numbered row by row, KV head by KV head, block of query
// rows by block, FP16 tiles before middle tiles; every CTA takes consecutive ones. Everything is derived
// from the counts where it is needed, on the device by the kernel, so that a captured launch follows
// the cache (and on the host by its test).
//
// CTA c of P takes the tiles whose place on a line of costs lies in [X c / P, X (c + 1) / P): a block
// costs its tiles and a charge before them, X is all blocks' cost. A CTA lists its segments (its part
// of a block) in shared memory, kMaxSeg at most. With equal tiles alone it could have any number of them:
// beside long rows a CTA's share is hundreds of tiles, and blocks of short rows have one each. Blocks
// wholly inside a share cost charge + 1 at least, so a share of (kMaxSeg - 2) (charge + 1) holds; that
// is N + charge K <= (kMaxSeg - 2) P (charge + 1) for N tiles in K blocks. While a share is kMaxSeg - 2
// tiles or less, nothing is charged; else what the list needs, and kStartTiles at least, about what a
// segment's start costs (its Q, its FP16 rows, its epilogue, beside 1.3 us a tile): 64 rows, half of
// 16384 and half of 60 tokens, take 669 us with the least charge the list needs, 358 with 3, 304 with 4,
// 312 with 5, and 292 without the short rows.
#pragma once

#ifdef __CUDACC__
#define FADE_SCHED __host__ __device__ __forceinline__
#else
#define FADE_SCHED inline
#endif

namespace fade {

constexpr int kTok = 128;      // tokens of a tile
constexpr int kMaxSeg = 128;   // segments of a CTA at most
constexpr int kStartTiles = 4;   // the least charge

struct RowTiles {
  int n;        // nodes
  int blocks;   // blocks of query rows of a unit
  int f16;      // FP16 tiles
  int tiles;    // tiles of one block
};
// A row of n nodes, G query heads a KV head, `rows` query rows a block, held16 FP16 and n_mid middle
// tokens.
FADE_SCHED RowTiles make_row_tiles(int n, int G, int rows, int held16, int n_mid) {
  RowTiles r;
  r.n = n;
  r.blocks = (n * G + rows - 1) / rows;
  r.f16 = (held16 + n + kTok - 1) / kTok;
  r.tiles = r.f16 + (n_mid + kTok - 1) / kTok;
  return r;
}
// CTAs for at most K blocks where `wanted` would be taken: K is half of what they may list, so that what
// the list needs stays below a 60th of a CTA's tiles.
FADE_SCHED int tree_ctas(long long K, int wanted) {
  const long long least = (K + kMaxSeg / 2 - 1) / (kMaxSeg / 2);
  return (int)(least > wanted ? least : wanted);
}
// The tiles that P CTAs take without a charge; the charge for N tiles in K blocks (K <= P kMaxSeg / 2).
FADE_SCHED int tree_hold(int P) { return (kMaxSeg - 2) * P; }
FADE_SCHED int tree_charge(int N, int K, int P) {
  const int hold = tree_hold(P);
  if (N <= hold) return 0;
  const int least = (N - hold - 1) / (hold - K) + 1;
  return least > kStartTiles ? least : kStartTiles;
}
// Prefix sums of the rows: tiles and blocks of the rows before row b; `charge` makes them costs.
struct Rows {
  const int *tiles, *blocks;   // [B + 1]
  int B, charge;
  FADE_SCHED long long cost(int b) const { return tiles[b] + (long long)charge * blocks[b]; }
};
FADE_SCHED int row_of(const Rows& r, int g) {   // tiles[b] <= g < tiles[b + 1]
  int lo = 0, hi = r.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (r.tiles[mid + 1] > g) hi = mid; else lo = mid + 1;
  }
  return lo;
}
// The first tile of CTA c of P: without a charge, and with one.
FADE_SCHED int equal_start(int N, int P, int c) { return (int)((long long)N * c / P); }
FADE_SCHED int cta_start(const Rows& r, int P, int c) {
  if (r.charge == 0) return equal_start(r.tiles[r.B], P, c);
  const long long X = r.cost(r.B), x = X * c / P;
  if (x == X) return r.tiles[r.B];
  int lo = 0, hi = r.B - 1;   // the row whose costs hold x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (r.cost(mid + 1) > x) hi = mid; else lo = mid + 1;
  }
  const int blocks = r.blocks[lo + 1] - r.blocks[lo];
  const int tiles = (r.tiles[lo + 1] - r.tiles[lo]) / blocks;
  const int at = (int)(x - r.cost(lo)), blk = at / (tiles + r.charge);
  const int in = at - blk * (tiles + r.charge) - r.charge;
  return r.tiles[lo] + blk * tiles + (in > 0 ? in : 0);
}
// The CTA that takes tile g without a charge; the one that takes tile t of the block that begins at tile
// g0 of row b.
FADE_SCHED int equal_cta_of(int N, int P, int g) { return (int)((((long long)g + 1) * P - 1) / N); }
FADE_SCHED int cta_of(const Rows& r, int P, int b, int g0, int tiles, int t) {
  if (r.charge == 0) return equal_cta_of(r.tiles[r.B], P, g0 + t);
  const long long charges = (long long)r.blocks[b] + (g0 - r.tiles[b]) / tiles + 1;
  return (int)(((g0 + t + r.charge * charges + 1) * P - 1) / r.cost(r.B));
}

// The k-th block of query rows from the one that holds tile g: row b, its blk-th block, first tile
// g0; g0 >= g_end if it lies at or past tile g_end. row(b): the RowTiles of row b.
struct Place {
  int b, blk, g0;
  RowTiles rt;
};
template <class Row>
FADE_SCHED Place block_from(const Row& row, const Rows& r, int H, int g, int k, int g_end) {
  Place p;
  p.b = row_of(r, g);
  p.rt = row(p.b);
  p.blk = (g - r.tiles[p.b]) / p.rt.tiles;
  while (p.blk + k >= H * p.rt.blocks) {   // on to the row that holds it
    k -= H * p.rt.blocks - p.blk;
    p.blk = 0;
    if (r.tiles[++p.b] >= g_end) {
      p.g0 = g_end;
      return p;
    }
    p.rt = row(p.b);
  }
  p.blk += k;
  p.g0 = r.tiles[p.b] + p.blk * p.rt.tiles;
  return p;
}

}  // namespace fade
