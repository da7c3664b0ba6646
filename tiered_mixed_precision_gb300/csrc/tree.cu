// Drafted tokens around the attention call: the tree's masks and positions, and the commit of the
// accepted path (its tokens appended with the demotions they cause, its attention mass added to
// the scores). Page "FADE：面向LLM推理的注意力感知分层KV缓存压缩技术", §第一层 and §第二层 (FP16 recent
// window, mid-aged tokens quantised), §四种驱逐策略详解 1 and 2 (H2O, EMA scores).
#include <math.h>

#include "tree.cuh"

namespace fade {

fade_status_t validate_tree(const fade_config_t* c, int32_t T) {
  fade_status_t st = validate_config(c);
  if (st) return st;
  if (T < 1 || T > FADE_TREE_MAX_NODES)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "%d tree nodes outside [1, %d]", T,
                     FADE_TREE_MAX_NODES);
  return FADE_OK;
}

fade_status_t validate_heads(const fade_heads_t* h, const char* name) {
  if (!h || !h->x) return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL %s", name);
  if ((reinterpret_cast<uintptr_t>(h->x) & 15) || h->row_stride % 8 || h->token_stride % 8 ||
      h->head_stride % 8)
    return set_error(FADE_ERR_INVALID_ARGUMENT,
                     "%s: vectors must start 16-byte aligned (strides in multiples of 8 elements)",
                     name);
  return FADE_OK;
}

fade_status_t validate_tree_layer(const fade_config_t* c, const fade_layer_t* L) {
  fade_status_t st = validate_layer(c, L);
  if (st) return st;
  uintptr_t any = 0;
  for (const void* p : {(const void*)L->mid_k_scales[0], (const void*)L->mid_k_scales[1],
                        (const void*)L->mid_v_scales[0], (const void*)L->mid_v_scales[1],
                        (const void*)L->sink_k, (const void*)L->sink_v, (const void*)L->recent_k,
                        (const void*)L->recent_v, (const void*)L->mid_k_codes[0],
                        (const void*)L->mid_k_codes[1], (const void*)L->mid_v_codes[0],
                        (const void*)L->mid_v_codes[1]})
    any |= reinterpret_cast<uintptr_t>(p);
  if (any & 15)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "the layer's K and V buffers must be 16-byte aligned");
  if (!aligned(L->sink_scores, 4) || !aligned(L->mid_scores[0], 4) || !aligned(L->mid_scores[1], 4) ||
      !aligned(L->recent_scores, 4) || !aligned(L->meta, 4) || !aligned(L->status, 4))
    return set_error(FADE_ERR_INVALID_ARGUMENT,
                     "the layer's scores, meta and status must be 4-byte aligned");
  return FADE_OK;
}

namespace {

// One CTA per row, one thread per node. Pointer doubling: after k rounds a node's mask holds its
// 2^k nearest ancestors and `up` is the 2^k-th, so six rounds reach every root of 64 nodes (a walk
// up the parents would take 64 dependent shared loads on a chain).
__global__ void __launch_bounds__(FADE_TREE_MAX_NODES)
    tree_layout_kernel(int T, const int32_t* __restrict__ parents,
                       const int32_t* __restrict__ n_nodes, const int32_t* __restrict__ base_pos,
                       uint64_t* __restrict__ mask, int32_t* __restrict__ pos) {
  __shared__ unsigned long long sm[FADE_TREE_MAX_NODES];
  __shared__ int su[FADE_TREE_MAX_NODES];
  const int b = blockIdx.x, i = threadIdx.x;
  const int n = n_nodes ? min(max(n_nodes[b], 0), T) : T;
  const bool live = i < n;
  int up = live ? parents[(size_t)b * T + i] : -1;
  if (up < 0 || up >= i) up = -1;
  unsigned long long m = live ? 1ull << i : 0ull;
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    sm[i] = m;
    su[i] = up;
    __syncthreads();
    if (up >= 0) {
      m |= sm[up];
      up = su[up];
    }
    __syncthreads();
  }
  if (i < T) {
    mask[(size_t)b * T + i] = m;
    pos[(size_t)b * T + i] = base_pos[b] + (live ? __popcll(m) - 1 : 0);
  }
}

// ----------------------------------------------------------------- commit
// The path's attention mass. Mathematics: with the path's nodes 0 .. n-1 and their G query rows as
// columns c (node i = c / G), token j's score becomes decay^k score + sum_c w_c exp(s_jc - lse_c),
// k the nodes that see it (all n; n - j for the j-th path token, which starts at 0), w_c = 1 and
// decay = 1 (H2O) or w_c = (1 - delta) delta^(n-1-i) and decay = delta (EMA): the accumulation node
// by node, written as one sum.
//
// Products on mma.sync: 16 tokens are the rows, 8 columns the columns of an instruction. Few
// columns and every key read once make this a stream over the codes, not a contraction for tcgen05;
// and it keeps the keys exact: codes are exact fp16 integers (halved), each 32-channel group is
// summed on its own and meets its scale (with log2 e / sqrt d) in fp32. A column's weight goes into
// its exponent: w exp(s - lse) = 2^(s' - (lse' - log2 w)). Thread (row g = lane / 4, t = lane % 4)
// holds channels 8t .. 8t+7 of every group of rows g and g + 8, as the pairs (8t+i, 8t+i+4) its
// code word unpacks into; the columns are laid out in shared memory in the same order.
//
// Measured at 4 rows of 16384 middle tokens, 8 KV heads of d = 128, INT4 keys, paths of 1 to 6
// nodes of 4 queries: 28 us for 43 MB (the copy rate's 6 us). Instruction issue bounds it,
// unpacking first and the products next; equal stretches of cost rather than of tiles took 10 us
// off (paths of different lengths, and a second wave of CTAs), weights in the exponents 5.
constexpr int kScoreCols = 64;   // columns staged at a time: longer paths take more passes

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t sub_h2(uint32_t x, uint32_t y) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Channels 8t .. 8t+7 of a group as the pairs (i, i + 4), i = 0 .. 3: half the codes of a middle row's
// word, or the values of an fp16 row.
template <int KB>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&p)[4]) {
  if constexpr (KB == 4) {
    const uint32_t h = w >> 8;
    p[0] = sub_h2((w & 0x000f000fu) ^ 0x60086008u, 0x60086008u);
    p[1] = sub_h2((w & 0x00f000f0u) ^ 0x50805080u, 0x50805080u);
    p[2] = sub_h2((h & 0x000f000fu) ^ 0x60086008u, 0x60086008u);
    p[3] = sub_h2((h & 0x00f000f0u) ^ 0x50805080u, 0x50805080u);
  } else {
    w |= (w >> 8) << 16;   // crumbs 0..3 in the low half, 4..7 in the high one
    p[0] = sub_h2((w & 0x00030003u) ^ 0x60026002u, 0x60026002u);
    p[1] = sub_h2((w & 0x000c000cu) ^ 0x58085808u, 0x58085808u);
    p[2] = sub_h2((w & 0x00300030u) ^ 0x50205020u, 0x50205020u);
    p[3] = sub_h2((w & 0x00c000c0u) ^ 0x48804880u, 0x48804880u);
  }
}
__device__ __forceinline__ void value_pairs(uint4 x, uint32_t (&p)[4]) {
  p[0] = prmt(x.x, x.z, 0x5410);
  p[1] = prmt(x.x, x.z, 0x7632);
  p[2] = prmt(x.y, x.w, 0x5410);
  p[3] = prmt(x.y, x.w, 0x7632);
}

// A warp's tiles come through a ring of kScoreStages in shared memory of its own (cp.async), since a
// tile is little work beside the latency of its 1 KB of codes. A row's 16-byte chunks are stored
// xor-ed with the row, so that the 32 words a warp reads lie in 32 banks.
constexpr int kScoreStages = 3;
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// The tokens of a path of n_path that become sinks, and those that the ring then demotes.
struct PathPlan {
  int to_sink, dem;
};
__device__ __forceinline__ PathPlan path_plan(const TreeArgs& a, const int32_t* m, int n_path) {
  PathPlan p;
  p.to_sink = min(max(a.S - m[FADE_META_N_SINK], 0), n_path);
  p.dem = max(0, m[FADE_META_N_RECENT] + n_path - p.to_sink - a.W);
  return p;
}
// Whether the commit takes a unit's path: its counts index the tiers and the middle tier holds the
// demotions (a captured commit may be replayed past what the host checked). Both kernels ask, so that a
// unit that is refused keeps its scores, too.
__device__ __forceinline__ bool takes_path(const TreeArgs& a, const int32_t* m, int n_path) {
  const int n_sink = m[FADE_META_N_SINK], n_mid = m[FADE_META_N_MID];
  const int n_rec = m[FADE_META_N_RECENT], head = m[FADE_META_HEAD], cur = m[FADE_META_CUR];
  return n_sink >= 0 && n_sink <= a.S && n_rec >= 0 && n_rec <= a.W && head >= 0 && head < a.W &&
         (cur & ~1) == 0 && n_mid >= 0 && n_mid <= a.C - path_plan(a, m, n_path).dem;
}

// What a CTA takes: row b's tiles cost kTileCost + 1 a block of eight columns each (a pass over the
// tile's codes, then two products a group a block), the costs of all rows and heads form one line,
// and every CTA takes an equal stretch of it. Paths differ in length, so equal tiles would not be
// equal work.
constexpr int kTileCost = 2;
struct ScoreRow {
  int n_sink, n_mid, n_rec;
  int mid_tiles, tiles, cost;
};
__device__ __forceinline__ ScoreRow score_row(const TreeArgs& a, int b, int n_path) {
  const int32_t* m = a.meta + (size_t)b * a.H * FADE_META_FIELDS;   // a row's heads agree
  ScoreRow r;
  r.n_sink = m[FADE_META_N_SINK];
  r.n_mid = m[FADE_META_N_MID];
  r.n_rec = m[FADE_META_N_RECENT];
  r.mid_tiles = (r.n_mid + 15) / 16;
  r.tiles = n_path && takes_path(a, m, n_path)
                ? r.mid_tiles + (r.n_sink + r.n_rec + n_path + 15) / 16 : 0;
  const int cols = n_path * a.G;
  r.cost = (cols + kScoreCols - 1) / kScoreCols * kTileCost + (cols + 7) / 8;
  return r;
}

template <int D, int KB>
__global__ void __launch_bounds__(256, 2) tree_scores_kernel(TreeArgs a, RowLens lens, int policy,
                                                          float delta,
                                                          const float* __restrict__ lse,
                                                          const int32_t* __restrict__ path,
                                                          float* __restrict__ path_sc) {
  constexpr int GR = D / 32, ROW = D * KB / 8, CH = ROW / 16;   // groups, bytes and chunks of a row
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kScale = kLog2e * (D == 64 ? 0.125f : 0.08838834764831845f);   // log2 e / sqrt D
  struct Stage {
    uint8_t codes[16][ROW];
    uint16_t scales[16][GR];
    float scores[16];
  };
  __shared__ uint4 sq[kScoreCols][GR][4];   // column's pairs of group, t
  __shared__ float sl[kScoreCols];          // lse of the column less its weight's logarithm, base 2
  extern __shared__ __align__(16) uint8_t ring_raw[];
  __shared__ long long pre[FADE_MAX_BATCH + 1];   // costs of the rows before
  __shared__ long long wsum[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  Stage* ring = reinterpret_cast<Stage*>(ring_raw) + warp * kScoreStages;
  {
    const int b = threadIdx.x;   // B <= 256
    long long v = 0;
    if (b < a.B && lens.v[b]) {
      const ScoreRow r = score_row(a, b, lens.v[b]);
      v = (long long)a.H * r.tiles * r.cost;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += wsum[w];
    pre[b + 1] = v;
    if (b == 0) pre[0] = 0;
    __syncthreads();
  }
  const long long x0 = pre[a.B] * blockIdx.x / gridDim.x;
  const long long x1 = pre[a.B] * (blockIdx.x + 1) / gridDim.x;
  const float decay = policy == FADE_EVICT_H2O ? 1.f : delta;
  const float gain = policy == FADE_EVICT_H2O ? 1.f : 1.f - delta;
  for (int b = 0; b < a.B; ++b) {
    if (pre[b + 1] <= x0 || pre[b] == pre[b + 1]) continue;
    if (pre[b] >= x1) break;
    const int n_path = lens.v[b], cols = n_path * a.G;
    const ScoreRow sr = score_row(a, b, n_path);
    // the row's tiles of 16 middle tokens, then of 16 FP16 tokens (sinks, ring, path), head by head;
    // a CTA's warps take its tiles of a head in turn
    const int mid_tiles = sr.mid_tiles, n_mid = sr.n_mid;
    const int n_sink = sr.n_sink, n_rec = sr.n_rec, n16 = n_sink + n_rec + n_path;
    const int first_tile = (int)((max(x0 - pre[b], 0ll) + sr.cost - 1) / sr.cost);
    const int end_tile = (int)((min(x1, pre[b + 1]) - pre[b] + sr.cost - 1) / sr.cost);
    float keep = 1.f;
    for (int e = 0; e < n_path; ++e) keep *= decay;
    for (int at_tile = first_tile; at_tile < end_tile;) {
      const int h = at_tile / sr.tiles, unit = b * a.H + h;
      const int tile0 = at_tile - h * sr.tiles, tile1 = min(sr.tiles, end_tile - h * sr.tiles);
      at_tile = h * sr.tiles + tile1;
      if (!takes_path(a, a.meta + (size_t)unit * FADE_META_FIELDS, n_path)) continue;   // uniform
      const int head = a.meta[unit * FADE_META_FIELDS + FADE_META_HEAD];
      const int cur = a.meta[unit * FADE_META_FIELDS + FADE_META_CUR];
      const uint8_t* codes = a.mk[cur] + (size_t)unit * a.C * ROW;
      const uint16_t* scales = a.mks[cur] + (size_t)unit * a.C * GR;
      float* scores = a.mid_sc[cur] + (size_t)unit * a.C;
      // a middle tile into its stage (rows past the tier lie within the unit's stride, a multiple
      // of 64)
      auto fetch = [&](int tile) {
        if (tile < min(tile1, mid_tiles)) {
          Stage& st = ring[((tile - tile0) >> 3) % kScoreStages];
          const size_t row = (size_t)16 * tile;
#pragma unroll
          for (int i = lane; i < 16 * CH; i += 32) {
            const int rr = i / CH, c = i % CH;
            cp_async16(smem_u32(&st.codes[rr][16 * (c ^ ((rr >> 1) & (CH - 1)))]),
                       codes + (row + rr) * ROW + 16 * c);
          }
          constexpr int SW = 16 * GR / 2;   // words of the tile's scales
#pragma unroll
          for (int i = lane; i < SW; i += 32)
            cp_async4(smem_u32(&st.scales[0][0]) + 4 * i, scales + row * GR + 2 * i);
          if (lane < 16) cp_async4(smem_u32(&st.scores[lane]), scores + row + lane);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      for (int c0 = 0; c0 < cols; c0 += kScoreCols) {
        const int n = min(kScoreCols, cols - c0);
        for (int i = 0; i < kScoreStages - 1; ++i) fetch(tile0 + warp + 8 * i);
        __syncthreads();   // the columns before are read
        for (int i = threadIdx.x; i < (n + 7) / 8 * 8 * GR * 4; i += 256) {
          // (columns past the last repeat it with an offset of inf, which adds nothing to the sum;
          // zeros would add NaN where they meet an infinite key)
          const int c = i / (GR * 4), gr = (i / 4) % GR, col = min(c0 + c, cols - 1);
          const int node = tree_node(a, path, b, col >> a.log_g);
          const size_t q = (((size_t)b * a.T + node) * a.Hq + h * a.G + (col & (a.G - 1)));
          uint32_t p[4];
          value_pairs(
              __ldg(reinterpret_cast<const uint4*>(a.q + q * D + 32 * gr + 8 * (i & 3))), p);
          sq[c][gr][i & 3] = make_uint4(p[0], p[1], p[2], p[3]);
          if (gr == 0 && (i & 3) == 0) {
            float wc = gain;
            for (int e = col >> a.log_g; e < n_path - 1; ++e) wc *= decay;
            sl[c] = c0 + c < cols ? fmaf(lse[q], kLog2e, -log2f(wc)) : INFINITY;
          }
        }
        __syncthreads();
#pragma unroll 1
        for (int tile = tile0 + warp; tile < tile1; tile += 8) {
          fetch(tile + 8 * (kScoreStages - 1));
          asm volatile("cp.async.wait_group %0;" ::"n"(kScoreStages - 1) : "memory");
          __syncwarp();
          const bool mid = tile < mid_tiles;
          const Stage& st = ring[((tile - tile0) >> 3) % kScoreStages];
          // rows g and g + 8 of the tile: their pairs and scales (twice, the codes are halved), the
          // score and its place, the first column (less c0 and 2t) whose node sees the token
          uint32_t k[2][GR][4];
          float sc[2][GR], old[2], *at[2];
          int first[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            first[r] = 0;
            if (mid) {
              at[r] = 16 * tile + row < n_mid ? scores + 16 * tile + row : nullptr;
              old[r] = st.scores[row];
#pragma unroll
              for (int e = 0; e < GR; ++e) {
                const int byte = e * (4 * KB) + t * KB, c = byte / 16;
                const uint8_t* w = &st.codes[row][16 * (c ^ ((row >> 1) & (CH - 1))) + byte % 16];
                code_pairs<KB>(KB == 4 ? *reinterpret_cast<const uint32_t*>(w)
                                       : *reinterpret_cast<const uint16_t*>(w),
                               k[r][e]);
                sc[r][e] = 2.f * kScale * h2f(st.scales[row][e]);
              }
            } else {
              const int i = 16 * (tile - mid_tiles) + row, j = min(i, n16 - 1);
              const uint16_t* x;
              if (j < n_sink) {
                x = a.sink_k + ((size_t)unit * a.S + j) * D;
                at[r] = a.sink_sc + (size_t)unit * a.S + j;
              } else if (j < n_sink + n_rec) {
                const size_t slot = (size_t)unit * a.W + (head + (j - n_sink)) % a.W;
                x = a.rec_k + slot * D;
                at[r] = a.rec_sc + slot;
              } else {
                const int i_path = j - n_sink - n_rec;
                first[r] = (i_path << a.log_g) - c0 - 2 * t;
                x = a.tk.x + b * a.tk.row_stride + h * a.tk.head_stride +
                    tree_node(a, path, b, i_path) * a.tk.token_stride;
                at[r] = path_sc + (size_t)unit * a.T + i_path;
              }
              // a path token starts at 0
              old[r] = c0 == 0 && j >= n_sink + n_rec ? 0.f : *at[r];
              if (i != j) at[r] = nullptr;
#pragma unroll
              for (int e = 0; e < GR; ++e) {
                value_pairs(*reinterpret_cast<const uint4*>(x + 32 * e + 8 * t), k[r][e]);
                sc[r][e] = kScale;
              }
            }
          }
          float sum[2] = {0.f, 0.f};
#pragma unroll 1
          for (int nb = 0; nb < n; nb += 8) {
            float s[4] = {};
#pragma unroll
            for (int e = 0; e < GR; ++e) {
              const uint4 q = sq[nb + g][e][t];   // column g of the eight: the B operand's column
              float d[4] = {};
              const uint32_t a0[4] = {k[0][e][0], k[1][e][0], k[0][e][1], k[1][e][1]};
              const uint32_t a1[4] = {k[0][e][2], k[1][e][2], k[0][e][3], k[1][e][3]};
              mma_16816(d, a0, q.x, q.y);
              mma_16816(d, a1, q.z, q.w);
#pragma unroll
              for (int v = 0; v < 4; ++v) s[v] = fmaf(d[v], sc[v >> 1][e], s[v]);
            }
            const float2 off = *reinterpret_cast<const float2*>(&sl[nb + 2 * t]);
#pragma unroll
            for (int v = 0; v < 4; ++v) {   // row g + 8 (v / 2), column 2t + v % 2
              const float p = exp2_approx(s[v] - (v & 1 ? off.y : off.x));
              if (nb + (v & 1) >= first[v >> 1]) sum[v >> 1] += p;
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float v = sum[r];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            // the first pass decays the score, later ones add to it
            if (t == 0 && at[r]) *at[r] = c0 == 0 ? fmaf(old[r], keep, v) : old[r] + v;
          }
          __syncwarp();   // the stage is read: the next round fills it
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
    }
  }
}

// One CTA of 8 warps per unit. The unit's ring followed by the path's non-sink tokens is one
// sequence; its first `dem` entries leave for the middle tier (whether they came from the ring or
// from the path), the rest end in ring slots head, head + 1, ... Demotions first (two warps a
// token, K and V side by side), then, after a barrier, the new tokens into the slots they freed.
template <int D, int KB, int VB>
__global__ void __launch_bounds__(256) tree_commit_kernel(TreeArgs a, RowLens lens,
                                                          const int32_t* __restrict__ path,
                                                          const float* __restrict__ path_sc) {
  const int h = blockIdx.x, b = blockIdx.y, unit = b * a.H + h;
  const int n_path = lens.v[b];
  if (n_path == 0) return;   // uniform per CTA, as are the returns below
  int32_t* m = a.meta + unit * FADE_META_FIELDS;
  const int n_sink = m[FADE_META_N_SINK], n_mid = m[FADE_META_N_MID];
  const int n_rec = m[FADE_META_N_RECENT], head = m[FADE_META_HEAD], cur = m[FADE_META_CUR];
  const auto [to_sink, dem] = path_plan(a, m, n_path);
  if (!takes_path(a, m, n_path)) {
    if (threadIdx.x == 0) record_status(a.status, kCheckTreeSlot);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0)
    for (int i = lane; i < n_path; i += 32) {
      const int node = path[(size_t)b * a.T + i];
      if (node < 0 || node >= a.T) record_status(a.status, kCheckTreePath);
    }
  auto tree_row = [&](const fade_heads_t& t, int i) {
    return t.x + b * t.row_stride + tree_node(a, path, b, i) * t.token_stride +
           h * t.head_stride;
  };
  for (int w = warp; w < 2 * dem; w += 8) {
    const int i = w >> 1, isv = w & 1;
    const size_t mrow = (size_t)unit * a.C + n_mid + i;
    const bool old = i < n_rec;
    const size_t rrow = (size_t)unit * a.W + (head + i) % a.W;
    const int pi = to_sink + i - n_rec;
    if (!isv) {
      warp_quantize_row<D, KB>(old ? a.rec_k + rrow * D : tree_row(a.tk, pi),
                               a.mk[cur] + mrow * (D * KB / 8), a.mks[cur] + mrow * (D / kGroup));
      if (lane == 0)
        a.mid_sc[cur][mrow] =
            old ? a.rec_sc[rrow] : (path_sc ? path_sc[(size_t)unit * a.T + pi] : 0.f);
    } else {
      const uint16_t* x = old ? a.rec_v + rrow * D : tree_row(a.tv, pi);
      uint16_t* scl = a.mvs[cur] + mrow * (D / kGroup);
      if (a.pq_cb)
        warp_pq_encode_row<D>(x, a.pq_cb, a.mv[cur] + mrow * (D / 4), scl);
      else
        warp_quantize_row<D, VB>(x, a.mv[cur] + mrow * (D * VB / 8), scl);
    }
  }
  __syncthreads();   // the demoted slots and every count have been read
  for (int i = warp; i < n_path; i += 8) {
    const int seq = n_rec + i - to_sink;   // the token's place in the ring's sequence
    if (i >= to_sink && seq < dem) continue;   // demoted above
    const size_t row = i < to_sink ? (size_t)unit * a.S + n_sink + i
                                   : (size_t)unit * a.W + (head + seq) % a.W;
    uint16_t* dk = (i < to_sink ? a.sink_k : a.rec_k) + row * D;
    uint16_t* dv = (i < to_sink ? a.sink_v : a.rec_v) + row * D;
    const uint16_t *sk = tree_row(a.tk, i), *sv = tree_row(a.tv, i);
    if (lane < D / 8)
      *reinterpret_cast<uint4*>(dk + 8 * lane) = *reinterpret_cast<const uint4*>(sk + 8 * lane);
    else if (lane >= 16 && lane - 16 < D / 8)
      *reinterpret_cast<uint4*>(dv + 8 * (lane - 16)) =
          *reinterpret_cast<const uint4*>(sv + 8 * (lane - 16));
    if (lane == 0)
      (i < to_sink ? a.sink_sc : a.rec_sc)[row] =
          path_sc ? path_sc[(size_t)unit * a.T + i] : 0.f;
  }
  if (threadIdx.x == 0) {
    m[FADE_META_N_SINK] = n_sink + to_sink;
    m[FADE_META_N_MID] = n_mid + dem;
    m[FADE_META_N_RECENT] = n_rec + n_path - to_sink - dem;
    m[FADE_META_HEAD] = (head + dem) % a.W;
  }
}

template <int D, int KB>
fade_status_t launch_scores(const fade_config_t* c, const TreeArgs& a, const RowLens& lens,
                            long long tiles, const float* lse, const int32_t* path, float* path_sc,
                            cudaStream_t st) {
  // two CTAs an SM (152 SMs; three measured the same), each with at least one tile a warp
  const long long most = (tiles + 7) / 8, fill = 2 * 152;
  constexpr int kRing = 8 * kScoreStages * 16 * (D * KB / 8 + D / 32 * 2 + 4);
  static_assert(kRing + kScoreCols * (D / 32 * 64 + 4) + 8 * (FADE_MAX_BATCH + 9) <= 48 * 1024,
                "the default shared memory");
  tree_scores_kernel<D, KB>
      <<<(unsigned)(fill < most ? fill : most), 256, kRing, st>>>(
          a, lens, c->policy, c->ema_decay, lse, path, path_sc);
  return launch_status("fade_tree_commit scores");
}

template <int D, int KB, int VB>
fade_status_t launch_commit(const fade_config_t* c, const TreeArgs& a, const RowLens& lens,
                            const int32_t* path, const float* path_sc, cudaStream_t st) {
  tree_commit_kernel<D, KB, VB>
      <<<dim3(c->num_kv_heads, c->batch), 256, 0, st>>>(a, lens, path, path_sc);
  return launch_status("fade_tree_commit");
}

}  // namespace

TreeArgs make_tree_args(const fade_config_t* c, const fade_layer_t* L, int T, const uint16_t* q,
                        const fade_heads_t* tk, const fade_heads_t* tv) {
  TreeArgs a{};
  a.sink_k = L->sink_k;
  a.sink_v = L->sink_v;
  a.rec_k = L->recent_k;
  a.rec_v = L->recent_v;
  for (int i = 0; i < 2; ++i) {
    a.mk[i] = L->mid_k_codes[i];
    a.mv[i] = L->mid_v_codes[i];
    a.mks[i] = L->mid_k_scales[i];
    a.mvs[i] = L->mid_v_scales[i];
    a.mid_sc[i] = L->mid_scores[i];
  }
  a.sink_sc = L->sink_scores;
  a.rec_sc = L->recent_scores;
  a.meta = L->meta;
  a.status = L->status;
  a.pq_cb = c->v_codec == FADE_V_PQ ? L->pq_codebook : nullptr;
  a.q = q;
  a.tk = *tk;
  a.tv = *tv;
  a.B = c->batch;
  a.H = c->num_kv_heads;
  a.Hq = c->num_q_heads;
  a.G = c->num_q_heads / c->num_kv_heads;
  while ((1 << a.log_g) < a.G) ++a.log_g;   // G is 1, 2, 4 or 8
  a.S = c->n_sink;
  a.W = c->recent_window;
  a.C = mid_stride(c);
  a.T = T;
  return a;
}

}  // namespace fade

using namespace fade;

extern "C" fade_status_t fade_tree_layout(const fade_config_t* c, int32_t T,
                                          const int32_t* parents, const int32_t* n_nodes,
                                          const int32_t* base_pos, uint64_t* mask, int32_t* pos,
                                          void* stream) {
  clear_error();
  FADE_RANGE("fade_tree_layout");
  fade_status_t st = validate_tree(c, T);
  if (st) return st;
  if (!parents || !base_pos || !mask || !pos)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL parents, base_pos, mask or pos");
  if (!aligned(mask, 8) || !aligned(parents, 4) || !aligned(n_nodes, 4) || !aligned(base_pos, 4) ||
      !aligned(pos, 4))
    return set_error(FADE_ERR_INVALID_ARGUMENT,
                     "mask must be 8-byte aligned, parents, n_nodes, base_pos and pos 4-byte");
  tree_layout_kernel<<<c->batch, FADE_TREE_MAX_NODES, 0, as_stream(stream)>>>(
      T, parents, n_nodes, base_pos, mask, pos);
  return launch_status("fade_tree_layout");
}

extern "C" size_t fade_tree_ws_bytes(const fade_config_t* c, int32_t T) {
  clear_error();
  if (validate_tree(c, T)) return 0;
  const size_t scores = (size_t)c->batch * c->num_kv_heads * T * 4;
  const size_t attn = tree_attention_ws(c, T);
  return ((scores > attn ? scores : attn) + 15) / 16 * 16;
}

extern "C" fade_status_t fade_tree_commit(const fade_config_t* c, fade_layer_t* L, int32_t T,
                                          const uint16_t* q_rot, const float* lse,
                                          const fade_heads_t* tree_k, const fade_heads_t* tree_v,
                                          const int32_t* path, const int32_t* h_n_path, void* ws,
                                          size_t ws_bytes, void* stream) {
  clear_error();
  FADE_RANGE("fade_tree_commit");
  fade_status_t st = validate_tree(c, T);
  if (!st) st = validate_tree_layer(c, L);
  if (!st) st = validate_heads(tree_k, "tree_k");
  if (!st) st = validate_heads(tree_v, "tree_v");
  if (st) return st;
  if (!path || !h_n_path)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL path or path lengths");
  if (!aligned(path, 4)) return set_error(FADE_ERR_INVALID_ARGUMENT, "path must be 4-byte aligned");
  const bool scored = c->policy == FADE_EVICT_H2O || c->policy == FADE_EVICT_EMA;
  if (scored && (!q_rot || !lse || !ws))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "H2O and EMA need q_rot, lse and a workspace");
  if (scored && ((reinterpret_cast<uintptr_t>(q_rot) | reinterpret_cast<uintptr_t>(ws)) & 15))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "q_rot and the workspace must be 16-byte aligned");
  if (scored && !aligned(lse, 4))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "lse must be 4-byte aligned");
  const size_t need = (size_t)c->batch * c->num_kv_heads * T * 4;
  if (scored && ws_bytes < need)
    return set_error(FADE_ERR_CAPACITY, "tree workspace %zu bytes, %zu needed", ws_bytes, need);
  RowLens lens{}, to_sink{}, dem{};
  int any = 0;
  long long tiles = 0;   // of 16 tokens, one more than every row's at most
  for (int b = 0; b < c->batch; ++b) {
    const int n = h_n_path[b];
    if (n < 0 || n > T)
      return set_error(FADE_ERR_INVALID_ARGUMENT, "row %d: path length %d outside [0, %d]", b, n,
                       T);
    if (c->shared_rows && n != h_n_path[0])
      return set_error(FADE_ERR_INVALID_ARGUMENT,
                       "rows sharing their tier decisions need equal path lengths (row %d)", b);
    const int room = c->n_sink - L->h_n_sink[b];
    to_sink.v[b] = n < room ? n : (room > 0 ? room : 0);
    const int over = L->h_n_recent[b] + n - to_sink.v[b] - c->recent_window;
    dem.v[b] = over > 0 ? over : 0;
    if (n && L->h_n_mid[b] + dem.v[b] > c->mid_capacity)
      return set_error(FADE_ERR_CAPACITY, "row %d needs %d middle slots, capacity %d", b,
                       L->h_n_mid[b] + dem.v[b], c->mid_capacity);
    if (n == 0) dem.v[b] = 0;
    lens.v[b] = n;
    any |= n;
    if (n)
      tiles += (long long)c->num_kv_heads *
               ((L->h_n_sink[b] + (long long)L->h_n_mid[b] + L->h_n_recent[b] + n) / 16 + 2);
  }
  if (!any) return FADE_OK;
  const TreeArgs a = make_tree_args(c, L, T, q_rot, tree_k, tree_v);
  cudaStream_t s = as_stream(stream);
  float* path_sc = scored ? static_cast<float*>(ws) : nullptr;
  const int d = c->head_dim, kb = c->middle_k_bits, vb = c->middle_v_bits;
  if (scored) {
    st = d == 64 ? (kb == 4 ? launch_scores<64, 4>(c, a, lens, tiles, lse, path, path_sc, s)
                            : launch_scores<64, 2>(c, a, lens, tiles, lse, path, path_sc, s))
                 : (kb == 4 ? launch_scores<128, 4>(c, a, lens, tiles, lse, path, path_sc, s)
                            : launch_scores<128, 2>(c, a, lens, tiles, lse, path, path_sc, s));
    if (st) return st;
  }
  if (d == 64)
    st = kb == 4 ? (vb == 4 ? launch_commit<64, 4, 4>(c, a, lens, path, path_sc, s)
                            : launch_commit<64, 4, 2>(c, a, lens, path, path_sc, s))
                 : (vb == 4 ? launch_commit<64, 2, 4>(c, a, lens, path, path_sc, s)
                            : launch_commit<64, 2, 2>(c, a, lens, path, path_sc, s));
  else
    st = kb == 4 ? (vb == 4 ? launch_commit<128, 4, 4>(c, a, lens, path, path_sc, s)
                            : launch_commit<128, 4, 2>(c, a, lens, path, path_sc, s))
                 : (vb == 4 ? launch_commit<128, 2, 4>(c, a, lens, path, path_sc, s)
                            : launch_commit<128, 2, 2>(c, a, lens, path, path_sc, s));
  if (st) return st;
  for (int b = 0; b < c->batch; ++b) {
    L->h_n_sink[b] += to_sink.v[b];
    L->h_n_mid[b] += dem.v[b];
    L->h_n_recent[b] += lens.v[b] - to_sink.v[b] - dem.v[b];
  }
  return FADE_OK;
}
