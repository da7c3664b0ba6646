// Attention of a tree of drafted tokens over the tiered cache and over itself.
// Page "FADE：面向LLM推理的注意力感知分层KV缓存压缩技术", §项目结构与代码质量 (kernels/: fused INT4 dequant
// + SDPA): attention runs on the packed tiers.
//
// Mathematics: the query rows of a unit (row b, KV head h) are its nodes' G heads, r = node * G + g.
// Over tiles of 128 tokens, S = Q K^T, P = 2^(c S - m) with c = log2(e)/sqrt(d) and a running
// reference m per row, O += P V, L += rowsum P; out = O / L. The reference is put 6 below a maximum,
// so that the largest P is at least 2^6 and fp16 loses only what is 2^-31 of it, and moves only when
// a tile's maximum passes it by more than 14 (P stays below 2^15 with the factor 2 of halved values;
// sums in fp32), which spares most rescalings of O.
//
// Why the 5th-generation tensor cores: T * G query rows share every dequantised key, so the
// contraction (4 d flops a row and token) is no longer the thin one of a single decode token. The
// codes are unpacked once per tile into shared memory (fp16, the 128-byte swizzle), S and O live in
// tensor memory, P goes back to tensor memory as the A operand of the second product.
#include <math.h>

#include "tree.cuh"

namespace fade {
namespace {

constexpr int kTok = 128;            // tokens of a tile
constexpr int kThr = 256;            // threads of a CTA
constexpr int kRefBelow = 6;         // log2 a new reference lies below the maximum it follows
constexpr int kRefSlack = 14;        // log2 a row's logits may pass its reference by
constexpr int kBlk = kTok * 128;     // bytes of a [128 rows][64 channels] fp16 block
constexpr int kMaxSM = 160;          // SMs the workspace is sized for

// Channel order of an unpacked row. Two codes of one 32-bit word leave it as one fp16 pair: INT4
// pairs channels (i, i + 4) of 8, INT2 (i, i + 8) of 16. Keys and queries share an order, which
// their product does not see; values' order is undone at the output.
enum Order { kNatural = 0, kPair4 = 4, kPair8 = 8 };
constexpr int kPQ = 0;               // VB of product-quantised values
constexpr Order order_of(int bits) { return bits == 4 ? kPair4 : bits == 2 ? kPair8 : kNatural; }
template <int ORDER>
__host__ __device__ constexpr int channel_of(int p) {
  return ORDER == kPair4 ? (p & ~7) + ((p & 7) >> 1) + 4 * (p & 1)
         : ORDER == kPair8 ? (p & ~15) + ((p & 15) >> 1) + 8 * (p & 1)
                           : p;
}

template <int D, int VB>
struct Shape {
  static constexpr bool PQ = VB == kPQ;
  static constexpr int BLOCKS = D / 64;                       // 64-channel blocks of a tile
  static constexpr int TILE = BLOCKS * kBlk;                  // bytes of Q, K or V
  static constexpr int CODEBOOK = PQ ? 256 * D * 2 : 0;
  static constexpr int SMEM = 3 * TILE + CODEBOOK + 4096 + 1024;   // + small arrays + alignment
  static constexpr int PER_SM = SMEM <= 110 * 1024 ? 2 : 1;   // resident CTAs
  static constexpr int TMEM = 256;                            // columns: S 128, O D
};

struct AttnTreeArgs {
  TreeArgs a;
  const uint64_t* mask;
  const int32_t* n_nodes;
  uint16_t* out;
  float* lse;
  float* part;   // per CTA two partials: [rows][2] (m, L), then [rows][D] O
};

// ---------------------------------------------------------------- schedule
// Tiles are numbered row by row, KV head by KV head, block of query rows by block, FP16 tiles
// before middle tiles; CTA c of P takes tiles [N c / P, N (c + 1) / P). Everything is derived on
// the device from the counts, so a captured launch follows the cache.
struct RowTiles {
  int n;        // nodes
  int blocks;   // blocks of query rows
  int f16;      // FP16 tiles
  int tiles;    // tiles of one block
};
template <int ROWS>
__device__ __forceinline__ RowTiles row_tiles(const TreeArgs& a, const int32_t* n_nodes, int b) {
  RowTiles r;
  r.n = n_nodes ? min(max(n_nodes[b], 0), a.T) : a.T;
  const int32_t* m = a.meta + (size_t)b * a.H * FADE_META_FIELDS;
  r.blocks = (r.n * a.G + ROWS - 1) / ROWS;
  r.f16 = (m[FADE_META_N_SINK] + m[FADE_META_N_RECENT] + r.n + kTok - 1) / kTok;
  r.tiles = r.f16 + (m[FADE_META_N_MID] + kTok - 1) / kTok;
  return r;
}
// Inclusive prefix of the rows' tiles into pre[1 .. B] (pre[0] = 0), by the whole CTA of 256.
template <int ROWS>
__device__ __forceinline__ void tile_prefix(const TreeArgs& a, const int32_t* n_nodes, int* pre) {
  __shared__ int wsum[8];
  const int b = threadIdx.x, lane = b & 31, warp = b >> 5;
  int v = 0;
  if (b < a.B) {
    const RowTiles r = row_tiles<ROWS>(a, n_nodes, b);
    v = a.H * r.blocks * r.tiles;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) wsum[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += wsum[w];
  pre[b + 1] = v;
  if (b == 0) pre[0] = 0;
  __syncthreads();
}
__device__ __forceinline__ int row_of(const int* pre, int B, int g) {   // pre[b] <= g < pre[b+1]
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] > g) hi = mid; else lo = mid + 1;
  }
  return lo;
}
__device__ __forceinline__ int cta_start(int N, int P, int c) {
  return (int)((long long)N * c / P);
}
__device__ __forceinline__ int cta_of(int N, int P, int g) {
  return (int)((((long long)g + 1) * P - 1) / N);
}

// ---------------------------------------------------------------- tensor memory and products
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
         ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);   // 128-byte swizzle
}
// fp16 operands, fp32 accumulator, M = 128; B's N rows K-major, or (mn) channels contiguous.
__host__ __device__ constexpr uint32_t instr_desc(int n, bool mn) {
  return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, int acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, int acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 16 lanes x 32 fp32 columns: v[4i .. 4i+1] row lane/4, columns 8i + 2(lane%4) + {0, 1};
// v[4i+2 .. 4i+3] the same columns of row lane/4 + 8.
__device__ __forceinline__ void tm_ld32(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
// 16 lanes x 32 fp16 (16 columns): word 2i row lane/4, column 4i + lane%4; word 2i+1 row lane/4+8.
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tm_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- tiles in shared memory
// Rows of 64 channels (128 bytes) under the 128-byte swizzle, one [128][64] block per 64 channels.
__device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {   // chunk: 8 channels
  return (uint32_t)((chunk >> 3) * kBlk + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}
__device__ __forceinline__ void st_chunk(char* tile, int row, int chunk, uint32_t x, uint32_t y,
                                         uint32_t z, uint32_t w) {
  *reinterpret_cast<uint4*>(tile + chunk_at(row, chunk)) = make_uint4(x, y, z, w);
}
// 32 fp16 channels (one quantisation group) of a row, stored in ORDER.
template <int ORDER>
__device__ __forceinline__ void store_f16(char* tile, int row, int g, const uint4 (&x)[4]) {
  if constexpr (ORDER == kNatural) {
#pragma unroll
    for (int c = 0; c < 4; ++c) st_chunk(tile, row, 4 * g + c, x[c].x, x[c].y, x[c].z, x[c].w);
  } else if constexpr (ORDER == kPair4) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      st_chunk(tile, row, 4 * g + c, prmt(x[c].x, x[c].z, 0x5410), prmt(x[c].x, x[c].z, 0x7632),
               prmt(x[c].y, x[c].w, 0x5410), prmt(x[c].y, x[c].w, 0x7632));
  } else {
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
      const uint4 &p = x[c], &q = x[c + 1];
      st_chunk(tile, row, 4 * g + c, prmt(p.x, q.x, 0x5410), prmt(p.x, q.x, 0x7632),
               prmt(p.y, q.y, 0x5410), prmt(p.y, q.y, 0x7632));
      st_chunk(tile, row, 4 * g + c + 1, prmt(p.z, q.z, 0x5410), prmt(p.z, q.z, 0x7632),
               prmt(p.w, q.w, 0x5410), prmt(p.w, q.w, 0x7632));
    }
  }
}
// Half the code times the scale, for two codes at once: the codes (offset binary, the sign bits
// flipped by the xor) land in the mantissas of 2^k with unit 1/2, so one subtraction leaves code / 2
// exactly; the product rounds once to fp16. Half the value, because 7 times the largest scale
// would pass fp16's range; the caller's constants take the factor back.
__device__ __forceinline__ uint32_t scaled(uint32_t u, uint32_t off, __half2 s) {
  const __half2 h = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&u),
                                    *reinterpret_cast<const __half2*>(&off)), s);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A group of 32 codes: INT4 in four words (x), INT2 in two.
template <int BITS>
__device__ __forceinline__ void store_codes(char* tile, int row, int g, const uint32_t* x,
                                            uint16_t scale) {
  const __half2 s = __half2half2(__ushort_as_half(scale));
  if constexpr (BITS == 4) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // nibbles at bits 0..3: 512 + u/2; at bits 4..7: 32 + u/2 (u = code + 8)
      const uint32_t w = x[c], h = w >> 8;
      st_chunk(tile, row, 4 * g + c, scaled((w & 0x000f000fu) ^ 0x60086008u, 0x60086008u, s),
               scaled((w & 0x00f000f0u) ^ 0x50805080u, 0x50805080u, s),
               scaled((h & 0x000f000fu) ^ 0x60086008u, 0x60086008u, s),
               scaled((h & 0x00f000f0u) ^ 0x50805080u, 0x50805080u, s));
    }
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // crumbs at bits 0, 2, 4, 6, 8 of a half: 512, 128, 32, 8, 2 + u/2 (u = code + 2)
      const uint32_t w = x[c], h = w >> 8;
      st_chunk(tile, row, 4 * g + 2 * c, scaled((w & 0x00030003u) ^ 0x60026002u, 0x60026002u, s),
               scaled((w & 0x000c000cu) ^ 0x58085808u, 0x58085808u, s),
               scaled((w & 0x00300030u) ^ 0x50205020u, 0x50205020u, s),
               scaled((w & 0x00c000c0u) ^ 0x48804880u, 0x48804880u, s));
      st_chunk(tile, row, 4 * g + 2 * c + 1,
               scaled((w & 0x03000300u) ^ 0x42004200u, 0x42004200u, s),
               scaled((h & 0x000c000cu) ^ 0x58085808u, 0x58085808u, s),
               scaled((h & 0x00300030u) ^ 0x50205020u, 0x50205020u, s),
               scaled((h & 0x00c000c0u) ^ 0x48804880u, 0x48804880u, s));
    }
  }
}

// Elements of a V row that are not finite, cleared from x; returns whether there were any.
__device__ __forceinline__ bool clear_nonfinite(uint4 (&x)[4]) {
  uint32_t* w = reinterpret_cast<uint32_t*>(x);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t lo = (w[i] & 0x7c00u) == 0x7c00u ? 0x0000ffffu : 0u;
    const uint32_t hi = (w[i] & 0x7c000000u) == 0x7c000000u ? 0xffff0000u : 0u;
    bad |= (lo | hi) != 0u;
    w[i] &= ~(lo | hi);
  }
  return bad;
}

// The item (token, group) of a tile that thread `tid` takes in round i: a quarter warp holds eight
// tokens of one group, so its 16-byte stores hit eight different chunks of the swizzle.
template <int D>
__device__ __forceinline__ void item_of(int i, int& tok, int& g) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = i * 8 + warp;
  if constexpr (D == 128) {
    tok = 8 * w + (lane & 7);
    g = lane >> 3;
  } else {
    tok = 16 * w + 8 * (lane >> 4) + (lane & 7);
    g = (lane >> 3) & 1;
  }
}

// A tile's middle codes and scales on their way to shared memory.
template <int D, int KB, int VB>
struct Codes {
  static constexpr int ITEMS = kTok * (D / 32) / kThr;
  static constexpr int KW = KB, VW = VB == kPQ ? 2 : VB;   // 32-bit words of a group
  uint32_t k[ITEMS][KW], v[ITEMS][VW];
  uint16_t ks[ITEMS], vs[ITEMS];
};
template <int W>
__device__ __forceinline__ void ld_words(const uint8_t* p, uint32_t* w) {
  if constexpr (W == 4) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = x.x; w[1] = x.y;
  }
}
// Tokens past the tier read its last row (masked in S); their V is zeroed by the caller.
template <int D, int KB, int VB>
__device__ __forceinline__ void load_codes(const TreeArgs& a, int unit, int cur, int n_mid, int t0,
                                           Codes<D, KB, VB>& c) {
  constexpr int G = D / 32;
#pragma unroll
  for (int i = 0; i < Codes<D, KB, VB>::ITEMS; ++i) {
    int tok, g;
    item_of<D>(i, tok, g);
    const size_t r = (size_t)unit * a.C + min(t0 + tok, n_mid - 1);
    ld_words<Codes<D, KB, VB>::KW>(a.mk[cur] + (r * G + g) * (4 * KB), c.k[i]);
    ld_words<Codes<D, KB, VB>::VW>(
        a.mv[cur] + (r * G + g) * (4 * Codes<D, KB, VB>::VW), c.v[i]);
    c.ks[i] = __ldg(a.mks[cur] + r * G + g);
    if (VB != kPQ) c.vs[i] = __ldg(a.mvs[cur] + r * G + g);
  }
}

// The key or value row of FP16 token j of a unit (sinks, then the ring oldest first, then nodes).
__device__ __forceinline__ const uint16_t* f16_row(const TreeArgs& a, int D, int b, int h, int unit,
                                                   int n_sink, int n_rec, int head, int j, bool v) {
  if (j < n_sink) return (v ? a.sink_v : a.sink_k) + ((size_t)unit * a.S + j) * D;
  j -= n_sink;
  if (j < n_rec) return (v ? a.rec_v : a.rec_k) + ((size_t)unit * a.W + (head + j) % a.W) * D;
  j -= n_rec;
  const fade_heads_t& t = v ? a.tv : a.tk;
  return t.x + b * t.row_stride + j * t.token_stride + h * t.head_stride;
}

// A CTA of 8 warps walks its tiles; per tile: K unpacked into shared memory, S = Q K^T issued, V
// unpacked while it runs, softmax, O += P V issued, which the next tile's K overlaps. Two CTAs share
// an SM (one with a codebook), so one's products run under the other's unpacking. R: 16-row halves
// of each 32-lane quarter of tensor memory in use: up to 64 query rows take lanes 0..15 of every
// quarter (R = 1), so that all eight warps have a share of the softmax; otherwise 128 (R = 2).
template <int D, int KB, int VB, int R>
__global__ void __launch_bounds__(kThr, (Shape<D, VB>::PER_SM))
    tree_attention_kernel(const __grid_constant__ AttnTreeArgs p) {
  using Sh = Shape<D, VB>;
  constexpr int ROWS = 64 * R, KO = order_of(KB), VO = order_of(VB);
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ char raw[];
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  char *sQ = base, *sK = base + Sh::TILE, *sV = base + 2 * Sh::TILE;
  uint2* sCB = reinterpret_cast<uint2*>(base + 3 * Sh::TILE);   // [256][D/4], centroid-major
  char* small = base + 3 * Sh::TILE + Sh::CODEBOOK;
  uint64_t* bars = reinterpret_cast<uint64_t*>(small);          // [0] S ready, [1] O ready
  uint32_t* sTm = reinterpret_cast<uint32_t*>(small + 16);
  uint32_t* sBad = reinterpret_cast<uint32_t*>(small + 24);     // [2] nodes with non-finite V
  float* sMax = reinterpret_cast<float*>(small + 64);           // [R][8 warps][16 rows]
  int* sPre = reinterpret_cast<int*>(small + 64 + 1024);        // [257]
  const TreeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quarter = warp & 3;
  const int colhalf = warp >> 2;   // which half of S's (and O's) columns this warp takes
  const uint32_t barS = smem_u32(bars), barO = smem_u32(bars + 1);

  tile_prefix<ROWS>(a, p.n_nodes, sPre);
  const int N = sPre[a.B];
  int g = cta_start(N, gridDim.x, blockIdx.x);
  const int g_end = cta_start(N, gridDim.x, blockIdx.x + 1), g_first = g;
  if (g >= g_end) return;   // uniform over the CTA; nothing allocated yet
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(sTm)),
                 "r"(Sh::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    mbar_init(barS, 1);
    mbar_init(barO, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if constexpr (Sh::PQ) {
    // the codebook [D/4][256] of 8-byte centroids, transposed
    const uint2* cb = reinterpret_cast<const uint2*>(a.pq_cb);
    for (int i = tid; i < 256 * (D / 4); i += kThr)
      sCB[(i & 255) * (D / 4) + (i >> 8)] = __ldg(cb + i);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *sTm, tmO = tm + 128;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  uint32_t phS = 0, phO = 0;
  bool dead = false;   // a wait gave up: later ones are skipped, the flow stays the same
  auto wait = [&](uint32_t bar, uint32_t& ph) {
    if (!dead && !mbar_wait(bar, ph, a.status, 1)) dead = true;
    ph ^= 1;
    __syncwarp();
    fence_after();
  };
  const float cscale = kLog2e * rsqrtf((float)D);

  while (g < g_end) {
    // ------------------------------------------------ the segment: tiles of one block of rows
    const int b = row_of(sPre, a.B, g);
    const RowTiles rt = row_tiles<ROWS>(a, p.n_nodes, b);
    const int rel = g - sPre[b], blk = rel / rt.tiles, t_begin = rel % rt.tiles;
    const int t_end = min(rt.tiles, t_begin + (g_end - g));
    const int h = blk / rt.blocks, qb = blk % rt.blocks, unit = b * a.H + h;
    const int r0 = qb * ROWS, rows = min(ROWS, rt.n * a.G - r0);   // query rows of the block
    const int32_t* m = a.meta + (size_t)unit * FADE_META_FIELDS;
    const int n_sink = m[FADE_META_N_SINK], n_mid = m[FADE_META_N_MID];
    const int n_rec = m[FADE_META_N_RECENT], head = m[FADE_META_HEAD], cur = m[FADE_META_CUR];
    const int n16 = n_sink + n_rec;   // cached FP16 tokens, then the nodes
    // a warp whose rows are all past the block's takes no part in the softmax
    const bool active = quarter * (16 * R) < rows;

    if (tid < 2) sBad[tid] = 0;
    // Q: matrix row 32 q + i holds query row 16 q + i (R = 1, i < 16) or 32 q + i
    for (int i = 0; i < Codes<D, KB, VB>::ITEMS; ++i) {
      int row, gq;
      item_of<D>(i, row, gq);
      const int in = row & 31, r = (row >> 5) * (16 * R) + in;
      uint4 x[4] = {};
      if (in < 16 * R && r < rows) {
        const int node = (r0 + r) / a.G, gh = (r0 + r) % a.G;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + (((size_t)b * a.T + node) * a.Hq + h * a.G + gh) * D + 32 * gq);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = __ldg(src + c);
      }
      store_f16<KO>(sQ, row, gq, x);
    }
    float mref[R][2], lsum[R][2];
#pragma unroll
    for (int f = 0; f < R; ++f)
      for (int e = 0; e < 2; ++e) {
        mref[f][e] = -INFINITY;
        lsum[f][e] = 0.f;
      }
    Codes<D, KB, VB> codes;
    if (t_begin >= rt.f16)
      load_codes<D, KB, VB>(a, unit, cur, n_mid, (t_begin - rt.f16) * kTok, codes);

    for (int t = t_begin; t < t_end; ++t) {
      const bool f16 = t < rt.f16, first = t == t_begin;
      const int tok0 = (f16 ? t : t - rt.f16) * kTok;
      const int count = min(kTok, (f16 ? n16 + rt.n : n_mid) - tok0);   // tokens of the tile
      // ---- K (its buffer is free: the last S has been waited for)
#pragma unroll
      for (int i = 0; i < Codes<D, KB, VB>::ITEMS; ++i) {
        int tok, gq;
        item_of<D>(i, tok, gq);
        if (f16) {
          uint4 x[4] = {};
          if (tok < count) {
            const uint4* src = reinterpret_cast<const uint4*>(
                f16_row(a, D, b, h, unit, n_sink, n_rec, head, tok0 + tok, false) + 32 * gq);
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = src[c];
          }
          store_f16<KO>(sK, tok, gq, x);
        } else {
          store_codes<KB>(sK, tok, gq, codes.k[i], codes.ks[i]);
        }
      }
      fence_proxy_async_smem();
      fence_before();
      __syncthreads();
      // ---- O of the last tile is complete: P's columns (S's) and V's buffer are free
      if (!first) wait(barO, phO);
      if (tid == 0) {
        fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * kBlk + (k & 3) * 32;
          mma_ss(tm, smem_desc(smem_u32(sQ) + off, 16, 1024),
                 smem_desc(smem_u32(sK) + off, 16, 1024), instr_desc(kTok, false), k > 0);
        }
        mma_commit(barS);
      }
      // ---- V while S is computed
#pragma unroll
      for (int i = 0; i < Codes<D, KB, VB>::ITEMS; ++i) {
        int tok, gq;
        item_of<D>(i, tok, gq);
        if (f16) {
          uint4 x[4] = {};
          if (tok < count) {
            const uint4* src = reinterpret_cast<const uint4*>(
                f16_row(a, D, b, h, unit, n_sink, n_rec, head, tok0 + tok, true) + 32 * gq);
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = src[c];
            // a node's infinities and NaN would reach the rows that do not see it (0 * inf):
            // they are left out of the product and put into the rows that see it at the end
            const int node = tok0 + tok - n16;
            if (node >= 0 && clear_nonfinite(x)) atomicOr(sBad + (node >> 5), 1u << (node & 31));
          }
          store_f16<VO>(sV, tok, gq, x);
        } else if constexpr (Sh::PQ) {
          // lane-dependent order of the eight sub-spaces: the 32 lanes of a warp read 32 different
          // sub-spaces of the centroid-major codebook, two wavefronts whatever the codes
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int s = (e + tok) & 7, code = (codes.v[i][s >> 2] >> (8 * (s & 3))) & 255;
            const uint2 x = tok < count ? sCB[code * (D / 4) + 8 * gq + s] : make_uint2(0u, 0u);
            *reinterpret_cast<uint2*>(sV + chunk_at(tok, 4 * gq + (s >> 1)) + 8 * (s & 1)) = x;
          }
        } else {
          store_codes<VB>(sV, tok, gq, codes.v[i], tok < count ? codes.vs[i] : (uint16_t)0);
        }
      }
      if (t + 1 < t_end && t + 1 >= rt.f16)   // the next tile's codes, in flight over the softmax
        load_codes<D, KB, VB>(a, unit, cur, n_mid, (t + 1 - rt.f16) * kTok, codes);
      fence_proxy_async_smem();
      wait(barS, phS);
      // ---- softmax: 16 rows x 64 columns a warp, two rows a thread
      if (active) {
        const float c = f16 ? cscale : 2.f * cscale;   // middle keys are stored halved
#pragma unroll
        for (int f = 0; f < R; ++f) {
          float s[32];
          const uint32_t at = tm + lanes + ((uint32_t)(16 * f) << 16) + 64 * colhalf;
          tm_ld32(at, s);
          tm_ld32(at + 32, s + 16);
          tm_wait_ld();
          const int col0 = 64 * colhalf + 2 * (lane & 3);
          if (f16) {
            uint64_t see[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = quarter * (16 * R) + 16 * f + (lane >> 2) + 8 * e;
              see[e] = r < rows ? p.mask[(size_t)b * a.T + (r0 + r) / a.G] : 0ull;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int col = col0 + 8 * (i >> 2) + (i & 1), node = tok0 + col - n16;
              const bool in = col < count && (node < 0 || ((see[(i >> 1) & 1] >> (node & 63)) & 1));
              s[i] = in ? s[i] : -INFINITY;
            }
          } else if (count < kTok) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (col0 + 8 * (i >> 2) + (i & 1) >= count) s[i] = -INFINITY;
          }
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; ++i) mx[(i >> 1) & 1] = fmaxf(mx[(i >> 1) & 1], s[i]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
          }
          float* mine = sMax + (f * 8 + warp) * 16;
          const float* other = sMax + (f * 8 + (warp ^ 4)) * 16;
          if ((lane & 3) == 0) {
            mine[lane >> 2] = mx[0];
            mine[(lane >> 2) + 8] = mx[1];
          }
          __syncwarp();
          asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");   // the quarter's two warps
          float ref[2], fac[2];
          bool move = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], other[(lane >> 2) + 8 * e]) * c;
            const bool up = mx[e] > mref[f][e] + kRefSlack;   // true from -inf
            const float to = up ? mx[e] - kRefBelow : mref[f][e];
            fac[e] = up ? ex2(mref[f][e] - to) : 1.f;
            mref[f][e] = to;
            lsum[f][e] *= fac[e];
            ref[e] = to == -INFINITY ? 0.f : to;
            move |= up;
          }
          // both warps of a quarter decide alike; each rescales its half of O's columns
          if (!first && __any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int q = 0; q < D / 64; ++q) {
              float o[16];
              const uint32_t ao = tmO + lanes + ((uint32_t)(16 * f) << 16) + colhalf * (D / 2) + 32 * q;
              tm_ld32(ao, o);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= fac[(i >> 1) & 1];
              tm_st32(ao, o);
            }
          }
          // P: twice the probability where V is stored halved
          const float add = (!f16 && !Sh::PQ) ? 1.f : 0.f;
          float sum[2] = {0.f, 0.f};
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int e = i & 1;
            const float x = ex2(fmaf(s[2 * i], c, add - ref[e]));
            const float y = ex2(fmaf(s[2 * i + 1], c, add - ref[e]));
            sum[e] += x + y;
            const __half2 h2 = __floats2half2_rn(x, y);
            pk[i] = *reinterpret_cast<const uint32_t*>(&h2);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) lsum[f][e] = fmaf(sum[e], add != 0.f ? 0.5f : 1.f, lsum[f][e]);
          // over S's first 64 columns: the quarter's two warps have both read S
          const uint32_t ap = tm + lanes + ((uint32_t)(16 * f) << 16) + 32 * colhalf;
          tm_st16(ap, pk);
          tm_st16(ap + 16, pk + 8);
        }
        tm_wait_st();
      }
      fence_before();
      __syncthreads();
      if (tid == 0) {
        fence_after();
#pragma unroll
        for (int k = 0; k < kTok / 16; ++k)
          mma_ts(tmO, tm + 8 * k, smem_desc(smem_u32(sV) + k * 2048, kBlk, 1024),
                 instr_desc(D, true), !(first && k == 0));
        mma_commit(barO);
      }
    }
    wait(barO, phO);

    // ------------------------------------------------ the segment's result
    const bool whole = t_begin == 0 && t_end == rt.tiles;
    // rows' sums: over the quad, then over the quarter's two warps
    float L[R][2];
#pragma unroll
    for (int f = 0; f < R; ++f)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = lsum[f][e];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        L[f][e] = v;
        if ((lane & 3) == 0) sMax[(f * 8 + warp) * 16 + (lane >> 2) + 8 * e] = v;
      }
    __syncthreads();
    const unsigned long long bad = sBad[0] | ((unsigned long long)sBad[1] << 32);
    float* part = p.part + ((size_t)blockIdx.x * 2 + (g == g_first ? 0 : 1)) * ROWS * (D + 2);
    if (active) {
#pragma unroll
      for (int f = 0; f < R; ++f) {
        int row[2];
        size_t vec[2];
        float inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int o = (lane >> 2) + 8 * e, r = quarter * (16 * R) + 16 * f + o;
          row[e] = r;
          // added in the same order by both warps
          L[f][e] = sMax[(f * 8 + quarter) * 16 + o] + sMax[(f * 8 + quarter + 4) * 16 + o];
          const int rr = r0 + min(r, rows - 1);
          vec[e] = ((size_t)b * a.T + rr / a.G) * a.Hq + h * a.G + rr % a.G;
          const float mm = mref[f][e];
          inv[e] = mm == -INFINITY ? 0.f : 1.f / L[f][e];
          if (colhalf == 0 && (lane & 3) == 0 && r < rows) {
            if (whole)
              p.lse[vec[e]] = mm == -INFINITY ? -INFINITY
                                              : (mm + log2f(L[f][e])) * 0.6931471805599453f;
            else
              *reinterpret_cast<float2*>(part + 2 * r) = make_float2(mm, L[f][e]);
          }
        }
#pragma unroll
        for (int q = 0; q < D / 64; ++q) {
          float o[16];
          const int c0 = colhalf * (D / 2) + 32 * q;
          tm_ld32(tmO + lanes + ((uint32_t)(16 * f) << 16) + c0, o);
          tm_wait_ld();
          for (unsigned long long left = bad; left; left &= left - 1) {
            const int node = __ffsll((long long)left) - 1;
            const uint16_t* v = a.tv.x + b * a.tv.row_stride + node * a.tv.token_stride +
                                h * a.tv.head_stride;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int e = (i >> 1) & 1;
              if (row[e] >= rows ||
                  !((p.mask[(size_t)b * a.T + (r0 + row[e]) / a.G] >> node) & 1))
                continue;
              const float x = h2f(v[channel_of<VO>(c0 + 8 * (i >> 2) + 2 * (lane & 3) + (i & 1))]);
              if (!isfinite(x)) o[i] += x;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const int e = (i >> 1) & 1, col = c0 + 8 * (i >> 2) + 2 * (lane & 3);
            if (row[e] >= rows) continue;
            if (whole) {
              p.out[vec[e] * D + channel_of<VO>(col)] = f2h(o[i] * inv[e]);
              p.out[vec[e] * D + channel_of<VO>(col + 1)] = f2h(o[i + 1] * inv[e]);
            } else {
              *reinterpret_cast<float2*>(part + 2 * ROWS + (size_t)row[e] * D + col) =
                  make_float2(o[i], o[i + 1]);
            }
          }
        }
      }
    }
    fence_before();
    __syncthreads();   // sMax, sBad, Q and O may be written again
    fence_after();
    g += t_end - t_begin;
  }
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(Sh::TMEM));
}

// Joins the partials of a block of query rows that several CTAs shared, in the order of their
// tiles: one warp a row, lane l its channels (in V's order) 2l + 64 i and the next.
template <int D, int VB, int R>
__global__ void __launch_bounds__(kThr) tree_combine_kernel(const __grid_constant__ AttnTreeArgs p,
                                                            int P) {
  constexpr int ROWS = 64 * R, VO = order_of(VB);
  __shared__ int pre[257];
  const TreeArgs& a = p.a;
  tile_prefix<ROWS>(a, p.n_nodes, pre);
  const int N = pre[a.B], b = blockIdx.z;
  const RowTiles rt = row_tiles<ROWS>(a, p.n_nodes, b);
  const int h = blockIdx.y, qb = blockIdx.x / (ROWS / 8);
  if (qb >= rt.blocks) return;
  const int begin = pre[b] + (h * rt.blocks + qb) * rt.tiles, end = begin + rt.tiles;
  const int c0 = cta_of(N, P, begin), c1 = cta_of(N, P, end - 1);
  if (c0 == c1) return;   // written by its CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = (blockIdx.x % (ROWS / 8)) * 8 + warp, rr = qb * ROWS + row;
  if (rr >= rt.n * a.G) return;
  float M = -INFINITY, L = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int c = c0; c <= c1; ++c) {
    const int g0 = cta_start(N, P, c);
    if (g0 == cta_start(N, P, c + 1)) continue;   // a CTA without tiles
    const float* part = p.part + ((size_t)c * 2 + (g0 >= begin ? 0 : 1)) * ROWS * (D + 2);
    const float2 ml = *reinterpret_cast<const float2*>(part + 2 * row);
    const float Mn = fmaxf(M, ml.x);
    const float fo = M == -INFINITY ? 0.f : ex2(M - Mn);
    const float fn = ml.x == -INFINITY ? 0.f : ex2(ml.x - Mn);
    L = fmaf(L, fo, ml.y * fn);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 x =
          *reinterpret_cast<const float2*>(part + 2 * ROWS + (size_t)row * D + 64 * i + 2 * lane);
      o[2 * i] = fmaf(o[2 * i], fo, x.x * fn);
      o[2 * i + 1] = fmaf(o[2 * i + 1], fo, x.y * fn);
    }
    M = Mn;
  }
  const size_t vec = ((size_t)b * a.T + rr / a.G) * a.Hq + h * a.G + rr % a.G;
  const float inv = M == -INFINITY ? 0.f : 1.f / L;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    p.out[vec * D + channel_of<VO>(64 * (i >> 1) + 2 * lane + (i & 1))] = f2h(o[i] * inv);
  if (lane == 0)
    p.lse[vec] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n < kMaxSM ? n : kMaxSM;
}

int rows_of(const fade_config_t* c, int T) {   // query rows of a block: 64 where they are enough
  return T * (c->num_q_heads / c->num_kv_heads) <= 64 ? 64 : 128;
}

template <int D, int KB, int VB, int R>
fade_status_t launch(const fade_config_t* c, const AttnTreeArgs& p, cudaStream_t st) {
  using Sh = Shape<D, VB>;
  const int sms = sm_count();
  if (sms == 0) return launch_status("fade_tree_attention device query");
  // no more CTAs than the configuration can have tiles (not the present counts: see the header)
  const long long blocks = ceil_div((long long)p.a.T * p.a.G, 64 * R);
  const long long most = (long long)p.a.B * p.a.H * blocks *
                         (ceil_div(p.a.C, kTok) + ceil_div(p.a.S + p.a.W + p.a.T, kTok));
  const int P = (int)(most < sms * Sh::PER_SM ? most : sms * Sh::PER_SM);
  auto kern = tree_attention_kernel<D, KB, VB, R>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM) !=
      cudaSuccess)
    return launch_status("fade_tree_attention shared-memory opt-in");
  kern<<<P, kThr, Sh::SMEM, st>>>(p);
  fade_status_t s = launch_status("fade_tree_attention");
  if (s) return s;
  tree_combine_kernel<D, VB, R>
      <<<dim3((unsigned)(blocks * 8 * R), p.a.H, p.a.B), kThr, 0, st>>>(p, P);
  return launch_status("fade_tree_attention combine");
}

template <int D, int KB, int VB>
fade_status_t launch_rows(const fade_config_t* c, const AttnTreeArgs& p, cudaStream_t st) {
  return rows_of(c, p.a.T) == 64 ? launch<D, KB, VB, 1>(c, p, st) : launch<D, KB, VB, 2>(c, p, st);
}

}  // namespace

size_t tree_attention_ws(const fade_config_t* c, int T) {
  return (size_t)kMaxSM * 2 * 2 * rows_of(c, T) * (c->head_dim + 2) * 4;
}

}  // namespace fade

using namespace fade;

extern "C" fade_status_t fade_tree_attention(const fade_config_t* c, const fade_layer_t* L,
                                             int32_t T, const uint16_t* q_rot,
                                             const fade_heads_t* tree_k,
                                             const fade_heads_t* tree_v, const uint64_t* mask,
                                             const int32_t* n_nodes, uint16_t* out, float* lse,
                                             void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  FADE_RANGE("fade_tree_attention");
  fade_status_t st = validate_tree(c, T);
  if (!st) st = validate_tree_layer(c, L);
  if (!st) st = validate_heads(tree_k, "tree_k");
  if (!st) st = validate_heads(tree_v, "tree_v");
  if (st) return st;
  if (!q_rot || !mask || !out || !lse || !ws)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL q_rot, mask, out, lse or ws");
  if ((reinterpret_cast<uintptr_t>(q_rot) | reinterpret_cast<uintptr_t>(out) |
       reinterpret_cast<uintptr_t>(ws)) & 15)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "q_rot, out and ws must be 16-byte aligned");
  if (ws_bytes < tree_attention_ws(c, T))
    return set_error(FADE_ERR_CAPACITY, "tree workspace %zu bytes, %zu needed", ws_bytes,
                     tree_attention_ws(c, T));
  AttnTreeArgs p{};
  p.a = make_tree_args(c, L, T, q_rot, tree_k, tree_v);
  p.mask = mask;
  p.n_nodes = n_nodes;
  p.out = out;
  p.lse = lse;
  p.part = static_cast<float*>(ws);
  cudaStream_t s = as_stream(stream);
  const int kb = c->middle_k_bits, vb = c->v_codec == FADE_V_PQ ? kPQ : c->middle_v_bits;
#define FADE_TREE_CASE(D_, KB_, VB_)               \
  if (c->head_dim == D_ && kb == KB_ && vb == VB_) return launch_rows<D_, KB_, VB_>(c, p, s);
  FADE_TREE_CASE(64, 4, 2) FADE_TREE_CASE(64, 4, 4) FADE_TREE_CASE(64, 2, 2)
  FADE_TREE_CASE(64, 2, 4) FADE_TREE_CASE(128, 4, 2) FADE_TREE_CASE(128, 4, 4)
  FADE_TREE_CASE(128, 2, 2) FADE_TREE_CASE(128, 2, 4) FADE_TREE_CASE(64, 4, kPQ)
  FADE_TREE_CASE(64, 2, kPQ) FADE_TREE_CASE(128, 4, kPQ) FADE_TREE_CASE(128, 2, kPQ)
#undef FADE_TREE_CASE
  return set_error(FADE_ERR_UNSUPPORTED, "unsupported (head_dim, k_bits, v_bits)");
}
