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
//
// Roundings to fewer than 32 bits: P and dequantised INT4 values to fp16 (2^-11 relative). INT4
// keys keep all their bits: code * scale has at most 14, its fp16 rounding leaves a remainder of at
// most 3, which E5M2 holds exactly; the remainder meets an E5M2 copy of the query in a second
// product (at the doubled 8-bit rate), so a logit is off by about 2^-15 of its terms, not 2^-12.
#include <math.h>

#include "tree.cuh"

namespace fade {
namespace {

constexpr int kTok = 128;            // tokens of a tile
constexpr int kRefBelow = 6;         // log2 a new reference lies below the maximum it follows
constexpr int kRefSlack = 14;        // log2 a row's logits may pass its reference by
constexpr int kAhead = 4;            // tiles that L2 is asked for ahead of their use
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

template <int D, int KB, int VB, int R>
struct Shape {
  static constexpr bool PQ = VB == kPQ, LOW = KB == 4;        // LOW: remainders of the keys
  static constexpr int TILE = D / 64 * kBlk;                  // bytes of Q, K or V in fp16
  static constexpr int LOWB = LOW ? kBlk : 0;                 // of Q or K in E5M2: 128-byte rows
  static constexpr int CODEBOOK = PQ ? 256 * D * 2 : 0;
  static constexpr int STAGE = 2 * TILE + LOWB;               // K, V, K's remainders
  static constexpr int FIXED = TILE + LOWB + CODEBOOK + 2048 + 1024;   // Q, small arrays, alignment
  static constexpr int STAGES = FIXED + 2 * STAGE <= 226 * 1024 ? 2 : 1;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
  static constexpr int SOFT = 128 * R;                        // softmax threads: 16 rows a warp
  static constexpr int UNPACK = 4 * D;                        // one group of 32 channels a thread
  static constexpr int THREADS = SOFT + UNPACK + 128;         // and four warps, one issues products
  // Registers a thread: at the launch, then by role (multiples of 8; the sum over the roles stays
  // within the launch's).
  static constexpr int REGS = 65536 / THREADS / 8 * 8;
  static constexpr int REGS_MMA = 40;
  static constexpr int REGS_UNPACK = THREADS == 896 ? 64 : REGS > 128 ? 128 : REGS;
  static constexpr int REGS_SOFT_ =
      (REGS * THREADS - REGS_MMA * 128 - REGS_UNPACK * UNPACK) / SOFT / 8 * 8;
  static constexpr int REGS_SOFT = REGS_SOFT_ > 160 ? 160 : REGS_SOFT_;
  static_assert(REGS_SOFT * SOFT + REGS_UNPACK * UNPACK + REGS_MMA * 128 <= REGS * THREADS, "");
  static constexpr int TMEM = 512;                            // columns: S 2 x 128, O D
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
// Inclusive prefix of the rows' tiles into pre[1 .. B] (pre[0] = 0), by the whole CTA (256 threads at least).
template <int ROWS>
__device__ __forceinline__ void tile_prefix(const TreeArgs& a, const int32_t* n_nodes, int* pre) {
  __shared__ int wsum[8];
  const int b = threadIdx.x, lane = b & 31, warp = b >> 5;
  int v = 0;
  if (b < a.B) {   // B <= 256
    const RowTiles r = row_tiles<ROWS>(a, n_nodes, b);
    v = a.H * r.blocks * r.tiles;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31 && warp < 8) wsum[warp] = v;
  __syncthreads();
  if (b < FADE_MAX_BATCH) {
    for (int w = 0; w < warp; ++w) v += wsum[w];
    pre[b + 1] = v;
    if (b == 0) pre[0] = 0;
  }
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
// E5M2 operands, fp32 accumulator.
__host__ __device__ constexpr uint32_t instr_desc_low(int n) {
  return instr_desc(n, false) | (1u << 7) | (1u << 10);
}
__device__ __forceinline__ void mma_low(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
  asm volatile("tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, 1;" ::"r"(d), "l"(a),
               "l"(b), "r"(id)
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
// exactly; the product rounds once to fp16, and LOW keeps what the rounding dropped (exact, one
// fused operation). Half the value, because 7 times the largest scale would pass fp16's range; the
// caller's constants take the factor back.
template <bool LOW>
__device__ __forceinline__ uint32_t scaled(uint32_t u, uint32_t off, __half2 s, uint32_t& rest) {
  const __half2 t = __hsub2(*reinterpret_cast<const __half2*>(&u),
                            *reinterpret_cast<const __half2*>(&off));
  const __half2 h = __hmul2(t, s);
  if constexpr (LOW) {
    const __half2 l = __hfma2(t, s, __hneg2(h));
    rest = *reinterpret_cast<const uint32_t*>(&l);
  }
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A group of 32 codes: INT4 in four words (x), INT2 in two. LOW (INT4): the remainders as E5M2, the
// upper bytes of their fp16 form, in the same order.
template <int BITS, bool LOW>
__device__ __forceinline__ void store_codes(char* tile, char* low, int row, int g,
                                            const uint32_t* x, uint16_t scale) {
  const __half2 s = __half2half2(__ushort_as_half(scale));
  if constexpr (BITS == 4) {
    uint32_t lo[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // nibbles at bits 0..3: 512 + u/2; at bits 4..7: 32 + u/2 (u = code + 8)
      const uint32_t w = x[c], h = w >> 8;
      uint32_t r[4] = {};
      const uint32_t a = scaled<LOW>((w & 0x000f000fu) ^ 0x60086008u, 0x60086008u, s, r[0]);
      const uint32_t b = scaled<LOW>((w & 0x00f000f0u) ^ 0x50805080u, 0x50805080u, s, r[1]);
      const uint32_t d = scaled<LOW>((h & 0x000f000fu) ^ 0x60086008u, 0x60086008u, s, r[2]);
      const uint32_t e = scaled<LOW>((h & 0x00f000f0u) ^ 0x50805080u, 0x50805080u, s, r[3]);
      st_chunk(tile, row, 4 * g + c, a, b, d, e);
      lo[2 * c] = prmt(r[0], r[1], 0x7531);
      lo[2 * c + 1] = prmt(r[2], r[3], 0x7531);
    }
    if constexpr (LOW) {
      st_chunk(low, row, 2 * g, lo[0], lo[1], lo[2], lo[3]);
      st_chunk(low, row, 2 * g + 1, lo[4], lo[5], lo[6], lo[7]);
    }
  } else {
    uint32_t none;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // crumbs at bits 0, 2, 4, 6, 8 of a half: 512, 128, 32, 8, 2 + u/2 (u = code + 2)
      const uint32_t w = x[c], h = w >> 8;
      auto sc = [&](uint32_t u, uint32_t off) { return scaled<false>(u, off, s, none); };
      st_chunk(tile, row, 4 * g + 2 * c, sc((w & 0x00030003u) ^ 0x60026002u, 0x60026002u),
               sc((w & 0x000c000cu) ^ 0x58085808u, 0x58085808u),
               sc((w & 0x00300030u) ^ 0x50205020u, 0x50205020u),
               sc((w & 0x00c000c0u) ^ 0x48804880u, 0x48804880u));
      st_chunk(tile, row, 4 * g + 2 * c + 1, sc((w & 0x03000300u) ^ 0x42004200u, 0x42004200u),
               sc((h & 0x000c000cu) ^ 0x58085808u, 0x58085808u),
               sc((h & 0x00300030u) ^ 0x50205020u, 0x50205020u),
               sc((h & 0x00c000c0u) ^ 0x48804880u, 0x48804880u));
    }
  }
}
// Two fp16 values as E5M2 bytes.
__device__ __forceinline__ uint32_t to_e5m2(uint32_t x) {
  uint16_t y;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(y) : "r"(x));
  return y;
}
// The E5M2 copy of 32 fp16 channels in the order of INT4 keys.
__device__ __forceinline__ void store_low(char* low, int row, int g, const uint4 (&x)[4]) {
#pragma unroll
  for (int c = 0; c < 4; c += 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4& y = x[c + i];
      w[2 * i] = to_e5m2(prmt(y.x, y.z, 0x5410)) | (to_e5m2(prmt(y.x, y.z, 0x7632)) << 16);
      w[2 * i + 1] = to_e5m2(prmt(y.y, y.w, 0x5410)) | (to_e5m2(prmt(y.y, y.w, 0x7632)) << 16);
    }
    st_chunk(low, row, 2 * g + (c >> 1), w[0], w[1], w[2], w[3]);
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

// The (token, group of 32 channels) of a tile that an unpacking thread takes: a quarter warp holds
// eight tokens of one group, so its 16-byte stores hit eight different chunks of the swizzle.
template <int D>
__device__ __forceinline__ void item_of(int thread, int& tok, int& g) {
  const int lane = thread & 31, w = thread >> 5;
  if constexpr (D == 128) {
    tok = 8 * w + (lane & 7);
    g = lane >> 3;
  } else {
    tok = 16 * w + 8 * (lane >> 4) + (lane & 7);
    g = (lane >> 3) & 1;
  }
}

// A thread's codes and scales of a middle tile on their way to shared memory.
template <int D, int KB, int VB>
struct Codes {
  static constexpr int KW = KB, VW = VB == kPQ ? 2 : VB;   // 32-bit words of a group
  uint32_t k[KW], v[VW];
  uint16_t ks, vs;
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
// Where a thread's codes of a segment's middle tiles lie (token `tok` of tile 0, group g).
template <int D, int KB, int VB>
struct CodePtrs {
  static constexpr int G = D / 32, KW = Codes<D, KB, VB>::KW, VW = Codes<D, KB, VB>::VW;
  const uint8_t *k, *v;
  const uint16_t *ks, *vs;
  int last;   // tokens from `tok` to the tier's last
  __device__ __forceinline__ CodePtrs(const TreeArgs& a, int unit, int cur, int n_mid, int tok,
                                      int g) {
    const size_t r = ((size_t)unit * a.C + tok) * G + g;
    k = a.mk[cur] + r * (4 * KW);
    v = a.mv[cur] + r * (4 * VW);
    ks = a.mks[cur] + r;
    vs = a.mvs[cur] + r;
    last = n_mid - 1 - tok;
  }
  // Tokens past the tier read its last row (masked in S); their V is zeroed by the caller.
  __device__ __forceinline__ void load(int tile, Codes<D, KB, VB>& c) const {
    const int r = min(tile * kTok, last) * G;
    ld_words<KW>(k + r * (4LL * KW), c.k);
    ld_words<VW>(v + r * (4LL * VW), c.v);
    c.ks = __ldg(ks + r);
    if (VB != kPQ) c.vs = __ldg(vs + r);
  }
};

// Ask for a tile's codes and scales to be in L2 (contiguous runs of 16-byte multiples; the stride of
// a unit is a multiple of 64 rows, so a run may pass the tier's end but not the buffer's).
template <int D, int KB, int VB>
__device__ __forceinline__ void prefetch_codes(const TreeArgs& a, int unit, int cur, int n_mid,
                                               int t0) {
  constexpr int G = D / 32, VW = Codes<D, KB, VB>::VW;
  const int rows = min(kTok, (n_mid - t0 + 7) & ~7);   // scales: 2 G bytes a row
  const size_t r = (size_t)unit * a.C + t0;
  auto run = [](const void* x, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(x), "r"(bytes) : "memory");
  };
  run(a.mk[cur] + r * (G * 4 * KB), rows * G * 4 * KB);
  run(a.mv[cur] + r * (G * 4 * VW), rows * G * 4 * VW);
  run(a.mks[cur] + r * G, rows * G * 2);
  if (VB != kPQ) run(a.mvs[cur] + r * G, rows * G * 2);
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

// The calling warpgroup's share of the CTA's registers (HAVE a thread at the launch).
template <int N, int HAVE>
__device__ __forceinline__ void reg_set() {
  if constexpr (N > HAVE)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else if constexpr (N < HAVE)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Waits for the phase-th completion of an mbarrier, suspended by the hardware for up to 1 ms at a
// time and bounded to about 2 s; false, with the layer's status set, when it gives up.
__device__ __forceinline__ bool wait_phase(uint32_t bar, int phase, int32_t* status) {
#pragma unroll 1
  for (int i = 0; i < 2000; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"((uint32_t)phase & 1), "r"(1000000)
        : "memory");
    if (ok) return true;
  }
  record_status(status, 1);
  return false;
}

// The lowest n bits; x moved up by n places (down for a negative n). Any n.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ uint64_t shifted(uint64_t x, int n) {
  return n >= 64 || n <= -64 ? 0ull : n >= 0 ? x << n : x >> -n;
}

// One segment of a CTA's tiles: consecutive tiles of one block of query rows. Every role walks the
// same segments.
struct Segment {
  int b, h, unit, r0, rows, n, f16, tiles;   // f16, tiles: of the whole block
  int begin, end;                            // its tiles in this segment
  int n_sink, n_mid, n_rec, head, cur;
};
template <int ROWS>
__device__ __forceinline__ Segment segment_at(const AttnTreeArgs& p, const int* pre, int g,
                                              int g_end) {
  const TreeArgs& a = p.a;
  Segment s;
  s.b = row_of(pre, a.B, g);
  const RowTiles rt = row_tiles<ROWS>(a, p.n_nodes, s.b);
  const int rel = g - pre[s.b], blk = rel / rt.tiles;
  s.begin = rel % rt.tiles;
  s.end = min(rt.tiles, s.begin + (g_end - g));
  s.h = blk / rt.blocks;
  s.r0 = (blk % rt.blocks) * ROWS;
  s.rows = min(ROWS, rt.n * a.G - s.r0);
  s.n = rt.n;
  s.f16 = rt.f16;
  s.tiles = rt.tiles;
  s.unit = s.b * a.H + s.h;
  const int32_t* m = a.meta + (size_t)s.unit * FADE_META_FIELDS;
  s.n_sink = m[FADE_META_N_SINK];
  s.n_mid = m[FADE_META_N_MID];
  s.n_rec = m[FADE_META_N_RECENT];
  s.head = m[FADE_META_HEAD];
  s.cur = m[FADE_META_CUR];
  return s;
}

// One CTA per SM, three roles that meet at mbarriers. D / 8 warps unpack tiles into a ring of STAGES
// (the next tile's codes already in registers); one thread issues the products, S of the
// next tile before O of the present one, so that S is computed under the softmax; 4 R warps do the
// softmax, 16 query rows each (two rows a thread, a row spread over four lanes: no exchange between
// warps). S has two buffers; P overwrites the first columns of its own. R: 16-row halves of each
// 32-lane quarter of tensor memory in use: up to 64 query rows take lanes 0..15 of every quarter
// (R = 1), which gives each scheduler of the SM a share of the softmax; otherwise 128 (R = 2).
template <int D, int KB, int VB, int R>
__global__ void __launch_bounds__((Shape<D, KB, VB, R>::THREADS), 1)
    tree_attention_kernel(const __grid_constant__ AttnTreeArgs p) {
  using Sh = Shape<D, KB, VB, R>;
  using Cd = Codes<D, KB, VB>;
  constexpr int ROWS = 64 * R, KO = order_of(KB), VO = order_of(VB), ST = Sh::STAGES;
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ char raw[];
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  char *sQ = base, *sQL = base + Sh::TILE, *stages = sQL + Sh::LOWB;
  uint2* sCB = reinterpret_cast<uint2*>(stages + ST * Sh::STAGE);   // [256][D/4], centroid-major
  char* small = stages + ST * Sh::STAGE + Sh::CODEBOOK;
  uint64_t* bars = reinterpret_cast<uint64_t*>(small);
  uint32_t* sTm = reinterpret_cast<uint32_t*>(small + 128);
  uint32_t* sBad = reinterpret_cast<uint32_t*>(small + 160);   // [8 segments][2] see below
  int* sPre = reinterpret_cast<int*>(small + 256);             // [257]
  auto kTile = [&](int st) { return stages + st * Sh::STAGE; };
  auto vTile = [&](int st) { return stages + st * Sh::STAGE + Sh::TILE; };
  auto kLow = [&](int st) { return stages + st * Sh::STAGE + 2 * Sh::TILE; };
  const uint32_t bar0 = smem_u32(bars);
  const uint32_t kFull = bar0, kFree = bar0 + 16, vFull = bar0 + 32, vFree = bar0 + 48;   // [2]
  const uint32_t sFull = bar0 + 64, pFull = bar0 + 80;                                    // [2]
  const uint32_t oFull = bar0 + 96, oRead = bar0 + 104;
  const TreeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  tile_prefix<ROWS>(a, p.n_nodes, sPre);
  const int N = sPre[a.B];
  const int g_first = cta_start(N, gridDim.x, blockIdx.x);
  const int g_end = cta_start(N, gridDim.x, blockIdx.x + 1);
  if (g_first >= g_end) return;   // uniform over the CTA; nothing allocated yet
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(sTm)),
                 "r"(Sh::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(kFull + 8 * i, Sh::UNPACK / 32);
      mbar_init(vFull + 8 * i, Sh::UNPACK / 32);
      mbar_init(kFree + 8 * i, 1);
      mbar_init(vFree + 8 * i, 1);
      mbar_init(sFull + 8 * i, 1);
      mbar_init(pFull + 8 * i, Sh::SOFT / 32);
    }
    mbar_init(oFull, 1);
    mbar_init(oRead, Sh::SOFT / 32);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if constexpr (Sh::PQ) {
    // the codebook [D/4][256] of 8-byte centroids, transposed
    const uint2* cb = reinterpret_cast<const uint2*>(a.pq_cb);
    for (int i = tid; i < 256 * (D / 4); i += Sh::THREADS)
      sCB[(i & 255) * (D / 4) + (i >> 8)] = __ldg(cb + i);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *sTm, tmO = tm + 256;
  bool dead = false;   // a wait gave up: later ones are skipped, the flow stays the same
  auto wait = [&](uint32_t bar, int phase) {   // until the bar's phase-th completion
    if (!dead && !wait_phase(bar, phase, a.status)) dead = true;
  };
  auto arrive = [&](uint32_t bar) {   // once per warp
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp >= Sh::SOFT / 32 && warp < (Sh::SOFT + Sh::UNPACK) / 32) {
    // ================================================================ unpacking
    reg_set<Sh::REGS_UNPACK, Sh::REGS>();
    int it = 0, seg = 0, tok, gq;
    item_of<D>(tid - Sh::SOFT, tok, gq);
    for (int g = g_first; g < g_end; ++seg) {
      const Segment s = segment_at<ROWS>(p, sPre, g, g_end);
      const int n16 = s.n_sink + s.n_rec;   // cached FP16 tokens, then the nodes
      uint32_t* bad = sBad + 2 * (seg & 7);
      const CodePtrs<D, KB, VB> ptrs(a, s.unit, s.cur, s.n_mid, tok, gq);
      Cd codes, next;
      auto fetch = [&](int t, Cd& c) {   // the codes of middle tile t of the segment
        if (t >= s.f16 && t < s.end)
          ptrs.load(t - s.f16, c);
      };
      auto ahead = [&](int t) {   // tile t into L2
        if (tid == Sh::SOFT && t >= s.f16 && t < s.end)
          prefetch_codes<D, KB, VB>(a, s.unit, s.cur, s.n_mid, (t - s.f16) * kTok);
      };
      fetch(s.begin, codes);
      for (int t = 1; t < kAhead; ++t) ahead(s.begin + t);
      // Q, once the last product that reads the old one is done: matrix row 32 q + i holds query
      // row 16 q + i (R = 1, i < 16) or 32 q + i
      if (it > 0) wait(kFree + 8 * ((it - 1) % ST), (it - 1) / ST);
      if (tid == Sh::SOFT) bad[0] = bad[1] = 0;
      {
        const int in = tok & 31, r = (tok >> 5) * (16 * R) + in;
        uint4 x[4] = {};
        if (in < 16 * R && r < s.rows) {
          const int node = (s.r0 + r) >> a.log_g, gh = (s.r0 + r) & (a.G - 1);
          const uint4* src = reinterpret_cast<const uint4*>(
              a.q + (((size_t)s.b * a.T + node) * a.Hq + s.h * a.G + gh) * D + 32 * gq);
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = __ldg(src + c);
        }
        store_f16<KO>(sQ, tok, gq, x);
        if constexpr (Sh::LOW) store_low(sQL, tok, gq, x);
      }
      for (int t = s.begin; t < s.end; ++t, ++it) {
        const bool f16 = t < s.f16;
        const int st = it % ST, use = it / ST;
        const int tok0 = (f16 ? t : t - s.f16) * kTok;
        const int count = min(kTok, (f16 ? n16 + s.n : s.n_mid) - tok0);   // tokens of the tile
        ahead(t + kAhead);
        fetch(t + 1, next);
        if (use > 0) wait(kFree + 8 * st, use - 1);
        {
          if (f16) {
            uint4 x[4] = {};
            if (tok < count) {
              const uint4* src = reinterpret_cast<const uint4*>(
                  f16_row(a, D, s.b, s.h, s.unit, s.n_sink, s.n_rec, s.head, tok0 + tok, false) +
                  32 * gq);
#pragma unroll
              for (int c = 0; c < 4; ++c) x[c] = src[c];
            }
            store_f16<KO>(kTile(st), tok, gq, x);
          } else {
            store_codes<KB, Sh::LOW>(kTile(st), kLow(st), tok, gq, codes.k, codes.ks);
          }
        }
        fence_proxy_async_smem();
        arrive(kFull + 8 * st);
        if (use > 0) wait(vFree + 8 * st, use - 1);
        {
          if (f16) {
            uint4 x[4] = {};
            if (tok < count) {
              const uint4* src = reinterpret_cast<const uint4*>(
                  f16_row(a, D, s.b, s.h, s.unit, s.n_sink, s.n_rec, s.head, tok0 + tok, true) +
                  32 * gq);
#pragma unroll
              for (int c = 0; c < 4; ++c) x[c] = src[c];
              // a node's infinities and NaN would reach the rows that do not see it (0 * inf):
              // they are left out of the product and put into the rows that see it at the end
              const int node = tok0 + tok - n16;
              if (node >= 0 && clear_nonfinite(x)) atomicOr(bad + (node >> 5), 1u << (node & 31));
            }
            store_f16<VO>(vTile(st), tok, gq, x);
          } else if constexpr (Sh::PQ) {
            // lane-dependent order of the eight sub-spaces: the 32 lanes of a warp read 32
            // different sub-spaces of the centroid-major codebook, two wavefronts whatever the
            // codes
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int ss = (e + tok) & 7;
              const uint32_t w = (ss & 4) ? codes.v[1] : codes.v[0];
              const int code = (w >> (8 * (ss & 3))) & 255;
              const uint2 x = tok < count ? sCB[code * (D / 4) + 8 * gq + ss] : make_uint2(0u, 0u);
              *reinterpret_cast<uint2*>(vTile(st) + chunk_at(tok, 4 * gq + (ss >> 1)) +
                                        8 * (ss & 1)) = x;
            }
          } else {
            store_codes<VB, false>(vTile(st), nullptr, tok, gq, codes.v,
                                   tok < count ? codes.vs : (uint16_t)0);
          }
        }
        fence_proxy_async_smem();
        arrive(vFull + 8 * st);
        codes = next;
      }
      g += s.end - s.begin;
    }
  } else if (warp >= (Sh::SOFT + Sh::UNPACK) / 32) {
    // ================================================================ products
    reg_set<Sh::REGS_MMA, Sh::REGS>();
    if (warp == (Sh::SOFT + Sh::UNPACK) / 32 && lane == 0) {
      // two walks over the same tiles: S runs one tile ahead of O
      int s_left = 0, s_f16 = 0, o_left = 0, gs = g_first, go = g_first, seg = -1;
      const int total = g_end - g_first;
      for (int it = 0; it <= total; ++it) {
        if (it < total) {   // S of tile `it`
          const int st = it % ST;
          if (s_left == 0) {   // s_left tiles of the segment, s_f16 of them FP16 tiles
            const Segment s = segment_at<ROWS>(p, sPre, gs, g_end);
            s_left = s.end - s.begin;
            s_f16 = s.f16 - s.begin;
            gs += s_left;
          }
          wait(kFull + 8 * st, it / ST);
          if (it >= 2) wait(oFull, it - 2);   // P of this buffer has been read
          fence_after();
          const uint32_t d = tm + 128 * (it & 1);
          const uint32_t q = smem_u32(sQ), k = smem_u32(kTile(st));
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = (i >> 2) * kBlk + (i & 3) * 32;
            mma_ss(d, smem_desc(q + off, 16, 1024), smem_desc(k + off, 16, 1024),
                   instr_desc(kTok, false), i > 0);
          }
          if constexpr (Sh::LOW)
            if (s_f16 <= 0) {   // the remainders of a middle tile's keys
              const uint32_t ql = smem_u32(sQL), kl = smem_u32(kLow(st));
#pragma unroll
              for (int i = 0; i < D / 32; ++i)
                mma_low(d, smem_desc(ql + 32 * i, 16, 1024), smem_desc(kl + 32 * i, 16, 1024),
                        instr_desc_low(kTok));
            }
          mma_commit(kFree + 8 * st);
          mma_commit(sFull + 8 * (it & 1));
          --s_left;
          --s_f16;
        }
        if (it > 0) {   // O of the tile before
          const int jt = it - 1, st = jt % ST;
          const bool first = o_left == 0;
          if (first) {
            const Segment o = segment_at<ROWS>(p, sPre, go, g_end);
            o_left = o.end - o.begin;
            go += o_left;
            ++seg;
          }
          --o_left;
          wait(vFull + 8 * st, jt / ST);
          wait(pFull + 8 * (jt & 1), jt >> 1);
          if (first && seg > 0) wait(oRead, seg - 1);   // the last segment's O has been read
          fence_after();
          const uint32_t v = smem_u32(vTile(st)), pt = tm + 128 * (jt & 1);
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i)
            mma_ts(tmO, pt + 8 * i, smem_desc(v + i * 2048, kBlk, 1024), instr_desc(D, true),
                   !(first && i == 0));
          mma_commit(vFree + 8 * st);
          mma_commit(oFull);
        }
      }
    }
    __syncwarp();
  } else {
    // ================================================================ softmax
    reg_set<Sh::REGS_SOFT, Sh::REGS>();
    const int quarter = warp & 3, f = warp >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32 + 16 * f) << 16;
    const int row0 = quarter * (16 * R) + 16 * f + (lane >> 2);   // this thread's rows: row0, + 8
    const float cscale = kLog2e * rsqrtf((float)D);
    int it = 0, seg = 0;
    for (int g = g_first; g < g_end; ++seg) {
      const Segment s = segment_at<ROWS>(p, sPre, g, g_end);
      const int n16 = s.n_sink + s.n_rec;
      // a warp whose rows are all past the block's takes no part
      const bool active = quarter * (16 * R) + 16 * f < s.rows;
      float mref[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
      for (int t = s.begin; t < s.end; ++t, ++it) {
        const uint32_t tS = tm + 128 * (it & 1) + lanes;
        wait(sFull + 8 * (it & 1), it >> 1);
        __syncwarp();
        fence_after();
        if (active) {
          const bool f16 = t < s.f16;
          const int tok0 = (f16 ? t : t - s.f16) * kTok;
          const int count = min(kTok, (f16 ? n16 + s.n : s.n_mid) - tok0);
          const float c = f16 ? cscale : 2.f * cscale;   // middle keys are stored halved
          // what this thread's rows attend to of a tile that is not wholly visible, a bit a column
          const bool masked = f16 || count < kTok;
          uint64_t vis[2][2];   // [row][half of the columns]
          if (masked) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint64_t see = 0;
              if (f16 && row0 + 8 * e < s.rows)
                see = p.mask[(size_t)s.b * a.T + ((s.r0 + row0 + 8 * e) >> a.log_g)];
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const int c0 = tok0 + 64 * half;   // column 0 of the half as a token
                uint64_t v = low_bits(f16 ? n16 - c0 : 64) | shifted(see, f16 ? n16 - c0 : 64);
                vis[e][half] = (v & low_bits(count - 64 * half)) >> (2 * (lane & 3));
              }
            }
          }
          // 64 columns of S; -inf where a row does not attend
          auto load = [&](int half, float (&x)[32]) {
            tm_ld32(tS + 64 * half, x);
            tm_ld32(tS + 64 * half + 32, x + 16);
            tm_wait_ld();
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((vis[(i >> 1) & 1][half] >> (8 * (i >> 2) + (i & 1))) & 1)) x[i] = -INFINITY;
            }
          };
          // the upper half is read twice, so that only 32 logits are held at a time
          float x[32], mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int half = 1; half >= 0; --half) {
            load(half, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) mx[(i >> 1) & 1] = fmaxf(mx[(i >> 1) & 1], x[i]);
          }
          float ref[2], fac[2];
          bool move = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2)) * c;
            const bool up = mx[e] > mref[e] + kRefSlack;   // true from -inf
            const float to = up ? mx[e] - kRefBelow : mref[e];
            fac[e] = up ? ex2(mref[e] - to) : 1.f;
            mref[e] = to;
            lsum[e] *= fac[e];
            ref[e] = to == -INFINITY ? 0.f : to;
            move |= up;
          }
          // O of the last tile: waited for at every tile, so that no wait is two phases behind
          if (t > s.begin) {
            wait(oFull, it - 1);
            __syncwarp();
          }
          if (t > s.begin && __any_sync(0xffffffffu, move)) {
            fence_after();
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              float o[16];
              tm_ld32(tmO + lanes + 32 * q, o);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= fac[(i >> 1) & 1];
              tm_st32(tmO + lanes + 32 * q, o);
            }
          }
          // P: twice the probability where V is stored halved
          const float add = (!f16 && !Sh::PQ) ? 1.f : 0.f;
          float sum[2] = {0.f, 0.f};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (half) load(1, x);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t pk[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int e = i & 1;
                const float y = ex2(fmaf(x[16 * q + 2 * i], c, add - ref[e]));
                const float z = ex2(fmaf(x[16 * q + 2 * i + 1], c, add - ref[e]));
                sum[e] += y + z;
                const __half2 h2 = __floats2half2_rn(y, z);
                pk[i] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              // over S's lower columns, which this warp has read for its rows
              tm_st16(tS + 32 * half + 16 * q, pk);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) lsum[e] = fmaf(sum[e], add != 0.f ? 0.5f : 1.f, lsum[e]);
          tm_wait_st();
        } else if (t > s.begin) {
          wait(oFull, it - 1);
        }
        fence_before();
        arrive(pFull + 8 * (it & 1));
      }
      wait(oFull, it - 1);
      __syncwarp();
      fence_after();

      // ---------------------------------------------- the segment's result
      const bool whole = s.begin == 0 && s.end == s.tiles;
      if (active) {
        const unsigned long long bad = *reinterpret_cast<volatile unsigned long long*>(
            sBad + 2 * (seg & 7));
        float* part = p.part + ((size_t)blockIdx.x * 2 + (g == g_first ? 0 : 1)) * ROWS * (D + 2);
        size_t vec[2];
        float inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float L = lsum[e];
          L += __shfl_xor_sync(0xffffffffu, L, 1);
          L += __shfl_xor_sync(0xffffffffu, L, 2);
          const int r = row0 + 8 * e, rr = s.r0 + min(r, s.rows - 1);
          vec[e] = ((size_t)s.b * a.T + (rr >> a.log_g)) * a.Hq + s.h * a.G + (rr & (a.G - 1));
          inv[e] = mref[e] == -INFINITY ? 0.f : 1.f / L;
          if ((lane & 3) == 0 && r < s.rows) {
            if (whole)
              p.lse[vec[e]] = mref[e] == -INFINITY
                                  ? -INFINITY
                                  : (mref[e] + log2f(L)) * 0.6931471805599453f;
            else
              *reinterpret_cast<float2*>(part + 2 * r) = make_float2(mref[e], L);
          }
        }
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          float o[16];
          tm_ld32(tmO + lanes + 32 * q, o);
          tm_wait_ld();
          for (unsigned long long left = bad; left; left &= left - 1) {
            const int node = __ffsll((long long)left) - 1;
            const uint16_t* v = a.tv.x + s.b * a.tv.row_stride + node * a.tv.token_stride +
                                s.h * a.tv.head_stride;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int r = row0 + 8 * ((i >> 1) & 1);
              if (r >= s.rows || !((p.mask[(size_t)s.b * a.T + ((s.r0 + r) >> a.log_g)] >> node) & 1))
                continue;
              const float y =
                  h2f(v[channel_of<VO>(32 * q + 8 * (i >> 2) + 2 * (lane & 3) + (i & 1))]);
              if (!isfinite(y)) o[i] += y;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const int e = (i >> 1) & 1, col = 32 * q + 8 * (i >> 2) + 2 * (lane & 3);
            if (row0 + 8 * e >= s.rows) continue;
            if (whole) {
              p.out[vec[e] * D + channel_of<VO>(col)] = f2h(o[i] * inv[e]);
              p.out[vec[e] * D + channel_of<VO>(col + 1)] = f2h(o[i + 1] * inv[e]);
            } else {
              *reinterpret_cast<float2*>(part + 2 * ROWS + (size_t)(row0 + 8 * e) * D + col) =
                  make_float2(o[i], o[i + 1]);
            }
          }
        }
      }
      fence_before();
      arrive(oRead);
      g += s.end - s.begin;
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(Sh::TMEM));
}

// Joins the partials of a block of query rows that several CTAs shared, in the order of their
// tiles: one warp a row, lane l its channels (in V's order) 2l + 64 i and the next.
template <int D, int VB, int R>
__global__ void __launch_bounds__(256) tree_combine_kernel(const __grid_constant__ AttnTreeArgs p,
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
    const float* part =
        p.part + ((size_t)c * 2 + (g0 >= begin ? 0 : 1)) * ROWS * (D + 2);
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
  using Sh = Shape<D, KB, VB, R>;
  const int sms = sm_count();
  if (sms == 0) return launch_status("fade_tree_attention device query");
  // no more CTAs than the configuration can have tiles (not the present counts: see the header)
  const long long blocks = ceil_div((long long)p.a.T * p.a.G, 64 * R);
  const long long most = (long long)p.a.B * p.a.H * blocks *
                         (ceil_div(p.a.C, kTok) + ceil_div(p.a.S + p.a.W + p.a.T, kTok));
  const int P = (int)(most < sms ? most : sms);
  auto kern = tree_attention_kernel<D, KB, VB, R>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM) !=
      cudaSuccess)
    return launch_status("fade_tree_attention shared-memory opt-in");
  // the kernel's register split counts on the registers it is launched with
  static const int regs = [&] {
    cudaFuncAttributes at{};
    return cudaFuncGetAttributes(&at, kern) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < Sh::REGS)
    return set_error(FADE_ERR_UNSUPPORTED, "fade_tree_attention built with %d registers, not %d",
                     regs, Sh::REGS);
  kern<<<P, Sh::THREADS, Sh::SMEM, st>>>(p);
  fade_status_t s = launch_status("fade_tree_attention");
  if (s) return s;
  tree_combine_kernel<D, VB, R>
      <<<dim3((unsigned)(blocks * 8 * R), p.a.H, p.a.B), 256, 0, st>>>(p, P);
  return launch_status("fade_tree_attention combine");
}

template <int D, int KB, int VB>
fade_status_t launch_rows(const fade_config_t* c, const AttnTreeArgs& p, cudaStream_t st) {
  return rows_of(c, p.a.T) == 64 ? launch<D, KB, VB, 1>(c, p, st) : launch<D, KB, VB, 2>(c, p, st);
}

}  // namespace

size_t tree_attention_ws(const fade_config_t* c, int T) {
  return (size_t)kMaxSM * 2 * rows_of(c, T) * (c->head_dim + 2) * 4;
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
