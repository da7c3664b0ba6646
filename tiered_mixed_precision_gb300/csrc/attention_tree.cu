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
// Roundings to fewer than 32 bits: P and dequantised values to fp16 (2^-11 relative for INT4; values are
// held halved, so 2^-24 at least). INT4 keys: code * scale has at most 14 bits, its fp16 rounding leaves
// a remainder of at most 3, kept in E5M2; the remainder meets an E5M2 copy of the query in a second
// product (at the doubled 8-bit rate), so a logit is off by 2^-14 of its terms at most, not 2^-11. That
// holds for scales of 2^-5 and more. E5M2 ends at 2^-16, so below them a halved remainder, a multiple of
// its scale's last bit over two, loses what lies under 2^-16: a key is off by 2^-15 at most, and never by
// more than the 2^-11 of itself that fp16 alone would leave (2^-24 at least). Remainders scaled by 2^12
// (and the sum by 2^-12, which the product does for nothing) would keep every bit down to scales of
// 2^-13, but the multiplication is one more on the pipe that bounds the unpacking: 171 to 181 us at 64
// rows of 4096 tokens, 515 to 541 at the long ones.
#include <math.h>

#include "tensor_core.cuh"
#include "tree.cuh"
#include "tree_schedule.h"

namespace fade {
namespace {

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
  static constexpr int FIXED = TILE + LOWB + CODEBOOK + 11264 + 1024;   // Q, small arrays, alignment
  static constexpr int STAGES = FIXED + 2 * STAGE <= 226 * 1024 ? 2 : 1;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
  static constexpr int SOFT = 256;                            // softmax threads
  static constexpr int UNPACK = 256;                          // threads that unpack K and V
  static constexpr int THREADS = SOFT + UNPACK + 128;         // and four warps: two issue, one prefetches
  static constexpr int TMEM = 512;                            // columns: S (and P) 2 x 128, O 2 x D
};

// What a CTA leaves for the joining kernel: its tiles, and the block of query rows that begins in it
// and ends in CTA `last` (-1: none; a block within one CTA is finished there).
struct Joint {
  int tiles, last, slot, b, h, r0, rows, pad;
};

struct AttnTreeArgs {
  TreeArgs a;
  const uint64_t* mask;
  const int32_t* n_nodes;
  uint16_t* out;
  float* lse;
  Joint* joint;  // per CTA
  float* part;   // per CTA two partials: [rows][2] (m, L), then [rows][D] O
};

// ---------------------------------------------------------------- schedule
template <int ROWS>
__device__ __forceinline__ RowTiles row_tiles(const TreeArgs& a, const int32_t* n_nodes, int b) {
  const int32_t* m = a.meta + (size_t)b * a.H * FADE_META_FIELDS;
  return make_row_tiles(n_nodes ? min(max(n_nodes[b], 0), a.T) : a.T, a.G, ROWS,
                        m[FADE_META_N_SINK] + m[FADE_META_N_RECENT], m[FADE_META_N_MID]);
}
// Inclusive prefix over the rows of f(row) into pre[1 .. B] (pre[0] = 0), by the whole CTA (256 threads
// at least).
template <class F>
__device__ __forceinline__ void row_prefix(int B, int* pre, const F& f) {
  __shared__ int wsum[8];
  const int b = threadIdx.x, lane = b & 31, warp = b >> 5;
  int v = b < B ? f(b) : 0;   // B <= 256
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
// The CTA's first tile, the one after its last, and the charge, where shares are long (out of line:
// inline it took a small launch 19 to 21 us; so did the other, 173 to 176 at 64 rows of 4096 tokens).
template <int ROWS>
__device__ __noinline__ int3 long_share(const AttnTreeArgs* p, const int* pre, int* pre_blocks) {
  const TreeArgs& a = p->a;
  row_prefix(a.B, pre_blocks, [&](int b) { return a.H * row_tiles<ROWS>(a, p->n_nodes, b).blocks; });
  const int P = gridDim.x, c = blockIdx.x;
  const Rows r{pre, pre_blocks, a.B, tree_charge(pre[a.B], pre_blocks[a.B], P)};
  return make_int3(cta_start(r, P, c), cta_start(r, P, c + 1), r.charge);
}

// The CTA that takes the last tile of a block of row b that begins at tile g0, likewise.
__device__ __noinline__ int long_last(const Rows* r, int b, int g0, int tiles) {
  return cta_of(*r, gridDim.x, b, g0, tiles, tiles - 1);
}

// ---------------------------------------------------------------- tensor memory and products
// E5M2 operands, fp32 accumulator.
__host__ __device__ constexpr uint32_t instr_desc_low(int n) {
  return instr_desc(n, false) | (1u << 7) | (1u << 10);
}
__device__ __forceinline__ void mma_low(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
  asm volatile("tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, 1;" ::"r"(d), "l"(a),
               "l"(b), "r"(id)
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
// ---------------------------------------------------------------- tiles in shared memory
// Rows of 64 channels (128 bytes) under the 128-byte swizzle, one [128][64] block per 64 channels.
// An unpacking thread always writes the same group of 32 channels of the same row: four 16-byte
// chunks, chunk c at `at` ^ 16 c (`at`: the tile's address plus the thread's offset, whose bits 4..6
// already hold the swizzle).
__device__ __forceinline__ uint32_t group_at(int row, int g) {
  return (uint32_t)((g >> 1) * kBlk + row * 128 + (((4 * (g & 1)) ^ (row & 7)) << 4));
}
// The same in a tile of E5M2 (32 bytes a group): chunks 0 and 1.
__device__ __forceinline__ uint32_t low_at(int row, int g) {
  return (uint32_t)(row * 128 + (((2 * g) ^ (row & 7)) << 4));
}
__device__ __forceinline__ void st_shared8(uint32_t at, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void st_chunk(uint32_t at, int c, uint32_t x, uint32_t y, uint32_t z,
                                         uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (16 * c)), "r"(x), "r"(y),
               "r"(z), "r"(w)
               : "memory");
}
// 32 fp16 channels (one quantisation group) of a row, stored in ORDER.
template <int ORDER>
__device__ __forceinline__ void store_f16(uint32_t at, const uint4 (&x)[4]) {
  if constexpr (ORDER == kNatural) {
#pragma unroll
    for (int c = 0; c < 4; ++c) st_chunk(at, c, x[c].x, x[c].y, x[c].z, x[c].w);
  } else if constexpr (ORDER == kPair4) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      st_chunk(at, c, prmt(x[c].x, x[c].z, 0x5410), prmt(x[c].x, x[c].z, 0x7632),
               prmt(x[c].y, x[c].w, 0x5410), prmt(x[c].y, x[c].w, 0x7632));
  } else {
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
      const uint4 &p = x[c], &q = x[c + 1];
      st_chunk(at, c, prmt(p.x, q.x, 0x5410), prmt(p.x, q.x, 0x7632), prmt(p.y, q.y, 0x5410),
               prmt(p.y, q.y, 0x7632));
      st_chunk(at, c + 1, prmt(p.z, q.z, 0x5410), prmt(p.z, q.z, 0x7632),
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
// Masks of the code fields in registers the compiler does not see through: a logic operation takes
// one literal, and the offsets are it.
template <int BITS>
struct Fields {
  uint32_t m[BITS == 4 ? 2 : 5];
  __device__ __forceinline__ Fields() {
#pragma unroll
    for (int i = 0; i < (BITS == 4 ? 2 : 5); ++i) {
      m[i] = BITS == 4 ? 0x000f000fu << (4 * i) : 0x00030003u << (2 * i);
      asm volatile("" : "+r"(m[i]));
    }
  }
};
// A group of 32 codes: INT4 in four words (x), INT2 in two. LOW (INT4): the remainders as E5M2, the
// upper bytes of their fp16 form, in the same order.
template <int BITS, bool LOW>
__device__ __forceinline__ void store_codes(uint32_t at, uint32_t low, const Fields<BITS>& f,
                                            const uint32_t* x, uint32_t scale) {
  const __half2 s = __half2half2(__ushort_as_half((unsigned short)scale));
  if constexpr (BITS == 4) {
    uint32_t lo[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // nibbles at bits 0..3: 512 + u/2; at bits 4..7: 32 + u/2 (u = code + 8)
      const uint32_t w = x[c], h = w >> 8;
      uint32_t r[4] = {};
      const uint32_t a = scaled<LOW>((w & f.m[0]) ^ 0x60086008u, 0x60086008u, s, r[0]);
      const uint32_t b = scaled<LOW>((w & f.m[1]) ^ 0x50805080u, 0x50805080u, s, r[1]);
      const uint32_t d = scaled<LOW>((h & f.m[0]) ^ 0x60086008u, 0x60086008u, s, r[2]);
      const uint32_t e = scaled<LOW>((h & f.m[1]) ^ 0x50805080u, 0x50805080u, s, r[3]);
      st_chunk(at, c, a, b, d, e);
      lo[2 * c] = prmt(r[0], r[1], 0x7531);
      lo[2 * c + 1] = prmt(r[2], r[3], 0x7531);
    }
    if constexpr (LOW) {
      st_chunk(low, 0, lo[0], lo[1], lo[2], lo[3]);
      st_chunk(low, 1, lo[4], lo[5], lo[6], lo[7]);
    }
  } else {
    uint32_t none;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // crumbs at bits 0, 2, 4, 6, 8 of a half: 512, 128, 32, 8, 2 + u/2 (u = code + 2)
      const uint32_t w = x[c], h = w >> 8;
      auto sc = [&](uint32_t u, uint32_t off) { return scaled<false>(u, off, s, none); };
      st_chunk(at, 2 * c, sc((w & f.m[0]) ^ 0x60026002u, 0x60026002u),
               sc((w & f.m[1]) ^ 0x58085808u, 0x58085808u),
               sc((w & f.m[2]) ^ 0x50205020u, 0x50205020u),
               sc((w & f.m[3]) ^ 0x48804880u, 0x48804880u));
      st_chunk(at, 2 * c + 1, sc((w & f.m[4]) ^ 0x42004200u, 0x42004200u),
               sc((h & f.m[1]) ^ 0x58085808u, 0x58085808u),
               sc((h & f.m[2]) ^ 0x50205020u, 0x50205020u),
               sc((h & f.m[3]) ^ 0x48804880u, 0x48804880u));
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
__device__ __forceinline__ void store_low(uint32_t low, const uint4 (&x)[4]) {
#pragma unroll
  for (int c = 0; c < 4; c += 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4& y = x[c + i];
      w[2 * i] = to_e5m2(prmt(y.x, y.z, 0x5410)) | (to_e5m2(prmt(y.x, y.z, 0x7632)) << 16);
      w[2 * i + 1] = to_e5m2(prmt(y.y, y.w, 0x5410)) | (to_e5m2(prmt(y.y, y.w, 0x7632)) << 16);
    }
    st_chunk(low, c >> 1, w[0], w[1], w[2], w[3]);
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

// The (token, group of 32 channels) of a tile that an unpacking thread takes first (the others lie
// 128 / ITEMS tokens on): a quarter warp holds eight tokens of one group, so its 16-byte stores hit
// eight different chunks of the swizzle.
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

// Loads that stay where they are written: the compiler would sink them to their use, a tile later.
template <int W>
__device__ __forceinline__ void ld_words(const uint8_t* p, uint32_t* w) {
  if constexpr (W == 4)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
  else
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
}
__device__ __forceinline__ uint32_t ld_half(const uint16_t* p) {
  uint32_t x;   // a whole register: packing it would wait for the load
  asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

// A thread's codes and scales of a middle tile, K's or V's (W 32-bit words a group). An item's
// registers take the next tile's codes as soon as they have been unpacked.
template <int D, int W, bool SCALED, int ITEMS>
struct Codes {
  static constexpr int G = D / 32, APART = kTok / ITEMS;
  uint32_t w[ITEMS][W];
  uint32_t sc[ITEMS];
  const uint8_t* codes;
  const uint16_t* scales;
  int last;   // tokens from the thread's first row of the tile to come to the tier's last
  __device__ __forceinline__ void start(const uint8_t* c, const uint16_t* s, size_t unit_row,
                                        int n_mid, int tok, int g) {
    const size_t r = (unit_row + tok) * G + g;
    codes = c + r * (4 * W);
    scales = s + r;
    last = n_mid - 1 - tok;
  }
  // Item i of the tile to come. Tokens past the tier read its last row: their keys are masked in S,
  // their values zeroed.
  __device__ __forceinline__ void load(int i) {
    const int at = min(APART * i, last) * G;
    ld_words<W>(codes + (long long)at * (4 * W), w[i]);
    if constexpr (SCALED) sc[i] = ld_half(scales + at);
  }
  __device__ __forceinline__ void next_tile() {
    codes += kTok * G * 4 * W;
    scales += kTok * G;
    last -= kTok;
  }
  __device__ __forceinline__ void load_all() {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) load(i);
    next_tile();
  }
};

// The key and value rows of FP16 token j of a unit (sinks, then the ring oldest first, then nodes).
struct Rows16 {
  const uint16_t *k, *v;
};
__device__ __forceinline__ Rows16 f16_rows(const TreeArgs& a, int D, int b, int h, int unit,
                                           int n_sink, int n_rec, int head, int j) {
  if (j < n_sink) {
    const size_t at = ((size_t)unit * a.S + j) * D;
    return {a.sink_k + at, a.sink_v + at};
  }
  j -= n_sink;
  if (j < n_rec) {
    const size_t at = ((size_t)unit * a.W + (head + j) % a.W) * D;
    return {a.rec_k + at, a.rec_v + at};
  }
  j -= n_rec;
  return {a.tk.x + b * a.tk.row_stride + j * a.tk.token_stride + h * a.tk.head_stride,
          a.tv.x + b * a.tv.row_stride + j * a.tv.token_stride + h * a.tv.head_stride};
}

// The lowest n bits; x moved up by n places (down for a negative n). Any n.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ uint64_t shifted(uint64_t x, int n) {
  return n >= 64 || n <= -64 ? 0ull : n >= 0 ? x << n : x >> -n;
}

// One segment of a CTA's tiles: consecutive tiles of one block of query rows. The list of a CTA's
// segments is made once, in shared memory, a thread a segment.
struct Segment {
  int b, h, unit, r0, rows, n, f16, tiles;   // f16, tiles: of the whole block
  int begin, end;                            // its tiles in this segment
  int n_sink, n_mid, n_rec, head, cur;
};
template <int ROWS>
__device__ __forceinline__ int list_segments(const AttnTreeArgs& p, const Rows& rows, int g_first,
                                             int g_end, Segment* list) {
  const TreeArgs& a = p.a;
  __shared__ int count;
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  if (threadIdx.x < kMaxSeg) {
    const Place at = block_from([&](int b) { return row_tiles<ROWS>(a, p.n_nodes, b); }, rows, a.H,
                                g_first, threadIdx.x, g_end);
    const RowTiles& rt = at.rt;
    if (at.g0 < g_end) {
      Segment s;
      s.b = at.b;
      s.begin = max(g_first - at.g0, 0);
      s.end = min(rt.tiles, g_end - at.g0);
      s.h = at.blk / rt.blocks;
      s.r0 = (at.blk % rt.blocks) * ROWS;
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
      list[threadIdx.x] = s;
      atomicMax(&count, threadIdx.x + 1);
    }
  }
  __syncthreads();
  return count;
}

// What tile t of a segment needs, asked for in L2 by one warp; with a segment's first tile, its Q.
template <int D, int KB, int VB>
__device__ __forceinline__ void tile_to_l2(const AttnTreeArgs& p, const Segment& s, int t) {
  const TreeArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  auto line = [](const void* x) { asm volatile("prefetch.global.L2 [%0];" ::"l"(x)); };
  if (t == s.begin)
#pragma unroll 1
    for (int i = lane; i < s.rows; i += 32) {
      const int r = s.r0 + i;
      const uint16_t* q = a.q + (((size_t)s.b * a.T + (r >> a.log_g)) * a.Hq + s.h * a.G +
                                 (r & (a.G - 1))) * D;
      line(q);
      if (D == 128) line(q + 64);
    }
  if (t < s.f16) {
    const int end = min((t + 1) * kTok, s.n_sink + s.n_rec + s.n);
#pragma unroll 1
    for (int j = t * kTok + lane; j < end; j += 32) {
      const Rows16 x = f16_rows(a, D, s.b, s.h, s.unit, s.n_sink, s.n_rec, s.head, j);
      line(x.k);
      line(x.v);
      if (D == 128) {
        line(x.k + 64);
        line(x.v + 64);
      }
    }
  } else {
    // contiguous runs of codes and scales, a 128-byte line a lane; the stride of a unit is a multiple
    // of 64 rows, so a run may pass the tier's end but not the buffer's
    constexpr int G = D / 32, KW = KB, VW = VB == kPQ ? 2 : VB;   // 32-bit words of a group
    const int t0 = (t - s.f16) * kTok, rows = min(kTok, (s.n_mid - t0 + 63) & ~63);
    const size_t r = ((size_t)s.unit * a.C + t0) * G;
    const int cur = s.cur;
    auto run = [&](const void* x, int bytes) {
#pragma unroll 1
      for (int i = lane * 128; i < bytes; i += 32 * 128) line(static_cast<const char*>(x) + i);
    };
    run(a.mk[cur] + r * (4 * KW), rows * G * 4 * KW);
    run(a.mv[cur] + r * (4 * VW), rows * G * 4 * VW);
    run(a.mks[cur] + r, rows * G * 2);
    if (VB != kPQ) run(a.mvs[cur] + r, rows * G * 2);
  }
}

// One CTA per SM, roles that meet at mbarriers. Eight warps unpack a tile's K, then its V, into
// rings of STAGES, the next tile's codes on their way into the registers; one warp issues
// S = Q K^T, one O += P V, one asks for coming tiles in L2; 8 warps do the softmax, 16 query rows at
// a time (a thread: two rows, spread over four lanes). A tile's chain (S, softmax, P V) is long and
// mostly waiting, so even and odd tiles run as two streams, each with its softmax warps, its S (over
// which P is written), its references and its own O; the segment's end joins them. R: 16-row halves
// of each 32-lane quarter of tensor memory in use: up to 64 query rows take lanes 0..15 of every
// quarter (R = 1), which gives each scheduler of the SM a share of the softmax; otherwise 128 (R = 2).
//
// What bounds it: the unpacking warps, which wait for others 8 to 11 % of the time (the softmax warps
// 43 to 65 %); a tile costs them some 800 instructions a scheduler, and every segment the latencies of
// its FP16 tile and its Q. More than 128 query rows a unit are several blocks, each of which unpacks the
// unit's tiles anew: twice at 256 rows (the long rows below), four times at 512.
// Four warps for K and four for V left the K side as the slower one: 188 and 568 us where all
// eight on both take 184 and 524 (the two workloads below). Without softmax and products the kernel
// still takes 157 and 385, without the unpacking arithmetic, stores and loads as well 105 and 221.
// Measured, unpacking and joining included: 64 rows of 4096 middle tokens, 8 KV heads of d = 128,
// INT4 K and INT2 V, 16 nodes of 4 query heads: 173 us (271 MB, 61 GFLOP, of which the copy rate
// asks 41 us). 4 rows of 65 to 131 thousand tokens, 64 nodes: 514 us (409 GFLOP: 211 us at the rate
// of a large matrix product).
template <int D, int KB, int VB, int R>
__global__ void __launch_bounds__((Shape<D, KB, VB, R>::THREADS), 1)
    tree_attention_kernel(const __grid_constant__ AttnTreeArgs p) {
  using Sh = Shape<D, KB, VB, R>;
  constexpr int ROWS = 64 * R, KO = order_of(KB), VO = order_of(VB), ST = Sh::STAGES;
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ char raw[];
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  constexpr int kStages = Sh::TILE + Sh::LOWB;   // after Q
  const uint32_t sQ = smem_u32(base), sQL = sQ + Sh::TILE, stages = sQ + kStages;
  uint2* sCB = reinterpret_cast<uint2*>(base + kStages + ST * Sh::STAGE);   // [256][D/4]: centroid-major
  char* small = base + kStages + ST * Sh::STAGE + Sh::CODEBOOK;
  uint64_t* bars = reinterpret_cast<uint64_t*>(small);
  uint32_t* sTm = reinterpret_cast<uint32_t*>(small + 128);
  volatile int* sDone = reinterpret_cast<volatile int*>(small + 136);   // tiles unpacked
  volatile int* sDead = reinterpret_cast<volatile int*>(small + 140);   // a wait gave up
  uint32_t* sBad = reinterpret_cast<uint32_t*>(small + 160);   // [8 segments][2] see below
  int* sPre = reinterpret_cast<int*>(small + 256);             // [257] rows' first tiles
  float* sMax = reinterpret_cast<float*>(small + 1296);        // [softmax warps][2][16 rows]
  int* sBlocks = reinterpret_cast<int*>(small + 2320);         // [257] rows' blocks before
  Segment* sSeg = reinterpret_cast<Segment*>(small + 3584);    // [kMaxSeg]
  auto kTile = [&](int st) { return stages + st * Sh::STAGE; };
  auto vTile = [&](int st) { return stages + st * Sh::STAGE + Sh::TILE; };
  auto kLow = [&](int st) { return stages + st * Sh::STAGE + 2 * Sh::TILE; };
  const uint32_t bar0 = smem_u32(bars);
  const uint32_t kFull = bar0, kFree = bar0 + 16, vFull = bar0 + 32, vFree = bar0 + 48;   // [2]
  const uint32_t sFull = bar0 + 64, pFull = bar0 + 80;                                    // [2]
  const uint32_t oFull = bar0 + 96, oRead = bar0 + 112, qFull = bar0 + 120;               // [2], 1, 1
  const TreeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  // the combine kernel may be scheduled as this one drains
  asm volatile("griddepcontrol.launch_dependents;");
  row_prefix(a.B, sPre, [&](int b) {
    const RowTiles r = row_tiles<ROWS>(a, p.n_nodes, b);
    return a.H * r.blocks * r.tiles;
  });
  const int N = sPre[a.B];
  int3 share = make_int3(equal_start(N, gridDim.x, blockIdx.x),
                         equal_start(N, gridDim.x, blockIdx.x + 1), 0);
  if (N > tree_hold(gridDim.x)) share = long_share<ROWS>(&p, sPre, sBlocks);
  const int g_first = share.x, g_end = share.y;
  const Rows all{sPre, sBlocks, a.B, share.z};
  if (g_first >= g_end) {   // uniform over the CTA; nothing allocated yet
    if (tid == 0) p.joint[blockIdx.x] = Joint{0, -1};
    return;
  }
  const int n_seg = list_segments<ROWS>(p, all, g_first, g_end, sSeg);
  if (tid == Sh::THREADS - 32) {
    const Segment& s = sSeg[n_seg - 1];
    Joint j{g_end - g_first, -1, n_seg == 1 ? 0 : 1, s.b, s.h, s.r0, s.rows, 0};
    if (s.begin == 0 && s.end < s.tiles)
      j.last = all.charge ? long_last(&all, s.b, g_end - s.end, s.tiles)
                          : equal_cta_of(N, gridDim.x, g_end - s.end + s.tiles - 1);
    p.joint[blockIdx.x] = j;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(sTm)),
                 "r"(Sh::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    *sDone = 0;
    *sDead = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(kFull + 8 * i, Sh::UNPACK / 32);
      mbar_init(vFull + 8 * i, Sh::UNPACK / 32);
      mbar_init(kFree + 8 * i, 1);
      mbar_init(vFree + 8 * i, 1);
      mbar_init(sFull + 8 * i, 1);
      mbar_init(pFull + 8 * i, Sh::SOFT / 64);
      mbar_init(oFull + 8 * i, 1);
    }
    mbar_init(oRead, Sh::SOFT / 32);
    mbar_init(qFull, Sh::UNPACK / 32);
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
  auto pair_sync = [&](int pair) {   // the two softmax warps of the same rows
    __syncwarp();
    asm volatile("bar.sync %0, 64;" ::"r"(4 + pair) : "memory");
  };
  auto wait = [&](uint32_t bar, int phase) {
    wait_phase(bar, phase, bar0 + 140);
    __syncwarp();
  };
  auto arrive = [&](uint32_t bar) {   // once per warp
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp >= Sh::SOFT / 32 && warp < (Sh::SOFT + Sh::UNPACK) / 32) {
    // ================================================================ unpacking
    // every warp its share of a tile's K, then of its V: K asks for more instructions than V, and
    // half the items a thread are half the code
    constexpr int NI = kTok * (D / 32) / Sh::UNPACK, APART = kTok / NI, ROWB = APART * 128;
    const bool first = tid == Sh::SOFT;
    int it = 0, tok, gq;
    item_of<D>(tid - Sh::SOFT, tok, gq);
    const uint32_t at16 = group_at(tok, gq), at8 = low_at(tok, gq);
    // a thread's 32 channels of a row (zeros without one)
    auto load_row = [&](const uint16_t* row, uint4 (&x)[4]) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[c] = row ? *reinterpret_cast<const uint4*>(row + 32 * gq + 8 * c)
                   : make_uint4(0u, 0u, 0u, 0u);
    };
    auto f16_row = [&](const Segment& s, int j) {
      return j < s.n_sink + s.n_rec + s.n
                 ? f16_rows(a, D, s.b, s.h, s.unit, s.n_sink, s.n_rec, s.head, j)
                 : Rows16{nullptr, nullptr};
    };
    const Fields<KB> kf;
    const Fields<Sh::PQ ? 4 : VB> vf;
#pragma unroll 1
    for (int seg = 0; seg < n_seg; ++seg) {
      const Segment& s = sSeg[seg];
      const int f16 = s.f16, t_end = s.end, n_mid = s.n_mid, n16 = s.n_sink + s.n_rec;
      uint32_t* bad = sBad + 2 * (seg & 7);
      int t = s.begin;
      Codes<D, KB, true, NI> ck;
      Codes<D, Sh::PQ ? 2 : VB, !Sh::PQ, NI> cv;
      const int t0 = max(t - f16, 0) * kTok + tok;
      ck.start(a.mk[s.cur], a.mks[s.cur], (size_t)s.unit * a.C, n_mid, t0, gq);
      cv.start(a.mv[s.cur], a.mvs[s.cur], (size_t)s.unit * a.C, n_mid, t0, gq);
      if (t >= f16) {
        ck.load_all();
        cv.load_all();
      }
#pragma unroll 1
      for (; t < t_end; ++t, ++it) {
        const int st = it % ST, use = it / ST;
        // ---------------------------------------------- keys
        if (use > 0) wait(kFree + 8 * st, use - 1);
        const uint32_t k = kTile(st) + at16, v = vTile(st) + at16;
        if (t < f16) {
          uint4 x[NI][4];
#pragma unroll
          for (int i = 0; i < NI; ++i) load_row(f16_row(s, t * kTok + tok + APART * i).k, x[i]);
#pragma unroll
          for (int i = 0; i < NI; ++i) store_f16<KO>(k + i * ROWB, x[i]);
          if (t + 1 == f16 && t + 1 < t_end) {
            ck.load_all();
            cv.load_all();
          }
        } else {
          const uint32_t l = kLow(st) + at8;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            store_codes<KB, Sh::LOW>(k + i * ROWB, l + i * ROWB, kf, ck.w[i], ck.sc[i]);
            if (t + 1 < t_end) ck.load(i);
          }
          ck.next_tile();
        }
        fence_proxy_async_smem();
        arrive(kFull + 8 * st);
        if (first) *sDone = it + 1;
        // ---------------------------------------------- a segment's Q
        // matrix row 32 q + i holds query row 16 q + i (R = 1, i < 16) or 32 q + i; stored once the
        // last product that reads the old one is done
        if (t == s.begin) {
          uint4 xq[NI][4];
          if (first) bad[0] = bad[1] = 0;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int row = tok + APART * i, in = row & 31, qr = (row >> 5) * (16 * R) + in;
            const int node = (s.r0 + qr) >> a.log_g, gh = (s.r0 + qr) & (a.G - 1);
            load_row(in < 16 * R && qr < s.rows
                         ? a.q + (((size_t)s.b * a.T + node) * a.Hq + s.h * a.G + gh) * D
                         : nullptr,
                     xq[i]);
          }
          if (it > 0) wait(kFree + 8 * ((it - 1) % ST), (it - 1) / ST);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            store_f16<KO>(sQ + at16 + i * ROWB, xq[i]);
            if constexpr (Sh::LOW) store_low(sQL + at8 + i * ROWB, xq[i]);
          }
          fence_proxy_async_smem();
          arrive(qFull);
          asm volatile("bar.sync 2, %0;" ::"n"(Sh::UNPACK) : "memory");   // the nodes' bits are cleared
        }
        // ---------------------------------------------- values
        if (use > 0) wait(vFree + 8 * st, use - 1);
        if (t < f16) {
#pragma unroll 1
          for (int i = 0; i < NI; ++i) {
            uint4 x[4];
            load_row(f16_row(s, t * kTok + tok + APART * i).v, x);
            // a node's infinities and NaN would reach the rows that do not see it (0 * inf): they
            // are left out of the product and put into the rows that see it at the end
            const int node = t * kTok + tok + APART * i - n16;
            if (node >= 0 && clear_nonfinite(x)) atomicOr(bad + (node >> 5), 1u << (node & 31));
            store_f16<VO>(v + i * ROWB, x);
          }
        } else {
          const int left = n_mid - (t - f16) * kTok - tok;   // tokens from this row on
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const uint32_t vi = v + i * ROWB;
            const bool in = left > APART * i;
            if constexpr (Sh::PQ) {
              // lane-dependent order of the eight sub-spaces: the 32 lanes of a warp read 32
              // different sub-spaces of the centroid-major codebook, two wavefronts whatever the
              // codes
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int ss = (e + tok) & 7;
                const uint32_t w = (ss & 4) ? cv.w[i][1] : cv.w[i][0];
                const int code = (w >> (8 * (ss & 3))) & 255;
                const uint2 x = in ? sCB[code * (D / 4) + 8 * gq + ss] : make_uint2(0u, 0u);
                st_shared8((vi ^ (16 * (ss >> 1))) + 8 * (ss & 1), x.x, x.y);
              }
            } else {
              store_codes<VB, false>(vi, 0, vf, cv.w[i], in ? cv.sc[i] : 0u);
            }
            if (t + 1 < t_end) cv.load(i);
          }
          cv.next_tile();
        }
        fence_proxy_async_smem();
        arrive(vFull + 8 * st);
      }
    }
  } else if (warp >= (Sh::SOFT + Sh::UNPACK) / 32) {
    // ================================================================ products
    const int role = warp - (Sh::SOFT + Sh::UNPACK) / 32;
    // a warp walks as one and elects the thread that issues, so that addresses and descriptors stay
    // in uniform registers
    const bool issuer = elect_one();
    constexpr uint32_t kStage = Sh::STAGE >> 4;
    if (role == 0) {   // S = Q K^T
      const uint64_t dQ = smem_desc(sQ, 16, 1024);
      const uint64_t dK = smem_desc(kTile(0), 16, 1024);
      const uint64_t dQL = smem_desc(sQL, 16, 1024);
      const uint64_t dKL = smem_desc(kLow(0), 16, 1024);
      int it = 0;
#pragma unroll 1
      for (int seg = 0; seg < n_seg; ++seg) {
        const Segment& s = sSeg[seg];
        int f16 = s.f16 - s.begin;   // FP16 tiles left
        const int n = s.end - s.begin;
#pragma unroll 1
        for (int i = 0; i < n; ++i, --f16, ++it) {
          const int st = it % ST;
          if (it >= 2) wait(oFull + 8 * (it & 1), (it >> 1) - 1);   // the buffer's P has been read
          if (i == 0) wait(qFull, seg);
          wait(kFull + 8 * st, it / ST);
          fence_after();
          if (issuer) {
            const uint32_t d = tm + 128 * (it & 1);
            const uint64_t k = dK + st * kStage;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              const uint32_t off = ((j >> 2) * kBlk + (j & 3) * 32) >> 4;
              mma_ss(d, dQ + off, k + off, instr_desc(kTok, false), j > 0);
            }
            if constexpr (Sh::LOW)
              if (f16 <= 0) {   // the remainders of a middle tile's keys
                const uint64_t kl = dKL + st * kStage;
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                  mma_low(d, dQL + 2 * j, kl + 2 * j, instr_desc_low(kTok));
              }
            mma_commit(kFree + 8 * st);
            mma_commit(sFull + 8 * (it & 1));
          }
          __syncwarp();
        }
      }
    } else if (role == 1) {   // O += P V
      const uint64_t dV = smem_desc(vTile(0), kBlk, 1024);
      int it = 0, seg = 0;
#pragma unroll 1
      for (; seg < n_seg; ++seg) {
        const Segment& s = sSeg[seg];
        const int n = s.end - s.begin;
#pragma unroll 1
        for (int i = 0; i < n; ++i, ++it) {
          const int st = it % ST, stream = it & 1;
          wait(vFull + 8 * st, it / ST);
          wait(pFull + 8 * stream, it >> 1);
          if (i == 0 && seg > 0) wait(oRead, seg - 1);   // the last segment's O has been read
          __syncwarp();
          fence_after();
          if (issuer) {
            const uint64_t v = dV + st * kStage;
            const uint32_t pt = tm + 128 * stream, o = tmO + D * stream;
#pragma unroll
            for (int j = 0; j < kTok / 16; ++j)
              mma_ts(o, pt + 8 * j, v + ((j * 2048) >> 4), instr_desc(D, true), i > 1 || j > 0);
            mma_commit(vFree + 8 * st);
            mma_commit(oFull + 8 * stream);
          }
          __syncwarp();
        }
      }
    } else if (role == 2) {   // L2, kAhead tiles ahead of the unpacking
      int it = 0;
#pragma unroll 1
      for (int seg = 0; seg < n_seg; ++seg) {
        const Segment& s = sSeg[seg];
#pragma unroll 1
        for (int t = s.begin; t < s.end; ++t, ++it) {
          // no more than kAhead tiles before the unpacking (a pace, not an order: bounded)
#pragma unroll 1
          for (int i = 0; *sDone + kAhead < it && i < 1000; ++i) __nanosleep(200);
          tile_to_l2<D, KB, VB>(p, s, t);
        }
      }
    }
  } else {
    // ================================================================ softmax
    const int quarter = warp & 3, stream = warp >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float cscale = kLog2e * rsqrtf((float)D);
    int it0 = 0, seg = 0;   // the segment's first tile
#pragma unroll 1
    for (; seg < n_seg; ++seg) {
      const Segment& s = sSeg[seg];
      const int f16_tiles = s.f16, t_begin = s.begin, t_end = s.end, n_mid = s.n_mid, rows = s.rows;
      const int n16 = s.n_sink + s.n_rec, n_f16 = n16 + s.n;
      // 16-row groups of this warp with rows of the block
      const int groups = min(R, max(0, (rows - quarter * (16 * R) + 15) / 16));
      const int t0 = t_begin + ((it0 ^ stream) & 1);   // this stream's first tile, and every other
      // this thread's two rows' references and sums: the present group's, and the other one's (R = 2)
      float mref[2] = {-INFINITY, -INFINITY}, lsum[2] = {0.f, 0.f};
      float mref_[2] = {-INFINITY, -INFINITY}, lsum_[2] = {0.f, 0.f};
      auto other_group = [&]() {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m = mref[e], l = lsum[e];
          mref[e] = mref_[e], lsum[e] = lsum_[e];
          mref_[e] = m, lsum_[e] = l;
        }
      };
#pragma unroll 1
      for (int t = t0; t < t_end; t += 2) {
        // S of the tile; the stream's last O += P V is then complete, too
        wait(sFull + 8 * stream, (it0 + t - t_begin) >> 1);
        fence_after();
        const bool f16 = t < f16_tiles;
#pragma unroll 1
        for (int f = 0; f < groups; ++f) {
          const uint32_t at = lanes + ((uint32_t)(16 * f) << 16);
          const uint32_t tS = tm + 128 * stream + at;
          const int row0 = quarter * (16 * R) + 16 * f + (lane >> 2);   // the thread's rows: row0, + 8
          const int tok0 = (f16 ? t : t - f16_tiles) * kTok;
          const int count = min(kTok, (f16 ? n_f16 : n_mid) - tok0);
          const float c = f16 ? cscale : 2.f * cscale;   // middle keys are stored halved
          auto load = [&](int half, float (&x)[32]) {   // 64 columns of S
            tm_ld32(tS + 64 * half, x);
            tm_ld32(tS + 64 * half + 32, x + 16);
            tm_wait_ld();
          };
          float x[32], m8[8];
          if (f16 || count < kTok) {   // -inf where a row does not attend, written back into S
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              load(half, x);
              const int c0 = tok0 + 64 * half;   // the half's first column as a token
              uint64_t vis[2];                   // what the rows attend to, a bit a column
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint64_t see = 0;
                if (f16 && row0 + 8 * e < rows)
                  see = p.mask[(size_t)s.b * a.T + ((s.r0 + row0 + 8 * e) >> a.log_g)];
                const uint64_t v =
                    low_bits(f16 ? n16 - c0 : 64) | shifted(see, f16 ? n16 - c0 : 64);
                vis[e] = (v & low_bits(count - 64 * half)) >> (2 * (lane & 3));
              }
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((vis[(i >> 1) & 1] >> (8 * (i >> 2) + (i & 1))) & 1)) x[i] = -INFINITY;
              tm_st32(tS + 64 * half, x);
              tm_st32(tS + 64 * half + 32, x + 16);
            }
            tm_wait_st();
          }
          // the upper half is read twice, so that only 32 logits are held at a time
#pragma unroll
          for (int i = 0; i < 8; ++i) m8[i] = -INFINITY;
#pragma unroll
          for (int half = 1; half >= 0; --half) {
            load(half, x);
#pragma unroll
            for (int i = 0; i < 32; ++i) m8[i & 7] = fmaxf(m8[i & 7], x[i]);
          }
          float ref[2], fac[2];
          bool move = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(fmaxf(m8[2 * e], m8[2 * e + 1]), fmaxf(m8[2 * e + 4], m8[2 * e + 5]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * c;
            const bool up = mx > mref[e] + kRefSlack;   // true from -inf
            const float to = up ? mx - kRefBelow : mref[e];
            fac[e] = up ? ex2(mref[e] - to) : 1.f;
            mref[e] = to;
            lsum[e] *= fac[e];
            ref[e] = to == -INFINITY ? 0.f : to;
            move |= up;
          }
          if (t > t0 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              float o[16];
              const uint32_t ao = tmO + at + D * stream + 32 * q;
              tm_ld32(ao, o);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= fac[(i >> 1) & 1];
              tm_st32(ao, o);
            }
          }
          // P over S's lower columns: twice the probability where V is stored halved
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
              tm_st16(tS + 32 * half + 16 * q, pk);
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) lsum[e] = fmaf(sum[e], add != 0.f ? 0.5f : 1.f, lsum[e]);
          if (R == 2) other_group();
        }
        if (R == 2 && groups == 1) other_group();
        tm_wait_st();
        fence_before();
        arrive(pFull + 8 * stream);
      }
      // the stream's last O (S of its last tile said that the one before is complete)
      const int last = it0 + t_end - t_begin - 1;
      if (t0 < t_end) wait(oFull + 8 * stream, (last - ((last ^ stream) & 1)) >> 1);
      fence_after();

      // ---------------------------------------------- the segment's result: both streams joined
      const bool whole = s.begin == 0 && s.end == s.tiles;
#pragma unroll 1
      for (int f = 0; f < groups; ++f) {
        const uint32_t at = lanes + ((uint32_t)(16 * f) << 16);
        const int row0 = quarter * (16 * R) + 16 * f + (lane >> 2);
        // rows' references and sums, over the quad and exchanged with the other stream's warp
        float* mine16 = sMax + warp * 32;
        const float* other16 = sMax + (warp ^ 4) * 32;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          lsum[e] += __shfl_xor_sync(0xffffffffu, lsum[e], 1);
          lsum[e] += __shfl_xor_sync(0xffffffffu, lsum[e], 2);
          if ((lane & 3) == 0) {
            mine16[(lane >> 2) + 8 * e] = mref[e];
            mine16[(lane >> 2) + 8 * e + 16] = lsum[e];
          }
        }
        fence_before();
        pair_sync(quarter);
        fence_after();
        const unsigned long long bad =
            *reinterpret_cast<volatile unsigned long long*>(sBad + 2 * (seg & 7));
        float* part = p.part + ((size_t)blockIdx.x * 2 + (seg == 0 ? 0 : 1)) * ROWS * (D + 2);
        size_t vec[2];
        float w[2][2];   // [row][stream]: what its O counts for
        float inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m1 = other16[(lane >> 2) + 8 * e], l1 = other16[(lane >> 2) + 8 * e + 16];
          const float M = fmaxf(mref[e], m1);
          // (a row without a maximum has seen nothing, sum 0, or NaN alone, sum NaN)
          const float w0 = mref[e] == -INFINITY ? lsum[e] : ex2(mref[e] - M);
          const float w1 = m1 == -INFINITY ? l1 : ex2(m1 - M);
          // the same order of the sum in both warps
          const float L = stream ? fmaf(l1, w1, lsum[e] * w0) : fmaf(lsum[e], w0, l1 * w1);
          w[e][0] = stream ? w1 : w0;
          w[e][1] = stream ? w0 : w1;
          const int r = row0 + 8 * e, rr = s.r0 + min(r, rows - 1);
          vec[e] =
              ((size_t)s.b * a.T + (rr >> a.log_g)) * a.Hq + s.h * a.G + (rr & (a.G - 1));
          inv[e] = M == -INFINITY ? L : 1.f / L;
          if (stream == 0 && (lane & 3) == 0 && r < rows) {
            if (whole)
              p.lse[vec[e]] =
                  M == -INFINITY ? L - INFINITY : (M + log2f(L)) * 0.6931471805599453f;
            else
              *reinterpret_cast<float2*>(part + 2 * r) = make_float2(M, L);
          }
        }
#pragma unroll 1
        for (int q = 0; q < D / 64; ++q) {   // each stream's warp joins half of the columns
          float o[16], o1[16];
          const int c0 = stream * (D / 2) + 32 * q;
          tm_ld32(tmO + at + c0, o);
          tm_ld32(tmO + at + D + c0, o1);
          tm_wait_ld();
          if (q == D / 64 - 1 && f == groups - 1) {
            fence_before();
            arrive(oRead);
          }
          // (a stream without a tile, or a row that saw nothing, may hold anything)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int e = (i >> 1) & 1;
            o[i] = (w[e][0] == 0.f ? 0.f : o[i] * w[e][0]) + (w[e][1] == 0.f ? 0.f : o1[i] * w[e][1]);
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const int e = (i >> 1) & 1, col = c0 + 8 * (i >> 2) + 2 * (lane & 3);
            if (row0 + 8 * e >= rows) continue;
            if (whole) {
              p.out[vec[e] * D + channel_of<VO>(col)] = f2h(o[i] * inv[e]);
              p.out[vec[e] * D + channel_of<VO>(col + 1)] = f2h(o[i + 1] * inv[e]);
            } else {
              *reinterpret_cast<float2*>(part + 2 * ROWS + (size_t)(row0 + 8 * e) * D + col) =
                  make_float2(o[i], o[i + 1]);
            }
          }
        }
        // what was left out of the product: infinities and NaN of the nodes' values, into the rows
        // that see them (this thread's own elements; rare, so the code is kept small)
#pragma unroll 1
        for (unsigned long long left = bad; left; left &= left - 1) {
          const int node = __ffsll((long long)left) - 1;
          const uint16_t* v = a.tv.x + s.b * a.tv.row_stride + node * a.tv.token_stride +
                              s.h * a.tv.head_stride;
#pragma unroll 1
          for (int i = 0; i < D / 4; ++i) {   // D / 8 channels of two rows
            const int e = i & 1, r = row0 + 8 * e;
            const int col = stream * (D / 2) + 8 * (i >> 2) + 2 * (lane & 3) + ((i >> 1) & 1);
            if (r >= rows || !((p.mask[(size_t)s.b * a.T + ((s.r0 + r) >> a.log_g)] >> node) & 1))
              continue;
            const int ch = channel_of<VO>(col);
            const float y = h2f(v[ch]);
            if (isfinite(y)) continue;
            if (whole) {
              uint16_t* at16 = p.out + (e ? vec[1] : vec[0]) * D + ch;
              *at16 = f2h(h2f(*at16) + y);
            } else {
              part[2 * ROWS + (size_t)r * D + col] += y;
            }
          }
        }
        pair_sync(quarter);   // the exchange has been read
        if (R == 2) other_group();
      }
      if (groups == 0) arrive(oRead);
      it0 += t_end - t_begin;
    }
  }
  fence_before();
  __syncthreads();
  if (tid == 0 && *sDead) record_status(a.status, 1);
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(Sh::TMEM));
}

// Joins the partials of a block of query rows that several CTAs shared, in the order of their
// tiles. CTA x takes the block that begins in CTA x of the attention kernel and ends in a later one
// (what that CTA left says which; without it, the schedule's divisions and searches took longer than
// the sums): one warp a row, lane l its channels (in V's order) 2l + 64 i and the next. At one request
// (2 blocks of 33 partials) the attention call took 30.6 us with the schedule derived here and the
// last partials loaded one by one, 24 us now.
template <int D, int VB, int R>
__global__ void __launch_bounds__(256) tree_combine_kernel(const __grid_constant__ AttnTreeArgs p) {
  constexpr int ROWS = 64 * R, VO = order_of(VB);
  const TreeArgs& a = p.a;
  // a programmatic dependent of the attention kernel: its partials are complete from here on (and
  // no CTA ends before it, so that what follows on the stream finds it done)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x0 = blockIdx.x;
  const Joint jt = p.joint[x0];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y * 8 + warp;
  if (row >= jt.rows || jt.last < 0) return;
  float M = -INFINITY, L = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  // up to 32 partials at a time: lane l reads the (m, L) of the l-th and weighs it, then every lane
  // adds its channels, the loads of eight partials at a time independent of each other (lanes past
  // the last partial repeat its slot with weight 0)
  for (int base = x0; base <= jt.last; base += 32) {
    const int c = min(base + lane, jt.last);
    const int slot = 2 * c + (c == x0 ? jt.slot : 0);
    float2 ml = *reinterpret_cast<const float2*>(p.part + (size_t)slot * ROWS * (D + 2) + 2 * row);
    if (base + lane > jt.last || p.joint[c].tiles == 0) ml = make_float2(-INFINITY, 0.f);
    const float Mn = fmaxf(M, warp_max(ml.x));
    const float fo = M == -INFINITY ? 0.f : ex2(M - Mn);
    const float w = ml.x == -INFINITY ? ml.y : ex2(ml.x - Mn);   // (0, or NaN)
    L = fmaf(L, fo, warp_sum(ml.y * w));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= fo;
    const int n = min(32, jt.last - base + 1);
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += 8) {
#pragma unroll
      for (int j = j0; j < j0 + 8; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        const int sj = __shfl_sync(0xffffffffu, slot, j);
        const float* part = p.part + (size_t)sj * ROWS * (D + 2) + 2 * ROWS + (size_t)row * D;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const float2 x = *reinterpret_cast<const float2*>(part + 64 * i + 2 * lane);
          // (weight 0: nothing seen, or no tiles; what lies there does not matter)
          o[2 * i] = wj == 0.f ? o[2 * i] : fmaf(x.x, wj, o[2 * i]);
          o[2 * i + 1] = wj == 0.f ? o[2 * i + 1] : fmaf(x.y, wj, o[2 * i + 1]);
        }
      }
    }
    M = Mn;
  }
  const int rr = jt.r0 + row;
  const size_t vec =
      ((size_t)jt.b * a.T + (rr >> a.log_g)) * a.Hq + jt.h * a.G + (rr & (a.G - 1));
  const float inv = M == -INFINITY ? L : 1.f / L;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    p.out[vec * D + channel_of<VO>(64 * (i >> 1) + 2 * lane + (i & 1))] = f2h(o[i] * inv);
  if (lane == 0)
    p.lse[vec] = M == -INFINITY ? L - INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// SMs of the current device (cached: the query is not free); 0 on an error.
int sm_count(int* device) {
  static int known[64];
  if (cudaGetDevice(device) != cudaSuccess || *device >= 64) return 0;
  const int d = *device;
  if (known[d] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *device) != cudaSuccess)
      return 0;
    known[d] = n < kMaxSM ? n : kMaxSM;
  }
  return known[d];
}

int rows_of(const fade_config_t* c, int T) {   // query rows of a block: 64 where they are enough
  return T * (c->num_q_heads / c->num_kv_heads) <= 64 ? 64 : 128;
}

template <int D, int KB, int VB, int R>
fade_status_t launch(const fade_config_t* c, const AttnTreeArgs& p, cudaStream_t st) {
  using Sh = Shape<D, KB, VB, R>;
  int device = 0;
  const int sms = sm_count(&device);
  if (sms == 0)
    return set_error(FADE_ERR_CUDA, "fade_tree_attention: no device, or one past the 64th");
  // no more CTAs than the configuration can have tiles (not the present counts: see the header)
  const long long blocks = ceil_div((long long)p.a.T * p.a.G, 64 * R);
  const long long most = (long long)p.a.B * p.a.H * blocks *
                         (ceil_div(p.a.C, kTok) + ceil_div(p.a.S + p.a.W + p.a.T, kTok));
  const long long all = (long long)p.a.B * p.a.H * blocks;
  const int P = tree_ctas(all, most < sms ? (int)most : sms);   // one an SM
  auto kern = tree_attention_kernel<D, KB, VB, R>;
  static bool opted[64];   // per device: the kernel has its shared memory
  if (!opted[device]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM) !=
        cudaSuccess)
      return launch_status("fade_tree_attention shared-memory opt-in");
    opted[device] = true;
  }
  kern<<<P, Sh::THREADS, Sh::SMEM, st>>>(p);
  fade_status_t s = launch_status("fade_tree_attention");
  if (s) return s;
  if (P == 1) return FADE_OK;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(P - 1, 8 * R);
  lc.blockDim = dim3(256);
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, tree_combine_kernel<D, VB, R>, p);
  if (e != cudaSuccess)
    return set_error(FADE_ERR_CUDA, "fade_tree_attention combine: %s", cudaGetErrorString(e));
  return launch_status("fade_tree_attention combine");
}

template <int D, int KB, int VB>
fade_status_t launch_rows(const fade_config_t* c, const AttnTreeArgs& p, cudaStream_t st) {
  return rows_of(c, p.a.T) == 64 ? launch<D, KB, VB, 1>(c, p, st) : launch<D, KB, VB, 2>(c, p, st);
}

}  // namespace

size_t tree_attention_ws(const fade_config_t* c, int T) {
  const int rows = rows_of(c, T);
  const long long blocks = (long long)c->batch * c->num_kv_heads *
                           ceil_div((long long)T * (c->num_q_heads / c->num_kv_heads), rows);
  return (size_t)tree_ctas(blocks, kMaxSM) * (sizeof(Joint) + 2 * rows * (c->head_dim + 2) * 4);
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
  if (!aligned(mask, 8) || !aligned(lse, 4) || !aligned(n_nodes, 4))
    return set_error(FADE_ERR_INVALID_ARGUMENT,
                     "mask must be 8-byte aligned, lse and n_nodes 4-byte");
  if (ws_bytes < tree_attention_ws(c, T))
    return set_error(FADE_ERR_CAPACITY, "tree workspace %zu bytes, %zu needed", ws_bytes,
                     tree_attention_ws(c, T));
  AttnTreeArgs p{};
  p.a = make_tree_args(c, L, T, q_rot, tree_k, tree_v);
  p.mask = mask;
  p.n_nodes = n_nodes;
  p.out = out;
  p.lse = lse;
  // the workspace: a Joint a CTA, then the partials
  const long long blocks =
      (long long)c->batch * c->num_kv_heads * ceil_div((long long)T * p.a.G, rows_of(c, T));
  p.joint = static_cast<Joint*>(ws);
  p.part = reinterpret_cast<float*>(p.joint + tree_ctas(blocks, kMaxSM));
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
