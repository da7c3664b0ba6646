// Causal attention of a prompt, of a chunk of it, or of single tokens, over FP16 keys and values: every
// earlier token, or a sliding window and the first tokens ("sinks") that stay visible.
// Page "FADE：面向LLM推理的注意力感知分层KV缓存压缩技术", §第一层 (sink and recent tokens) and §核心机制:
// a position-evicted cache of S sinks and w other tokens shows a query what this attention does with
// n_sink = S and window = w.
//
// Mathematics: the query rows of a unit (row b, KV head h) are its tokens' G heads, r = token * G + g.
// Over tiles of 128 tokens, S = Q K^T, P = 2^(c S - m) with c = log2(e)/sqrt(d) and a running reference
// m per row, O += P V, L += rowsum P; out = O / L, lse = (m + log2 L) ln 2. The reference is put 6 below
// a maximum and moves only when a tile's maximum passes it by more than 14 (P stays below 2^15; fp16
// loses only what is 2^-31 of the largest P), which spares most rescalings of O.
//
// Roundings to fewer than 32 bits: P to fp16 before it meets V, the output. The tensor cores take P in 16
// bits, as V is; fp16 has three bits more than bf16, and the reference keeps P in its range. That is half a
// step, 2^-11, of every probability: errors of 2.5e-4 to 3.0e-4 of the output's norm against 64 bits, where
// the output's own rounding alone makes 2.0e-4. A second product, with what is lost of P, would take it away
// for half as many products again. L sums P before its rounding. Products of fp16 operands are exact in
// fp32, sums are fp32.
//
// What bounds it: at d = 128 the tensor cores, which a pair of tiles (256 query rows, 128 tokens) keeps
// busy for 2048 cycles of the 2700 to 3100 that the softmax's chain takes (wait, read S, maximum,
// exponentials, write P); at d = 64 the chain, 2300 to 2500 cycles against 1024 of products and as many
// of exponentials. 32 query and 8 KV heads: 16383 tokens of d = 128 1320 to 1510 us, as the clocks hold
// (1660 to 1460 TFLOP/s), of d = 64 1070 us; 2 prompts of 32768 tokens under a window of 4160 2.8 to
// 3.1 ms; 8 prompts of 1024 to 2048 tokens of d = 64 132 us, where an item's start and end cost as much
// as three of its six to eight tiles. Single tokens read their keys and values once: 64 rows of 4164
// tokens 175 us, 6.2 TB/s.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "prompt.cuh"
#include "tensor_core.cuh"
#include "tensor_map.cuh"

namespace fade {
namespace {

constexpr int kRefBelow = 6;     // log2 a new reference lies below the maximum it follows
constexpr int kRefSlack = 14;    // log2 a row's logits may pass its reference by
constexpr int kTile = kPromptTile;
constexpr int kBlk = kTile * 128;   // bytes of a [128][64] fp16 block
constexpr int kBadBufs = 8, kBadTiles = 8;   // see the checking warp

template <int D>
struct Shape {
  static constexpr int TILE = D / 64 * kBlk;            // bytes of a Q, K or V tile
  static constexpr int QBUFS = D == 128 ? 1 : 2;        // of each query tile
  static constexpr int STAGES = D == 128 ? 5 : 10;      // ring of K and V tiles
  static constexpr int SMALL = 2048;
  static constexpr int SMEM = 1024 + (2 * QBUFS + STAGES) * TILE + SMALL;
  static constexpr int THREADS = 384;   // 8 softmax warps, load, products of either tile, checks
  // Tensor memory, 512 columns: S 2 x 128, O 2 x D. P is written over S where nothing is left (d =
  // 128); otherwise it has columns of its own, and the next S need not wait for P V.
  static constexpr bool OVER = D == 128;
};

struct Args {
  CUtensorMap q, k, v;
  PromptShape s;
  PromptRows rows;
  const uint16_t* vx;            // values by address, for the rows that hold infinities or NaN
  int64_t v_row, v_tok, v_head;
  uint16_t* out;
  int64_t o_row, o_tok, o_head;
  float* lse;                    // NULL: not asked for
  float* part;                   // per CTA two partials: [part_rows][2] (m, L), then [part_rows][D] O
  int32_t* status;
  int part_rows;
  PromptUnits units;
  PromptSchedule sched;
};

// Whether a query of the block may not see all of tile kt. At most seven tiles of a block: the last
// tiles' positions and the window's first ones span at most 255 tokens each, and one tile holds the
// end of the sinks.
__device__ __forceinline__ bool is_masked(const Sight& s, const PromptItem& it, int kt) {
  const int t0 = kt * kTile, t1 = t0 + kTile - 1;
  return t1 > it.p0 || (s.window && t0 < it.p1 - s.window + 1 && t1 >= s.sink);
}
__device__ __forceinline__ bool sees(const Sight& s, int pos, int j) {
  return j <= pos && (!s.window || j > pos - s.window || j < s.sink);
}
// The lowest n bits; any n.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1;
}

// 32 lanes (a query row each) x 32 columns.
__device__ __forceinline__ void tm_ld_row(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_ld_row16(uint32_t addr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// Words w[i] of lane k of a quad become words w[k] of lane i.
__device__ __forceinline__ void transpose_quad(uint32_t (&w)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
    const bool high = lane & b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & b) continue;
      const uint32_t give = high ? w[i] : w[i | b];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, give, b);
      if (high)
        w[i] = got;
      else
        w[i | b] = got;
    }
  }
}
__device__ __forceinline__ void tm_st_row16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// One persistent CTA per SM; an item is two tiles of 128 query rows of a unit, which share every K and
// V tile. Roles meet at mbarriers: one warp loads (bulk tensor copies into a ring of K and V tiles), one
// for either query tile issues its products, four softmax warps a query tile (a thread a row) turn S
// into P. The two query tiles run free of each other but for the ring, and an item's first S is issued
// behind the last P V of the one before, while that one's result is written out. The two softmax warps
// of a scheduler take turns at the exponentials (d = 64, 16383 tokens: 1152 us without, 1123 with). What
// the loops run by comes from parameters and the block's index alone, which the compiler knows to be the
// same in a whole warp: with items told through shared memory the same loops took a quarter longer.
//
// Twice the softmax warps, in two streams of 64 tokens a query tile (d = 64): 1066 -> 1040 us at 16383
// tokens, 145 -> 167 at the short prompts, as instructions then fill two thirds of the slots.
//
// A value that is infinite or NaN would reach queries that do not see its token (0 * inf), so a warp
// looks through the V tiles that some query of the block sees only in part, clears such values and
// marks their tokens; at the end they are added for the rows that see them. Marks are kept per item, in
// kBadBufs buffers; the warp writes to a buffer only once every softmax warp is past its last user.
template <int D>
__global__ void __launch_bounds__(Shape<D>::THREADS, 1)
    prompt_attention_kernel(const __grid_constant__ Args a) {
  using Sh = Shape<D>;
  constexpr int NS = Sh::STAGES, QB = Sh::QBUFS;
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ char raw[];
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  char* tiles = base + 2 * QB * Sh::TILE;
  const uint32_t sQ = smem_u32(base), ring = smem_u32(tiles);
  char* small = tiles + NS * Sh::TILE;
  uint32_t* sBad = reinterpret_cast<uint32_t*>(small);   // [kBadBufs][kBadTiles][4]
  constexpr int kBad = kBadBufs * kBadTiles * 16;
  volatile int* sDone = reinterpret_cast<volatile int*>(small + kBad);   // [8] items behind each warp
  volatile int* sDead = sDone + 8;
  uint32_t* sTm = reinterpret_cast<uint32_t*>(small + kBad + 36);
  const uint32_t dead = smem_u32(small) + kBad + 32, bars = dead + 32;
  // [2] each, of the query tiles (Q: [QB][2])
  const uint32_t qFull = bars, qFree = qFull + 16 * QB, sFull = qFree + 16 * QB, sRead = sFull + 16,
                 pFull = sRead + 16, oDone = pFull + 16;
  const uint32_t full = oDone + 16, empty = full + 8 * NS, loaded = empty + 8 * NS;
  static_assert(kBad + 64 + 32 * QB + 64 + 24 * NS <= Sh::SMALL, "small arrays");
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const PromptShape& s = a.s;

  // (only the joining kernel may start early: nothing else after this call expects to)
  if (a.sched.join[0].last) asm volatile("griddepcontrol.launch_dependents;");
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(sTm)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    *sDead = 0;
    for (int i = 0; i < 2 * QB; ++i) {
      mbar_init(qFull + 8 * i, 1);
      mbar_init(qFree + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sFull + 8 * i, 1);
      mbar_init(sRead + 8 * i, 4);
      mbar_init(pFull + 8 * i, 4);
      mbar_init(oDone + 8 * i, 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 2);   // the products of either query tile
      mbar_init(loaded + 8 * i, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < kBad / 4) sBad[tid] = 0;
  if (tid < 8) sDone[tid] = 0;
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *sTm;
  auto wait = [&](uint32_t bar, int phase) {
    wait_phase(bar, phase, dead);
    __syncwarp();
  };
  PromptWalk<PromptItem> walk;
  PromptItem it;
  auto next = [&](PromptItem& x) {
    return walk.next(a.sched, gridDim.x, blockIdx.x,
                     [&](int index) { return prompt_item(s, a.rows, a.units, index); }, x);
  };

  // The softmax's warps take registers from the others: 4 x 80 + 8 x 208 of 12 x 168 a lane. What they
  // spilled otherwise lay in an item's end (d = 128, 8 short prompts: 172 us without, 157 with).
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 8) {
      // ================================================================ loads
      const bool issuer = elect_one();
      const int per = kTile >> s.log_g;
      int seq = 0, q_uses[2] = {0, 0};
#pragma unroll 1
      while (next(it)) {
#pragma unroll 1
        for (int j = 0; j < it.n; ++j) {
          const int kt = it.tile(j);
          const bool masked = is_masked(s.sight, it, kt);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++seq) {
            const int st = seq % NS, use = seq / NS;
            if (use > 0) wait(empty + 8 * st, use - 1);
            if (issuer) {
              const uint32_t bar = (kv && masked ? loaded : full) + 8 * st;
              mbar_expect_tx(bar, Sh::TILE);
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                load_box(ring + st * Sh::TILE + c * kBlk, kv ? &a.v : &a.k, 64 * c, kt * kTile,
                         it.h * s.kv_head[kv], it.b * s.kv_row[kv], bar);
            }
            __syncwarp();
          }
          if (j > 0) continue;
          // Q after the item's first tiles, whose copies need not wait for the last item
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t >= it.active) break;
            const int buf = 2 * (q_uses[t] % QB) + t, use = q_uses[t] / QB;
            ++q_uses[t];
            if (use > 0) wait(qFree + 8 * buf, use - 1);
            if (issuer) {
              mbar_expect_tx(qFull + 8 * buf, Sh::TILE);
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                load_box(sQ + buf * Sh::TILE + c * kBlk, &a.q, 64 * c, it.h * s.G, it.tok0 + t * per,
                         it.b * s.q_row, qFull + 8 * buf);
            }
            __syncwarp();
          }
        }
      }
    } else if (warp == 9 || warp == 10) {
      // ================================================================ products of query tile t
      const bool issuer = elect_one();
      const int t = warp - 9;
      const uint64_t dQ = smem_desc(sQ, 16, 1024), dK = smem_desc(ring, 16, 1024);
      const uint64_t dV = smem_desc(ring, kBlk, 1024);
      const uint32_t tS = tm + 128 * t, tO = tm + 256 + D * t, tP = Sh::OVER ? tS : tm + 384 + 64 * t;
      constexpr uint32_t kStage = Sh::TILE >> 4;
      int seq = 0, q_uses = 0, n_s = 0, n_p = 0;   // S issued, P taken
#pragma unroll 1
      while (next(it)) {
        if (t >= it.active) {   // (full first: a stage's next use has then begun)
#pragma unroll 1
          for (int j = 0; j < 2 * it.n; ++j, ++seq) {
            wait(full + 8 * (seq % NS), seq / NS);
            if (issuer) mbar_arrive(empty + 8 * (seq % NS));
            __syncwarp();
          }
          continue;
        }
        const int buf = 2 * (q_uses % QB) + t;
        wait(qFull + 8 * buf, q_uses / QB);
        ++q_uses;
        auto issue_s = [&](int at, bool last) {   // S = Q K^T of the tile whose K is at ring place `at`
          wait(full + 8 * (at % NS), at / NS);
          if (!Sh::OVER && n_s > 0) wait(sRead + 8 * t, n_s - 1);
          ++n_s;
          fence_after();
          if (issuer) {
            const uint64_t q = dQ + buf * kStage, kk = dK + (at % NS) * kStage;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t off = ((i >> 2) * kBlk + (i & 3) * 32) >> 4;
              mma_ss(tS, q + off, kk + off, instr_desc(kTile, false), i > 0);
            }
            mma_commit(sFull + 8 * t);
            mma_commit(empty + 8 * (at % NS));
            if (last) mma_commit(qFree + 8 * buf);
          }
          __syncwarp();
        };
        issue_s(seq, it.n == 1);
#pragma unroll 1
        for (int j = 0; j < it.n; ++j, seq += 2) {
          const int sv = (seq + 1) % NS;
          const bool more = j + 1 < it.n;
          if (!Sh::OVER && more) issue_s(seq + 2, j + 2 == it.n);
          wait(full + 8 * sv, (seq + 1) / NS);
          wait(pFull + 8 * t, n_p++);
          fence_after();
          if (issuer) {
            const uint64_t v = dV + sv * kStage;
#pragma unroll
            for (int i = 0; i < kTile / 16; ++i)
              mma_ts(tO, tP + 8 * i, v + ((i * 2048) >> 4), instr_desc(D, true), j > 0 || i > 0);
            mma_commit(oDone + 8 * t);
            mma_commit(empty + 8 * sv);
          }
          __syncwarp();
          if (Sh::OVER && more) issue_s(seq + 2, j + 2 == it.n);
        }
      }
    } else {
      // ================================================================ values that are not finite
      uint32_t phases = 0, dirty = 0;   // of `loaded`, a bit a stage; buffers that hold marks
      int seq = 0, count = 0;
#pragma unroll 1
      for (; next(it); ++count) {
        const int buf = count % kBadBufs;
        uint32_t* bad = sBad + buf * (kBadTiles * 4);
        bool ready = false;
        auto own = [&]() {   // the buffer's last user is done with it (a bounded wait)
          if (!ready && count >= kBadBufs) {
            const long long t0 = clock64();
            while (!*sDead && __any_sync(0xffffffffu, sDone[lane & 7] <= count - kBadBufs))
              if (clock64() - t0 > kWaitCycles) *sDead = 1;
          }
          ready = true;
        };
        if ((dirty >> buf) & 1) {
          own();
          bad[lane] = 0;
          dirty &= ~(1u << buf);
          __syncwarp();
        }
        int slot = 0;
#pragma unroll 1
        for (int j = 0; j < it.n; ++j, seq += 2) {
          if (!is_masked(s.sight, it, it.tile(j))) continue;
          const int st = (seq + 1) % NS;
          wait(loaded + 8 * st, (phases >> st) & 1);
          phases ^= 1u << st;
          uint4* tile = reinterpret_cast<uint4*>(tiles + st * Sh::TILE);
#pragma unroll 1
          for (int i0 = lane; i0 < Sh::TILE / 16; i0 += 8 * 32) {
            uint32_t inf[8];
            uint4 x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = tile[i0 + 32 * e];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              auto f = [](uint32_t w) { return (w & 0x7c007c00u) + 0x04000400u; };
              inf[e] = (f(x[e].x) | f(x[e].y) | f(x[e].z) | f(x[e].w)) & 0x80008000u;
            }
            if (!__any_sync(0xffffffffu, inf[0] | inf[1] | inf[2] | inf[3] | inf[4] | inf[5] | inf[6] |
                                             inf[7]))
              continue;
            own();
            dirty |= 1u << buf;
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
              const int i = i0 + 32 * e, row = (i >> 3) & 127;
              uint32_t w[4] = {tile[i].x, tile[i].y, tile[i].z, tile[i].w};
              bool any = false;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t lo = (w[q] & 0x7c00u) == 0x7c00u ? 0xffffu : 0u;
                const uint32_t hi = (w[q] & 0x7c000000u) == 0x7c000000u ? 0xffff0000u : 0u;
                any |= (lo | hi) != 0;
                w[q] &= ~(lo | hi);
              }
              if (any) {
                tile[i] = make_uint4(w[0], w[1], w[2], w[3]);
                atomicOr(bad + 4 * slot + (row >> 5), 1u << (row & 31));
              }
            }
          }
          ++slot;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + 8 * st);
        }
      }
    }
  } else {
    // ================================================================ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tm + 128 * t + lanes, tO = tm + 256 + D * t + lanes;
    const uint32_t tP = Sh::OVER ? tS : tm + 384 + 64 * t + lanes;
    const float c = kLog2e * rsqrtf((float)D);
    const f2x c2 = f2_pack(c, c);
    auto arrive = [&](uint32_t bar) {
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    const int turn = 1 + 2 * (warp & 3) + t, others = 1 + 2 * (warp & 3) + (t ^ 1);
    if (t == 1) asm volatile("bar.arrive %0, 64;" ::"r"(others) : "memory");
    int n_s = 0, count = 0;   // S waited for, items
    bool some = next(it);
#pragma unroll 1
    for (; some; ++count) {
      __syncwarp();
      if (lane == 0) sDone[warp] = count;
      if (t >= it.active) {
        some = next(it);
        continue;
      }
      const int per = kTile >> s.log_g, tok = it.tok0 + t * per + (r >> s.log_g);
      const int q_len = a.rows.q_len[it.b], pos = it.off + tok;
      // rows of this warp with a query, uniformly
      const bool live = it.tok0 + t * per + (((warp & 3) * 32) >> s.log_g) < q_len;
      const bool turns = it.active == 2 && it.tok0 + (((warp & 3) * 32 + 128) >> s.log_g) < q_len;
      float ref = -INFINITY, sum = 0.f;
      bool masks = false;
#pragma unroll 1
      for (int j = 0; j < it.n; ++j) {
        const int kt = it.tile(j);
        const bool masked = is_masked(s.sight, it, kt);
        masks |= masked;
        wait(sFull + 8 * t, n_s++);
        fence_after();
        float x[128];
        if (live) {
#pragma unroll
          for (int i = 0; i < 4; ++i) tm_ld_row(tS + 32 * i, x + 32 * i);
          tm_wait_ld();
        }
        if (!Sh::OVER) arrive(sRead + 8 * t);
        float fac = 1.f;
        bool up = false;
        if (live) {
          if (masked) {
            const int hi = pos - kt * kTile;
            const int lo = s.sight.window ? hi - s.sight.window : -1;   // the last one not seen
            const int si = s.sight.sink - kt * kTile;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t see = low_bits(hi + 1 - 32 * q) &
                                   (~low_bits(lo + 1 - 32 * q) | low_bits(si - 32 * q));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(see & (1u << i))) x[32 * q + i] = -INFINITY;
            }
          }
          float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i < 128; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              m4[e] = i + 4 + e < 128 ? fmaxf(fmaxf(m4[e], x[i + e]), x[i + 4 + e])
                                      : fmaxf(m4[e], x[i + e]);
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
          up = mx > ref + kRefSlack;   // true from -inf
          if (up) {
            fac = ex2(ref - (mx - kRefBelow));
            ref = mx - kRefBelow;
            sum *= fac;
          }
        }
        // the last P V is done: O may be scaled, P's columns written
        if (j > 0) {
          wait(oDone + 8 * t, n_s - 2);
          fence_after();
          if (__any_sync(0xffffffffu, up)) {
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              float o[16];
              tm_ld_row16(tO + 16 * q, o);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= fac;
              tm_st_row16(tO + 16 * q, reinterpret_cast<const uint32_t*>(o));
            }
          }
        }
        if (turns) asm volatile("bar.sync %0, 64;" ::"r"(turn) : "memory");
        if (live) {
          const float sub = ref == -INFINITY ? 0.f : -ref;
          const f2x sub2 = f2_pack(sub, sub);
          f2x acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const f2x y = f2_fma(f2_pack(x[32 * q + 2 * i], x[32 * q + 2 * i + 1]), c2, sub2);
              float y0, y1;
              f2_unpack(y, y0, y1);
              y0 = ex2(y0);
              y1 = ex2(y1);
              acc[i & 1] = f2_add(acc[i & 1], f2_pack(y0, y1));
              const __half2 h2 = __floats2half2_rn(y0, y1);
              pk[i] = *reinterpret_cast<const uint32_t*>(&h2);
            }
            tm_st_row16(tP + 16 * q, pk);
          }
          if (turns) asm volatile("bar.arrive %0, 64;" ::"r"(others) : "memory");
          float a0, a1, b0, b1;
          f2_unpack(acc[0], a0, a1);
          f2_unpack(acc[1], b0, b1);
          sum += (a0 + a1) + (b0 + b1);
          tm_wait_st();
        }
        arrive(pFull + 8 * t);
      }
      // the next item is worked out while the last P V runs
      const PromptItem now = it;
      some = next(it);
      wait(oDone + 8 * t, n_s - 1);
      fence_after();
      if (!live) continue;

      // ---------------------------------------------- the item's result
      // Read so that a quad of lanes holds consecutive channels of a row, and written 64 bytes a row:
      // with a thread a row, every 16-byte store met 32 lines (16383 tokens of d = 128: 1455 us, 1403 now;
      // 8 short prompts of d = 64: 162, 148 now).
      const bool whole = now.n == now.all;
      const uint32_t* bad = sBad + (count % kBadBufs) * (kBadTiles * 4);
      const bool any_bad =
          masks && __any_sync(0xffffffffu, reinterpret_cast<const volatile uint32_t*>(bad)[lane] != 0);
      float* part = a.part + ((size_t)blockIdx.x * 2 + (now.begin == 0 ? 1 : 0)) * a.part_rows * (D + 2);
      if (tok < q_len) {
        if (!whole)
          *reinterpret_cast<float2*>(part + 2 * (128 * t + r)) = make_float2(ref, sum);
        else if (a.lse)
          a.lse[((size_t)now.b * s.n_q + tok) * s.Hq + now.h * s.G + (r & (s.G - 1))] =
              (ref + log2f(sum)) * 0.6931471805599453f;
      }
      const float inv = 1.f / sum;
      part += 2 * a.part_rows;
      // A thread's rows are 8 apart, so by whole tokens (G <= 8) and with one head.
      const int row0 = (warp & 3) * 32 + (lane >> 2), step = 8 >> s.log_g;
      const int tk0 = now.tok0 + t * per + (row0 >> s.log_g);
      const int64_t at0 = now.b * a.o_row + tk0 * a.o_tok + (now.h * s.G + (row0 & (s.G - 1))) * a.o_head;
#pragma unroll 1
      for (int f = 0; f < 2; ++f) {   // 16 rows at a time, two of them in a thread
        float scale[2];
        bool mine[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mine[e] = tk0 + (2 * f + e) * step < q_len;
          scale[e] = __shfl_sync(0xffffffffu, inv, 16 * f + 8 * e + (lane >> 2));
        }
#pragma unroll 1
        for (int q = 0; q < D / 32; q += 2) {
          float o[2][16];
          __syncwarp();
#pragma unroll
          for (int z = 0; z < 2; ++z) tm_ld32(tO + ((uint32_t)(16 * f) << 16) + 32 * (q + z), o[z]);
          tm_wait_ld();
          if (any_bad) {   // what was left out of the products, into the rows that see it
            int slot = 0;
#pragma unroll 1
            for (int j = 0; j < now.n; ++j) {
              const int kt = now.tile(j);
              if (!is_masked(s.sight, now, kt)) continue;
#pragma unroll 1
              for (int w = 0; w < 4; ++w)
#pragma unroll 1
                for (uint32_t left = bad[4 * slot + w]; left; left &= left - 1) {
                  const int key = kt * kTile + 32 * w + __ffs(left) - 1;
                  const uint16_t* v = a.vx + now.b * a.v_row + key * a.v_tok + now.h * a.v_head +
                                      32 * q + 2 * (lane & 3);
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    if (!mine[e] || !sees(s.sight, now.off + tk0 + (2 * f + e) * step, key)) continue;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                      const float y = h2f(v[8 * (i >> 1) + (i & 1)]);
                      if (!isfinite(y)) o[i >> 3][4 * ((i & 7) >> 1) + 2 * e + (i & 1)] += y;
                    }
                  }
                }
              ++slot;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (whole) {
              uint16_t* out = a.out + at0 + (2 * f + e) * (step * a.o_tok) + 32 * q + 8 * (lane & 3);
              __syncwarp();
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __half2 h2 = __floats2half2_rn(o[z][4 * i + 2 * e] * scale[e],
                                                       o[z][4 * i + 2 * e + 1] * scale[e]);
                  w[i] = *reinterpret_cast<const uint32_t*>(&h2);
                }
                transpose_quad(w);
                if (mine[e])
                  *reinterpret_cast<uint4*>(out + 32 * z) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else if (mine[e]) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float2*>(part + (size_t)(128 * t + row0 + 8 * (2 * f + e)) * D + 32 * q +
                                           8 * i + 2 * (lane & 3)) =
                    make_float2(o[i >> 2][4 * (i & 3) + 2 * e], o[i >> 2][4 * (i & 3) + 2 * e + 1]);
            }
          }
        }
      }
      __syncwarp();
      fence_before();
    }
    __syncwarp();
    if (lane == 0) sDone[warp] = 1 << 30;
    if (t == 0) asm volatile("bar.sync %0, 64;" ::"r"(turn) : "memory");   // (the first turn again)
  }
  fence_before();
  __syncthreads();
  if (tid == 0 && *sDead) record_status(a.status, 1);
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
}

// Joins the partials of an item that several CTAs shared, in the order of its tiles: a warp a query
// row, lane l the channels 2l + 64 i and the next.
template <int D>
__global__ void __launch_bounds__(256) prompt_combine_kernel(const __grid_constant__ Args a) {
  const PromptShape& s = a.s;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const auto& jn = a.sched.join[blockIdx.x];
  const PromptItem it = prompt_item(s, a.rows, a.units, jn.item);
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int tok = it.tok0 + (row >> s.log_g);   // (query tile 1 begins at row 128)
  if (tok >= a.rows.q_len[it.b]) return;
  float M = -INFINITY, L = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  const size_t slot = (size_t)a.part_rows * (D + 2);
#pragma unroll 1
  for (int c0 = jn.first; c0 <= jn.last; c0 += 8) {
    float2 ml[8];
    float2 x[8][D / 64];
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      const int c = min(c0 + z, (int)jn.last);
      // (a CTA between them may have no share)
      const bool has = c0 + z <= jn.last && (a.sched.start[c].item != a.sched.start[c + 1].item ||
                                             a.sched.start[c].tile != a.sched.start[c + 1].tile);
      const float* p = a.part + (2 * c + (c == jn.first ? 1 : 0)) * slot;
      ml[z] = has ? *reinterpret_cast<const float2*>(p + 2 * row) : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        x[z][i] = has ? *reinterpret_cast<const float2*>(p + 2 * a.part_rows + (size_t)row * D +
                                                         64 * i + 2 * lane)
                      : make_float2(0.f, 0.f);
    }
    float Mn = M;
#pragma unroll
    for (int z = 0; z < 8; ++z) Mn = fmaxf(Mn, ml[z].x);
    const float f = M == -INFINITY ? 0.f : ex2(M - Mn);
    L *= f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= f;
#pragma unroll
    for (int z = 0; z < 8; ++z) {
      // without a maximum nothing was seen, sum 0, or NaN alone, sum NaN
      const float w = ml[z].x == -INFINITY ? ml[z].y : ex2(ml[z].x - Mn);
      // (a weight of 0 leaves nothing of numbers, but what is none reaches the result, as in a whole item)
      auto add = [&](float v, float sum) { return isfinite(v) ? fmaf(v, w, sum) : sum + v; };
      L = add(ml[z].y, L);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        o[2 * i] = add(x[z][i].x, o[2 * i]);
        o[2 * i + 1] = add(x[z][i].y, o[2 * i + 1]);
      }
    }
    M = Mn;
  }
  const int head = it.h * s.G + (row & (s.G - 1));
  uint16_t* out = a.out + it.b * a.o_row + tok * a.o_tok + head * a.o_head;
  const float inv = 1.f / L;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const __half2 h2 = __floats2half2_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
    *reinterpret_cast<uint32_t*>(out + 64 * i + 2 * lane) = *reinterpret_cast<const uint32_t*>(&h2);
  }
  if (lane == 0 && a.lse)
    a.lse[((size_t)it.b * s.n_q + tok) * s.Hq + head] = (M + log2f(L)) * 0.6931471805599453f;
}

// Blocks of two query tiles of a unit whose row has n queries.
int blocks_of(const fade_config_t* c, long long n) {
  return ceil_div(n * (c->num_q_heads / c->num_kv_heads), 2 * kTile);
}
// Query rows of a partial; a multiple of 8, so that its vectors start 16-byte aligned.
int partial_rows(const fade_config_t* c, int n_q) {
  const long long rows = (long long)n_q * (c->num_q_heads / c->num_kv_heads);
  return (int)std::min<long long>((rows + 7) / 8 * 8, 2 * kTile);
}

template <int D>
fade_status_t launch(const fade_config_t* c, Args& a, int blocks, cudaStream_t st) {
  using Sh = Shape<D>;
  int device = 0;
  const int sms = prompt_sms(&device);
  if (sms == 0) return FADE_ERR_CUDA;
  a.part_rows = partial_rows(c, a.s.n_q);
  a.units.set(a.s);
  int P = 0;
  const int joins = prompt_schedule(a.s, a.rows, blocks, sms, a.sched, &P);
  auto kern = prompt_attention_kernel<D>;
  static std::atomic<bool> opted[64];   // per device: the kernel has its shared memory
  if (!opted[device]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM) !=
        cudaSuccess)
      return launch_status("fade_prompt_attention shared-memory opt-in");
    opted[device] = true;
  }
  kern<<<P, Sh::THREADS, Sh::SMEM, st>>>(a);
  fade_status_t s = launch_status("fade_prompt_attention");
  if (s || joins == 0) return s;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(joins, a.part_rows / 8);
  lc.blockDim = dim3(256);
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, prompt_combine_kernel<D>, a);
  if (e != cudaSuccess)
    return set_error(FADE_ERR_CUDA, "fade_prompt_attention combine: %s", cudaGetErrorString(e));
  return launch_status("fade_prompt_attention combine");
}

}  // namespace

size_t prompt_attention_ws(const fade_config_t* c, int32_t n_q) {
  return (size_t)2 * kPromptSMs * partial_rows(c, n_q) * (c->head_dim + 2) * 4;
}

int prompt_sms(int* device) {
  static std::atomic<int> known[64];
  if (cudaGetDevice(device) != cudaSuccess || *device >= 64) {
    set_error(FADE_ERR_CUDA, "no device, or one past the 64th");
    return 0;
  }
  const int d = *device;
  int n = known[d];
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) {
      launch_status("SM count");
      return 0;
    }
    known[d] = n = n < kPromptSMs ? n : kPromptSMs;
  }
  return n;
}

fade_status_t prompt_shape(const fade_config_t* c, const fade_heads_t* q, const fade_heads_t* k,
                           const fade_heads_t* v, int32_t n_q, int32_t n_kv, const int32_t* h_q_len,
                           const int32_t* h_kv_len, int32_t n_sink, int32_t window,
                           PromptShape* shape, PromptRows* rows) {
  fade_status_t st = validate_config(c);
  if (st) return st;
  if (n_q < 1 || n_kv < 1 || n_q > FADE_PROMPT_MAX_TOKENS || n_kv > FADE_PROMPT_MAX_TOKENS)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "%d queries or %d tokens outside [1, %d]", n_q, n_kv,
                     FADE_PROMPT_MAX_TOKENS);
  if (n_sink < 0 || window < 0)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "n_sink %d or window %d below 0", n_sink, window);
  struct {
    const fade_heads_t* x;
    const char* name;
    int tokens, heads;
  } in[3] = {{q, "q", n_q, c->num_q_heads},
             {k, "k", n_kv, c->num_kv_heads},
             {v, "v", n_kv, c->num_kv_heads}};
  for (int i = 0; i < (v ? 3 : 2); ++i) {
    if ((st = validate_heads(in[i].x, in[i].name))) return st;
    const fade_heads_t& x = *in[i].x;
    if (x.row_stride < 0 || x.token_stride < 0 || x.head_stride < 0)
      return set_error(FADE_ERR_UNSUPPORTED, "%s: negative strides", in[i].name);
    if ((x.token_stride == 0 && in[i].tokens > 1) ||
        (i == 0 && x.head_stride == 0 && in[i].heads > 1))
      return set_error(FADE_ERR_UNSUPPORTED, "%s: the same vector for every token%s", in[i].name,
                       i == 0 ? " or head" : "");
  }
  PromptShape& s = *shape;
  s.B = c->batch;
  s.H = c->num_kv_heads;
  s.Hq = c->num_q_heads;
  s.G = s.Hq / s.H;
  s.log_g = 0;
  while ((1 << s.log_g) < s.G) ++s.log_g;   // G is 1, 2, 4 or 8
  s.n_q = n_q;
  s.n_kv = n_kv;
  s.sight.window = window < n_kv ? window : 0;   // (a window of all tokens hides none)
  s.sight.sink = s.sight.window ? std::min(n_sink, n_kv) : 0;
  s.q_row = q->row_stride != 0;
  s.kv_row[0] = k->row_stride != 0;
  s.kv_head[0] = k->head_stride != 0;
  s.kv_row[1] = v && v->row_stride != 0;
  s.kv_head[1] = v && v->head_stride != 0;
  for (int b = 0; b < s.B; ++b) {
    const int ql = h_q_len ? h_q_len[b] : n_q, kl = h_kv_len ? h_kv_len[b] : n_kv;
    if (ql < 0 || ql > n_q || kl < 0 || kl > n_kv || ql > kl)
      return set_error(FADE_ERR_INVALID_ARGUMENT,
                       "row %d: %d queries outside [0, %d], %d tokens outside [0, %d], or fewer tokens "
                       "than queries",
                       b, ql, n_q, kl, n_kv);
    rows->q_len[b] = ql;
    rows->kv_len[b] = kl;
    rows->order[b] = (uint8_t)b;
  }
  std::stable_sort(rows->order, rows->order + s.B,
                   [&](uint8_t x, uint8_t y) { return rows->kv_len[x] > rows->kv_len[y]; });
  return FADE_OK;
}

}  // namespace fade

using namespace fade;

extern "C" size_t fade_prompt_ws_bytes(const fade_config_t* c, int32_t n_q, int32_t n_kv) {
  clear_error();
  if (validate_config(c)) return 0;
  if (n_q < 1 || n_kv < 1 || n_q > FADE_PROMPT_MAX_TOKENS || n_kv > FADE_PROMPT_MAX_TOKENS) {
    set_error(FADE_ERR_INVALID_ARGUMENT, "%d queries or %d tokens outside [1, %d]", n_q, n_kv,
              FADE_PROMPT_MAX_TOKENS);
    return 0;
  }
  return std::max(prompt_attention_ws(c, n_q), prompt_mass_ws());
}

extern "C" fade_status_t fade_prompt_attention(const fade_config_t* c, const fade_heads_t* q,
                                               const fade_heads_t* k, const fade_heads_t* v,
                                               int32_t n_q, int32_t n_kv, const int32_t* h_q_len,
                                               const int32_t* h_kv_len, int32_t n_sink,
                                               int32_t window, const fade_heads_t* out, float* lse,
                                               int32_t* status, void* ws, size_t ws_bytes,
                                               void* stream) {
  clear_error();
  FADE_RANGE("fade_prompt_attention");
  if (!v || !v->x) return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL v");
  Args a{};
  fade_status_t st = prompt_shape(c, q, k, v, n_q, n_kv, h_q_len, h_kv_len, n_sink, window, &a.s,
                                  &a.rows);
  if (!st) st = validate_heads(out, "out");
  if (st) return st;
  if ((out->row_stride == 0 && a.s.B > 1) || (out->token_stride == 0 && n_q > 1) ||
      (out->head_stride == 0 && a.s.Hq > 1))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "out: rows, queries or heads share vectors");
  if (!ws || !aligned(ws, 16))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(status, 4))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "lse and status must be 4-byte aligned");
  if (ws_bytes < prompt_attention_ws(c, n_q))
    return set_error(FADE_ERR_CAPACITY, "prompt workspace %zu bytes, %zu needed", ws_bytes,
                     prompt_attention_ws(c, n_q));
  int blocks = 0;
  for (int b = 0; b < a.s.B; ++b) blocks = std::max(blocks, blocks_of(c, a.rows.q_len[b]));
  if (blocks == 0) return FADE_OK;
  if ((long long)blocks * a.s.B * a.s.H > (1 << 30))
    return set_error(FADE_ERR_UNSUPPORTED, "fade_prompt_attention: more than 2^30 blocks of queries");
  const int d = c->head_dim, per = kTile / a.s.G;
  st = encode_heads(&a.q, "q", *q, d, a.s.Hq, n_q, a.s.B, a.s.G, per, true);
  if (!st) st = encode_heads(&a.k, "k", *k, d, a.s.H, n_kv, a.s.B, 1, kTile, false);
  if (!st) st = encode_heads(&a.v, "v", *v, d, a.s.H, n_kv, a.s.B, 1, kTile, false);
  if (st) return st;
  a.vx = v->x;
  a.v_row = v->row_stride;
  a.v_tok = v->token_stride;
  a.v_head = v->head_stride;
  a.out = out->x;
  a.o_row = out->row_stride;
  a.o_tok = out->token_stride;
  a.o_head = out->head_stride;
  a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.status = status;
  return d == 64 ? launch<64>(c, a, blocks, as_stream(stream))
                 : launch<128>(c, a, blocks, as_stream(stream));
}
