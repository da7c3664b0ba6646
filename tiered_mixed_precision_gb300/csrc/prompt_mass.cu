// Column sums of a prompt's attention: the importance that its tokens start with.
// Pages "探秘Transformer系列之（25）--- KV Cache优化之处理长文本序列", §1.3.1 H2O (a token's importance is the
// column sum of the attention matrix) and FADE-zh §四种驱逐策略详解 1 (captured at prefill).
//
// Mathematics: mass[j] = sum over the query rows r of the unit that see key j of 2^(c S[r][j] - l[r]),
// c = log2(e)/sqrt(d), l = log2(e) lse. The attention's log-sum-exp makes it one pass: no maximum, no
// second sum. Products run transposed, S^T = K Q^T, so that a thread of a softmax warp owns a key and
// its sum stays in a register.
//
// A term is off by what scaling its logit and its lse rounds (2^-24 of either) and by ex2: 1.7e-7 to 2.8e-7
// of the masses' norm against 64 bits, where the elementary fp32 form has 0.5e-7 to 0.8e-7.
// Sums are fp32: 16 terms a key and lane in a tile, the tiles of a share, four lanes, two warps, the
// shares of the CTAs that took the key's tiles; each in one fixed order. No atomics: the same bits on
// every run.
//
// What bounds it: instruction issue, 0.66 to 0.70 a cycle and scheduler. Of some 260 instructions of a
// warp and tile, 140 are the 64 exponentials, their scaling and their sums. 32 query and 8 KV heads: 8
// prompts of 1024 to 2048 tokens of d = 64 94 us (the exponentials alone, 32 a clock and SM: 37); 32768
// tokens of d = 128 under a window of 4160 865 to 1050 us, as the clocks hold (1210 to 1000 TFLOP/s).
#include <math.h>

#include <algorithm>
#include <atomic>

#include "prompt.cuh"
#include "tensor_core.cuh"
#include "tensor_map.cuh"

namespace fade {
namespace {

constexpr int kTile = kPromptTile;   // keys of a tile, and query rows of one
constexpr int kBlk = kTile * 128;    // bytes of a [128][64] fp16 block
constexpr int kPair = 2 * kTile;     // keys of an item

template <int D>
struct Shape {
  static constexpr int TILE = D / 64 * kBlk;          // bytes of a K or Q tile
  static constexpr int STAGES = D == 128 ? 4 : 8;     // ring of Q tiles
  static constexpr int SMALL = 3 * 1024;   // barriers, lse, halves
  static constexpr int SMEM = 1024 + 2 * TILE + STAGES * TILE + SMALL;
  static constexpr int THREADS = 640;   // 16 warps that sum, load, products, 2 that scale lse
};

struct Args {
  CUtensorMap q, k;
  PromptShape s;
  PromptRows rows;
  const float* lse;
  float* mass;
  float* part;      // per CTA two partials of kPair sums
  int32_t* status;
  int add;
  PromptUnits units;
  PromptSchedule sched;
};

// One persistent CTA per SM; an item is two tiles of 128 keys of a unit, both met by every query tile of
// the ring. Roles meet at mbarriers: one warp loads (bulk tensor copies), two bring the rows' lse, one
// issues the products, four warps a key tile sum; S has two buffers a key tile, so products run ahead of
// the sums. A summing thread reads two columns of every eight of four keys: their lse, two words, serve
// all four (with a thread a key, every lse was read by every thread; with 8 summing warps the chain of a
// tile, wait, read, exponentials, was exposed: 8 prompts of up to 2048 tokens took 113 and 138 us).
template <int D>
__global__ void __launch_bounds__(Shape<D>::THREADS, 1)
    prompt_mass_kernel(const __grid_constant__ Args a) {
  using Sh = Shape<D>;
  constexpr int NS = Sh::STAGES;
  constexpr float kLog2e = 1.4426950408889634f;
  extern __shared__ char raw[];
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sK = smem_u32(base), ring = sK + 2 * Sh::TILE;
  char* small = base + (2 + NS) * Sh::TILE;
  float* sL = reinterpret_cast<float*>(small + 1024);   // [2 buffers][128]
  float* sHalf = sL + 2 * kTile;                        // [kPair] sums of the second halves
  const uint32_t bars = smem_u32(small);
  const uint32_t kFull = bars, kFree = bars + 8, sFull = bars + 16, sFree = bars + 48,
                 full = bars + 80, empty = full + 8 * NS, dead = empty + 8 * NS;
  static_assert(80 + 16 * NS + 8 <= 1024, "small arrays");
  volatile int* sDead = reinterpret_cast<volatile int*>(small + (dead - bars));
  uint32_t* sTm = reinterpret_cast<uint32_t*>(small + (dead - bars) + 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const PromptShape& s = a.s;
  const int per = kTile >> s.log_g;

  asm volatile("griddepcontrol.launch_dependents;");   // (the joining kernel always follows)
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(sTm)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    *sDead = 0;
    mbar_init(kFull, 1);
    mbar_init(kFree, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(sFull + 8 * i, 3);   // the products, two warps of lse
      mbar_init(sFree + 8 * i, 8);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *sTm;
  auto wait = [&](uint32_t bar, int phase) {
    wait_phase(bar, phase, dead);
    __syncwarp();
  };
  PromptWalk<MassItem> walk;
  MassItem it;
  auto next = [&]() {
    return walk.next(a.sched, gridDim.x, blockIdx.x,
                     [&](int index) { return mass_item(s, a.rows, a.units, index); }, it);
  };

  if (warp == 16) {
    // ================================================================ loads
    const bool issuer = elect_one();
    int seq = 0, count = 0;
#pragma unroll 1
    while (next()) {
#pragma unroll 1
      for (int j = 0; j < it.n; ++j, ++seq) {
        const int st = seq % NS, use = seq / NS;
        if (use > 0) wait(empty + 8 * st, use - 1);
        if (issuer) {
          mbar_expect_tx(full + 8 * st, Sh::TILE);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            load_box(ring + st * Sh::TILE + c * kBlk, &a.q, 64 * c, it.h * s.G,
                     (it.first + it.begin + j) * per, it.b * s.q_row, full + 8 * st);
        }
        __syncwarp();
        if (j > 0) continue;
        if (count > 0) wait(kFree, count - 1);
        if (issuer) {
          mbar_expect_tx(kFull, 2 * Sh::TILE);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              load_box(sK + t * Sh::TILE + c * kBlk, &a.k, 64 * c, it.k0 + t * kTile,
                       it.h * s.kv_head[0], it.b * s.kv_row[0], kFull);
        }
        __syncwarp();
      }
      ++count;
    }
  } else if (warp == 17) {
    // ================================================================ products
    const bool issuer = elect_one();
    const uint64_t dK = smem_desc(sK, 16, 1024), dQ = smem_desc(ring, 16, 1024);
    constexpr uint32_t kStage = Sh::TILE >> 4;
    int seq = 0, count = 0;
#pragma unroll 1
    while (next()) {
      wait(kFull, count);
#pragma unroll 1
      for (int j = 0; j < it.n; ++j, ++seq) {
        const int st = seq % NS, buf = seq & 1;
        wait(full + 8 * st, seq / NS);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (seq >= 2) wait(sFree + 16 * t + 8 * buf, (seq >> 1) - 1);
          fence_after();
          if (issuer) {
            const uint64_t kk = dK + t * kStage, q = dQ + st * kStage;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t o = ((i >> 2) * kBlk + (i & 3) * 32) >> 4;
              mma_ss(tm + 256 * t + 128 * buf, kk + o, q + o, instr_desc(kTile, false), i > 0);
            }
            mma_commit(sFull + 16 * t + 8 * buf);
          }
          __syncwarp();
        }
        if (issuer) {
          mma_commit(empty + 8 * st);
          if (j + 1 == it.n) mma_commit(kFree);
        }
        __syncwarp();
      }
      ++count;
    }
  } else if (warp >= 18) {
    // ================================================================ lse
    const int r0 = (warp - 18) * 64 + lane;
    int seq = 0;
#pragma unroll 1
    while (next()) {
#pragma unroll 1
      for (int j = 0; j < it.n; ++j, ++seq) {
        const int buf = seq & 1;
        float l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + 32 * e, tok = (it.first + it.begin + j) * per + (r >> s.log_g);
          l[e] = tok < it.q_len ? a.lse[((size_t)it.b * s.n_q + tok) * s.Hq + it.h * s.G +
                                        (r & (s.G - 1))]
                                : 0.f;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (seq >= 2) wait(sFree + 16 * t + 8 * buf, (seq >> 1) - 1);
#pragma unroll
        for (int e = 0; e < 2; ++e) sL[buf * kTile + r0 + 32 * e] = -kLog2e * l[e];
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(sFull + 8 * buf);
          mbar_arrive(sFull + 16 + 8 * buf);
        }
      }
    }
  } else {
    // ================================================================ sums
    // two warps a group of 32 keys, each with half of a tile's query rows
    const int t = warp >> 3, half = (warp >> 2) & 1, col = 2 * (lane & 3);
    const int key0 = t * kTile + (warp & 3) * 32 + (lane >> 2);   // the thread's keys: + 16 f + 8 e
    const uint32_t tS = tm + 256 * t + 64 * half + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = kLog2e * rsqrtf((float)D);
    const f2x c2 = f2_pack(c, c);
    // of the columns 64 half + 8 i + col + {0, 1}, those below n, a bit each
    auto below = [&](int n) {
      n -= 64 * half;
      const int bits = 2 * (n >> 3) + min(max((n & 7) - col, 0), 2);
      return n <= 0 ? 0u : bits >= 32 ? ~0u : (1u << bits) - 1;
    };
    int seq = 0;
#pragma unroll 1
    while (next()) {
      // Of the item's query tiles: every query of [all0, all1) sees every key of this key tile, none
      // outside [any0, any1) sees any (its key 0 is token a0, the item's query 0 at position `from`).
      // Told apart once an item: tile by tile, 32768 tokens under a window took 929 us instead of 864.
      const int a0 = it.k0 + t * kTile, w = s.sight.window;
      const int tile0 = it.first + it.begin, from = it.off + tile0 * per;
      const bool sinks = a0 < s.sight.sink, all_sinks = a0 + kTile - 1 < s.sight.sink;
      auto up = [&](int x) { return x <= 0 ? 0 : (x + per - 1) / per; };    // tiles that begin before x
      auto whole = [&](int x) { return x <= 0 ? 0 : x / per; };             // tiles that end before x
      const int all0 = up(a0 + kTile - 1 - from), any0 = whole(a0 - from);
      const int all1 = min(whole(it.q_len - tile0 * per), w && !all_sinks ? whole(a0 + w - from) : it.n);
      const int any1 = w && !sinks ? up(a0 + kTile - 1 + w - from) : it.n;
      f2x total[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) total[e] = f2_pack(0.f, 0.f);
#pragma unroll 1
      for (int i = 0; i < it.n; ++i, ++seq) {
        const int buf = seq & 1;
        wait(sFull + 16 * t + 8 * buf, seq >> 1);
        fence_after();
        if (i >= any0 && i < any1) {
          float x[2][2][16];
#pragma unroll
          for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int q = 0; q < 2; ++q)
              tm_ld32(tS + 128 * buf + 32 * q + ((uint32_t)(16 * f) << 16), x[f][q]);
          const float* l = sL + buf * kTile + 64 * half + col;
          f2x acc[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = f2_pack(0.f, 0.f);
          tm_wait_ld();
          auto sum_tile = [&](auto some) {
            uint32_t see[4];
            if constexpr (decltype(some)::value) {
              const int p0 = from + i * per, left = it.q_len - (tile0 + i) * per;
#pragma unroll
              for (int e = 0; e < 4; ++e) {   // queries that see the key: columns [lo, hi)
                const int j = it.k0 + key0 + 8 * e;
                const int end = min(w && j >= s.sight.sink ? j + w - p0 : per, left);
                see[e] = below(min(max(end, 0), per) << s.log_g) &
                         ~below(min(max(j - p0, 0), per) << s.log_g);
              }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int i8 = 0; i8 < 4; ++i8) {
                const float2 ll = *reinterpret_cast<const float2*>(l + 32 * q + 8 * i8);
                const f2x l2 = f2_pack(ll.x, ll.y);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float* y = &x[e >> 1][q][4 * i8 + 2 * (e & 1)];
                  float y0, y1;
                  f2_unpack(f2_fma(f2_pack(y[0], y[1]), c2, l2), y0, y1);
                  y0 = ex2(y0);
                  y1 = ex2(y1);
                  if constexpr (decltype(some)::value) {
                    const uint32_t bit = 1u << (2 * (4 * q + i8));
                    if (!(see[e] & bit)) y0 = 0.f;
                    if (!(see[e] & (bit << 1))) y1 = 0.f;
                  }
                  acc[e] = f2_add(acc[e], f2_pack(y0, y1));
                }
              }
          };
          if (i >= all0 && i < all1)
            sum_tile(std::false_type());
          else
            sum_tile(std::true_type());
#pragma unroll
          for (int e = 0; e < 4; ++e) total[e] = f2_add(total[e], acc[e]);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sFree + 16 * t + 8 * buf);
      }
      float* out = it.n == it.all
                       ? a.mass + ((size_t)it.b * s.H + it.h) * s.n_kv
                       : a.part + ((size_t)blockIdx.x * 2 + (it.begin == 0 ? 1 : 0)) * kPair - it.k0;
      const int end = it.n == it.all ? a.rows.kv_len[it.b] : it.k0 + kPair;
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y1;
        f2_unpack(total[e], y[e], y1);
        y[e] += y1;
        y[e] += __shfl_xor_sync(0xffffffffu, y[e], 1);
        y[e] += __shfl_xor_sync(0xffffffffu, y[e], 2);
        if (half && (lane & 3) == 0) sHalf[key0 + 8 * e] = y[e];
      }
      const int pair = 1 + 4 * t + (warp & 3);   // the two warps' named barrier
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
      if (!half && (lane & 3) == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = it.k0 + key0 + 8 * e;
          const float z = y[e] + sHalf[key0 + 8 * e];
          if (j < end) out[j] = it.n == it.all && a.add ? out[j] + z : z;
        }
      }
      __syncwarp();
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");   // (read: the next item may write)
    }
  }
  fence_before();
  __syncthreads();
  if (tid == 0 && *sDead) record_status(a.status, 1);
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
}

// The pairs that several CTAs shared, added in their order (block x < joins), and zeros where no query
// sees a key: pairs without tiles, keys past a row's length (block joins + pair * units + unit).
__global__ void __launch_bounds__(kPair) prompt_mass_join_kernel(const __grid_constant__ Args a,
                                                                 int joins) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PromptShape& s = a.s;
  const bool shared = (int)blockIdx.x < joins;
  const MassItem it =
      mass_item(s, a.rows, a.units, shared ? a.sched.join[blockIdx.x].item : blockIdx.x - joins);
  const int j = it.k0 + threadIdx.x, kv_len = a.rows.kv_len[it.b];
  float* m = a.mass + ((size_t)it.b * s.H + it.h) * s.n_kv + j;
  if (j >= s.n_kv) return;
  if (!shared) {
    if (!a.add && (it.all == 0 || j >= kv_len)) *m = 0.f;
    return;
  }
  if (j >= kv_len) return;
  float total = 0.f;
  const auto& jn = a.sched.join[blockIdx.x];
  for (int c = jn.first; c <= jn.last; ++c) {
    if (a.sched.start[c].item == a.sched.start[c + 1].item &&
        a.sched.start[c].tile == a.sched.start[c + 1].tile)
      continue;   // no share
    total += a.part[((size_t)c * 2 + (c == jn.first ? 1 : 0)) * kPair + threadIdx.x];
  }
  *m = a.add ? *m + total : total;
}

template <int D>
fade_status_t launch(Args& a, cudaStream_t st) {
  using Sh = Shape<D>;
  int device = 0;
  const int sms = prompt_sms(&device);
  if (sms == 0) return FADE_ERR_CUDA;
  auto kern = prompt_mass_kernel<D>;
  static std::atomic<bool> opted[64];   // per device: the kernel has its shared memory
  if (!opted[device]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM) !=
        cudaSuccess)
      return launch_status("fade_prompt_mass shared-memory opt-in");
    opted[device] = true;
  }
  int P = 0;
  a.units.set(a.s);
  const int joins = mass_schedule(a.s, a.rows, sms, a.sched, &P);
  kern<<<P, Sh::THREADS, Sh::SMEM, st>>>(a);
  fade_status_t s = launch_status("fade_prompt_mass");
  if (s) return s;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(joins + ceil_div(a.s.n_kv, kPair) * a.s.B * a.s.H);
  lc.blockDim = dim3(kPair);
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, prompt_mass_join_kernel, a, joins);
  if (e != cudaSuccess)
    return set_error(FADE_ERR_CUDA, "fade_prompt_mass join: %s", cudaGetErrorString(e));
  return launch_status("fade_prompt_mass join");
}

}  // namespace

size_t prompt_mass_ws() { return (size_t)2 * kPromptSMs * kPair * 4; }

}  // namespace fade

using namespace fade;

extern "C" fade_status_t fade_prompt_mass(const fade_config_t* c, const fade_heads_t* q,
                                          const fade_heads_t* k, int32_t n_q, int32_t n_kv,
                                          const int32_t* h_q_len, const int32_t* h_kv_len,
                                          int32_t n_sink, int32_t window, const float* lse,
                                          int32_t accumulate, float* mass, int32_t* status, void* ws,
                                          size_t ws_bytes, void* stream) {
  clear_error();
  FADE_RANGE("fade_prompt_mass");
  Args a{};
  fade_status_t st = prompt_shape(c, q, k, nullptr, n_q, n_kv, h_q_len, h_kv_len, n_sink, window,
                                  &a.s, &a.rows);
  if (st) return st;
  if (!lse || !mass) return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL lse or mass");
  if (!ws || !aligned(ws, 16))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
  if (!aligned(lse, 4) || !aligned(mass, 4) || !aligned(status, 4))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "lse, mass and status must be 4-byte aligned");
  if (ws_bytes < prompt_mass_ws())
    return set_error(FADE_ERR_CAPACITY, "prompt workspace %zu bytes, %zu needed", ws_bytes,
                     prompt_mass_ws());
  const int d = c->head_dim;
  st = encode_heads(&a.q, "q", *q, d, a.s.Hq, n_q, a.s.B, a.s.G, kTile / a.s.G, true);
  if (!st) st = encode_heads(&a.k, "k", *k, d, a.s.H, n_kv, a.s.B, 1, kTile, false);
  if (st) return st;
  a.lse = lse;
  a.mass = mass;
  a.part = static_cast<float*>(ws);
  a.status = status;
  if ((long long)ceil_div(n_kv, kPair) * a.s.B * a.s.H > (1 << 30))
    return set_error(FADE_ERR_UNSUPPORTED, "fade_prompt_mass: more than 2^30 blocks of keys");
  a.add = accumulate != 0;
  return d == 64 ? launch<64>(a, as_stream(stream)) : launch<128>(a, as_stream(stream));
}
