// Column sums of a prompt's attention: the importance that its tokens start with.
// Pages "探秘Transformer系列之（25）--- KV Cache优化之处理长文本序列", §1.3.1 H2O (a token's importance is the
// column sum of the attention matrix) and FADE-zh §四种驱逐策略详解 1 (captured at prefill).
//
// Mathematics: mass[j] = sum over the query rows r of the unit that see key j of 2^(c S[r][j] - l[r]),
// c = log2(e)/sqrt(d), l = log2(e) lse. The attention's log-sum-exp makes it one pass: no maximum, no
// second sum. Products run transposed, S^T = K Q^T, so that a thread of a softmax warp owns a key and
// its sum stays in a register.
//
// Sums are fp32, tile by tile (128 terms, then a tile's sum a term), in one fixed order: no atomics, the
// same bits on every run.
#include <math.h>

#include <algorithm>

#include "prompt.cuh"
#include "tensor_core.cuh"
#include "tensor_map.cuh"

namespace fade {
namespace {

constexpr int kTile = 128;          // keys of a tile, and query rows of one
constexpr int kBlk = kTile * 128;   // bytes of a [128][64] fp16 block
constexpr int kPair = 2 * kTile;    // keys of an item
constexpr int kMaxChunks = 16;      // pieces that a pair's queries are cut into at most
constexpr int kMinChunk = 8;        // query tiles of a piece at least
constexpr int kMaxSM = 160;         // SMs the workspace is sized for

template <int D>
struct Shape {
  static constexpr int TILE = D / 64 * kBlk;          // bytes of a K or Q tile
  static constexpr int STAGES = D == 128 ? 4 : 8;     // ring of Q tiles
  static constexpr int SMALL = 1024 + STAGES * 512;   // barriers, then the rows' -l of every stage
  static constexpr int SMEM = 1024 + 2 * TILE + STAGES * TILE + SMALL;
  static constexpr int THREADS = 384;   // 8 warps that sum, load, products, 2 that scale lse
};

struct Args {
  CUtensorMap q, k;
  PromptShape s;
  PromptRows rows;
  const float* lse;
  float* mass;
  float* part;      // chunks > 1: [chunk][unit][pairs * kPair]
  int32_t* status;
  int pairs, chunks, add;
};

// The query tiles [begin, begin + n) that see a pair of key tiles; a chunk of them.
struct Item {
  int b, h, u, k0, chunk, chunks, begin, n;
  int off, q_len;   // position of query token 0; the row's queries
};
__device__ __forceinline__ Item item_at(const Args& a, int index) {
  const PromptShape& s = a.s;
  const int units = s.B * s.H;
  Item it;
  it.chunk = index % a.chunks;
  index /= a.chunks;
  const int u = index % units;
  it.k0 = index / units * kPair;
  it.b = a.rows.order[u / s.H];
  it.h = u % s.H;
  it.u = it.b * s.H + it.h;
  it.q_len = a.rows.q_len[it.b];
  const int kv_len = a.rows.kv_len[it.b], per = kTile >> s.log_g;
  it.off = kv_len - it.q_len;
  const int first = max(it.k0 - it.off, 0);
  int last = it.q_len - 1;
  if (s.sight.window && it.k0 >= s.sight.sink)
    last = min(last, it.k0 + kPair - 1 + s.sight.window - 1 - it.off);
  const int all = it.k0 < kv_len && first <= last ? last / per - first / per + 1 : 0;
  it.chunks = min(a.chunks, max((all + kMinChunk - 1) / kMinChunk, 1));
  it.begin = 0;
  it.n = 0;
  if (it.chunk < it.chunks) {
    const int from = all * it.chunk / it.chunks;
    it.begin = first / per + from;
    it.n = all * (it.chunk + 1) / it.chunks - from;
  }
  return it;
}
__device__ __forceinline__ int item_index(int k) {   // forth and back over the CTAs
  const int P = gridDim.x, c = blockIdx.x;
  return k * P + ((k & 1) ? P - 1 - c : c);
}

__device__ __forceinline__ void tm_ld_row(uint32_t addr, float* v) {   // 32 lanes x 32 columns
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

// One persistent CTA per SM; an item is two tiles of 128 keys of a unit, both met by every query tile of
// the ring. Roles meet at mbarriers: one warp loads (bulk tensor copies), two bring the rows' lse, one
// issues the products, four warps a key tile (a thread a key) sum; S has two buffers a key tile, so
// products run ahead of the sums.
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
  float* sL = reinterpret_cast<float*>(small + 1024);   // [NS][128]
  const uint32_t bars = smem_u32(small);
  const uint32_t kFull = bars, kFree = bars + 8, sFull = bars + 16, sFree = bars + 48,
                 full = bars + 80, empty = full + 8 * NS, dead = empty + 8 * NS;
  static_assert(80 + 16 * NS + 8 <= 1024, "small arrays");
  volatile int* sDead = reinterpret_cast<volatile int*>(small + (dead - bars));
  uint32_t* sTm = reinterpret_cast<uint32_t*>(small + (dead - bars) + 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const PromptShape& s = a.s;
  const int items = a.pairs * a.chunks * s.B * s.H, per = kTile >> s.log_g;

  if (a.chunks > 1) asm volatile("griddepcontrol.launch_dependents;");
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
      mbar_init(sFull + 8 * i, 1);
      mbar_init(sFree + 8 * i, 4);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + 8 * i, 3);    // the copy, two warps of lse
      mbar_init(empty + 8 * i, 9);   // the products, eight warps that read lse
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

  if (warp == 8) {
    // ================================================================ loads
    const bool issuer = elect_one();
    int seq = 0, count = 0;
#pragma unroll 1
    for (int k = 0; k * gridDim.x < items; ++k) {
      const int index = item_index(k);
      if (index >= items) continue;
      const Item it = item_at(a, index);
      if (it.n == 0) continue;
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
#pragma unroll 1
      for (int j = 0; j < it.n; ++j, ++seq) {
        const int st = seq % NS, use = seq / NS;
        if (use > 0) wait(empty + 8 * st, use - 1);
        if (issuer) {
          mbar_expect_tx(full + 8 * st, Sh::TILE);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            load_box(ring + st * Sh::TILE + c * kBlk, &a.q, 64 * c, it.h * s.G, (it.begin + j) * per,
                     it.b * s.q_row, full + 8 * st);
        }
        __syncwarp();
      }
      ++count;
    }
  } else if (warp == 9) {
    // ================================================================ products
    const bool issuer = elect_one();
    const uint64_t dK = smem_desc(sK, 16, 1024), dQ = smem_desc(ring, 16, 1024);
    constexpr uint32_t kStage = Sh::TILE >> 4;
    int seq = 0, count = 0;
#pragma unroll 1
    for (int k = 0; k * gridDim.x < items; ++k) {
      const int index = item_index(k);
      if (index >= items) continue;
      const Item it = item_at(a, index);
      if (it.n == 0) continue;
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
  } else if (warp >= 10) {
    // ================================================================ lse
    const int r0 = (warp - 10) * 64 + lane;
    int seq = 0;
#pragma unroll 1
    for (int k = 0; k * gridDim.x < items; ++k) {
      const int index = item_index(k);
      if (index >= items) continue;
      const Item it = item_at(a, index);
#pragma unroll 1
      for (int j = 0; j < it.n; ++j, ++seq) {
        const int st = seq % NS, use = seq / NS;
        float l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + 32 * e, tok = (it.begin + j) * per + (r >> s.log_g);
          l[e] = tok < it.q_len ? a.lse[((size_t)it.b * s.n_q + tok) * s.Hq + it.h * s.G +
                                        (r & (s.G - 1))]
                                : 0.f;
        }
        if (use > 0) wait(empty + 8 * st, use - 1);
#pragma unroll
        for (int e = 0; e < 2; ++e) sL[st * kTile + r0 + 32 * e] = -kLog2e * l[e];
        __syncwarp();
        if (lane == 0) mbar_arrive(full + 8 * st);
      }
    }
  } else {
    // ================================================================ sums
    const int t = warp >> 2, key = t * kTile + (warp & 3) * 32 + lane;
    const uint32_t tS = tm + 256 * t + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = kLog2e * rsqrtf((float)D);
    const f2x c2 = f2_pack(c, c);
    int seq = 0;
#pragma unroll 1
    for (int k = 0; k * gridDim.x < items; ++k) {
      const int index = item_index(k);
      if (index >= items) continue;
      const Item it = item_at(a, index);
      if (it.chunk >= it.chunks) continue;
      const int j = it.k0 + key, k_end = it.k0 + t * kTile + kTile - 1;
      float total = 0.f;
#pragma unroll 1
      for (int i = 0; i < it.n; ++i, ++seq) {
        const int st = seq % NS, buf = seq & 1, tok0 = (it.begin + i) * per;
        const int p0 = it.off + tok0;
        // rows that see the key: columns [lo, hi)
        const int hi_tok = min(s.sight.window && j >= s.sight.sink ? j + s.sight.window - p0 : per,
                               it.q_len - tok0);
        const int lo = max(j - p0, 0) << s.log_g, hi = min(max(hi_tok, 0), per) << s.log_g;
        const bool all = k_end <= p0 && it.q_len - tok0 >= per &&
                         (!s.sight.window || k_end < s.sight.sink ||
                          k_end - kTile + 1 + s.sight.window >= p0 + per);   // uniform
        wait(sFull + 16 * t + 8 * buf, seq >> 1);
        wait(full + 8 * st, seq / NS);   // (complete: what was written there is seen from here on)
        fence_after();
        f2x acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        const float4* l4 = reinterpret_cast<const float4*>(sL + st * kTile);
        auto sum_tile = [&](auto some) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float x[32];
            tm_ld_row(tS + 128 * buf + 32 * q, x);
            tm_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 l = l4[8 * q + e];
              float y[4];
              f2_unpack(f2_fma(f2_pack(x[4 * e], x[4 * e + 1]), c2, f2_pack(l.x, l.y)), y[0], y[1]);
              f2_unpack(f2_fma(f2_pack(x[4 * e + 2], x[4 * e + 3]), c2, f2_pack(l.z, l.w)), y[2],
                        y[3]);
#pragma unroll
              for (int i4 = 0; i4 < 4; ++i4) {
                y[i4] = ex2(y[i4]);
                const int col = 32 * q + 4 * e + i4;
                if (decltype(some)::value && (col < lo || col >= hi)) y[i4] = 0.f;
              }
              acc[0] = f2_add(acc[0], f2_pack(y[0], y[1]));
              acc[1] = f2_add(acc[1], f2_pack(y[2], y[3]));
            }
          }
        };
        if (all)
          sum_tile(std::false_type());
        else
          sum_tile(std::true_type());
        fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(sFree + 16 * t + 8 * buf);
          mbar_arrive(empty + 8 * st);
        }
        float a0, a1, b0, b1;
        f2_unpack(acc[0], a0, a1);
        f2_unpack(acc[1], b0, b1);
        total += (a0 + a1) + (b0 + b1);
      }
      if (a.chunks > 1) {
        a.part[((size_t)it.chunk * s.B * s.H + it.u) * a.pairs * kPair + j] = total;
      } else if (j < s.n_kv) {
        float* m = a.mass + (size_t)it.u * s.n_kv + j;
        if (j >= a.rows.kv_len[it.b]) total = 0.f;   // (n > 0: whatever lies there)
        *m = a.add ? *m + total : total;
      }
    }
  }
  fence_before();
  __syncthreads();
  if (tid == 0 && *sDead) record_status(a.status, 1);
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512));
}

// The chunks of every pair, added in their order.
__global__ void __launch_bounds__(kPair) prompt_mass_join_kernel(const __grid_constant__ Args a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PromptShape& s = a.s;
  const Item it = item_at(a, blockIdx.x * a.chunks);
  const int j = it.k0 + threadIdx.x;
  if (j >= s.n_kv) return;
  float total = 0.f;
  if (j < a.rows.kv_len[it.b])
    for (int i = 0; i < it.chunks; ++i)
      total += a.part[((size_t)i * s.B * s.H + it.u) * a.pairs * kPair + j];
  float* m = a.mass + (size_t)it.u * s.n_kv + j;
  *m = a.add ? *m + total : total;
}

int pairs_of(int32_t n_kv) { return ceil_div(n_kv, kPair); }

// Pieces of a pair's queries: enough for several items an SM.
int most_chunks(const fade_config_t* c, int32_t n_q, int32_t n_kv) {
  const long long items = (long long)c->batch * c->num_kv_heads * pairs_of(n_kv);
  const int tiles = ceil_div((long long)n_q * (c->num_q_heads / c->num_kv_heads), kTile);
  return std::min({kMaxChunks, (int)std::min<long long>(ceil_div(8 * kMaxSM, items), kMaxChunks),
                   ceil_div(tiles, kMinChunk)});
}

template <int D>
fade_status_t launch(Args& a, cudaStream_t st) {
  using Sh = Shape<D>;
  int device = 0;
  const int sms = prompt_sms(&device);
  if (sms == 0) return FADE_ERR_CUDA;
  auto kern = prompt_mass_kernel<D>;
  static bool opted[64];   // per device: the kernel has its shared memory
  if (!opted[device]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM) !=
        cudaSuccess)
      return launch_status("fade_prompt_mass shared-memory opt-in");
    opted[device] = true;
  }
  const long long items = (long long)a.pairs * a.chunks * a.s.B * a.s.H;
  if (items > (1 << 30))
    return set_error(FADE_ERR_UNSUPPORTED, "fade_prompt_mass: more than 2^30 blocks of keys");
  kern<<<(unsigned)std::min<long long>(items, sms), Sh::THREADS, Sh::SMEM, st>>>(a);
  fade_status_t s = launch_status("fade_prompt_mass");
  if (s || a.chunks == 1) return s;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3((unsigned)(items / a.chunks));
  lc.blockDim = dim3(kPair);
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, prompt_mass_join_kernel, a);
  if (e != cudaSuccess)
    return set_error(FADE_ERR_CUDA, "fade_prompt_mass join: %s", cudaGetErrorString(e));
  return launch_status("fade_prompt_mass join");
}

}  // namespace

size_t prompt_mass_ws(const fade_config_t* c, int32_t n_q, int32_t n_kv) {
  const int chunks = most_chunks(c, n_q, n_kv);
  return chunks == 1 ? 0
                     : (size_t)chunks * c->batch * c->num_kv_heads * pairs_of(n_kv) * kPair * 4;
}

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
  if (ws_bytes < prompt_mass_ws(c, n_q, n_kv))
    return set_error(FADE_ERR_CAPACITY, "prompt workspace %zu bytes, %zu needed", ws_bytes,
                     prompt_mass_ws(c, n_q, n_kv));
  const int d = c->head_dim;
  st = encode_heads(&a.q, "q", *q, d, a.s.Hq, n_q, a.s.B, a.s.G, kTile / a.s.G, true);
  if (!st) st = encode_heads(&a.k, "k", *k, d, a.s.H, n_kv, a.s.B, 1, kTile, false);
  if (st) return st;
  a.lse = lse;
  a.mass = mass;
  a.part = static_cast<float*>(ws);
  a.status = status;
  a.pairs = pairs_of(n_kv);
  a.chunks = most_chunks(c, n_q, n_kv);
  a.add = accumulate != 0;
  return d == 64 ? launch<64>(a, as_stream(stream)) : launch<128>(a, as_stream(stream));
}
