// Per-head RMS norm of queries and keys with the rotation to their positions in one pass.
// Mathematics, per vector x of d channels: y = x / sqrt(mean(x^2) + eps) * w in fp32, the pairs
// (i, i + r/2) of y rotated by the table's cos and sin of the token's position, one rounding to
// fp16. Page "FADE：面向LLM推理的注意力感知分层KV缓存压缩技术", §RoPE重计算 (float32 RoPE math, cast
// through the model dtype) and §RoPE方案兼容性 (the schemes the table holds).
#include <math.h>

#include "fade_internal.cuh"

namespace fade {
namespace {

struct NormSide {
  const uint16_t* x;
  uint16_t* y;
  const uint16_t* w;   // nullptr: no norm
  long long xr, xt, xh, yr, yt, yh;   // element strides: row, token, head
  int heads, chunks;   // chunks of V vectors per token
};

struct NormArgs {
  NormSide q, k;
  const float* table;  // nullptr: no rotation
  const int32_t* pos;  // nullptr: the token's index
  float eps;
  int max_pos, rh, n_tokens;
  long long n_items;   // tokens x chunks of both sides
};

__device__ __forceinline__ uint32_t pack_h2(float x, float y) {
  return f2h(x) | ((uint32_t)f2h(y) << 16);
}
__device__ __forceinline__ void unpack_h2(uint32_t u, float* f) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u));
  f[0] = v.x;
  f[1] = v.y;
}

// A group of D / (2 SL) lanes takes one vector, lane l its rotation slots SL l .. SL l + SL - 1: slot
// s < rh is the pair (s, s + rh), a slot s >= rh the two unrotated channels 2s and 2s + 1. A pair
// never leaves its lane, so only the sum of squares is exchanged. SL = 8 (rh a multiple of 8): a
// lane's slots are all rotated or all not, its 16 channels two 16-byte words; SL = 4 (rh even): slots
// go by twos, in 4-byte words.
template <int SL>
__device__ __forceinline__ void load_slots(const uint16_t* x, int l, int rh, float (&a)[SL],
                                           float (&b)[SL]) {
  if constexpr (SL == 8) {
    const int s = 8 * l;
    const uint4 lo = *reinterpret_cast<const uint4*>(x + (s < rh ? s : 2 * s));
    const uint4 hi = *reinterpret_cast<const uint4*>(x + (s < rh ? s + rh : 2 * s + 8));
    unpack_h2(lo.x, a); unpack_h2(lo.y, a + 2); unpack_h2(lo.z, a + 4); unpack_h2(lo.w, a + 6);
    unpack_h2(hi.x, b); unpack_h2(hi.y, b + 2); unpack_h2(hi.z, b + 4); unpack_h2(hi.w, b + 6);
  } else {
#pragma unroll
    for (int p = 0; p < SL; p += 2) {   // two slots: both rotated or neither
      const int s = SL * l + p;
      unpack_h2(*reinterpret_cast<const uint32_t*>(x + (s < rh ? s : 2 * s)), a + p);
      unpack_h2(*reinterpret_cast<const uint32_t*>(x + (s < rh ? s + rh : 2 * s + 2)), b + p);
    }
  }
}
template <int SL>
__device__ __forceinline__ void store_slots(uint16_t* y, int l, int rh, const float (&a)[SL],
                                            const float (&b)[SL]) {
  if constexpr (SL == 8) {
    const int s = 8 * l;
    *reinterpret_cast<uint4*>(y + (s < rh ? s : 2 * s)) =
        make_uint4(pack_h2(a[0], a[1]), pack_h2(a[2], a[3]), pack_h2(a[4], a[5]), pack_h2(a[6], a[7]));
    *reinterpret_cast<uint4*>(y + (s < rh ? s + rh : 2 * s + 8)) =
        make_uint4(pack_h2(b[0], b[1]), pack_h2(b[2], b[3]), pack_h2(b[4], b[5]), pack_h2(b[6], b[7]));
  } else {
#pragma unroll
    for (int p = 0; p < SL; p += 2) {
      const int s = SL * l + p;
      *reinterpret_cast<uint32_t*>(y + (s < rh ? s : 2 * s)) = pack_h2(a[p], a[p + 1]);
      *reinterpret_cast<uint32_t*>(y + (s < rh ? s + rh : 2 * s + 2)) = pack_h2(b[p], b[p + 1]);
    }
  }
}

// One warp per (token, chunk): a chunk is U rounds of 64 SL / D vectors of one side, which share the
// token's table row and the weights. Bound by DRAM (2 bytes read and written a channel), so what
// counts is bytes in flight: every load of a warp is issued before the first is waited for, 64
// registers keep 32 warps an SM. 4 x 8191 tokens of 32 + 8 heads of 128 (684 MB): 150 us, 4.56 TB/s,
// 0.68 of the copy rate; one round a warp 166 us, four (2 CTAs' registers) 210 us, CTAs of 256
// threads 155 us, 8-byte loads (4 slots a lane) 185 us. Rotary widths that are no multiple of 16 (SL = 4,
// 4-byte words): 194 us at 44 of the 128 channels. Every load goes to a register here, so registers
// limit the bytes in flight; staging tokens in shared memory was not tried.
constexpr int kNormThreads = 128, kNormRounds = 2;
template <int D, int SL, int U>
__global__ void __launch_bounds__(kNormThreads, 8) qk_norm_rope_kernel(const __grid_constant__ NormArgs a) {
  constexpr int LV = D / (2 * SL), NV = 32 / LV;   // lanes a vector, vectors a round
  const uint32_t item = blockIdx.x * (kNormThreads / 32u) + (threadIdx.x >> 5);   // below 2^31 (the host checks)
  if (item >= (uint32_t)a.n_items) return;   // uniform over the warp
  const int lane = threadIdx.x & 31, l = lane % LV, sub = lane / LV;
  const uint32_t per = a.q.chunks + a.k.chunks;
  const uint32_t tok = item / per;
  const int c = (int)(item - tok * per);
  const bool isq = c < a.q.chunks;
  const NormSide& s = isq ? a.q : a.k;
  const uint32_t row = tok / (uint32_t)a.n_tokens, t = tok - row * (uint32_t)a.n_tokens;
  const int h0 = (isq ? c : c - a.q.chunks) * (U * NV) + sub;
  const uint16_t* x = s.x + row * s.xr + t * s.xt;
  uint16_t* y = s.y + row * s.yr + t * s.yt;
  // the position and the lane's part of the table row are asked for before anything is waited for
  const float* tab = nullptr;
  if (a.table) {
    const int p = min(max(a.pos ? a.pos[tok] : (int)t, 0), a.max_pos - 1);
    tab = a.table + (size_t)p * D + 2 * SL * l;
  }
  float A[U][SL], B[U][SL];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * NV;
    if (h < s.heads) {
      load_slots<SL>(x + h * s.xh, l, a.rh, A[u], B[u]);
    } else {
#pragma unroll
      for (int e = 0; e < SL; ++e) A[u][e] = B[u][e] = 0.f;
    }
  }
  if (tab && SL * l < a.rh) asm volatile("prefetch.global.L1 [%0];" ::"l"(tab));
  if (s.w) {
    float wa[SL], wb[SL];
    load_slots<SL>(s.w, l, a.rh, wa, wb);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < SL; ++e) q = fmaf(A[u][e], A[u][e], fmaf(B[u][e], B[u][e], q));
#pragma unroll
      for (int o = LV / 2; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      const float r = rsqrtf(fmaf(q, 1.0f / D, a.eps));
#pragma unroll
      for (int e = 0; e < SL; ++e) {
        A[u][e] *= r * wa[e];
        B[u][e] *= r * wb[e];
      }
    }
  }
  if (tab) {
#pragma unroll
    for (int e = 0; e < SL; e += 2) {   // a block of the table row: two pairs
      if ((SL == 8 ? SL * l : SL * l + e) >= a.rh) continue;
      const float4 cs = *reinterpret_cast<const float4*>(tab + 2 * e);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float p0 = A[u][e], q0 = B[u][e], p1 = A[u][e + 1], q1 = B[u][e + 1];
        rotate_pair(p0, q0, cs.x, cs.z, A[u][e], B[u][e]);
        rotate_pair(p1, q1, cs.y, cs.w, A[u][e + 1], B[u][e + 1]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (h0 + u * NV < s.heads) store_slots<SL>(y + (h0 + u * NV) * s.yh, l, a.rh, A[u], B[u]);
}

template <int D, int SL>
void launch(const NormArgs& a0, long long tokens, cudaStream_t st) {
  constexpr int NV = 64 * SL / D;
  NormArgs a = a0;
  auto items = [&](int per) {
    a.q.chunks = a.q.x ? ceil_div(a.q.heads, per) : 0;
    a.k.chunks = a.k.x ? ceil_div(a.k.heads, per) : 0;
    a.n_items = tokens * (a.q.chunks + a.k.chunks);
  };
  items(kNormRounds * NV);
  // one round a warp where two would leave schedulers without a warp (152 SMs x 32 warps)
  const bool deep = a.n_items >= 4864;
  if (!deep) items(NV);
  const unsigned grid = (unsigned)ceil_div(a.n_items, kNormThreads / 32);
  if (deep)
    qk_norm_rope_kernel<D, SL, kNormRounds><<<grid, kNormThreads, 0, st>>>(a);
  else
    qk_norm_rope_kernel<D, SL, 1><<<grid, kNormThreads, 0, st>>>(a);
}

bool side_strides_ok(const fade_heads_t* h) {
  return !(reinterpret_cast<uintptr_t>(h->x) & 15) && h->row_stride % 8 == 0 &&
         h->token_stride % 8 == 0 && h->head_stride % 8 == 0;
}

// The vectors of an output must be apart: no stride shorter than a vector where it is used.
bool apart(const fade_heads_t* h, long long rows, long long tokens, int heads, int d) {
  auto far = [d](long long s, long long n) { return n <= 1 || s >= d || s <= -d; };
  return far(h->row_stride, rows) && far(h->token_stride, tokens) && far(h->head_stride, heads);
}

}  // namespace
}  // namespace fade

using namespace fade;

extern "C" fade_status_t fade_qk_norm_rope(const fade_config_t* c, const float* table,
                                           int32_t max_pos, const fade_heads_t* q_in,
                                           const fade_heads_t* q_out, const uint16_t* q_weight,
                                           const fade_heads_t* k_in, const fade_heads_t* k_out,
                                           const uint16_t* k_weight, float eps,
                                           const int32_t* pos, int64_t n_rows, int32_t n_tokens,
                                           void* stream) {
  clear_error();
  FADE_RANGE("fade_qk_norm_rope");
  fade_status_t st = validate_config(c);
  if (st) return st;
  if (n_rows < 0 || n_tokens < 0)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "negative n_rows or n_tokens");
  const long long tokens = (long long)n_rows * n_tokens;
  if (tokens == 0) return FADE_OK;
  if ((!q_in && !k_in) || (q_in && (!q_in->x || !q_out || !q_out->x)) ||
      (k_in && (!k_in->x || !k_out || !k_out->x)))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL q or k, or no output for one of them");
  const bool rope = c->rope.kind != FADE_ROPE_NONE;
  if (rope && (!table || max_pos < 1 || (reinterpret_cast<uintptr_t>(table) & 15)))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL or unaligned RoPE table, or max_pos < 1");
  if (rope && !pos && n_tokens > max_pos)
    return set_error(FADE_ERR_CAPACITY, "positions up to %d exceed the table (%d)", n_tokens - 1,
                     max_pos);
  if (reinterpret_cast<uintptr_t>(pos) & 3)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "pos must be 4-byte aligned");
  const uint16_t* w[2] = {q_in ? q_weight : nullptr, k_in ? k_weight : nullptr};
  if ((w[0] || w[1]) && !(eps > 0.f && isfinite(eps)))
    return set_error(FADE_ERR_INVALID_ARGUMENT, "eps must be positive and finite");
  const fade_heads_t* in[2] = {q_in, k_in};
  const fade_heads_t* out[2] = {q_out, k_out};
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) continue;
    if (!side_strides_ok(in[i]) || !side_strides_ok(out[i]) ||
        (reinterpret_cast<uintptr_t>(w[i]) & 15))
      return set_error(FADE_ERR_INVALID_ARGUMENT,
                       "%s: vectors and weights must start 16-byte aligned (strides in multiples "
                       "of 8 elements)", i ? "k" : "q");
    if (!apart(out[i], n_rows, n_tokens, i ? c->num_kv_heads : c->num_q_heads, c->head_dim))
      return set_error(FADE_ERR_INVALID_ARGUMENT, "%s: the output's vectors overlap",
                       i ? "k" : "q");
  }
  if (tokens > (1LL << 31) / (c->num_q_heads + c->num_kv_heads))
    return set_error(FADE_ERR_UNSUPPORTED, "%lld tokens in one call", tokens);
  NormArgs a{};
  for (int i = 0; i < 2; ++i) {
    NormSide& s = i ? a.k : a.q;
    if (!in[i]) continue;
    s = NormSide{in[i]->x, out[i]->x, w[i], in[i]->row_stride, in[i]->token_stride,
                 in[i]->head_stride, out[i]->row_stride, out[i]->token_stride,
                 out[i]->head_stride, i ? c->num_kv_heads : c->num_q_heads, 0};
  }
  a.table = rope ? table : nullptr;
  a.pos = pos;
  a.eps = eps;
  a.max_pos = max_pos;
  a.rh = rope ? rotary_width(c) / 2 : c->head_dim / 2;
  a.n_tokens = n_tokens;
  cudaStream_t s = as_stream(stream);
  const bool wide = a.rh % 8 == 0;
  if (c->head_dim == 64)
    wide ? launch<64, 8>(a, tokens, s) : launch<64, 4>(a, tokens, s);
  else
    wide ? launch<128, 8>(a, tokens, s) : launch<128, 4>(a, tokens, s);
  return launch_status("fade_qk_norm_rope");
}
