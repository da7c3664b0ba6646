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

// A group of D/8 lanes takes one vector, lane l its rotation slots 4l .. 4l+3: slot s < rh is the
// pair (s, s + rh), a slot s >= rh the two unrotated channels 2s and 2s + 1. FULL (rh = D/2): a
// lane's eight channels are two runs of four, read and written as 8-byte words; otherwise (rh
// even) as 4-byte words. A pair never leaves its lane, so only the sum of squares is exchanged.
template <int D, bool FULL>
__device__ __forceinline__ void load_slots(const uint16_t* x, int l, int rh, float (&a)[4],
                                           float (&b)[4]) {
  if constexpr (FULL) {
    const uint2 lo = *reinterpret_cast<const uint2*>(x + 4 * l);
    const uint2 hi = *reinterpret_cast<const uint2*>(x + D / 2 + 4 * l);
    const float2 l0 = __half22float2(*reinterpret_cast<const __half2*>(&lo.x));
    const float2 l1 = __half22float2(*reinterpret_cast<const __half2*>(&lo.y));
    const float2 h0 = __half22float2(*reinterpret_cast<const __half2*>(&hi.x));
    const float2 h1 = __half22float2(*reinterpret_cast<const __half2*>(&hi.y));
    a[0] = l0.x; a[1] = l0.y; a[2] = l1.x; a[3] = l1.y;
    b[0] = h0.x; b[1] = h0.y; b[2] = h1.x; b[3] = h1.y;
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {   // two slots: both rotated or neither (rh is even)
      const int s = 4 * l + 2 * p;
      const uint32_t u = *reinterpret_cast<const uint32_t*>(x + (s < rh ? s : 2 * s));
      const uint32_t v = *reinterpret_cast<const uint32_t*>(x + (s < rh ? s + rh : 2 * s + 2));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
      const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&v));
      a[2 * p] = f.x; a[2 * p + 1] = f.y;
      b[2 * p] = g.x; b[2 * p + 1] = g.y;
    }
  }
}

__device__ __forceinline__ uint32_t pack_h2(float x, float y) {
  return f2h(x) | ((uint32_t)f2h(y) << 16);
}

template <int D, bool FULL>
__device__ __forceinline__ void store_slots(uint16_t* y, int l, int rh, const float (&a)[4],
                                            const float (&b)[4]) {
  if constexpr (FULL) {
    *reinterpret_cast<uint2*>(y + 4 * l) = make_uint2(pack_h2(a[0], a[1]), pack_h2(a[2], a[3]));
    *reinterpret_cast<uint2*>(y + D / 2 + 4 * l) =
        make_uint2(pack_h2(b[0], b[1]), pack_h2(b[2], b[3]));
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int s = 4 * l + 2 * p;
      *reinterpret_cast<uint32_t*>(y + (s < rh ? s : 2 * s)) = pack_h2(a[2 * p], a[2 * p + 1]);
      *reinterpret_cast<uint32_t*>(y + (s < rh ? s + rh : 2 * s + 2)) =
          pack_h2(b[2 * p], b[2 * p + 1]);
    }
  }
}

// One warp per (token, chunk): a chunk is U rounds of 256/D vectors of one side. The table row and
// the weights stay in registers over the rounds, and every round's loads are issued first.
template <int D, bool FULL, int U>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const __grid_constant__ NormArgs a) {
  constexpr int LV = D / 8, NV = 32 / LV;   // lanes a vector, vectors a round
  const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (item >= a.n_items) return;   // uniform over the warp
  const int lane = threadIdx.x & 31, l = lane % LV, sub = lane / LV;
  const int per = a.q.chunks + a.k.chunks;
  const long long tok = item / per;
  const int c = (int)(item % per);
  const bool isq = c < a.q.chunks;
  const NormSide& s = isq ? a.q : a.k;
  const long long row = tok / a.n_tokens, t = tok % a.n_tokens;
  const int h0 = (isq ? c : c - a.q.chunks) * (U * NV) + sub;
  const uint16_t* x = s.x + row * s.xr + t * s.xt;
  uint16_t* y = s.y + row * s.yr + t * s.yt;
  float A[U][4], B[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * NV;
    if (h < s.heads) {
      load_slots<D, FULL>(x + h * s.xh, l, a.rh, A[u], B[u]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) A[u][e] = B[u][e] = 0.f;
    }
  }
  float wa[4], wb[4], cs[4], sn[4];
  if (s.w) load_slots<D, FULL>(s.w, l, a.rh, wa, wb);
  if (a.table) {
    long long p = a.pos ? a.pos[tok] : t;
    p = min(max(p, 0LL), (long long)a.max_pos - 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {   // block 2l + e of the table row: two pairs
      const int sl = 4 * l + 2 * e;
      float4 r = make_float4(1.f, 1.f, 0.f, 0.f);
      if (FULL || sl < a.rh)
        r = *reinterpret_cast<const float4*>(a.table + p * D + 2 * sl);
      cs[2 * e] = r.x; cs[2 * e + 1] = r.y;
      sn[2 * e] = r.z; sn[2 * e + 1] = r.w;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * NV;
    if (s.w) {
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) q = fmaf(A[u][e], A[u][e], fmaf(B[u][e], B[u][e], q));
#pragma unroll
      for (int o = LV / 2; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      const float r = rsqrtf(fmaf(q, 1.0f / D, a.eps));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        A[u][e] *= r * wa[e];
        B[u][e] *= r * wb[e];
      }
    }
    if (a.table) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (FULL || 4 * l + e < a.rh) {
          const float p = A[u][e], q = B[u][e];
          rotate_pair(p, q, cs[e], sn[e], A[u][e], B[u][e]);
        }
    }
    if (h < s.heads) store_slots<D, FULL>(y + h * s.yh, l, a.rh, A[u], B[u]);
  }
}

template <int D, bool FULL>
void launch(const NormArgs& a0, long long tokens, cudaStream_t st) {
  constexpr int NV = 256 / D;
  NormArgs a = a0;
  auto items = [&](int per) {
    a.q.chunks = a.q.x ? ceil_div(a.q.heads, per) : 0;
    a.k.chunks = a.k.x ? ceil_div(a.k.heads, per) : 0;
    a.n_items = tokens * (a.q.chunks + a.k.chunks);
  };
  items(4 * NV);
  const bool deep = a.n_items >= 4096;
  if (!deep) items(NV);
  const unsigned grid = (unsigned)((a.n_items + 7) / 8);
  if (deep)
    qk_norm_rope_kernel<D, FULL, 4><<<grid, 256, 0, st>>>(a);
  else
    qk_norm_rope_kernel<D, FULL, 1><<<grid, 256, 0, st>>>(a);
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
  const bool full = a.rh == c->head_dim / 2;
  if (c->head_dim == 64)
    full ? launch<64, true>(a, tokens, s) : launch<64, false>(a, tokens, s);
  else
    full ? launch<128, true>(a, tokens, s) : launch<128, false>(a, tokens, s);
  return launch_status("fade_qk_norm_rope");
}
