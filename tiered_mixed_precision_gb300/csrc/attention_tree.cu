// Attention of a tree of drafted tokens over the tiered cache and over itself.
// Page "FADE：面向LLM推理的注意力感知分层KV缓存压缩技术", §项目结构与代码质量 (kernels/: fused INT4 dequant
// + SDPA): attention runs on the packed tiers.
#include <math.h>

#include "tree.cuh"

namespace fade {

size_t tree_attention_ws(const fade_config_t*, int) { return 16; }

namespace {

// One CTA per (query head, node, row): its 8 warps take the tokens in turn, lane l owning channels
// l, l + 32, ..; each warp keeps a running maximum and sum, merged in shared memory at the end.
template <int D, int KB, int VB>
__global__ void __launch_bounds__(256) tree_attention_kernel(TreeArgs a,
                                                             const uint64_t* __restrict__ mask,
                                                             const int32_t* __restrict__ n_nodes,
                                                             uint16_t* __restrict__ out,
                                                             float* __restrict__ lse) {
  constexpr int E = D / 32;
  const int hq = blockIdx.x, t = blockIdx.y, b = blockIdx.z, h = hq / a.G, unit = b * a.H + h;
  const int n = n_nodes ? min(max(n_nodes[b], 0), a.T) : a.T;
  if (t >= n) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t* m = a.meta + unit * FADE_META_FIELDS;
  const int n_sink = m[FADE_META_N_SINK], n_mid = m[FADE_META_N_MID];
  const int n_rec = m[FADE_META_N_RECENT], head = m[FADE_META_HEAD], cur = m[FADE_META_CUR];
  const int held = n_sink + n_mid + n_rec;
  const size_t vec = ((size_t)b * a.T + t) * a.Hq + hq;
  const uint64_t seen = mask[(size_t)b * a.T + t];
  const float scale = rsqrtf((float)D);
  float q[E], o[E], M = -INFINITY, L = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = h2f(a.q[vec * D + 32 * e + lane]);
    o[e] = 0.f;
  }
  for (int j = warp; j < held + n; j += 8) {
    float k[E], v[E];
    if (j >= n_sink && j < n_sink + n_mid) {
      const size_t r = (size_t)unit * a.C + (j - n_sink);
      const uint8_t* kc = a.mk[cur] + r * (D * KB / 8);
      const uint8_t* vc = a.mv[cur] + r * (D * VB / 8);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = 32 * e + lane;
        k[e] = (float)unpack_code<KB>(kc, c) * h2f(a.mks[cur][r * E + e]);
        v[e] = a.pq_cb ? h2f(a.pq_cb[((size_t)(c >> 2) * 256 + vc[c >> 2]) * 4 + (c & 3)])
                       : (float)unpack_code<VB>(vc, c) * h2f(a.mvs[cur][r * E + e]);
      }
    } else {
      const uint16_t *xk, *xv;
      if (j < n_sink) {
        xk = a.sink_k + ((size_t)unit * a.S + j) * D;
        xv = a.sink_v + ((size_t)unit * a.S + j) * D;
      } else if (j < held) {
        const size_t r = (size_t)unit * a.W + (head + (j - n_sink - n_mid)) % a.W;
        xk = a.rec_k + r * D;
        xv = a.rec_v + r * D;
      } else {
        if (!((seen >> (j - held)) & 1)) continue;
        xk = a.tk.x + b * a.tk.row_stride + (j - held) * a.tk.token_stride + h * a.tk.head_stride;
        xv = a.tv.x + b * a.tv.row_stride + (j - held) * a.tv.token_stride + h * a.tv.head_stride;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = h2f(xk[32 * e + lane]);
        v[e] = h2f(xv[32 * e + lane]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
    s = warp_sum(s) * scale;
    const float Mn = fmaxf(M, s), r = __expf(M - Mn), p = __expf(s - Mn);
    L = fmaf(L, r, p);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], r, p * v[e]);
    M = Mn;
  }
  __shared__ float sm[8], sl[8], so[8][D];
  if (lane == 0) {
    sm[warp] = M;
    sl[warp] = L;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][32 * e + lane] = o[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float Mx = -INFINITY, Ls = 0.f, acc = 0.f;
    for (int w = 0; w < 8; ++w) Mx = fmaxf(Mx, sm[w]);
    for (int w = 0; w < 8; ++w) {
      const float r = sm[w] == -INFINITY ? 0.f : __expf(sm[w] - Mx);
      Ls = fmaf(sl[w], r, Ls);
      acc = fmaf(so[w][threadIdx.x], r, acc);
    }
    out[vec * D + threadIdx.x] = f2h(Mx == -INFINITY ? 0.f : acc / Ls);
    if (threadIdx.x == 0) lse[vec] = Mx == -INFINITY ? -INFINITY : Mx + logf(Ls);
  }
}

template <int D, int KB, int VB>
fade_status_t launch(const fade_config_t* c, const TreeArgs& a, const uint64_t* mask,
                     const int32_t* n_nodes, uint16_t* out, float* lse, cudaStream_t st) {
  tree_attention_kernel<D, KB, VB><<<dim3(c->num_q_heads, a.T, c->batch), 256, 0, st>>>(
      a, mask, n_nodes, out, lse);
  return launch_status("fade_tree_attention");
}

}  // namespace
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
  if (!st) st = validate_layer(c, L);
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
  const TreeArgs a = make_tree_args(c, L, T, q_rot, tree_k, tree_v);
  cudaStream_t s = as_stream(stream);
  const int kb = c->middle_k_bits, vb = c->middle_v_bits;
#define FADE_TREE_CASE(D_, KB_, VB_)               \
  if (c->head_dim == D_ && kb == KB_ && vb == VB_) \
    return launch<D_, KB_, VB_>(c, a, mask, n_nodes, out, lse, s);
  FADE_TREE_CASE(64, 4, 2) FADE_TREE_CASE(64, 4, 4) FADE_TREE_CASE(64, 2, 2)
  FADE_TREE_CASE(64, 2, 4) FADE_TREE_CASE(128, 4, 2) FADE_TREE_CASE(128, 4, 4)
  FADE_TREE_CASE(128, 2, 2) FADE_TREE_CASE(128, 2, 4)
#undef FADE_TREE_CASE
  return set_error(FADE_ERR_UNSUPPORTED, "unsupported (head_dim, k_bits, v_bits)");
}
