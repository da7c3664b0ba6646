// Shared by the drafted-token translation units (and, through prompt.cuh, the prompts): what their kernels
// read, 2^x, and the host checks.
#pragma once

#include "fade_internal.cuh"

namespace fade {

struct TreeArgs {
  uint16_t *sink_k, *sink_v, *rec_k, *rec_v;
  uint8_t *mk[2], *mv[2];
  uint16_t *mks[2], *mvs[2];
  float *sink_sc, *mid_sc[2], *rec_sc;
  int32_t *meta, *status;
  const uint16_t* pq_cb;   // nullptr: integer-coded V
  const uint16_t* q;       // [B][T][Hq][D]
  fade_heads_t tk, tv;     // the nodes' keys and values, H heads
  int B, H, Hq, G, log_g, S, W, C, T;   // G = 1 << log_g
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The i-th node of row b's path; a node outside the tree reads as node 0 (the commit records it).
__device__ __forceinline__ int tree_node(const TreeArgs& a, const int32_t* path, int b, int i) {
  const int n = path[(size_t)b * a.T + i];
  return n >= 0 && n < a.T ? n : 0;
}

// Whether a pointer (NULL included) starts on a multiple of `bytes`.
inline bool aligned(const void* p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}
fade_status_t validate_tree(const fade_config_t* c, int32_t T);
// validate_layer, and the 16-byte alignment that vector loads of the tiers need.
fade_status_t validate_tree_layer(const fade_config_t* c, const fade_layer_t* L);
fade_status_t validate_heads(const fade_heads_t* h, const char* name);
TreeArgs make_tree_args(const fade_config_t* c, const fade_layer_t* L, int T, const uint16_t* q,
                        const fade_heads_t* tk, const fade_heads_t* tv);
// Workspace bytes of the attention call for a valid configuration and T.
size_t tree_attention_ws(const fade_config_t* c, int T);

}  // namespace fade
