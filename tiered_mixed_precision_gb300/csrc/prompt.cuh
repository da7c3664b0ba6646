// Shared by the prompt translation units (attention and its column sums): rows, what a query sees,
// host checks.
#pragma once

#include "tree.cuh"

namespace fade {

// The rows of a call. Queries are the last q_len of a row's kv_len tokens.
struct PromptRows {
  int32_t q_len[FADE_MAX_BATCH], kv_len[FADE_MAX_BATCH];
  uint8_t order[FADE_MAX_BATCH];   // rows, the most tokens first
};

// What queries see: token j of position i's past if window is 0, j > i - window or j < sink.
struct Sight {
  int sink, window;   // window 0: sink 0, too
};

struct PromptShape {
  int B, H, G, log_g, Hq, n_q, n_kv;
  Sight sight;
  // 0 where a stride is 0 (a broadcast dimension): the tensor map's extent is 1 there
  int q_row, kv_row[2], kv_head[2];
};

// Checks what the prompt calls share and fills rows and shape. v: NULL where the call has none.
fade_status_t prompt_shape(const fade_config_t* c, const fade_heads_t* q, const fade_heads_t* k,
                           const fade_heads_t* v, int32_t n_q, int32_t n_kv, const int32_t* h_q_len,
                           const int32_t* h_kv_len, int32_t n_sink, int32_t window,
                           PromptShape* shape, PromptRows* rows);
// SMs of the current device (0: an error, which is set).
int prompt_sms(int* device);
size_t prompt_attention_ws(const fade_config_t* c, int32_t n_q);
size_t prompt_mass_ws(const fade_config_t* c, int32_t n_q, int32_t n_kv);

}  // namespace fade
