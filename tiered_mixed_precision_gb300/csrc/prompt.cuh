// Shared by the prompt translation units (attention and its column sums): rows, what a query sees,
// host checks.
#pragma once

#include "prompt_schedule.h"
#include "tree.cuh"

namespace fade {

// Checks what the prompt calls share and fills rows and shape. v: NULL where the call has none.
fade_status_t prompt_shape(const fade_config_t* c, const fade_heads_t* q, const fade_heads_t* k,
                           const fade_heads_t* v, int32_t n_q, int32_t n_kv, const int32_t* h_q_len,
                           const int32_t* h_kv_len, int32_t n_sink, int32_t window,
                           PromptShape* shape, PromptRows* rows);
// SMs of the current device (0: an error, which is set).
int prompt_sms(int* device);
size_t prompt_attention_ws(const fade_config_t* c, int32_t n_q);
size_t prompt_mass_ws();

}  // namespace fade
