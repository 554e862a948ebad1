// attn_internal.h -- host-side helpers the attention sources share.
#pragma once

#include "attn_core.h"
#include "tp_attention.h"

namespace ringc {

constexpr long long kMaxRow = 1LL << 21;       // elements from one token's row to the next

bool fill_prompt_args(PromptArgs& p, const void* const* q, const void* const* k, const void* const* v, const int* cu_q,
                      const int* cu_k, int P, int B, int Tq, int Tk, int Hq, int Hkv, int D, long long q_stride,
                      long long k_stride, long long v_stride, int causal, float scale);
int prompt_shape(int P, int B, int Tq, int Tk, int Hq, int Hkv, int D, float scale);
// The kernels work with scale log2(e), which has to be finite too.
inline bool scale_ok(float scale) { return scale > 0.0f && scale * kLog2e <= 3.4e38f; }
bool row_stride_ok(long long stride, int heads, int D);
int prompt_slots(int B, int total, int per, int rows, int units);

}  // namespace ringc
