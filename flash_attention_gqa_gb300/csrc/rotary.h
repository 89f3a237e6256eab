// Internal interface of the rotary positions (rotary.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "paged.h"

namespace fa {

constexpr int kMaxRotaryAxes = 16;
constexpr int kMaxRotaryTokens = 1 << 30;   // B * T of one call

// A tensor [B, T, heads, H] of bf16, its byte strides.
struct RotaryRows {
  void* at;
  int64_t batch, token, head;
};

struct RotaryArgs {
  RotaryRows q, q_out, k, k_out, v;   // k_out: no append; v: append
  const int32_t* positions;           // of (axis, b, t), strides in elements
  int64_t pos_axis, pos_batch, pos_token;
  const float* inv_freq;              // [pairs]
  const int32_t* axes;                // [pairs] or null: axis 0
  int pairs, n_axes;
  bool adjacent, inverse;
  float q_scale;
  int B, T, QH, KH, H;
  // append: where keys and values go
  const int64_t* slots;               // [B * T]
  void *k_cache, *v_cache;
  const float *k_scale, *v_scale;     // [KH] or null
  PagedLayout lay;
  uint32_t* err;
};

enum RotaryTo { ROTARY_PLAIN, ROTARY_BF16, ROTARY_E4M3 };   // rows; pages of either type
cudaError_t launch_rotary(const RotaryArgs& a, RotaryTo to, int sm_count, cudaStream_t st);

}  // namespace fa
