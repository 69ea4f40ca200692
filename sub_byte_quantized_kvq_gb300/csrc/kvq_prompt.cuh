// kvq_prompt.cuh -- launch interfaces of the calls before the cache: per-head
// norms with rotary positions, and attention of whole prompts.
#pragma once
#include "kvq_common.cuh"

namespace kvq {

struct NormRopeArgs {
  const void* in[2];        // q, k: rows of heads x D, `stride` elements apart (null: absent)
  void* out[2];
  long long in_stride[2], out_stride[2];
  int heads[2];
  const float* weight[2];   // gains [D], or null: ones
  const int32_t* positions; // [axes][rows]
  const float* inv_freq;    // [rot / 2]
  int rows, axes, rot;
  int interleaved;          // pairs (2i, 2i + 1), else (i, i + rot / 2)
  float eps;                // negative: no norm
  uint8_t pair_axis[64];    // the axis of each pair
};
// in_dtype, out_dtype: kvq_dtype.
cudaError_t norm_rope_launch(const NormRopeArgs& a, int D, int in_dtype, int out_dtype, cudaStream_t st);

struct PromptArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;
  const int32_t* first;     // [B] first row of each sequence, or null: b t_new
  const int32_t* lens;      // [B] tokens of each sequence, or null: t_new
  uint32_t* status;
  long long q_stride, k_stride, v_stride, out_stride;   // elements from a row to the next
  int B, Hkv, Hq, G, rows, t_new, causal;
  int out32;                // out is fp32, else of the inputs' type
  float scale;
};
// dtype: KVQ_BF16 or KVQ_F16.
cudaError_t prompt_launch(const PromptArgs& a, int D, int dtype, cudaStream_t st);

// The rows of sequence b: false where it has none, or where they do not fit the
// call's bounds (bad).
__device__ __forceinline__ bool prompt_rows(const PromptArgs& a, int b, long long& first, int& n, bool& bad) {
  n = a.lens ? a.lens[b] : a.t_new;
  first = a.first ? a.first[b] : (long long)b * a.t_new;
  bad = n > 0 && (n > a.t_new || first < 0 || first + n > a.rows);
  return n > 0 && !bad;
}

}  // namespace kvq
