// kvq_tree.cuh -- argument blocks and launches of tree attention, page mass and
// page eviction (not part of the public ABI).
#pragma once
#include "kvq_internal.cuh"

namespace kvq {

// Rows of a (sequence, kv head): r = t * G + g, node t's query of the group's
// head g; R = T * G of them.
struct TreeArgs {
  const uint8_t* pool;
  const uint8_t* tier_pool;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const float* staging;
  uint32_t* status;
  const __nv_bfloat16* q;        // [B][T][Hq][D]
  const __nv_bfloat16* kv[2];    // [B][T][Hkv][D], or null: no tree
  const uint64_t* mask;          // [B or 1][T] ancestor words, or null: a chain
  int mask_stride;               // T, or 0 when every sequence has the same tree
  const int32_t* nodes;          // [B] live nodes, or null: T
  float* part_o;                 // [B][Hkv][S][R][D]
  float2* part_ml;               // [B][Hkv][S][R] (m in log2 units, l)
  void* out;                     // [B][T][Hq][D] in out_dtype
  int out_dtype;
  float* lse;                    // [B][T][Hq], or null
  float* page_lse;               // [B][T][Hq][P], or null
  int B, Hkv, Hq, G, T, R, P;
  int fmt, ppsm, num_pages, num_tier_pages, n_static;
  int S, pps;                    // splits, pages per split (S * pps >= P)
  int max_seq_len;
  float scale_log2;              // softmax_scale * log2(e)
};

struct EvictArgs {
  const int32_t* table_in;
  const int32_t* lens_in;
  const float* mass_in;
  int32_t* table_out;
  int32_t* lens_out;
  float* mass_out;
  int32_t* evicted;              // [B], or null
  int B, ppsm;
  int unit;                      // pages evicted together (4 for the group format)
  int keep, sink, recent;        // units
};

constexpr float kLn2 = 0.69314718055994531f;
constexpr int kTreeRows = 128;      // rows of a CTA
constexpr int kTreeTilePages = 8;   // a split is whole tiles of this many pages

__host__ __device__ constexpr bool page_format(int f) { return f >= KVQ_FMT_CB2_OUTLIER; }
__host__ __device__ constexpr int unit_tokens(int f) { return f == KVQ_FMT_CB2_GROUP4 ? kPage * kGroupPages : kPage; }

// What of a sequence is visible, and where it lies.
struct SeqView {
  int len;       // visible tokens
  int blocks;    // pages of them that lie in blocks
  int nodes;     // live tree nodes
};
__device__ __forceinline__ SeqView seq_view(const TreeArgs& a, int b) {
  const int L = max(a.seq_lens[b], 0);
  SeqView v;
  v.len = min(L, a.max_seq_len);
  const int pages = (v.len + kPage - 1) / kPage, u = unit_tokens(a.fmt);
  v.blocks = page_format(a.fmt) ? min(pages, L / u * (u / kPage)) : pages;
  v.nodes = a.nodes ? min(max(a.nodes[b], 0), a.T) : a.T;
  return v;
}
// Visible tokens that wait in staging (the merge kernel's).
__device__ __forceinline__ int staged_tokens(const TreeArgs& a, const SeqView& v) {
  return page_format(a.fmt) ? max(v.len - v.blocks * kPage, 0) : 0;
}
__device__ __forceinline__ float* page_lse_row(const TreeArgs& a, int b, int h, int r) {
  return a.page_lse + (((size_t)b * a.T + r / a.G) * a.Hq + (size_t)h * a.G + r % a.G) * a.P;
}

// One translation unit per format instantiates its kernels; the one for R rows:
struct TreeKernel {
  void* fn;
  size_t smem;
  int threads;
};
TreeKernel tree_kernel_int4(int D, int R);
TreeKernel tree_kernel_e2m1(int D, int R);
TreeKernel tree_kernel_cb2(int D, int R);
TreeKernel tree_kernel_tiered(int D, int R);
TreeKernel tree_kernel_cb2s(int D, int R);
TreeKernel tree_kernel_a3(int D, int R);
TreeKernel tree_kernel_cb2g(int D, int R);

cudaError_t tree_launch(const TreeArgs& a, int D, cudaStream_t st);
// Splits tree_launch's first kernel is given when the caller leaves the choice.
int tree_auto_splits(int B, int Hkv, int R, int max_seq_len, int sms);
// The largest count that choice takes for any bound on the lengths up to max_seq_len (grows with it).
int tree_most_splits(int B, int Hkv, int R, int max_seq_len, int sms);

cudaError_t page_mass_launch(const float* lse, const float* page_lse, const uint64_t* nodes, float decay, const float* in,
                             float* out, int B, int T, int Hq, int P, int ppsm, cudaStream_t st);

// Longest page-table row evict_launch takes (it holds the row and its mass in shared memory).
constexpr int kEvictMaxPages = 28672;
cudaError_t evict_launch(const EvictArgs& a, cudaStream_t st);

}  // namespace kvq
