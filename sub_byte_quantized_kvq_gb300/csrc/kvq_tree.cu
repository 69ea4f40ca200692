// kvq_tree.cu -- attention of a tree of drafted tokens over the quantized cache.
//
// For row r = (node t, head g of the kv head's group) of sequence b:
//   a[r][j] = scale * q_r . k_j   over the cached tokens j < L and the nodes
//                                 that t's ancestor word names
//   out[r]  = sum_j e^a[r][j] v_j / sum_j e^a[r][j]
//   lse[r]  = ln sum_j e^a[r][j],   page_lse[r][p] = ln sum over page p
// in two launches: split kernels turn the cached pages into partial states
// (m, l, o) per (row, split); the merge kernel adds what is not in blocks (the
// fp32 staging tail and the drafted tokens' bf16 K and V), joins the splits and
// writes the results.
#include <algorithm>
#include <mutex>

#include "kvq_tree.cuh"

namespace kvq {

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// ----------------------------------------------------------------------------- rows on the CUDA cores
// A warp's state for kWR rows: channel c = 32 i + lane of row w in o[w][i].
constexpr int kWR = 4;
template <int D>
struct RowState {
  float m[kWR], l[kWR], o[kWR][D / 32];
};
template <int D>
__device__ __forceinline__ void row_state_init(RowState<D>& st) {
#pragma unroll
  for (int w = 0; w < kWR; ++w) {
    st.m[w] = -INFINITY;
    st.l[w] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) st.o[w][i] = 0.f;
  }
}

// One chunk of up to 16 tokens (ks, vs: fp32 [16][D + 1] in shared memory) for
// the warp's rows: lane = (half of the channels, token) for the scores, a
// channel slice for the outputs.  seen[w]: bit t set where row w attends to
// token t.  page[w] is set to the chunk's log2-sum-exp.  Tokens a row does not
// see are left out, whatever their K and V hold.
template <int D>
__device__ __forceinline__ void rows_chunk(RowState<D>& st, const float (*qs)[D], const float (*ks)[D + 1],
                                           const float (*vs)[D + 1], const uint32_t (&seen)[kWR], float scale_log2,
                                           float (&page)[kWR], int lane) {
  const int t = lane & 15, c0 = (lane >> 4) * (D / 2);
  float s[kWR];
#pragma unroll
  for (int w = 0; w < kWR; ++w) s[w] = 0.f;
#pragma unroll 8
  for (int c = 0; c < D / 2; ++c) {
    const float k = ks[t][c0 + c];
#pragma unroll
    for (int w = 0; w < kWR; ++w) s[w] = fmaf(qs[w][c0 + c], k, s[w]);
  }
#pragma unroll
  for (int w = 0; w < kWR; ++w) {
    s[w] += __shfl_xor_sync(0xffffffffu, s[w], 16);
    s[w] = (seen[w] >> t) & 1u ? s[w] * scale_log2 : -INFINITY;
    float mx = s[w];
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float mp = mx == -INFINITY ? 0.f : mx;
    const float p = exp2_approx(s[w] - mp);
    float sum = p;
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    page[w] = seen[w] ? mx + log2f(sum) : -INFINITY;
    // join: the chunk's state relative to its own maximum, the rows' to theirs
    const float mn = fmaxf(st.m[w], mx), mb = mn == -INFINITY ? 0.f : mn;
    const float fo = exp2_approx(st.m[w] - mb), fp = exp2_approx(mp - mb);
    st.m[w] = mn;
    st.l[w] = st.l[w] * fo + sum * (mx == -INFINITY ? 0.f : fp);
    s[w] = mx == -INFINITY ? 0.f : p * fp;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) st.o[w][i] *= fo;
  }
#pragma unroll 4
  for (int tt = 0; tt < kPage; ++tt) {
    float v[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) v[i] = vs[tt][32 * i + lane];
#pragma unroll
    for (int w = 0; w < kWR; ++w) {
      const float p = __shfl_sync(0xffffffffu, s[w], tt);
      if ((seen[w] >> tt) & 1u) {   // uniform over the warp
#pragma unroll
        for (int i = 0; i < D / 32; ++i) st.o[w][i] = fmaf(p, v[i], st.o[w][i]);
      }
    }
  }
}

// The CTA's query rows r0 .. r0 + n - 1 in fp32 (zeros past the live rows).
template <int D>
__device__ __forceinline__ void load_queries(const TreeArgs& a, int b, int h, int r0, int n, int live, float (*qs)[D]) {
  for (int i = threadIdx.x; i < n * D; i += blockDim.x) {
    const int r = r0 + i / D, t = r / a.G, g = r % a.G;
    qs[i / D][i % D] =
        r < live ? __bfloat162float(a.q[(((size_t)b * a.T + t) * a.Hq + (size_t)h * a.G + g) * D + i % D]) : 0.f;
  }
}

// ----------------------------------------------------------------------------- tail, tree and merge
// Grid (ceil(R / kMRows), Hkv, B), 4 warps of kWR rows: the staged tail and the
// drafted tokens in chunks of 16 on the CUDA cores (K and V of a token that a
// row does not see never reach the row, so a branch may hold infinities or NaN
// without touching its siblings), then the splits in ascending order.
constexpr int kMRows = 4 * kWR;
template <int D>
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeArgs a) {
  __shared__ float qs[kMRows][D];
  __shared__ float kvs[2][kPage][D + 1];
  const int r0 = blockIdx.x * kMRows, h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const SeqView v = seq_view(a, b);
  const int live = v.nodes * a.G;
  load_queries<D>(a, b, h, r0, kMRows, live, qs);
  RowState<D> st;
  row_state_init(st);
  if (r0 < live) {
    const int staged = v.len - v.blocks * kPage;   // <= 0 for per-token formats
    const int su = unit_tokens(a.fmt), off = v.blocks * kPage % su;   // rows of staging before the first of them
    const int cs = staged > 0 ? (staged + kPage - 1) / kPage : 0;
    const int cn = a.kv[0] ? (v.nodes + kPage - 1) / kPage : 0;
    for (int ch = 0; ch < cs + cn; ++ch) {
      const bool tail = ch < cs;
      const int t0 = kPage * (tail ? ch : ch - cs), n = min(kPage, (tail ? staged : v.nodes) - t0);
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * n * D; i += blockDim.x) {
        const int role = i / (n * D), t = i / D % n, c = i % D;
        kvs[role][t][c] = tail ? a.staging[((((size_t)b * a.Hkv + h) * 2 + role) * su + off + t0 + t) * D + c]
                               : __bfloat162float(a.kv[role][(((size_t)b * a.T + t0 + t) * a.Hkv + h) * D + c]);
      }
      __syncthreads();
      uint32_t seen[kWR];
      float page[kWR];
#pragma unroll
      for (int w = 0; w < kWR; ++w) {
        const int r = r0 + warp * kWR + w, t = r / a.G;
        uint32_t bits = (1u << n) - 1u;
        if (!tail)
          bits &= (uint32_t)((a.mask ? (r < live ? a.mask[(size_t)b * a.mask_stride + t] : 0ull) : (2ull << t) - 1ull) >> t0);
        seen[w] = r < live ? bits : 0u;
      }
      rows_chunk<D>(st, qs + warp * kWR, kvs[0], kvs[1], seen, a.scale_log2, page, lane);
      if (tail && a.page_lse && lane == 0)
#pragma unroll
        for (int w = 0; w < kWR; ++w) {
          const int r = r0 + warp * kWR + w;
          if (r < live) page_lse_row(a, b, h, r)[v.blocks + ch] = page[w] * kLn2;
        }
    }
  }
#pragma unroll
  for (int w = 0; w < kWR; ++w) {
    const int r = r0 + warp * kWR + w;
    if (r >= a.R) continue;
    const size_t base = ((size_t)b * a.Hkv + h) * a.S * a.R + r;
    if (r < live)
      for (int s = 0; s < a.S; ++s) {
        const size_t row = base + (size_t)s * a.R;
        const float2 ml = a.part_ml[row];
        if (ml.x == -INFINITY) continue;   // nothing in this split
        const float mn = fmaxf(st.m[w], ml.x);
        const float f0 = exp2_approx(st.m[w] - mn), f1 = exp2_approx(ml.x - mn);
        st.m[w] = mn;
        st.l[w] = st.l[w] * f0 + ml.y * f1;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          st.o[w][i] = fmaf(a.part_o[row * D + 32 * i + lane], f1, st.o[w][i] * f0);
      }
    const size_t o = ((size_t)b * a.T + r / a.G) * a.Hq + (size_t)h * a.G + r % a.G;
    const bool empty = st.m[w] == -INFINITY;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float x = empty ? 0.f : st.o[w][i] / st.l[w];
      if (a.out_dtype == KVQ_BF16) static_cast<__nv_bfloat16*>(a.out)[o * D + 32 * i + lane] = __float2bfloat16_rn(x);
      else static_cast<float*>(a.out)[o * D + 32 * i + lane] = x;
    }
    if (a.lse && lane == 0) a.lse[o] = empty ? -INFINITY : (st.m[w] + log2f(st.l[w])) * kLn2;
  }
}

// ----------------------------------------------------------------------------- host side
static TreeKernel tree_kernel(int fmt, int D) {
  switch (fmt) {
    case KVQ_FMT_INT4_G32: return tree_kernel_int4(D);
    case KVQ_FMT_FP4_E2M1_S16: return tree_kernel_e2m1(D);
    case KVQ_FMT_CB2_OUTLIER: return tree_kernel_cb2(D);
    case KVQ_FMT_CB2_STATIC: return tree_kernel_cb2s(D);
    case KVQ_FMT_ASYM3_OUTLIER: return tree_kernel_a3(D);
    case KVQ_FMT_CB2_GROUP4: return tree_kernel_cb2g(D);
    default: return tree_kernel_tiered(D);
  }
}

// One CTA runs per SM, so the cached pages of the call take
// waves(S) x (tiles of a split + what a CTA costs besides, about three tiles:
// barriers, tensor memory, the query, the pipeline's fill and drain, the
// partial state) -- the smallest product, and among equals the fewest splits.
int tree_auto_splits(int B, int Hkv, int R, int max_seq_len, int sms) {
  const long long tiles = (max_seq_len + kPage * kTreeTilePages - 1) / (kPage * kTreeTilePages);
  const long long units = (long long)B * Hkv * ((R + kTreeRows - 1) / kTreeRows);
  long long best = 1, cost = -1;
  for (long long s = 1; s <= std::min<long long>(std::max<long long>(tiles, 1), 256); ++s) {
    const long long c = (units * s + sms - 1) / sms * ((tiles + s - 1) / s + 3);
    if (cost < 0 || c < cost) {
      cost = c;
      best = s;
    }
  }
  return (int)best;
}

// The split kernels' dynamic shared memory, allowed once per kernel and device.
static cudaError_t allow_smem(const TreeKernel& k) {
  static std::mutex mutex;
  static struct { void* fn; int dev; } done[256];
  static int n = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mutex);
  for (int i = 0; i < n; ++i)
    if (done[i].fn == k.fn && done[i].dev == dev) return cudaSuccess;
  e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
  if (e == cudaSuccess && n < 256) {
    done[n].fn = k.fn;
    done[n++].dev = dev;
  }
  return e;
}

template <int D>
static cudaError_t tree_launch_d(const TreeArgs& a, cudaStream_t st) {
  const TreeKernel k = tree_kernel(a.fmt, D);
  cudaError_t e = allow_smem(k);
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<TreeArgs*>(&a)};
  e = cudaLaunchKernel(k.fn, dim3(a.S, a.Hkv * ((a.R + kTreeRows - 1) / kTreeRows), a.B), dim3(k.threads), args, k.smem, st);
  if (e != cudaSuccess) return e;
  tree_merge_kernel<D><<<dim3((a.R + kMRows - 1) / kMRows, a.Hkv, a.B), 128, 0, st>>>(a);
  return cudaGetLastError();
}
cudaError_t tree_launch(const TreeArgs& a, int D, cudaStream_t st) {
  return D == 64 ? tree_launch_d<64>(a, st) : tree_launch_d<128>(a, st);
}

}  // namespace kvq
