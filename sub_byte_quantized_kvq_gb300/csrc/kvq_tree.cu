// kvq_tree.cu -- attention of a tree of drafted tokens over the quantized cache.
//
// For row r = (node t, head g of the kv head's group) of sequence b:
//   a[r][j] = scale * q_r . k_j   over the cached tokens j < L and the nodes
//                                 that t's ancestor word names
//   out[r]  = sum_j e^a[r][j] v_j / sum_j e^a[r][j]
//   lse[r]  = ln sum_j e^a[r][j],   page_lse[r][p] = ln sum over page p
// in two launches: a split kernel (kvq_tree_split.cuh) turns the cached pages
// into partial states (m, l, o) per (row, split); the merge kernel adds what is
// not in blocks (the fp32 staging tail and the drafted tokens' bf16 K and V),
// joins the splits and writes the results.
#include <algorithm>
#include <mutex>

#include "kvq_tree.cuh"

namespace kvq {

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// ----------------------------------------------------------------------------- tail, tree and merge
// What is not in blocks, and the joining of the splits.  Grid (ceil(R / (8 WR)),
// Hkv, B), 8 warps of WR rows.
//
// The staged tail (up to 15 tokens, 63 for the group format) and the drafted
// tokens go in chunks of 16 through shared memory in fp32 and are computed on
// the CUDA cores: K and V of a token that a row does not see never reach the
// row, so a branch may hold infinities or NaN without touching its siblings,
// and bf16 K and V keep their whole range.  It is little work (16 nodes: 1/2000
// of the cached pages' at 32k tokens), done before the split kernel's results
// are waited for.  The merge reads each partial state once, four or more rows'
// or splits' loads in flight; splits are joined in ascending order.
template <int D, int WR>
struct RowState {
  float m[WR], l[WR], o[WR][D / 32];   // lane's channels (D / 32) lane ..
};

template <int N>
struct Vec;
template <>
struct Vec<2> { using T = float2; };
template <>
struct Vec<4> { using T = float4; };
template <int N>
__device__ __forceinline__ void load_vec(float (&v)[N], const float* p) {
  *reinterpret_cast<typename Vec<N>::T*>(v) = *reinterpret_cast<const typename Vec<N>::T*>(p);
}

// One chunk of up to 16 tokens (ks, vs: fp32 rows of D + 4) for the warp's rows:
// lane = (half of the channels, token) for the scores, D / 32 channels for the
// outputs.  seen[w]: bit t set where row w attends to token t.  page[w] is set
// to the chunk's log2-sum-exp.
template <int D, int WR>
__device__ __forceinline__ void rows_chunk(RowState<D, WR>& st, const float (*qs)[D], const float (*ks)[D + 4],
                                           const float (*vs)[D + 4], const uint32_t (&seen)[WR], float scale_log2,
                                           float (&page)[WR], int lane) {
  constexpr int VEC = D / 32;
  const int t = lane & 15, c0 = (lane >> 4) * (D / 2);
  float s[WR];
#pragma unroll
  for (int w = 0; w < WR; ++w) s[w] = 0.f;
#pragma unroll 4
  for (int c = c0; c < c0 + D / 2; c += 4) {
    const float4 k = *reinterpret_cast<const float4*>(&ks[t][c]);
#pragma unroll
    for (int w = 0; w < WR; ++w) {
      const float4 q = *reinterpret_cast<const float4*>(&qs[w][c]);
      s[w] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[w]))));
    }
  }
#pragma unroll
  for (int w = 0; w < WR; ++w) {
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
    page[w] = seen[w] ? mx + __log2f(sum) : -INFINITY;
    // join: the chunk's state relative to its own maximum, the rows' to theirs
    const float mn = fmaxf(st.m[w], mx), mb = mn == -INFINITY ? 0.f : mn;
    const float fo = exp2_approx(st.m[w] - mb), fp = exp2_approx(mp - mb);
    st.m[w] = mn;
    st.l[w] = st.l[w] * fo + sum * (mx == -INFINITY ? 0.f : fp);
    s[w] = mx == -INFINITY ? 0.f : p * fp;
#pragma unroll
    for (int i = 0; i < VEC; ++i) st.o[w][i] *= fo;
  }
  uint32_t any = 0u;
#pragma unroll
  for (int w = 0; w < WR; ++w) any |= seen[w];
  for (; any; any &= any - 1u) {   // tokens that a row of the warp sees (uniform over the warp)
    const int tt = __ffs((int)any) - 1;
    float v[VEC];
    load_vec(v, &vs[tt][VEC * lane]);
#pragma unroll
    for (int w = 0; w < WR; ++w) {
      const float p = __shfl_sync(0xffffffffu, s[w], tt);
      if ((seen[w] >> tt) & 1u) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) st.o[w][i] = fmaf(p, v[i], st.o[w][i]);
      }
    }
  }
}

// 8 bf16 as fp32.
__device__ __forceinline__ void widen8(uint4 x, float* o) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(u[i] << 16);
    o[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

constexpr int kMergeWarps = 8;
template <int D, int WR>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeArgs a) {
  constexpr int ROWS = kMergeWarps * WR, VEC = D / 32;
  __shared__ __align__(16) float qs[ROWS][D];
  __shared__ __align__(16) float kvs[2][kPage][D + 4];
  const int r0 = blockIdx.x * ROWS, h = blockIdx.y, b = blockIdx.z;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rw = r0 + warp * WR;
  const SeqView v = seq_view(a, b);
  const int live = v.nodes * a.G;
  RowState<D, WR> st;
#pragma unroll
  for (int w = 0; w < WR; ++w) {
    st.m[w] = -INFINITY;
    st.l[w] = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) st.o[w][i] = 0.f;
  }
  const int staged = staged_tokens(a, v), cs = (staged + kPage - 1) / kPage;
  const int cn = a.kv[0] ? (v.nodes + kPage - 1) / kPage : 0;
  if (r0 < live && cs + cn > 0) {
    for (int i = threadIdx.x; i < ROWS * D / 8; i += 32 * kMergeWarps) {
      const int r = r0 + i / (D / 8), t = r / a.G;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (r < live)
        x = *reinterpret_cast<const uint4*>(a.q + (((size_t)b * a.T + t) * a.Hq + (size_t)h * a.G + r % a.G) * D + i % (D / 8) * 8);
      widen8(x, &qs[i / (D / 8)][i % (D / 8) * 8]);
    }
    const int su = unit_tokens(a.fmt), off = v.blocks * kPage % su;   // rows of staging before the first of the tail
    uint64_t sees[WR];
#pragma unroll
    for (int w = 0; w < WR; ++w) {
      const int r = rw + w, t = r / a.G;
      sees[w] = r >= live ? 0ull : a.mask ? a.mask[(size_t)b * a.mask_stride + t] : (2ull << t) - 1ull;
    }
    for (int ch = 0; ch < cs + cn; ++ch) {
      const bool tail = ch < cs;
      const int t0 = kPage * (tail ? ch : ch - cs), n = min(kPage, (tail ? staged : v.nodes) - t0);
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * n * D / 8; i += 32 * kMergeWarps) {
        const int role = i / (n * D / 8), t = i / (D / 8) % n, c = i % (D / 8) * 8;
        float x[8];
        if (tail) {
          const float* src = a.staging + ((((size_t)b * a.Hkv + h) * 2 + role) * su + off + t0 + t) * D + c;
          *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
          *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(src + 4);
        } else {
          widen8(*reinterpret_cast<const uint4*>(a.kv[role] + (((size_t)b * a.T + t0 + t) * a.Hkv + h) * D + c), x);
        }
        *reinterpret_cast<float4*>(&kvs[role][t][c]) = *reinterpret_cast<const float4*>(x);
        *reinterpret_cast<float4*>(&kvs[role][t][c + 4]) = *reinterpret_cast<const float4*>(x + 4);
      }
      __syncthreads();
      uint32_t seen[WR], any = 0u;
#pragma unroll
      for (int w = 0; w < WR; ++w) {
        const uint32_t all = (1u << n) - 1u;
        seen[w] = rw + w >= live ? 0u : tail ? all : (uint32_t)(sees[w] >> t0) & all;
        any |= seen[w];
      }
      if (!any) continue;   // no row of the warp sees the chunk
      float page[WR];
      rows_chunk<D, WR>(st, qs + warp * WR, kvs[0], kvs[1], seen, a.scale_log2, page, lane);
      if (tail && a.page_lse && lane == 0)
#pragma unroll
        for (int w = 0; w < WR; ++w)
          if (rw + w < live) page_lse_row(a, b, h, rw + w)[v.blocks + ch] = page[w] * kLn2;
    }
  }

  asm volatile("griddepcontrol.wait;" ::: "memory");   // the split kernel's partial states
  const int nr = min(WR, live - rw);   // live rows of the warp
  if (nr > 0 && v.blocks > 0) {
    const size_t base = ((size_t)b * a.Hkv + h) * a.S * a.R + rw;
    float M[WR];
#pragma unroll
    for (int w = 0; w < WR; ++w) M[w] = st.m[w];
    for (int s = lane; s < a.S; s += 32)
#pragma unroll
      for (int w = 0; w < WR; ++w)
        if (w < nr) M[w] = fmaxf(M[w], a.part_ml[base + (size_t)s * a.R + w].x);
#pragma unroll
    for (int w = 0; w < WR; ++w) {
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) M[w] = fmaxf(M[w], __shfl_xor_sync(0xffffffffu, M[w], x));
      const float f = M[w] == -INFINITY ? 0.f : exp2_approx(st.m[w] - M[w]);
      st.m[w] = M[w];
      st.l[w] *= f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) st.o[w][i] *= f;
    }
    for (int s0 = 0; s0 < a.S; s0 += 32) {
      float wt[WR];   // split s0 + lane's weight (0 without tokens: its sum is 0, or NaN where a wait gave up)
#pragma unroll
      for (int w = 0; w < WR; ++w) {
        const float2 ml = s0 + lane < a.S && w < nr ? a.part_ml[base + (size_t)(s0 + lane) * a.R + w] : make_float2(-INFINITY, 0.f);
        wt[w] = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - M[w]);
        float sum = wt[w] * ml.y;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        st.l[w] += sum;
      }
      const int n = min(32, a.S - s0);
      constexpr int U = WR >= 4 ? 2 : 8;   // splits in flight
      for (int s = 0; s < n; s += U) {
        float x[U][WR][VEC], f[U][WR];
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int w = 0; w < WR; ++w) {
            f[k][w] = s + k < n ? __shfl_sync(0xffffffffu, wt[w], (s + k) & 31) : 0.f;
            if (f[k][w] != 0.f) load_vec(x[k][w], a.part_o + (base + (size_t)(s0 + s + k) * a.R + w) * D + VEC * lane);
          }
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int w = 0; w < WR; ++w)
            if (f[k][w] != 0.f)
#pragma unroll
              for (int i = 0; i < VEC; ++i) st.o[w][i] = fmaf(f[k][w], x[k][w][i], st.o[w][i]);
      }
    }
  }
#pragma unroll
  for (int w = 0; w < WR; ++w) {
    const int r = rw + w;
    if (r >= a.R) continue;
    const size_t o = ((size_t)b * a.T + r / a.G) * a.Hq + (size_t)h * a.G + r % a.G;
    const bool empty = st.l[w] == 0.f;   // (a row of NaN scores has no maximum either, but its sum is NaN)
    float y[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) y[i] = empty ? 0.f : st.o[w][i] / st.l[w];
    if (a.out_dtype == KVQ_BF16) {
      uint32_t u[VEC / 2];
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(y[i], y[i + 1]);
        u[i / 2] = *reinterpret_cast<const uint32_t*>(&p);
      }
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + o * D + VEC * lane);
      if (VEC == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[VEC / 2 - 1]);
      else dst[0] = u[0];
    } else {
      float* dst = static_cast<float*>(a.out) + o * D + VEC * lane;
      *reinterpret_cast<typename Vec<VEC>::T*>(dst) = *reinterpret_cast<const typename Vec<VEC>::T*>(y);
    }
    if (a.lse && lane == 0) a.lse[o] = empty ? -INFINITY : (st.m[w] + __log2f(st.l[w])) * kLn2;
  }
}

// ----------------------------------------------------------------------------- host side
static TreeKernel tree_kernel(int fmt, int D, int R) {
  switch (fmt) {
    case KVQ_FMT_INT4_G32: return tree_kernel_int4(D, R);
    case KVQ_FMT_FP4_E2M1_S16: return tree_kernel_e2m1(D, R);
    case KVQ_FMT_CB2_OUTLIER: return tree_kernel_cb2(D, R);
    case KVQ_FMT_CB2_STATIC: return tree_kernel_cb2s(D, R);
    case KVQ_FMT_ASYM3_OUTLIER: return tree_kernel_a3(D, R);
    case KVQ_FMT_CB2_GROUP4: return tree_kernel_cb2g(D, R);
    default: return tree_kernel_tiered(D, R);
  }
}

static long long tree_tiles(int max_seq_len) {
  return (max_seq_len + kPage * kTreeTilePages - 1) / (kPage * kTreeTilePages);
}
static long long tree_units(int B, int Hkv, int R) { return (long long)B * Hkv * ((R + kTreeRows - 1) / kTreeRows); }
int tree_most_splits(int B, int Hkv, int R, int max_seq_len, int sms) {   // (never over 8 waves)
  const long long units = tree_units(B, Hkv, R);
  return (int)std::min({std::max(tree_tiles(max_seq_len), 1ll), (8ll * sms + units - 1) / units, 256ll});
}
// One CTA runs per SM, so the cached pages of the call take
// waves(S) x (tiles of a split + what a CTA costs besides: barriers, tensor
// memory, the query, the pipeline's fill and drain, the partial state; measured
// 4 us or three tiles with 8 rows, 8 us or five and a half with 128; counted as
// five for any rows and any format, INT4 with its tiles of 64 tokens included) --
// the smallest product, and among equals the fewest splits.
int tree_auto_splits(int B, int Hkv, int R, int max_seq_len, int sms) {
  const long long tiles = tree_tiles(max_seq_len), units = tree_units(B, Hkv, R);
  const long long most = tree_most_splits(B, Hkv, R, max_seq_len, sms);
  long long best = 1, cost = -1;
  for (long long s = 1; s <= most; ++s) {
    const long long c = (units * s + sms - 1) / sms * ((tiles + s - 1) / s + 5);
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
  const TreeKernel k = tree_kernel(a.fmt, D, a.R);
  cudaError_t e = allow_smem(k);
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<TreeArgs*>(&a)};
  e = cudaLaunchKernel(k.fn, dim3(a.S, a.Hkv * ((a.R + kTreeRows - 1) / kTreeRows), a.B), dim3(k.threads), args, k.smem, st);
  if (e != cudaSuccess) return e;
  // The merge is launched while the split kernel runs (programmatic dependent launch): that hides its launch, and its work
  // on the tail and the nodes where an SM has no split CTA (beside one, no merge CTA fits).  A warp takes four rows,
  // which share the loads of the tail's and the nodes' K and V, or one where that would leave most SMs idle (up to
  // two CTAs of 8 one-row warps on each of 152; measured with 8 of them: 4096 rows 46 us a call instead of 42).
  const bool few = (long long)a.B * a.Hkv * a.R <= 152 * 8 * 2;
  const int rows = kMergeWarps * (few ? 1 : 4);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.R + rows - 1) / rows, a.Hkv, a.B);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 1>, a) : cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 4>, a);
}
cudaError_t tree_launch(const TreeArgs& a, int D, cudaStream_t st) {
  return D == 64 ? tree_launch_d<64>(a, st) : tree_launch_d<128>(a, st);
}

}  // namespace kvq
