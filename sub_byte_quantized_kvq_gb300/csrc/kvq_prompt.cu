// kvq_prompt.cu -- attention of whole prompts (causal or full, grouped heads,
// padded or packed sequences):
//   a_ij = scale q_i . k_j for the tokens j that i sees,
//   out_i = sum_j e^a_ij v_j / sum_j e^a_ij,  lse_i = ln sum_j e^a_ij
// One CTA per (tile of 64 tokens, query head, sequence), 32 keys at a time in
// fp32 on the CUDA cores, the running maximum and sum of each row in registers.
#include "kvq_prompt.cuh"

namespace kvq {

template <class T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }

template <int D, class T, class O>
__global__ void __launch_bounds__(256) prompt_plain_kernel(const PromptArgs a) {
  constexpr int KT = 32, XS = D + 4;
  extern __shared__ float sm[];
  float(*qs)[XS] = reinterpret_cast<float(*)[XS]>(sm);
  float(*ks)[XS] = qs + 64;
  float(*vs)[XS] = ks + KT;
  float(*ps)[KT + 1] = reinterpret_cast<float(*)[KT + 1]>(vs + KT);
  const int h = blockIdx.y, b = blockIdx.z, kvh = h / a.G, r = threadIdx.x >> 2, part = threadIdx.x & 3;
  long long f;
  int n;
  bool bad;
  const bool has = prompt_rows(a, b, f, n, bad);
  if (bad && h == 0 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, KVQ_STATUS_BAD_ROWS);
  const int t0 = blockIdx.x * 64, t = t0 + r;
  if (!has || t0 >= n) return;
  const T *q = static_cast<const T*>(a.q), *k = static_cast<const T*>(a.k), *v = static_cast<const T*>(a.v);
  for (int i = threadIdx.x; i < 64 * D; i += 256)
    qs[i / D][i % D] = t0 + i / D < n ? widen(q[(f + t0 + i / D) * a.q_stride + (long long)h * D + i % D]) : 0.f;
  float m = -INFINITY, l = 0.f, o[D / 4] = {};
  const int top = a.causal ? min(n, t0 + 64) : n, lim = a.causal ? min(n, t + 1) : n;   // keys the CTA, the row sees
  for (int j0 = 0; j0 < top; j0 += KT) {
    __syncthreads();
    for (int i = threadIdx.x; i < KT * D; i += 256) {
      const int j = j0 + i / D;
      ks[i / D][i % D] = j < n ? widen(k[(f + j) * a.k_stride + (long long)kvh * D + i % D]) : 0.f;
      vs[i / D][i % D] = j < n ? widen(v[(f + j) * a.v_stride + (long long)kvh * D + i % D]) : 0.f;
    }
    __syncthreads();
    float s[KT / 4], mx = m;
    for (int x = 0; x < KT / 4; ++x) {
      float dot = 0.f;
      for (int c = 0; c < D; ++c) dot = fmaf(qs[r][c], ks[part + 4 * x][c], dot);
      s[x] = j0 + part + 4 * x < lim ? dot * a.scale : -INFINITY;
      mx = fmaxf(mx, s[x]);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float mb = mx == -INFINITY ? 0.f : mx, fo = expf(m - mb);
    m = mx;
    l *= fo;
    for (int x = 0; x < KT / 4; ++x) {
      const float p = expf(s[x] - mb);
      l += p;
      ps[r][part + 4 * x] = p;
    }
    __syncwarp();
    for (int c = 0; c < D / 4; ++c) o[c] *= fo;
    for (int j = 0; j < KT && j0 + j < lim; ++j)
      for (int c = 0; c < D / 4; ++c) o[c] = fmaf(ps[r][j], vs[j][part + 4 * c], o[c]);
  }
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (t >= n) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  O* dst = static_cast<O*>(a.out) + (f + t) * a.out_stride + (long long)h * D;
  for (int c = 0; c < D / 4; ++c) dst[part + 4 * c] = (O)(l == 0.f ? 0.f : o[c] * inv);
  if (a.lse && part == 0) a.lse[(f + t) * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <int D, class T, class O>
static cudaError_t launch(const PromptArgs& a, cudaStream_t st) {
  const int smem = (64 + 64) * (D + 4) * 4 + 64 * 33 * 4;
  const cudaError_t e = cudaFuncSetAttribute(prompt_plain_kernel<D, T, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prompt_plain_kernel<D, T, O><<<dim3((a.t_new + 63) / 64, a.Hq, a.B), 256, smem, st>>>(a);
  return cudaGetLastError();
}
cudaError_t prompt_launch(const PromptArgs& a, int D, int dtype, int out_dtype, cudaStream_t st) {
  if (dtype == KVQ_BF16)
    return out_dtype == KVQ_F32 ? (D == 64 ? launch<64, __nv_bfloat16, float>(a, st) : launch<128, __nv_bfloat16, float>(a, st))
                                : (D == 64 ? launch<64, __nv_bfloat16, __nv_bfloat16>(a, st) : launch<128, __nv_bfloat16, __nv_bfloat16>(a, st));
  return out_dtype == KVQ_F32 ? (D == 64 ? launch<64, __half, float>(a, st) : launch<128, __half, float>(a, st))
                              : (D == 64 ? launch<64, __half, __half>(a, st) : launch<128, __half, __half>(a, st));
}

}  // namespace kvq
