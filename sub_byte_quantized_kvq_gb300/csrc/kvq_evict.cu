// kvq_evict.cu -- the attention mass of the cache's pages, and eviction by it.
#include "kvq_tree.cuh"

namespace kvq {

// ----------------------------------------------------------------------------- page mass
// out[b][p] = decay * in[b][p] + sum over the marked nodes t and heads h of
// e^(page_lse[b][t][h][p] - lse[b][t][h]); one thread a page, rows in ascending
// order.  A row without a token (lse = -inf) adds nothing.
__global__ void __launch_bounds__(128) page_mass_kernel(const float* __restrict__ lse, const float* __restrict__ page_lse,
                                                        const uint64_t* __restrict__ nodes, float decay, const float* in,
                                                        float* out, int T, int Hq, int P, int ppsm) {
  const int p = blockIdx.x * 128 + threadIdx.x, b = blockIdx.y;
  if (p >= ppsm) return;
  const uint64_t on = nodes ? nodes[b] : ~0ull;
  float w = 0.f;
  if (p < P)
    for (int t = 0; t < T; ++t) {
      if (!((on >> t) & 1ull)) continue;
      for (int h = 0; h < Hq; ++h) {
        const size_t r = ((size_t)b * T + t) * Hq + h;
        const float z = lse[r];
        if (z != -INFINITY) w += __expf(page_lse[r * P + p] - z);
      }
    }
  const size_t i = (size_t)b * ppsm + p;
  out[i] = fmaf(decay, in[i], w);
}

cudaError_t page_mass_launch(const float* lse, const float* page_lse, const uint64_t* nodes, float decay, const float* in,
                             float* out, int B, int T, int Hq, int P, int ppsm, cudaStream_t st) {
  page_mass_kernel<<<dim3((ppsm + 127) / 128, B), 128, 0, st>>>(lse, page_lse, nodes, decay, in, out, T, Hq, P, ppsm);
  return cudaGetLastError();
}

// ----------------------------------------------------------------------------- eviction
constexpr int kEvThreads = 1024;

// Exclusive prefix sum of x over the CTA; `total` gets the sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  __syncthreads();   // warp_sums may still be read by the previous call
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kEvThreads / 32; ++w) {
    const int y = warp_sums[w];
    before += w < warp ? y : 0;
    total += y;
  }
  return before + s - x;
}

// The order of page masses as unsigned keys: larger mass, larger key; -0 as +0,
// NaN below everything.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

// One CTA per sequence.  The row and its masses are first copied to shared
// memory, so the outputs may be the inputs.  A radix select over 8-bit digits
// finds the key of the last free unit to stay; ties go to the lowest index.
__global__ void __launch_bounds__(kEvThreads) evict_kernel(const EvictArgs a) {
  extern __shared__ uint8_t dyn[];
  int32_t* row = reinterpret_cast<int32_t*>(dyn);
  float* mass = reinterpret_cast<float*>(row + a.ppsm);
  __shared__ int hist[256], sums[kEvThreads / 32], pick[2];
  const int b = blockIdx.x, tid = threadIdx.x;
  const size_t at = (size_t)b * a.ppsm;
  for (int i = tid; i < a.ppsm; i += kEvThreads) {
    row[i] = a.table_in[at + i];
    mass[i] = a.mass_in[at + i];
  }
  const int L = a.lens_in[b];
  const int len = min(max(L, 0), a.ppsm * kPage);
  const int used = (len + kPage - 1) / kPage, full = len / (kPage * a.unit);   // full units
  const int first = a.sink, last = full - a.recent;                            // free units: [first, last)
  __syncthreads();
  auto key_of = [&](int u) {
    float m = mass[u * a.unit];
    for (int j = 1; j < a.unit; ++j) m += mass[u * a.unit + j];
    return mass_key(m);
  };
  const bool evict = full > a.keep;
  uint32_t cut = 0u;
  int need = 0;   // units with the cut's own key that stay
  if (evict) {
    need = a.keep - a.sink - a.recent;   // free units that stay; >= 0, and fewer than there are
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
      for (int i = tid; i < 256; i += kEvThreads) hist[i] = 0;
      __syncthreads();
      for (int u = first + tid; u < last; u += kEvThreads) {
        const uint32_t k = key_of(u);
        if (shift == 24 || (k >> (shift + 8)) == (cut >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1);
      }
      __syncthreads();
      // digits in descending order, one a thread: the first whose running count reaches `need`
      int total;
      const int n = tid < 256 ? hist[255 - tid] : 0;
      const int before = block_scan(n, sums, total);
      if (tid < 256 && before < need && before + n >= need) {
        pick[0] = 255 - tid;
        pick[1] = need - before;
      }
      __syncthreads();
      cut |= (uint32_t)pick[0] << shift;
      need = pick[1];
      __syncthreads();
    }
    if (a.keep == a.sink + a.recent) cut = 0xFFFFFFFFu;
  }
  // each thread's consecutive units, so that ranks follow the page order
  const int per = (full + kEvThreads - 1) / kEvThreads, u0 = min(tid * per, full), u1 = min(u0 + per, full);
  auto is_free = [&](int u) { return evict && u >= first && u < last; };
  int ties = 0, total, n_kept;
  for (int u = u0; u < u1; ++u) ties += is_free(u) && key_of(u) == cut;
  const int tie0 = block_scan(ties, sums, total);
  int kept = 0, tie = tie0;
  for (int u = u0; u < u1; ++u) {
    if (!is_free(u)) ++kept;
    else {
      const uint32_t k = key_of(u);
      kept += k > cut || (k == cut && tie++ < need);
    }
  }
  const int kept0 = block_scan(kept, sums, n_kept);
  const int gone = full - n_kept, dropped = gone * a.unit;
  int k = kept0, e = u0 - kept0;
  tie = tie0;
  for (int u = u0; u < u1; ++u) {
    bool stay = !is_free(u);
    if (!stay) {
      const uint32_t key = key_of(u);
      stay = key > cut || (key == cut && tie++ < need);
    }
    const int to = stay ? k++ * a.unit : a.ppsm - dropped + e++ * a.unit;
    for (int j = 0; j < a.unit; ++j) {
      a.table_out[at + to + j] = row[u * a.unit + j];
      a.mass_out[at + to + j] = stay ? mass[u * a.unit + j] : 0.f;
    }
  }
  for (int i = full * a.unit + tid; i < a.ppsm; i += kEvThreads) {   // the partial unit, then unused entries
    a.table_out[at + i - dropped] = row[i];
    a.mass_out[at + i - dropped] = i < used ? mass[i] : 0.f;
  }
  if (tid == 0) {
    a.lens_out[b] = L - dropped * kPage;
    if (a.evicted) a.evicted[b] = dropped;
  }
}

cudaError_t evict_launch(const EvictArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)a.ppsm * 8;
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(evict_kernel),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictMaxPages * 8);
  if (e != cudaSuccess) return e;
  evict_kernel<<<a.B, kEvThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
