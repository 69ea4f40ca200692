// kvq_evict.cu -- the attention mass of the cache's pages, and eviction by it.
#include <mutex>

#include "kvq_tree.cuh"

namespace kvq {

// ----------------------------------------------------------------------------- page mass
// out[b][p] = decay * in[b][p] + sum over the marked nodes t and heads h of
// e^(page_lse[b][t][h][p] - lse[b][t][h]).
//
// One pass over page_lse, which is all there is to read: a CTA takes 128 pages
// of a sequence, its 16 warps every 16th marked (node, head) row, four
// coalesced loads of four rows in flight each: 11.5 us for the 67 MB of 16
// sequences x 512 rows x 2048 pages, half of them marked (15 with a division per
// row and bounds in every block; 19 so and with 8 warps).  The warps' sums are
// added in ascending order, so results do not depend on timing.  A row without a
// token (lse = -inf) adds nothing.
constexpr int kMassWarps = 16, kMassPages = 128, kMassPer = kMassPages / 32;
__global__ void __launch_bounds__(32 * kMassWarps) page_mass_kernel(const float* __restrict__ lse,
                                                                    const float* __restrict__ page_lse,
                                                                    const uint64_t* __restrict__ nodes, float decay,
                                                                    const float* in, float* out, int T, int Hq, int P,
                                                                    int ppsm) {
  __shared__ int marked[64];
  __shared__ float part[kMassWarps][kMassPages];
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, p0 = blockIdx.x * kMassPages + lane;
  const uint64_t on = (nodes ? nodes[b] : ~0ull) & (T == 64 ? ~0ull : (1ull << T) - 1ull);
  if (threadIdx.x < T && ((on >> threadIdx.x) & 1ull)) marked[__popcll(on & ((1ull << threadIdx.x) - 1ull))] = threadIdx.x;
  __syncthreads();
  const int n = blockIdx.x * kMassPages < P ? __popcll(on) : 0;   // marked nodes
  const bool whole = (blockIdx.x + 1) * kMassPages <= P;
  float w[kMassPer] = {};
  constexpr int U = 4;
  int i = 0, h = warp;   // this warp's next row: head h of the i-th marked node (h may pass Hq: the node's successors)
  auto settle = [&]() {
    while (h >= Hq && i < n) {
      h -= Hq;
      ++i;
    }
  };
  for (settle(); i < n;) {
    float z[U], x[U][kMassPer];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      z[k] = -INFINITY;
      if (i < n) {
        const size_t r = ((size_t)b * T + marked[i]) * Hq + h;
        const float* row = page_lse + r * P + p0;
        z[k] = lse[r];
#pragma unroll
        for (int c = 0; c < kMassPer; ++c) x[k][c] = whole || p0 + 32 * c < P ? row[32 * c] : -INFINITY;
        h += kMassWarps;
        settle();
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (z[k] != -INFINITY)
#pragma unroll
        for (int c = 0; c < kMassPer; ++c) w[c] += __expf(x[k][c] - z[k]);
  }
#pragma unroll
  for (int c = 0; c < kMassPer; ++c) part[warp][32 * c + lane] = w[c];
  __syncthreads();
  const int p = blockIdx.x * kMassPages + threadIdx.x;
  if (threadIdx.x < kMassPages && p < ppsm) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kMassWarps; ++k) sum += part[k][threadIdx.x];
    const size_t i = (size_t)b * ppsm + p;
    out[i] = fmaf(decay, in[i], sum);
  }
}

cudaError_t page_mass_launch(const float* lse, const float* page_lse, const uint64_t* nodes, float decay, const float* in,
                             float* out, int B, int T, int Hq, int P, int ppsm, cudaStream_t st) {
  page_mass_kernel<<<dim3((ppsm + kMassPages - 1) / kMassPages, B), 32 * kMassWarps, 0, st>>>(lse, page_lse, nodes, decay, in,
                                                                                             out, T, Hq, P, ppsm);
  return cudaGetLastError();
}

// ----------------------------------------------------------------------------- eviction
// The order of page masses as unsigned keys: larger mass, larger key; -0 as +0,
// NaN below everything.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

// One CTA per sequence; latency is all that counts (two words a page to read
// and to write), so barriers are few.  The row and its masses are first copied
// to shared memory, so the outputs may be the inputs.  A radix select over
// 8-bit digits (a histogram by the CTA, its scan by one warp) finds the key of
// the last free unit to stay; ties go to the lowest index.  One scan over the
// threads' consecutive units then gives every page its place.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) evict_kernel(const EvictArgs a) {
  extern __shared__ uint8_t dyn[];
  int32_t* row = reinterpret_cast<int32_t*>(dyn);
  float* mass = reinterpret_cast<float*>(row + a.ppsm);
  constexpr int W = THREADS / 32;
  __shared__ int hist[2][256], sums[W], pick[2];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t at = (size_t)b * a.ppsm;
  const int L = a.lens_in[b];
  for (int i = tid; i < a.ppsm; i += THREADS) {
    row[i] = a.table_in[at + i];
    mass[i] = a.mass_in[at + i];
  }
  for (int i = tid; i < 256; i += THREADS) hist[1][i] = 0;   // the first digit's (d = 3)
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
  int need = evict ? a.keep - a.sink - a.recent : 0;   // free units that stay: >= 0, and fewer than there are
  if (evict && need == 0) cut = 0xFFFFFFFFu;           // (above every key)
  // after each digit, `need` is the number of units to stay among those whose key starts as the cut does
  for (int d = 3; d >= 0 && need > 0; --d) {
    int* h = hist[d & 1];
    const int shift = 8 * d;
    for (int u = first + tid; u < last; u += THREADS) {
      const uint32_t k = key_of(u);
      if (d == 3 || (k >> (shift + 8)) == (cut >> (shift + 8))) atomicAdd(&h[(k >> shift) & 255u], 1);
    }
    for (int i = tid; i < 256; i += THREADS) hist[(d & 1) ^ 1][i] = 0;
    __syncthreads();
    if (warp == 0) {   // lane: 8 digits from 255 - 8 lane down; the first digit whose running count reaches `need`
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = h[255 - 8 * lane - i];
      int before = sum;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, x);
        if (lane >= x) before += y;
      }
      before -= sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < need && before + c[i] >= need) {
          pick[0] = 255 - 8 * lane - i;
          pick[1] = need - before;
        }
        before += c[i];
      }
    }
    __syncthreads();
    cut |= (uint32_t)pick[0] << shift;
    need = pick[1];   // (written again only after the next digit's barrier)
  }
  // each thread's consecutive units, so that ranks follow the page order: those that stay for sure
  // (low half of the count) and those with the cut's own key (high half), of which the first `need` stay
  const int per = (full + THREADS - 1) / THREADS, u0 = min(tid * per, full), u1 = min(u0 + per, full);
  auto kind = [&](int u) -> uint32_t {
    if (!evict || u < first || u >= last) return 1u;
    const uint32_t k = key_of(u);
    return k > cut ? 1u : k == cut ? 0x10000u : 0u;
  };
  uint32_t count = 0u;
  for (int u = u0; u < u1; ++u) count += kind(u);
  uint32_t before = count;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, before, x);
    if (lane >= x) before += y;
  }
  if (lane == 31) sums[warp] = (int)before;
  __syncthreads();
  uint32_t other = lane < warp ? (uint32_t)sums[lane < W ? lane : 0] : 0u;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) other += __shfl_xor_sync(0xffffffffu, other, x);
  before += other - count;
  const int dropped = evict ? (full - a.keep) * a.unit : 0;
  int ties = (int)(before >> 16), kept = (int)(before & 0xFFFFu) + min(ties, need), gone = u0 - kept;
  for (int u = u0; u < u1; ++u) {
    const uint32_t x = kind(u);
    const bool stay = x == 1u || (x != 0u && ties < need);
    ties += x >> 16;
    const int to = stay ? kept++ * a.unit : a.ppsm - dropped + gone++ * a.unit;
    for (int j = 0; j < a.unit; ++j) {
      a.table_out[at + to + j] = row[u * a.unit + j];
      a.mass_out[at + to + j] = stay ? mass[u * a.unit + j] : 0.f;
    }
  }
  for (int i = full * a.unit + tid; i < a.ppsm; i += THREADS) {   // the partial unit, then unused entries
    a.table_out[at + i - dropped] = row[i];
    a.mass_out[at + i - dropped] = i < used ? mass[i] : 0.f;
  }
  if (tid == 0) {
    a.lens_out[b] = L - dropped * kPage;
    if (a.evicted) a.evicted[b] = dropped;
  }
}

// A row beyond 48 KB of shared memory needs the kernel's attribute, set once per device.
static cudaError_t allow_long_rows() {
  static std::mutex mutex;
  static bool done[64] = {};
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mutex);
  if (dev < 64 && done[dev]) return cudaSuccess;
  const cudaError_t f = cudaFuncSetAttribute(reinterpret_cast<const void*>(evict_kernel<1024>),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictMaxPages * 8);
  if (f == cudaSuccess && dev < 64) done[dev] = true;
  return f;
}

cudaError_t evict_launch(const EvictArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)a.ppsm * 8;
  if (a.ppsm <= 1024) {   // fewer warps, shorter barriers
    evict_kernel<256><<<a.B, 256, smem, st>>>(a);
  } else {
    if (smem > 32 * 1024) {
      const cudaError_t e = allow_long_rows();
      if (e != cudaSuccess) return e;
    }
    evict_kernel<1024><<<a.B, 1024, smem, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace kvq
