// kvq_rope.cu -- per-head RMS norms of queries and keys and their rotary
// positions, in one pass over the rows.
//
//   n_c = x_c w_c / sqrt(1/D sum x^2 + eps)
//   pair (a, b) of the first R channels, phi = position[axis] * inv_freq:
//   y_a = n_a cos phi - n_b sin phi,  y_b = n_b cos phi + n_a sin phi
//
// Angles: a product in binary32 would be off by 2^-24 phi radians, 0.008 at 128k
// tokens.  Only phi modulo a turn counts, so a pair's frequency is turned once
// into a 64-bit fixed-point fraction of a turn per position (its 24 bits times 96 of
// 1 / (2 pi), off by at most 2^-63), and position x fraction modulo 2^64 is one
// integer product: the phase is off by less than 2^-32 of a turn at position 2^31.
// It is cut to 32 bits; their top gives the quadrant, the rest an angle within an
// eighth of a turn, which binary32 holds to 2^-28 of a turn.
//
// What bounds it: memory.  Each value is read once and written once, 16 bytes a
// lane; D / 16 lanes hold a head (chunks of 8 channels l and l + R / 16, so a
// pair's two channels are in one lane in either order of pairs), so a warp does
// 32 / (D / 16) heads a step and shares the sines and cosines of its row, each
// computed by one lane.  131072 rows of 40 heads of 128, bf16 (2.7 GB): 419 us, 6.4
// TB/s; 8 x 4096 rows: 112 us, 6.0 TB/s; one row: 3.8 to 4.2 us, a launch and the
// latency of positions, sines and one load.  Items are groups of one role: heads
// that do not fill the last group of q or of k leave lanes without work (D = 64, 4
// query heads and 1 kv head: 5 of 16 places are used).
#include <algorithm>
#include <atomic>

#include "kvq_prompt.cuh"

namespace kvq {

constexpr int kRopeWarps = 8;

template <int DT>
struct Elem;
template <>
struct Elem<KVQ_F32> { static constexpr int kWords = 8; };    // 32-bit words of 8 values
template <>
struct Elem<KVQ_F16> { static constexpr int kWords = 4; };
template <>
struct Elem<KVQ_BF16> { static constexpr int kWords = 4; };

template <int DT>
__device__ __forceinline__ void unpack8(const uint32_t (&u)[Elem<DT>::kWords], float* x) {
#pragma unroll
  for (int i = 0; i < Elem<DT>::kWords; ++i) {
    if (DT == KVQ_F32) {
      x[i] = __uint_as_float(u[i]);
    } else if (DT == KVQ_BF16) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(u32_as_h2(u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
template <int DT>
__device__ __forceinline__ void pack8(const float* x, uint32_t (&u)[Elem<DT>::kWords]) {
#pragma unroll
  for (int i = 0; i < Elem<DT>::kWords; ++i) {
    if (DT == KVQ_F32) {
      u[i] = __float_as_uint(x[i]);
    } else if (DT == KVQ_BF16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      u[i] = h2_as_u32(__floats2half2_rn(x[2 * i], x[2 * i + 1]));
    }
  }
}
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&u)[N], const uint8_t* p) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4*>(u + i) = __ldcs(reinterpret_cast<const uint4*>(p + 4 * i));   // (read once)
}
template <int N>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4*>(p + 4 * i) = *reinterpret_cast<const uint4*>(u + i);
}

// A frequency m 2^-s as a fraction of a turn per position, modulo 2^64: m times the first 96 bits of 1 / (2 pi), in whole
// numbers (off by less than 2^-63 below a frequency of 64, by 2^-32 at 2^55).  In binary64, 1 / (2 pi) rounded once, the
// fraction is off by up to 2^-52.9 and the phase at position 2^31 by more than 2^-22 of a turn; as two binary64 numbers it
// takes a decode step 0.5 us longer.
__device__ __forceinline__ uint64_t turn_per_position(float inv_freq) {
  const uint32_t u = __float_as_uint(inv_freq), e = u >> 23 & 255u, m = (u & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int s = max(150 - (int)max(e, 1u), -31);
  const uint64_t a1 = (uint64_t)m * 0x9391054Au + ((uint64_t)m * 0x7F09D5F4u >> 32), a2 = (uint64_t)m * 0x28BE60DBu + (a1 >> 32);
  const uint64_t per = s >= 32 ? a2 >> min(s - 32, 63) : a2 << (32 - s) | (a1 << 32) >> (32 + s);
  return u >> 31 ? 0ull - per : per;
}
// sin and cos of position * frequency.
__device__ __forceinline__ void turn_sincos(int pos, uint64_t per, float& s, float& c) {
  const int32_t turn = (int32_t)(((uint64_t)(int64_t)pos * per + 0x80000000ull) >> 32);   // in 2^-32 turns
  const int32_t quad = (int32_t)((uint32_t)turn + 0x20000000u) >> 30;                     // the nearest quarter
  const float rest = (float)(int32_t)((uint32_t)turn - ((uint32_t)quad << 30)) * 0x1p-31f;   // within +-1/4, in half turns
  float a, b;
  sincospif(rest, &a, &b);
  const bool odd = quad & 1;
  s = odd ? b : a;
  c = odd ? a : b;
  if (quad & 2) s = -s;
  if ((quad + 1) & 2) c = -c;
}

// CTAs an SM: 80 registers a thread for fp32 rows, 64 for the others, where at most 48 bytes a thread are spilled (none of
// fp32 rows but for fp32 results, 32).
template <int IN>
constexpr int rope_ctas() { return IN == KVQ_F32 ? 3 : 4; }

// Item (row, g) is 32 / (D / 16) heads of one row: q's groups first, then k's.  A warp takes whole rows, as many as every
// warp can have, then a run of the items of the rows that are left; the next item's loads are in flight while one is
// computed.  (7777 rows of 10 items, 4864 warps: 15% longer with whole rows alone; 131072 rows: 5% longer where a warp's rows
// lie behind one another.)
template <int D, int IN, int OUT>
__global__ void __launch_bounds__(32 * kRopeWarps, rope_ctas<IN>()) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int LPH = D / 16, HPW = 32 / LPH, PER = 8 / HPW;   // lanes a head, heads a step, pairs whose phase a lane computes
  constexpr int EI = IN == KVQ_F32 ? 4 : 2, EO = OUT == KVQ_F32 ? 4 : 2;
  __shared__ __align__(16) float gain[2][D];
  const int lane = threadIdx.x & 31, l = lane % LPH, hg = lane / LPH;
  const bool norm = a.eps >= 0.f;
  if (norm)
    for (int i = threadIdx.x; i < 2 * D; i += 32 * kRopeWarps) gain[i / D][i % D] = a.weight[i / D] ? a.weight[i / D][i % D] : 1.f;
  const int rc = a.rot / 16;                                   // chunks that hold a half of the rotated channels
  const bool turned = l < rc;
  const int c0 = turned ? l : 2 * rc + 2 * (l - rc), c1 = turned ? l + rc : c0 + 1;   // the lane's chunks of 8 channels
  // pair j = 0..7 of the lane: its index, and in registers x[j], y[j]: halves (c0, c1), or neighbours
  auto pair_of = [&](int j) { return a.interleaved ? 4 * (j < 4 ? c0 : c1) + (j & 3) : 8 * c0 + j; };
  uint64_t per[PER];
  const int32_t* where[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int p = turned ? pair_of(hg * PER + i) : 0;
    per[i] = turned ? turn_per_position(a.inv_freq[p]) : 0ull;
    where[i] = turned ? a.positions + (size_t)a.pair_axis[p] * a.rows : nullptr;
  }
  __syncthreads();
  const int gq = (a.heads[0] + HPW - 1) / HPW, groups = gq + (a.heads[1] + HPW - 1) / HPW;
  const int warps = gridDim.x * kRopeWarps, w = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const int rounds = a.rows / warps;                                   // rows of each warp
  const int over = a.rows - rounds * warps;                            // rows that are left, and their items
  const long long rest = (long long)over * groups, run = (rest + warps - 1) / warps, run0 = min(w * run, rest);
  long long left = (long long)rounds * groups + min(run, rest - run0);   // items of this warp
  uint32_t u0[Elem<IN>::kWords], u1[Elem<IN>::kWords];
  int h = 0, role = 0;
  auto place = [&](int g, int& r, int& head) {
    r = g >= gq;
    head = (g - (r ? gq : 0)) * HPW + hg;
    return head < a.heads[r];
  };
  auto fetch = [&](int row, int g) {
    if (place(g, role, h)) {
      const uint8_t* p = static_cast<const uint8_t*>(a.in[role]) + (row * a.in_stride[role] + (long long)h * D) * EI;
      load_words(u0, p + 8 * EI * c0);
      load_words(u1, p + 8 * EI * c1);
    }
  };
  if (left == 0) return;
  const int run_row = rounds * warps + (int)(run0 / groups), run_g = (int)(run0 % groups);
  int row = rounds > 0 ? w : run_row, g = rounds > 0 ? 0 : run_g;
  auto next_row = [&]() { return row >= (rounds - 1) * warps ? (row >= rounds * warps ? row + 1 : run_row) : row + warps; };
  fetch(row, g);
  while (true) {
    float cs[8], sn[8];
    {
      float s[PER], c[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        s[i] = 0.f;
        c[i] = 1.f;
        if (turned) turn_sincos(where[i][row], per[i], s[i], c[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sn[j] = __shfl_sync(0xffffffffu, s[j % PER], j / PER * LPH + l);
        cs[j] = __shfl_sync(0xffffffffu, c[j % PER], j / PER * LPH + l);
      }
    }
    for (; g < groups; ++g) {
      float x[8], y[8];
      unpack8<IN>(u0, x);
      unpack8<IN>(u1, y);
      int r, head;
      const bool live = place(g, r, head);
      const bool more = --left > 0;
      if (more) {
        if (g + 1 < groups) fetch(row, g + 1);
        else fetch(next_row(), row >= (rounds - 1) * warps && row < rounds * warps ? run_g : 0);
      }
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float m = fmaf(ss, 1.f / D, a.eps);
        float f = rsqrtf(m);
        if (m > 0.f && m < INFINITY) f = fmaf(0.5f * f, fmaf(-m * f, f, 1.f), f);   // one Newton step: rsqrtf alone is good to 2^-22.9
        float wx[8], wy[8];
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          *reinterpret_cast<float4*>(wx + j) = *reinterpret_cast<const float4*>(&gain[r][8 * c0 + j]);
          *reinterpret_cast<float4*>(wy + j) = *reinterpret_cast<const float4*>(&gain[r][8 * c1 + j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[j] = x[j] * f * wx[j];
          y[j] = y[j] * f * wy[j];
        }
      }
      if (turned) {
        if (a.interleaved) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float& p = j < 4 ? x[2 * j & 7] : y[2 * j & 7];
            float& q = j < 4 ? x[(2 * j + 1) & 7] : y[(2 * j + 1) & 7];
            const float t = fmaf(p, cs[j], -q * sn[j]);
            q = fmaf(q, cs[j], p * sn[j]);
            p = t;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float t = fmaf(x[j], cs[j], -y[j] * sn[j]);
            y[j] = fmaf(y[j], cs[j], x[j] * sn[j]);
            x[j] = t;
          }
        }
      }
      if (live) {
        uint32_t o[Elem<OUT>::kWords];
        uint8_t* p = static_cast<uint8_t*>(a.out[r]) + (row * a.out_stride[r] + (long long)head * D) * EO;
        pack8<OUT>(x, o);
        store_words(p + 8 * EO * c0, o);
        pack8<OUT>(y, o);
        store_words(p + 8 * EO * c1, o);
      }
      if (!more) return;
    }
    g = row >= (rounds - 1) * warps && row < rounds * warps ? run_g : 0;
    row = next_row();
  }
}

// The SMs of the current device (looked up once for each).
static cudaError_t sms_of_device(int& sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  }
  return e;
}

template <int D, int IN, int OUT>
static cudaError_t launch(const NormRopeArgs& a, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = sms_of_device(sms);
  if (e != cudaSuccess) return e;
  constexpr int HPW = 32 / (D / 16);
  const int groups = (a.heads[0] + HPW - 1) / HPW + (a.heads[1] + HPW - 1) / HPW;
  const long long items = (long long)a.rows * groups, ctas = std::min<long long>((items + kRopeWarps - 1) / kRopeWarps, sms * rope_ctas<IN>());
  norm_rope_kernel<D, IN, OUT><<<(unsigned)ctas, 32 * kRopeWarps, 0, st>>>(a);
  return cudaGetLastError();
}
template <int D, int IN>
static cudaError_t launch_out(const NormRopeArgs& a, int out_dtype, cudaStream_t st) {
  return out_dtype == KVQ_BF16 ? launch<D, IN, KVQ_BF16>(a, st)
       : out_dtype == KVQ_F16  ? launch<D, IN, KVQ_F16>(a, st)
                               : launch<D, IN, KVQ_F32>(a, st);
}
template <int D>
static cudaError_t launch_in(const NormRopeArgs& a, int in_dtype, int out_dtype, cudaStream_t st) {
  return in_dtype == KVQ_BF16 ? launch_out<D, KVQ_BF16>(a, out_dtype, st)
       : in_dtype == KVQ_F16  ? launch_out<D, KVQ_F16>(a, out_dtype, st)
                              : launch_out<D, KVQ_F32>(a, out_dtype, st);
}
cudaError_t norm_rope_launch(const NormRopeArgs& a, int D, int in_dtype, int out_dtype, cudaStream_t st) {
  return D == 64 ? launch_in<64>(a, in_dtype, out_dtype, st) : launch_in<128>(a, in_dtype, out_dtype, st);
}

}  // namespace kvq
