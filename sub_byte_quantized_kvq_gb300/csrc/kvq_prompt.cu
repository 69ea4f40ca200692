// kvq_prompt.cu -- attention of whole prompts (causal or full, grouped heads,
// padded or packed sequences) on the tensor cores:
//   a_ij = scale q_i . k_j for the tokens j that i sees,
//   out_i = sum_j e^a_ij v_j / sum_j e^a_ij,  lse_i = ln sum_j e^a_ij
//
// A tile is 128 rows: 128 / P consecutive tokens of P query heads of one kv head
// (P: the power of two in the group size), so short prompts fill tiles too.  A
// CTA takes two tiles, one behind the other, and goes once over the keys that
// they see, 128 at a time:
//
//   load warp     Q, K and V tiles by tiled TMA with 128-byte swizzle, straight
//                 from the caller's rows (any row stride); K and V in one ring
//   MMA warp      S = Q K^T (both from shared memory), O += P V with P from tensor
//                 memory and V as it lies, [token][channel].  Tile 0's and tile
//                 1's MMAs alternate: one's run while the other's softmax does
//   2 x 4 softmax warps, one row a thread: the row of S in registers, its maximum,
//                 p = 2^(a - m), P into tensor memory.  m is raised only when a row
//                 passes it by more than 2^8 (rare after the first keys); the
//                 warp then scales O.  At the end O / l goes to global memory
//   2 cleaning warps  V tiles with rows that not all of the CTA's tokens see: a
//                 weight of 0 times what may lie there (infinities, NaN, stale
//                 memory) has to stay 0.  Rows past the sequence become zeros;
//                 infinities and NaN in rows of later tokens too, and the tokens
//                 that do see them get them added at the end
//
// Precision: products of the inputs are exact in fp32, S, m, l and O are fp32; P
// is rounded to the inputs' type (fp16 biased by 2^6, so that small p keep their
// bits: p <= 2^14).
#include <algorithm>

#include "kvq_prompt.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace prompt {

constexpr int kM = 128, kKeys = 128;      // rows and keys of a tile
constexpr int kThreads = 384;
// Registers a thread: the launch has 168 each; the softmax warps take what the others give up.
constexpr int kRegsSoftmax = 208, kRegsRest = 88;
static_assert(256 * kRegsSoftmax + 128 * kRegsRest <= kThreads * 168, "setmaxnreg shares exceed what the launch has");
constexpr float kLag = 8.f;               // log2 of how far a row's scores may pass its reference m
constexpr float kLn2f = 0.69314718055994531f, kLog2e = 1.4426950408889634f;

template <int D>
struct Plan {
  static constexpr int kTile = kM * D * 2;            // bytes of a Q, K or V tile
  static constexpr int kBlock = kM * 128;             // of its 64 channels
  static constexpr int kStages = D == 128 ? 5 : 8;    // the ring of K and V tiles
  static constexpr int kSmem = 1024 + (2 + kStages) * kTile + 512;   // 1024: alignment slack
  // tensor memory: S of tile x at 128 x, O at 256 + D x, P over S (D = 128) or behind O
  static constexpr bool kOverS = D == 128;
  static __device__ __forceinline__ uint32_t p_at(int x) { return kOverS ? 128 * x : 384 + 64 * x; }
};
static_assert(Plan<128>::kSmem <= 227 * 1024, "shared memory");

struct Launch {
  CUtensorMap q, k, v;
  PromptArgs a;
  int P, tokens, tiles;   // heads and tokens of a tile, tiles of a CTA
  int units;              // Hq / P
};

struct Wait {
  volatile int* stop;
  // A bounded wait: gives up after 2e8 cycles (100 ms), or when another role has.
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait_sleep(bar, parity, 20000u))
      if (*stop || clock64() - t0 > 200000000ll) {
        *stop = 1;
        return false;
      }
    return true;
  }
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  if (BF) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  return h2_as_u32(__floats2half2_rn(lo, hi));
}

// The CTA's sequence and the first of its tokens, by its rank among all CTAs of a head: those with the most keys first
// (later CTAs then fill the gaps that they leave), none for what a sequence does not have.  With T_b tiles of `span`
// tokens in sequence b, count(L) = sum_b max(0, T_b - L) tiles lie at L or later in their sequences; the rank-th is
// the largest L with count(L) > rank.  By one warp, the first 128 sequences in registers.
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int span, long long rank, int lane, int& b, int& t0) {
  constexpr int R = 4;
  auto tiles_of = [&](int s) {
    long long f;
    int n;
    bool bad;
    return s < a.B && prompt_rows(a, s, f, n, bad) ? (n + span - 1) / span : 0;
  };
  int T[R];
#pragma unroll
  for (int k = 0; k < R; ++k) T[k] = tiles_of(lane + 32 * k);
  auto count = [&](int L) {
    long long c = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) c += max(0, T[k] - L);
    for (int s = lane + 32 * R; s < a.B; s += 32) c += max(0, tiles_of(s) - L);
    // (a sequence has at most 2^31 tiles; their sum over a warp in two halves)
    const unsigned lo = __reduce_add_sync(0xffffffffu, (unsigned)c & 0xFFFFFFu), hi = __reduce_add_sync(0xffffffffu, (unsigned)(c >> 24));
    return (long long)lo + ((long long)hi << 24);
  };
  if (count(0) <= rank) return false;
  int lo = 0, hi = (a.t_new - 1) / span + 1;   // count(lo) > rank >= count(hi) = 0
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (count(mid) > rank) lo = mid;
    else hi = mid;
  }
  int left = (int)(rank - count(lo + 1));      // which of the sequences with more than lo tiles
  for (int s0 = 0; s0 < a.B; s0 += 32) {
    const unsigned has = __ballot_sync(0xffffffffu, tiles_of(s0 + lane) > lo);
    const int n = __popc(has);
    if (left < n) {
      const unsigned at = __fns(has, 0, left + 1);
      b = s0 + (int)at;
      t0 = lo * span;
      return true;
    }
    left -= n;
  }
  return false;
}

template <int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Launch p) {
  using Pl = Plan<D>;
  constexpr int NS = Pl::kStages, KC = D / 64;
  extern __shared__ uint8_t raw_smem[];
  const PromptArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = raw_smem + (((smem_u32(raw_smem) + 1023u) & ~1023u) - smem_u32(raw_smem));
  uint8_t* ring = smem + 2 * Pl::kTile;
  uint64_t *q_full = reinterpret_cast<uint64_t*>(ring + NS * Pl::kTile), *full = q_full + 2, *empty = full + NS, *s_full = empty + NS,
           *p_full = s_full + 2, *o_done = p_full + 2, *v_raw = o_done + 2, *v_clean = v_raw + 4, *drained = v_clean + 4;
  volatile int* found = reinterpret_cast<volatile int*>(drained + 1);   // [0] b or -1, [1] t0, [2] stop, [3] bad V
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + 1) + 4;
  static_assert((2 + 2 * NS + 2 + 2 + 2 + 4 + 4 + 1) * 8 + 20 <= 512 && NS <= 8, "barriers");

  if (warp == 0) {
    int b = -1, t0 = 0;
    if (!find_tile(a, p.tiles * p.tokens, blockIdx.x / p.units, lane, b, t0)) b = -1;
    if (lane == 0) {
      found[0] = b;
      found[1] = t0;
    }
  } else if (warp == 8 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&v_raw[i], 1);
      mbar_init(&v_clean[i], 2);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
    found[2] = found[3] = 0;
  } else if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 10 && blockIdx.x == 0) {
    for (int s = lane; s < a.B; s += 32) {
      long long f;
      int n;
      bool bad;
      prompt_rows(a, s, f, n, bad);
      if (bad) atomicOr(a.status, KVQ_STATUS_BAD_ROWS);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tslot;
  const int b = found[0], t0 = found[1];
  bool ok = true;
  if (b >= 0) {
    const Wait wait{found + 2};
    long long first;
    int n;
    bool bad;
    prompt_rows(a, b, first, n, bad);
    const int u = blockIdx.x % p.units, head0 = u * p.P, kvh = head0 / a.G;
    // keys that tile x's tokens see, in tiles; the first of them that not every token sees whole
    auto n_keys = [&](int x) {
      const int t = t0 + x * p.tokens;
      return x < p.tiles && t < n ? ((a.causal ? min(n, t + p.tokens) : n) + kKeys - 1) / kKeys : 0;
    };
    const int n0 = n_keys(0), n1 = n_keys(1), most = max(n0, n1);
    auto masked_from = [&](int t) { return a.causal ? min(t + 1, n) / kKeys : n / kKeys; };
    const int clean0 = masked_from(t0);   // V tiles from here on are cleaned

    if (warp < 8) {
      // ---------------------------------------------------------------- softmax, one tile a warpgroup
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
      const int x = warp >> 2, row = tid & 127, nx = x ? n1 : n0, tx = t0 + x * p.tokens;
      const int token = tx + row / p.P, head = head0 + row % p.P;
      const int lim = a.causal ? min(n, token + 1) : n, mask0 = masked_from(tx);
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t ts = tmem + lanes + 128 * x, to = tmem + lanes + 256 + D * x, tp = tmem + lanes + Pl::p_at(x);
      const bool neg = a.scale < 0.f;
      const float f = fmaxf(fabsf(a.scale) * kLog2e, 1e-36f);   // (not 0: what is masked is -inf times it)
      constexpr float bias = BF ? 0.f : 6.f;
      float m = -INFINITY;
      uint64_t l2 = 0ull;
      for (int it = 0; it < nx; ++it) {
        ok = __all_sync(0xffffffffu, wait(&s_full[x], it & 1));
        if (!ok) break;
        tc::fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld32_issue(ts + 32 * c, s[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::wait_ld(s[c]);
        if (neg)
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) s[c][j] ^= 0x80000000u;
        if (it >= mask0) {
          const int k = lim - it * kKeys;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j >= k) s[c][j] = 0xFF800000u;
        }
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          top[c] = __uint_as_float(s[c][0]);
#pragma unroll
          for (int j = 1; j < 31; j += 2) top[c] = fmaxf(fmaxf(top[c], __uint_as_float(s[c][j])), __uint_as_float(s[c][j + 1]));
          top[c] = fmaxf(top[c], __uint_as_float(s[c][31]));
        }
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if (it == 0) {
          m = mx;
        } else {
          if (!Pl::kOverS) {   // PV(it - 1) reads P (over S, S(it) was issued after it)
            ok = __all_sync(0xffffffffu, wait(&o_done[x], (it - 1) & 1));
            if (!ok) break;
            tc::fence_after();
          }
          const bool raise = (mx - m) * f > kLag;
          if (__any_sync(0xffffffffu, raise)) {
            const float alpha = raise ? ex2f((m - mx) * f) : 1.f;
            if (raise) m = mx;
            const float2 l = unpack2(l2);
            l2 = pack2(l.x * alpha, l.y * alpha);
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tc::ld16(to + c, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tc::st16(to + c, o);
            }
          }
        }
        const float mb = m == -INFINITY ? bias : bias - m * f;
        const uint64_t f2 = pack2(f, f), mb2 = pack2(mb, mb);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 y = unpack2(fma2(pack2u(s[c][j], s[c][j + 1]), f2, mb2));
            const float e0 = ex2f(y.x), e1 = ex2f(y.y);
            l2 = add2(l2, pack2(e0, e1));
            w[j / 2] = pack_p<BF>(e0, e1);
          }
          tc::st16(tp + 16 * c, w);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      // ---- O / l, and the tile's log-sum-exp
      if (nx > 0) {
        ok = ok && __all_sync(0xffffffffu, wait(&o_done[x], (nx - 1) & 1));
        tc::fence_after();
        const float2 lp = unpack2(l2);
        const float l = lp.x + lp.y;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool live = token < n, patch = found[3] != 0;
        const long long r = first + token;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          if (ok) {
            tc::ld32(to + c, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = l == 0.f ? 0.f : o[j] * inv;
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = NAN;
          }
          if (__builtin_expect(patch && live, 0)) {   // infinities and NaN that the cleaning took out of the tiles
            for (int j = t0 + 1; j < lim; ++j) {
              const uint16_t* v = static_cast<const uint16_t*>(a.v) + (first + j) * a.v_stride + (long long)kvh * D + c;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = BF ? __uint_as_float((uint32_t)v[i] << 16) : __half2float(__ushort_as_half(v[i]));
                if (!isfinite(y)) o[i] += y;
              }
            }
          }
          if (!live) {
          } else if (a.out32) {
            float* dst = static_cast<float*>(a.out) + r * a.out_stride + (long long)head * D + c;
#pragma unroll
            for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(dst + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          } else {
            uint16_t* dst = static_cast<uint16_t*>(a.out) + r * a.out_stride + (long long)head * D + c;
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              *reinterpret_cast<uint4*>(dst + j) = make_uint4(pack_p<BF>(o[j], o[j + 1]), pack_p<BF>(o[j + 2], o[j + 3]),
                                                              pack_p<BF>(o[j + 4], o[j + 5]), pack_p<BF>(o[j + 6], o[j + 7]));
          }
          __syncwarp();
        }
        if (a.lse && live)
          a.lse[r * a.Hq + head] = !ok ? NAN : l == 0.f ? -INFINITY : (m * f - bias + __log2f(l)) * kLn2f;
        tc::fence_before();
      }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
      if (warp == 8 && lane == 0) {
        // -------------------------------------------------------------- loads: K(0), V(0), K(1), ... through the ring
        for (int x = 0; x < 2; ++x)
          if (x ? n1 : n0) {
            mbar_arrive_expect_tx(&q_full[x], Pl::kTile);
            for (int c = 0; c < KC; ++c)
              tc::tma3d(smem + x * Pl::kTile + c * Pl::kBlock, &p.q, 64 * c, head0, (int)first + t0 + x * p.tokens, &q_full[x]);
          }
        int i = 0;
        for (; i < 2 * most; ++i) {
          const int st = i % NS;
          if (i >= NS && !wait(&empty[st], (i / NS - 1) & 1)) {
            ok = false;
            break;
          }
          // a V tile that is cleaned lands on a barrier of its own (the ring holds at most four), so that the cleaning warps
          // see each of its phases
          const int w = (i >> 1) - clean0;
          uint64_t* bar = (i & 1) && w >= 0 ? &v_raw[w & 3] : &full[st];
          if (bar != &full[st]) mbar_arrive(&full[st]);
          mbar_arrive_expect_tx(bar, Pl::kTile);
          for (int c = 0; c < KC; ++c)
            tc::tma3d(ring + st * Pl::kTile + c * Pl::kBlock, i & 1 ? &p.v : &p.k, 64 * c, kvh, (int)first + (i >> 1) * kKeys, bar);
        }
        if (!ok) {   // what is in flight has to land before the CTA ends
          for (int x = 0; x < 2; ++x)
            if (x ? n1 : n0) mbar_wait_bounded(&q_full[x], 0, kWaitLimitNs);
          for (int j = max(0, i - NS); j < i; ++j) {
            const int w = (j >> 1) - clean0;
            if ((j & 1) && w >= 0) mbar_wait_bounded(&v_raw[w & 3], (w >> 2) & 1, kWaitLimitNs);
            else mbar_wait_bounded(&full[j % NS], (j / NS) & 1, kWaitLimitNs);
          }
        }
      } else if (warp == 9 && lane == 0) {
        // -------------------------------------------------------------- MMA
        constexpr uint32_t id_s = BF ? tc::idesc_bf16(kM, kKeys) : tc::idesc_f16(kM, kKeys);
        constexpr uint32_t id_o = (BF ? tc::idesc_bf16(kM, D) : tc::idesc_f16(kM, D)) | tc::kBMajorN;
        const uint64_t qd = tc::desc_sw128(smem_u32(smem)), kd = tc::desc_sw128(smem_u32(ring)),
                       vd = tc::desc_sw128_mn(smem_u32(ring), Pl::kBlock);
        const int total = 2 * most;
        auto full_wait = [&](int i) { return wait(&full[i % NS], (i / NS) & 1); };
        auto release = [&](int i) {   // (only where a later tile takes the place)
          if (i + NS < total) tc::commit(&empty[i % NS]);
        };
        auto scores = [&](int x, int it) {
          const uint64_t kt = kd + ((2 * it) % NS * Pl::kTile >> 4), qt = qd + (x * Pl::kTile >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = ((k >> 2) * Pl::kBlock + (k & 3) * 32) >> 4;
            tc::mma(tmem + 128 * x, qt + at, kt + at, id_s, k != 0);
          }
          tc::commit(&s_full[x]);
        };
        ok = full_wait(0);
        for (int x = 0; x < 2 && ok; ++x)
          if (x ? n1 : n0) {
            ok = wait(&q_full[x], 0);
            tc::fence_after();
            if (ok) scores(x, 0);
          }
        if (ok) release(0);
        for (int it = 0; it < most && ok; ++it) {
          const int w = it - clean0;
          ok = full_wait(2 * it + 1) && (w < 0 || (wait(&v_raw[w & 3], (w >> 2) & 1) && wait(&v_clean[w & 3], (w >> 2) & 1)));
          const int last = it < n1 ? 1 : 0;   // the last tile that uses K(it), V(it)
          for (int x = 0; x < 2 && ok; ++x) {
            const int nx = x ? n1 : n0;
            if (it >= nx) continue;
            ok = wait(&p_full[x], it & 1);
            if (!ok) break;
            tc::fence_after();
            const uint64_t vt = vd + ((2 * it + 1) % NS * Pl::kTile >> 4);
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              tc::mma_ta(tmem + 256 + D * x, tmem + Pl::p_at(x) + 8 * k, vt + (k * 2048 >> 4), id_o, (it | k) != 0);
            tc::commit(&o_done[x]);
            if (x == last) release(2 * it + 1);
            if (it + 1 < nx) {
              ok = full_wait(2 * it + 2);
              // S(it + 1) goes over P(it), which PV(it) reads: MMAs with different accumulators have no order of their own
              if (Pl::kOverS) ok = ok && wait(&o_done[x], it & 1);
              if (!ok) break;
              tc::fence_after();
              scores(x, it + 1);
              if (x == (it + 1 < n1 ? 1 : 0)) release(2 * it + 2);
            }
          }
        }
        if (!ok) {   // tensor memory may be freed, and shared memory given up, once what was issued is done
          tc::commit(drained);
          mbar_wait_bounded(drained, 0, kWaitLimitNs);
        }
      } else if (warp >= 10) {
        // -------------------------------------------------------------- V tiles that not every token sees whole
        int bad_v = 0;
        for (int it = clean0; it < most; ++it) {
          const int w = it - clean0;
          ok = __all_sync(0xffffffffu, wait(&v_raw[w & 3], (w >> 2) & 1));
          if (!ok) break;
          uint8_t* vt = ring + (2 * it + 1) % NS * Pl::kTile;
#pragma unroll 4
          for (int e = tid - 320; e < Pl::kTile / 16; e += 64) {
            const int j = it * kKeys + (e >> 3) % kKeys;   // (the swizzle keeps a row's 128 bytes together)
            uint4* at = reinterpret_cast<uint4*>(vt) + e;
            if (j >= n) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else if (j > t0 && a.causal) {
              // an exponent of all ones carries into its sign's place
              constexpr uint32_t ones = BF ? 0x7F807F80u : 0x7C007C00u, unit = BF ? 0x00800080u : 0x04000400u;
              uint4 y = *at;
              uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
              uint32_t any = 0u;
#pragma unroll
              for (int k = 0; k < 4; ++k) any |= (yw[k] & ones) + unit;
              if (__builtin_expect(any & 0x80008000u, 0)) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t c = ((yw[k] & ones) + unit) & 0x80008000u;   // 0x8000 in the halves to clear
                  yw[k] &= ~((c >> 15) * 0xFFFFu);
                }
                *at = y;
                bad_v = 1;
              }
            }
          }
          if (bad_v) found[3] = 1;
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_clean[w & 3]);
        }
      }
    }
    if (!ok && lane == 0) atomicOr(a.status, KVQ_STATUS_TIMEOUT);
  }
  __syncthreads();
  if (warp == 9) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Rows of `heads` x D 16-bit values, boxes of 64 channels x box_heads heads x box_rows rows, 128-byte swizzle.
static bool encode(CUtensorMap* map, const void* base, bool bf, int D, int heads, int rows, long long stride, int box_heads, int box_rows) {
  const tc::EncodeTiledFn enc = tc::encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows}, strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
  return enc(map, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF>
static cudaError_t launch(const PromptArgs& a, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(prompt_kernel<D, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<D>::kSmem);
  if (e != cudaSuccess) return e;
  Launch p;
  p.a = a;
  p.P = a.G & -a.G;
  p.tokens = kM / p.P;
  p.units = a.Hq / p.P;
  // CTAs of a head: every sequence may have a last tile that is not full, and no more rows than there are
  auto ctas = [&](int tiles) {
    const long long span = (long long)tiles * p.tokens;
    return std::min((long long)a.B * ((a.t_new + span - 1) / span), a.rows / span + a.B);
  };
  p.tiles = ctas(2) * p.units >= sms ? 2 : 1;   // one tile a CTA where two would leave SMs idle
  const long long grid = ctas(p.tiles) * p.units;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  if (!encode(&p.q, a.q, BF, D, a.Hq, a.rows, a.q_stride, p.P, p.tokens) || !encode(&p.k, a.k, BF, D, a.Hkv, a.rows, a.k_stride, 1, kKeys) ||
      !encode(&p.v, a.v, BF, D, a.Hkv, a.rows, a.v_stride, 1, kKeys))
    return cudaErrorInvalidValue;
  prompt_kernel<D, BF><<<(unsigned)grid, kThreads, Plan<D>::kSmem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace prompt

cudaError_t prompt_launch(const PromptArgs& a, int D, int dtype, cudaStream_t st) {
  if (dtype == KVQ_BF16) return D == 64 ? prompt::launch<64, true>(a, st) : prompt::launch<128, true>(a, st);
  return D == 64 ? prompt::launch<64, false>(a, st) : prompt::launch<128, false>(a, st);
}

}  // namespace kvq
