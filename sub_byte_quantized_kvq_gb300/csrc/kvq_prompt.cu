// kvq_prompt.cu -- attention of whole prompts (causal or full, grouped heads,
// padded or packed sequences) on the tensor cores:
//   a_ij = scale q_i . k_j for the tokens j that i sees,
//   out_i = sum_j e^a_ij v_j / sum_j e^a_ij,  lse_i = ln sum_j e^a_ij
//
// A tile is 128 rows: 128 / P consecutive tokens of P query heads of one kv head
// (P: the power of two in the group size), so short prompts fill tiles too.  One
// CTA an SM takes pairs of tiles, in parts whose keys stay in L2; a pair's two
// tiles lie behind one another and go once over the keys that they see, 128 at a
// time:
//
//   load warp     finds the pairs; Q, K and V tiles by tiled TMA with 128-byte
//                 swizzle, straight from the caller's rows (any row stride); K and
//                 V in one ring of five 32 KB tiles (D = 64: eight of 16 KB)
//   MMA warp      S = Q K^T (both from shared memory), O += P V with P from tensor
//                 memory and V as it lies, [token][channel]
//   2 x 4 softmax warps, a warpgroup a tile, one row a thread: 128 scores in
//                 registers, p = 2^(a - m), P into tensor memory.  m is raised only
//                 when the sums ask for it (rare after the first keys); the warp
//                 then scales O.  At the end O / l goes to global memory
//   2 cleaning warps  V tiles with rows that not all of the pair's tokens see: a
//                 weight of 0 times what may lie there (infinities, NaN, stale
//                 memory) has to stay 0.  Rows past the sequence become zeros;
//                 infinities and NaN in rows of later tokens too, and the tokens
//                 that do see them get them added at the end
//
// Precision: products of the inputs are exact in fp32, S, m, l and O are fp32.  P
// is rounded to the inputs' type, as the MMA takes it: off by at most 2^-8 (bf16) or
// 2^-11 (fp16) of each weight, as an output of that type is itself, and averaged
// over the keys; l adds the weights before they are rounded.  fp16 weights are
// biased by 2^6, so that small ones keep their bits (a half's sum stays below 2^15):
// those below 2^-20 of a row's largest are subnormal halves, off by up to 2^-31 of it,
// and those below 2^-31 become 0 in O.
//
// What bounds it: MMA time and the power limit for long prompts, the ends of pairs
// for shorter ones.  128 keys of a pair are 2048 cycles of MMAs (D = 128), measured
// as 2100 to 2300 (S reads both operands from shared memory), and take 2600: the
// softmax of a tile runs beside the other tile's MMAs (16384 exponentials at 32 a
// cycle and SM, measured, are 512 cycles; with the fused multiply-adds, sums and
// conversions about 700 for half the keys of both tiles, one warp of each on a
// scheduler), and each hand-over between the roles costs about 200.  A pair costs
// 5000 to 8000 cycles at its ends (first softmax, output of 64 KB, cleaning of the
// last V tiles).  With D = 64, 128 keys of a pair are 1024 cycles of MMAs, and the
// softmax's 1400 are the limit.
//   32768 tokens, 64 heads of 128, causal: 10.3 to 10.4 ms, 1.69 to 1.71 PFLOP/s (a
//   library product of 8192^3 holds 1.74 under the same power limit)
//   8 x 4096, 32 heads: 705 us, 1.56 PFLOP/s (772 without a pause);  17 tokens: 5.9 us
// What carried it: the MMAs issued by one elected lane of a converged warp (130 ->
// 64 cycles an MMA of N = 128; 12.2 -> 11.1 ms), one place for both tiles' S and no
// maximum in the common path (10.7 ms), S a step ahead of PV (17 tokens: 6.9 -> 5.7
// us), all weights computed before the wait for the last PV (10.4 ms), pairs in
// parts that L2 holds (8 x 4096: 746 -> 704 us, without a pause 854 -> 772).  The
// compiled softmax changes by up to 8% with code elsewhere in the kernel: time
// every change.
#include <algorithm>
#include <mutex>

#include "kvq_prompt.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace prompt {

constexpr int kM = 128, kKeys = 128;      // rows and keys of a tile
constexpr int kThreads = 384;
// Registers a thread: the launch has 168 each; the softmax warps take what the others give up.
constexpr int kRegsSoftmax = 208, kRegsRest = 88;
static_assert(256 * kRegsSoftmax + 128 * kRegsRest <= kThreads * 168, "setmaxnreg shares exceed what the launch has");
constexpr float kLn2f = 0.69314718055994531f, kLog2e = 1.4426950408889634f;

template <int D>
struct Plan {
  static constexpr int kTile = kM * D * 2;            // bytes of a Q, K or V tile
  static constexpr int kBlock = kM * 128;             // of its 64 channels
  static constexpr int kStages = D == 128 ? 5 : 8;    // the ring of K and V tiles
  static constexpr int kSmem = 1024 + (2 + kStages) * kTile + 512;   // 1024: alignment slack
  // Tensor memory: S at 0, P at 128 + 64 x, O at 256 + D x.  Both tiles' S go through one place, in turn: P then has one of
  // its own, and S(it + 1) need not wait for the PV that reads P(it).
  static constexpr int kP = 128, kO = 256;
};
static_assert(Plan<128>::kSmem <= 227 * 1024, "shared memory");

struct Launch {
  CUtensorMap q, k, v;
  PromptArgs a;
  int P, log_p, tokens, tiles;   // heads (a power of two) and tokens of a tile, tiles of a CTA
  int log_span;           // log2 of a pair's tokens
  int units;              // Hq / P
  int wide;               // rows of out are 32-byte aligned
  int pairs;              // tile pairs of all units, at most
  int seqs, hu, parts;    // sequences and units that are taken together; such parts of the units
};

struct Wait {
  volatile int* stop;
  // A bounded wait: gives up after 2e8 cycles (about 100 ms), or when another role has.
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

template <bool BF>
__device__ __forceinline__ float2 unpack_p(uint32_t u) {
  if (BF) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  return __half22float2(u32_as_h2(u));
}

// What the roles know of a tile pair: the sequence's first row and length (0: no more tiles), the first token, and the
// heads (unit u: query heads u P .. u P + P - 1).
struct Pair {
  int first, n, t0, unit;
};

// The order of the pairs.  `seqs` sequences and `heads` kv heads are taken at a time: their K and V are about 24 MB (one
// sequence and kv head at least), so that the CTAs, which go through them together, find them in L2.  Calls without a pause,
// under the power limit, on one GPU: 8 x 4096 tokens of 8 kv heads 840 us with all 134 MB, 780 with 64 MB at a time, 769 with
// 32, 764 with 24 and 16; 32768 tokens 10860, 10570, 10690, 10660 and 10660 us; 16 ragged sequences of up to 6007 1500, 1465,
// 1477, 1467 and 1497 us (shorter parts have more ends).  Within such a part the pairs with the most keys come first (later
// ones then fill the gaps that they leave); every other part goes backwards, so that the pairs of one round of CTAs are
// alike at its borders too, the last one forwards.
//
// Sequence b has T_b pairs of `span` tokens (none for what it does not have); count(L) = sum_b max(0, T_b - L) pairs of a head
// lie at L or later in their sequences, and the rank-th is at the largest L with count(L) > rank.  By one warp, the T_b of 256
// sequences in registers, however few are taken at a time: asked for rising indices, it reads each length once (2048
// sequences of up to 200 tokens: 1.03 ms; with the lengths behind the 256th read again for each pair 10.5 ms; 1024
// sequences of up to 64 tokens, padded to 4096 and so taken one at a time: 278 us; with a load for each of them 562 us).
struct Finder {
  static constexpr int R = 8;
  const Launch& p;
  const PromptArgs& a;
  int lane, most, T[R];
  int seq0;                    // the first of the `seqs` sequences
  int at, W[R];                // its place among those whose T_b are in registers
  unsigned item0 = 0, n = 0;   // their first item (pair x unit), and their pairs of a head
  bool even;                   // every sequence has t_new tokens
  __device__ __forceinline__ Finder(const Launch& launch, int ln) : p(launch), a(launch.a), lane(ln) {
    most = ((a.t_new - 1) >> p.log_span) + 1;
    seq0 = -p.seqs;
    at = 32 * R;
    even = !a.lens && !a.first && (long long)a.B * a.t_new <= a.rows;
#pragma unroll
    for (int k = 0; k < R; ++k) T[k] = 0;
  }
  __device__ __forceinline__ unsigned count(int L) const {
    unsigned c = 0;
#pragma unroll
    for (int k = 0; k < R; ++k) c += max(0, T[k] - L);
    return __reduce_add_sync(0xffffffffu, c);
  }
  // The pair of item i (indices below 2^31, checked by the launch).
  __device__ __forceinline__ bool find(unsigned i, Pair& r) {
    long long first;
    bool bad;
    if (even) {
      const unsigned per = (unsigned)most * p.seqs * p.units, g = i / per;
      seq0 = (int)g * p.seqs;
      item0 = g * per;
      if (seq0 >= a.B) return false;
      n = (unsigned)most * min(p.seqs, a.B - seq0);
    } else {
#pragma unroll 1
      while (i - item0 >= n * p.units) {
        if (a.B - seq0 <= p.seqs) return false;
        item0 += n * p.units;
        seq0 += p.seqs;
        at += p.seqs;
        if (at + p.seqs > 32 * R) {
          at = 0;
#pragma unroll
          for (int k = 0; k < R; ++k) {
            const int s = seq0 + lane + 32 * k;
            int len;
            W[k] = s < a.B && prompt_rows(a, s, first, len, bad) ? ((len - 1) >> p.log_span) + 1 : 0;
          }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) T[k] = (unsigned)(lane - at + 32 * k) < (unsigned)p.seqs ? W[k] : 0;
        n = count(0);
      }
    }
    const unsigned q = i - item0, part = q / (n * p.hu), inside = q - part * n * p.hu;
    const unsigned hw = min(p.hu, p.units - (int)part * p.hu);   // units of this part
    unsigned rank = inside / hw;
    r.unit = (int)(part * p.hu + inside - rank * hw);
    if (((a.B - 1 - seq0) / p.seqs + 1) * p.parts - 1 - (int)part & 1) rank = n - 1 - rank;
    int b;
    if (even) {
      const unsigned width = min(p.seqs, a.B - seq0), level = rank / width;
      b = seq0 + (int)(rank - level * width);
      r.t0 = (most - 1 - (int)level) << p.log_span;
    } else {
      int lo = 0, hi = most;     // count(lo) > rank >= count(hi)
      unsigned above = 0;        // count(hi)
#pragma unroll 1
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        const unsigned c = count(mid);
        if (c > rank) {
          lo = mid;
        } else {
          hi = mid;
          above = c;
        }
      }
      int left = (int)(rank - above);   // which of the sequences with more than lo pairs
      b = 0;
#pragma unroll 1
      for (int j = 0; j < p.seqs; j += 32) {
        const int s = seq0 + j + lane;
        int len;
        unsigned has = __ballot_sync(0xffffffffu, j + lane < p.seqs && s < a.B && prompt_rows(a, s, first, len, bad) && (len - 1) >> p.log_span >= lo);
        const int c = __popc(has);
        if (left < c) {
#pragma unroll 1
          for (; left > 0; --left) has &= has - 1;
          b = seq0 + j + __ffs((int)has) - 1;
          break;
        }
        left -= c;
      }
      r.t0 = lo << p.log_span;
    }
    prompt_rows(a, b, first, r.n, bad);
    r.first = (int)first;
    return true;
  }
};

// The k-th pair of this CTA: every round of the grid's CTAs takes the next ones in the finder's order, odd rounds
// backwards, so that no CTA has the longer one each time.
__device__ __forceinline__ Pair next_pair(const Launch& p, Finder& finder, unsigned k) {
  const unsigned i = k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);   // below 2^31 + 2 grids
  Pair r = {0, 0, 0, 0};
  if (i < (unsigned)p.pairs) finder.find(i, r);
  return r;
}

template <int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Launch p) {
  using Pl = Plan<D>;
  constexpr int NS = Pl::kStages, KC = D / 64;
  extern __shared__ uint8_t raw_smem[];
  const PromptArgs& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  uint8_t* smem = raw_smem + (((smem_u32(raw_smem) + 1023u) & ~1023u) - smem_u32(raw_smem));
  uint8_t* ring = smem + 2 * Pl::kTile;
  uint64_t *q_full = reinterpret_cast<uint64_t*>(ring + NS * Pl::kTile), *q_empty = q_full + 2, *full = q_empty + 2, *empty = full + NS,
           *s_full = empty + NS, *s_read = s_full + 2, *p_full = s_read + 1, *o_done = p_full + 2, *v_raw = o_done + 2, *v_clean = v_raw + 8,
           *info_full = v_clean + 8, *info_empty = info_full + 2, *drained = info_empty + 2;
  volatile int* info = reinterpret_cast<volatile int*>(drained + 1);   // [2] Pair
  volatile int* stop = info + 8;                                       // a wait gave up
  volatile int* bad_v = stop + 1;                                      // [2] pair's V has infinities or NaN that were cleaned
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + 1) + 11;
  static_assert((4 + 2 * NS + 2 + 1 + 2 + 2 + 8 + 8 + 2 + 2 + 1) * 8 + 48 <= 512 && NS <= 8, "barriers");

  if (warp == 8 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
      mbar_init(&info_full[i], 1);
      mbar_init(&info_empty[i], 11);   // softmax, MMA and cleaning warps
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(drained, 1);
    mbar_init(s_read, 4);
    for (int i = 0; i < 8; ++i) {
      mbar_init(&v_raw[i], 1);
      mbar_init(&v_clean[i], 2);
    }
    fence_mbar_init();
    stop[0] = bad_v[0] = bad_v[1] = 0;
  } else if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 10) {
    for (long long i = blockIdx.x * 32 + lane; i < a.B; i += gridDim.x * 32) {   // the sequences' rows are checked once
      long long f;
      int n;
      bool bad;
      prompt_rows(a, (int)i, f, n, bad);
      if (bad) atomicOr(a.status, KVQ_STATUS_BAD_ROWS);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tslot;
  const Wait wait{stop};
  bool ok = true;
  Pair pair = {0, 0, 0, 0};
  // keys that the tokens of the pair's tile x see, in tiles; the first tile that not every token from t on sees whole
  auto n_keys = [&](int x) {
    const int t = pair.t0 + x * p.tokens;
    return x < p.tiles && t < pair.n ? ((a.causal ? min(pair.n, t + p.tokens) : pair.n) + kKeys - 1) / kKeys : 0;
  };
  auto masked_from = [&](int t) { return (a.causal ? min(t + 1, pair.n) : pair.n) / kKeys; };
  // the k-th pair, published by the load warp (whole warps; false at the end)
  auto get_pair = [&](int k) {
    ok = __all_sync(0xffffffffu, wait(&info_full[k & 1], (k >> 1) & 1));
    if (!ok) return false;
    const volatile int* i = info + 4 * (k & 1);
    pair = {i[0], i[1], i[2], i[3]};
    return pair.n > 0;
  };
  auto give_pair_back = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&info_empty[k & 1]);
  };

  struct Place {   // of the ring, and the phase of its barriers' use
    int i, phase;
    __device__ __forceinline__ Place next() const { return i + 1 == NS ? Place{0, phase ^ 1} : Place{i + 1, phase}; }
  };

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax, one tile a warpgroup
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int x = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes, to = tmem + lanes + Pl::kO + D * x, tp = tmem + lanes + Pl::kP + 64 * x;
    const bool neg = a.scale < 0.f;
    const float f = fmaxf(fabsf(a.scale) * kLog2e, 1e-36f);   // (not 0: what is masked is -inf times it)
    constexpr float bias = BF ? 0.f : 6.f, kMost = BF ? 0x1p16f : 0x1p15f;   // m and the weights in log2 units: p = 2^(s f - m + bias)
    int done = 0;   // key tiles of earlier pairs
    for (int pk = 0; get_pair(pk); ++pk) {
      const int nx = n_keys(x), tx = pair.t0 + x * p.tokens;
      const int token = tx + (row >> p.log_p), mask0 = masked_from(tx);
      const int lim = a.causal ? min(pair.n, token + 1) : pair.n;
      float m = token < pair.n ? -INFINITY : 0.f, l = 0.f;   // (a row past the sequence asks for nothing)
      for (int it = 0; it < nx; ++it) {
        ok = __all_sync(0xffffffffu, wait(&s_full[x], (done + it) & 1));
        if (!ok) break;
        tc::fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld32_issue(ts + 32 * c, s[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::wait_ld(s[c]);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_read);   // the next S may come
        if (neg)
#pragma unroll
          for (int j = 0; j < 128; ++j) s[j / 32][j % 32] ^= 0x80000000u;
        if (it >= mask0) {
          const int k = lim - it * kKeys;   // keys from here on that the row sees
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j >= k) s[j / 32][j % 32] = 0xFF800000u;
        }
        if (it == 0) {   // m: the maximum of the first half (where that is -inf, the code below goes on looking)
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 64; ++j) top = fmaxf(top, __uint_as_float(s[j / 32][j % 32]));
          m = fmaxf(m, top * f);
        }
        // Half of the keys at a time.  No maximum is taken in the common path: a half whose sum passes kMost (rare; whatever P
        // could not hold is among them) raises m to its maximum, scales l, O and the first half's weights, and is computed
        // again.  (The first half's weights are then rounded a second time: half a step more, where m jumps within 128 keys.)
        // PV(it - 1), which reads P and adds to O, is waited for when the weights are ready to go over P.
        const int before = (done + it - 1) & 1;
        const uint64_t f2 = pack2(f, f);
        uint32_t w[4][16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sum;
#pragma unroll 1
          for (bool again = false;; again = true) {
            const float mb = m == -INFINITY ? bias : bias - m;
            const uint64_t mb2 = pack2(mb, mb);
            uint64_t sums = 0ull;
#pragma unroll
            for (int j = 64 * h; j < 64 * h + 64; j += 2) {
              const float2 y = unpack2(fma2(pack2u(s[j / 32][j % 32], s[j / 32][j % 32 + 1]), f2, mb2));
              const float e0 = ex2f(y.x), e1 = ex2f(y.y);
              sums = add2(sums, pack2(e0, e1));
              w[j / 32][j % 32 / 2] = pack_p<BF>(e0, e1);
            }
            const float2 y = unpack2(sums);
            sum = y.x + y.y;
            const bool raise = sum > kMost || m == -INFINITY;
            if (__builtin_expect(again || !__any_sync(0xffffffffu, raise), 1)) break;
            float top = -INFINITY;
#pragma unroll
            for (int j = 64 * h; j < 64 * h + 64; ++j) top = fmaxf(top, __uint_as_float(s[j / 32][j % 32]));
            const float to_m = raise ? fmaxf(m, top * f) : m;
            const float alpha = to_m == m ? 1.f : ex2f(m - to_m);
            m = to_m;
            l *= alpha;
            if (h)
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float2 v = unpack_p<BF>(w[j / 16][j % 16]);
                w[j / 16][j % 16] = pack_p<BF>(v.x * alpha, v.y * alpha);
              }
            if (it > 0) {   // (before that O holds nothing)
              ok = __all_sync(0xffffffffu, wait(&o_done[x], before));
              if (!ok) break;
              tc::fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tc::ld16(to + c, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                tc::st16(to + c, o);
              }
              tc::wait_st();   // the second half may scale O again: a load is behind a store only if that is waited for
            }
          }
          l += sum;
        }
        if (ok && it > 0) ok = __all_sync(0xffffffffu, wait(&o_done[x], before));
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::st16(tp + 16 * c, w[c]);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      if (nx > 0) {
        // ---- O / l, and the tile's log-sum-exp
        done += nx;
        ok = __all_sync(0xffffffffu, wait(&o_done[x], (done - 1) & 1));
        if (!ok) break;
        tc::fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool live = token < pair.n, patch = bad_v[pk & 1] != 0;
        const long long r = (long long)pair.first + token;
        const int head = pair.unit * p.P + (row & (p.P - 1));
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tc::ld32(to + c, o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = l == 0.f ? 0.f : o[j] * inv;
          if (__builtin_expect(patch && live, 0)) {   // infinities and NaN that the cleaning took out of the tiles
            for (int j = pair.t0 + 1; j < lim; ++j) {
              const uint16_t* v = static_cast<const uint16_t*>(a.v) + ((long long)pair.first + j) * a.v_stride + (long long)(head / a.G) * D + c;
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
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_p<BF>(o[2 * i], o[2 * i + 1]);
            if (p.wide) {   // 32 bytes a store: whole sectors
#pragma unroll
              for (int i = 0; i < 16; i += 8)
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 2 * i), "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]),
                             "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                             : "memory");
            } else {
#pragma unroll
              for (int i = 0; i < 16; i += 4) *reinterpret_cast<uint4*>(dst + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            }
          }
          __syncwarp();
        }
        if (a.lse && live) a.lse[r * a.Hq + head] = l == 0.f ? -INFINITY : (m - bias + __log2f(l)) * kLn2f;
        tc::fence_before();
      }
      give_pair_back(pk);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    int pos = 0, cleaned = 0;   // places of the ring and cleaned V tiles of earlier pairs
    if (warp == 8) {
      // ---------------------------------------------------------------- pairs, and loads through the ring
      int q_used[2] = {0, 0};
      Finder finder(p, lane);
      for (int pk = 0; ok; ++pk) {
        pair = next_pair(p, finder, pk);
        if (lane == 0) {
          if (pk >= 2) ok = wait(&info_empty[pk & 1], ((pk >> 1) - 1) & 1);
          if (ok) {
            volatile int* i = info + 4 * (pk & 1);
            i[0] = pair.first;
            i[1] = pair.n;
            i[2] = pair.t0;
            i[3] = pair.unit;
            bad_v[pk & 1] = 0;
            mbar_arrive(&info_full[pk & 1]);
          }
          const int n0 = n_keys(0), n1 = n_keys(1), most = max(n0, n1), clean0 = masked_from(pair.t0), head0 = pair.unit * p.P;
          uint64_t* v_bar = nullptr;
          for (int i = 0; ok && pair.n > 0 && i < 2 * most; ++i) {
            if (i == 0 || i == 1) {   // the tiles' queries: tile 0's before the first keys, tile 1's behind them
              if (i ? n1 : n0) {
                if (q_used[i]) ok = wait(&q_empty[i], (q_used[i] - 1) & 1);
                if (!ok) break;
                ++q_used[i];
                mbar_arrive_expect_tx(&q_full[i], Pl::kTile);
                for (int c = 0; c < KC; ++c)
                  tc::tma3d(smem + i * Pl::kTile + c * Pl::kBlock, &p.q, 64 * c, head0, pair.first + pair.t0 + i * p.tokens, &q_full[i]);
              }
            }
            const int st = pos % NS;
            if (pos >= NS) ok = wait(&empty[st], (pos / NS - 1) & 1);
            if (!ok) break;
            // the i-th tile: K(0), K(1), V(0), K(2), V(1), ..., V(most - 1)
            const bool is_v = i == 2 * most - 1 || (i > 0 && i % 2 == 0);
            const int j = is_v ? (i == 2 * most - 1 ? most - 1 : i / 2 - 1) : (i + 1) / 2;
            // K(0) and K(1) have their places' barriers; V(j) and K(j + 2) land on V's together.  A V tile that is cleaned lands
            // on a barrier of its own (the ring holds at most eight), so that the cleaning warps see each of its phases
            const bool raw = is_v && j >= clean0;
            if (is_v) {
              v_bar = &full[st];
              const int with = (raw ? 0 : Pl::kTile) + (j + 2 < most ? Pl::kTile : 0);
              if (with) mbar_arrive_expect_tx(v_bar, with);
              else mbar_arrive(v_bar);
            } else {
              if (j < 2) mbar_arrive_expect_tx(&full[st], Pl::kTile);
              else mbar_arrive(&full[st]);
            }
            uint64_t* bar = raw ? &v_raw[cleaned & 7] : !is_v && j < 2 ? &full[st] : v_bar;
            if (raw) {
              ++cleaned;
              mbar_arrive_expect_tx(bar, Pl::kTile);
            }
            for (int c = 0; c < KC; ++c)
              tc::tma3d(ring + st * Pl::kTile + c * Pl::kBlock, is_v ? &p.v : &p.k, 64 * c, head0 / a.G, pair.first + j * kKeys, bar);
            ++pos;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (pair.n == 0) break;
      }
      if (lane == 0) {   // what is in flight has to land before the CTA ends, whatever became of the other roles
        for (int i = 0; i < 2; ++i)
          if (q_used[i]) mbar_wait_bounded(&q_full[i], (q_used[i] - 1) & 1, kWaitLimitNs);
        for (int j = max(0, pos - NS); j < pos; ++j) mbar_wait_bounded(&full[j % NS], (j / NS) & 1, kWaitLimitNs);
        for (int j = max(0, cleaned - 8); j < cleaned; ++j) mbar_wait_bounded(&v_raw[j & 7], (j >> 3) & 1, kWaitLimitNs);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---------------------------------------------------------------- MMA
      constexpr uint32_t id_s = BF ? tc::idesc_bf16(kM, kKeys) : tc::idesc_f16(kM, kKeys);
      constexpr uint32_t id_o = (BF ? tc::idesc_bf16(kM, D) : tc::idesc_f16(kM, D)) | tc::kBMajorN;
      const uint64_t qd = tc::desc_sw128(smem_u32(smem)), kd = tc::desc_sw128(smem_u32(ring)),
                     vd = tc::desc_sw128_mn(smem_u32(ring), Pl::kBlock);
      // The whole warp goes along, and one lane of it (elect.sync) issues: the operands are then known to be the same in
      // all lanes.  Issued by one thread in a branch of its own, each MMA took 130 cycles instead of the 64 of its math.
      int done[2] = {0, 0}, q_used[2] = {0, 0}, issued = 0;   // key tiles of earlier pairs, pairs with a tile x; S so far
      Place base{0, 0};                           // of the pair's K(0)
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      auto all_wait = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
      for (int pk = 0; get_pair(pk); ++pk) {
        give_pair_back(pk);
        pair.n = __shfl_sync(0xffffffffu, pair.n, 0);
        pair.t0 = __shfl_sync(0xffffffffu, pair.t0, 0);
        const int n0 = n_keys(0), n1 = n_keys(1), most = max(n0, n1), clean0 = masked_from(pair.t0);
        auto await = [&](bool at_all, uint64_t* bar, int parity) { ok = ok && (!at_all || all_wait(bar, parity)); };
        // S(it) of tile x, K(it) at place ks, once the S before it is read
        auto scores = [&](int x, int it, const Place& ks) {
          await(issued > 0, s_read, (issued - 1) & 1);
          ++issued;
          tc::fence_after();
          const uint64_t kt = kd + (__shfl_sync(0xffffffffu, ks.i, 0) * Pl::kTile >> 4), qt = qd + (x * Pl::kTile >> 4);
          const bool last = it + 1 == (x ? n1 : n0), frees = x == (it < n1 ? 1 : 0);   // of the queries' uses; of K(it)'s
          if (ok && tc::elect()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t at = ((k >> 2) * Pl::kBlock + (k & 3) * 32) >> 4;
              tc::mma(tm, qt + at, kt + at, id_s, k != 0);
            }
            tc::commit(&s_full[x]);
            if (last) tc::commit(&q_empty[x]);
            if (frees) tc::commit(&empty[ks.i]);
          }
          __syncwarp();
        };
        // PV(it) of tile x, V(it) at place vs; known: its P is (an S read after it was written has been waited for)
        auto values = [&](int x, int it, const Place& vs, bool known) {
          await(!known, &p_full[x], (done[x] + it) & 1);
          tc::fence_after();
          const uint64_t vt = vd + (__shfl_sync(0xffffffffu, vs.i, 0) * Pl::kTile >> 4);
          const bool frees = x == (it < n1 ? 1 : 0);   // the last use of V(it)
          if (ok && tc::elect()) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              tc::mma_ta(tm + Pl::kO + D * x, tm + Pl::kP + 64 * x + 8 * k, vt + (k * 2048 >> 4), id_o, (it | k) != 0);
            tc::commit(&o_done[x]);
            if (frees) tc::commit(&empty[vs.i]);
          }
          __syncwarp();
        };
        const Place first = base;
        Place k1 = base.next();                         // K(it + 1)'s place
        Place vs = most > 1 ? k1.next() : k1;           // V(it)'s
        await(true, &full[first.i], first.phase);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (x ? n1 : n0) {
            await(true, &q_full[x], q_used[x] & 1);
            ++q_used[x];
            scores(x, 0, first);
          }
        await(most > 1, &full[k1.i], k1.phase);
        if (n1 > 0 && n0 > 1) scores(0, 1, k1);
        // Two tiles: S(it + 1) of tile 1, PV(it) of tile 0, S(it + 2) of tile 0, PV(it) of tile 1.  A softmax reads its next S when
        // it has written its P; the other tile's S then goes first, and the PV has the time that the softmax takes until it
        // has the next weights.  One tile: S(it + 1), PV(it).
        for (int it = 0; it < most && ok; ++it) {
          const Place k2 = vs.next();                   // K(it + 2)'s place
          if (n1 > 0) {
            if (it + 1 < n1) scores(1, it + 1, k1);
          } else if (it + 1 < n0) {
            scores(0, it + 1, k1);
          }
          await(true, &full[vs.i], vs.phase);           // V(it), and with it K(it + 2)
          if (it >= clean0) {
            const int w = cleaned + it - clean0;
            await(true, &v_raw[w & 7], (w >> 3) & 1);
            await(true, &v_clean[w & 7], (w >> 3) & 1);
          }
          if (it < n0) values(0, it, vs, n1 > 0 && it + 1 < n0);
          if (n1 > 0) {
            if (it + 2 < n0) scores(0, it + 2, k2);
            values(1, it, vs, it + 2 < n0);
          }
          vs = it + 2 < most ? k2.next() : k2;
          k1 = k2;
        }
        base = vs;
        if (!ok) break;
        pos += 2 * most;
        cleaned += max(0, most - clean0);
        done[0] += n0;
        done[1] += n1;
      }
      if (ok) {   // tensor memory may be freed, and shared memory given up, once what was issued is done
        for (int j = max(0, pos - NS); j < pos; ++j) ok = ok && all_wait(&empty[j % NS], (j / NS) & 1);
        for (int x = 0; x < 2; ++x)
          if (q_used[x]) ok = ok && all_wait(&q_empty[x], (q_used[x] - 1) & 1);
      }
      if (!ok) {
        if (tc::elect()) tc::commit(drained);
        __syncwarp();
        mbar_wait_bounded(drained, 0, kWaitLimitNs);
      }
    } else {
      // ---------------------------------------------------------------- V tiles that not every token sees whole
      for (int pk = 0; get_pair(pk); ++pk) {
        const int most = max(n_keys(0), n_keys(1)), clean0 = masked_from(pair.t0);
        int any_bad = 0;
        for (int it = clean0; it < most; ++it, ++cleaned) {
          ok = __all_sync(0xffffffffu, wait(&v_raw[cleaned & 7], (cleaned >> 3) & 1));
          if (!ok) break;
          uint8_t* vt = ring + (pos + (it == most - 1 ? 2 * most - 1 : 2 * it + 2)) % NS * Pl::kTile;
          const int whole = max(0, (a.causal ? min(pair.t0 + 1, pair.n) : pair.n) - it * kKeys);   // rows before it: every token sees them
          for (int c = 0; c < KC; ++c)
#pragma unroll 4
            for (int e = 8 * whole + (tid - 320); e < 8 * kKeys; e += 64) {   // (the swizzle keeps a row's 128 bytes together)
              uint4* at = reinterpret_cast<uint4*>(vt + c * Pl::kBlock) + e;
              if (it * kKeys + (e >> 3) >= pair.n) {
                *at = make_uint4(0u, 0u, 0u, 0u);
              } else {
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
                    const uint32_t z = ((yw[k] & ones) + unit) & 0x80008000u;   // 0x8000 in the halves to clear
                    yw[k] &= ~((z >> 15) * 0xFFFFu);
                  }
                  *at = y;
                  any_bad = 1;
                }
              }
            }
          if (any_bad) bad_v[pk & 1] = 1;
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_clean[cleaned & 7]);
        }
        if (!ok) break;
        pos += 2 * most;
        give_pair_back(pk);
      }
    }
  }
  if (!ok && lane == 0) {
    *stop = 1;
    atomicOr(a.status, KVQ_STATUS_TIMEOUT);
  }
  __syncthreads();
  if (warp == 9) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (*stop) {   // nothing that a wait gave up on is taken for a result
    Finder finder(p, lane);
    for (int pk = 0;; ++pk) {
      pair = next_pair(p, finder, pk);   // (every warp by itself)
      if (pair.n == 0) break;
      for (int i = warp; i < p.tiles * kM; i += kThreads / 32) {
        const int token = pair.t0 + (i >> p.log_p), head = pair.unit * p.P + (i & (p.P - 1));
        if (token >= pair.n) continue;
        const long long r = (long long)pair.first + token, at = r * a.out_stride + (long long)head * D;
        for (int c = lane; c < D; c += 32)
          if (a.out32) static_cast<float*>(a.out)[at + c] = NAN;
          else static_cast<uint16_t*>(a.out)[at + c] = 0x7FFF;   // NaN in bf16 and fp16
        if (a.lse && lane == 0) a.lse[r * a.Hq + head] = NAN;
      }
    }
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

// The SMs of the current device; the kernel's shared memory is allowed once for each.
template <int D, bool BF>
static cudaError_t sms_of_device(int& sms) {
  static std::mutex mutex;
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mutex);
  if (dev < 64 && known[dev]) {
    sms = known[dev];
    return cudaSuccess;
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(prompt_kernel<D, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<D>::kSmem);
  if (e == cudaSuccess && dev < 64) known[dev] = sms;
  return e;
}

template <int D, bool BF>
static cudaError_t launch(const PromptArgs& a, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = sms_of_device<D, BF>(sms);
  if (e != cudaSuccess) return e;
  Launch p;
  p.a = a;
  p.P = a.G & -a.G;
  for (p.log_p = 0; 1 << p.log_p < p.P; ++p.log_p) {}
  p.tokens = kM / p.P;
  p.units = a.Hq / p.P;
  p.wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_stride % 16 == 0;
  // CTAs of a head: every sequence may have a last tile that is not full, and no more rows than there are
  auto ctas = [&](int tiles) {
    const long long span = (long long)tiles * p.tokens;
    return std::min((long long)a.B * ((a.t_new + span - 1) / span), a.rows / span + a.B);
  };
  // One tile a CTA where pairs would leave SMs idle.  8 kv heads x 4, D 128, pairs and single tiles: 1024 tokens (128 pairs)
  // 19.1 and 18.2 us, 1536 (192 pairs) 26.3 and 31.0, 2048 32.0 and 42.9; one kv head of 64 channels, 2048 tokens 21.3 and 18.2.
  p.tiles = ctas(2) * p.units >= sms ? 2 : 1;
  const long long pairs = ctas(p.tiles) * p.units;
  if (pairs > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;   // (more rows or heads than memory holds)
  p.pairs = (int)pairs;
  p.log_span = 7 - p.log_p + (p.tiles == 2);
  const int tokens = std::max(1, (int)std::min((long long)a.t_new, (long long)a.rows / a.B));   // of a sequence, about
  const int at_once = std::max(1, (24 << 20) / (4 * D * a.Hkv));                                // whose K and V are 24 MB
  p.seqs = std::min({a.B, 256, std::max(1, at_once / tokens)});
  const int heads = a.Hkv / std::min(a.Hkv, (tokens - 1) / at_once + 1);                        // parts alike, but for the last
  p.hu = heads * (p.units / a.Hkv);
  p.parts = (a.Hkv + heads - 1) / heads;
  const unsigned grid = (unsigned)std::min(p.pairs, sms);
  if (!encode(&p.q, a.q, BF, D, a.Hq, a.rows, a.q_stride, p.P, p.tokens) || !encode(&p.k, a.k, BF, D, a.Hkv, a.rows, a.k_stride, 1, kKeys) ||
      !encode(&p.v, a.v, BF, D, a.Hkv, a.rows, a.v_stride, 1, kKeys))
    return cudaErrorInvalidValue;
  prompt_kernel<D, BF><<<grid, kThreads, Plan<D>::kSmem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace prompt

cudaError_t prompt_launch(const PromptArgs& a, int D, int dtype, cudaStream_t st) {
  if (dtype == KVQ_BF16) return D == 64 ? prompt::launch<64, true>(a, st) : prompt::launch<128, true>(a, st);
  return D == 64 ? prompt::launch<64, false>(a, st) : prompt::launch<128, false>(a, st);
}

}  // namespace kvq
