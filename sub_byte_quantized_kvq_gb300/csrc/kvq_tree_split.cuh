// kvq_tree_split.cuh -- tree attention over the cached pages on the tensor cores.
//
// One CTA per (split, kv head x tile of 128 rows, sequence).  A tile of 128
// rows (node, head of the group) x kTok tokens costs two MMAs, S = Q K^T and
// O += P V, and each page's codes are expanded once for all of the rows:
//
//   16 dequant warps  each takes one page's K or V of every tile: its own ring of
//                   asynchronous copies (16 bytes a lane; bulk copies are issued
//                   at one per 33 ns and SM, 90 ns and warp, whatever their size,
//                   and held the warp up for as long), then
//                   codes -> fp16 tiles in shared memory, K as [token][channel],
//                   V transposed as [channel][token], both K-major with 128-byte
//                   swizzle; the block layout holds mma fragments, which
//                   stmatrix turns into rows; outliers are stored over their slots
//   MMA warp        tcgen05.mma with Q and P from tensor memory, the tiles from
//                   shared memory; S(i + 1) is issued before PV(i), once PV(i - 1)
//                   is done with P(i - 1) in its columns, so the tensor cores work
//                   while the softmax warps do
//   4 softmax warps one row a thread (tensor-memory lane): p = 2^(s - m) with a
//                   reference m that is raised only when the sums ask for it,
//                   page sums for page_lse; P goes over S's own columns
//
// Precision: Q is scaled by a power of two into fp16 range and exact; K is
// exact in fp16 (INT4: an fp16 pair, two MMAs); S, m, l and O are fp32.  P is
// rounded to fp16 (at most 2^-11 relative; biased by 2^kPBias so that small
// p keep their bits), V to fp16 where the format's value has more (INT4, FP8
// tier): for a bf16 result both are below its own rounding.  An FP8 page's V may
// have any magnitude: v_shift moves a power of two of its scale to P.
//
// What bounds it: no unit alone.  A tile of 128 tokens is about 1024 cycles of MMA
// at 128 rows, 800-1200 of this SM's share of the measured HBM rate, and 6,600
// (FP4) to 7,200 (tiered) warp instructions, which take four schedulers 1,650 to
// 1,800 cycles; measured, it takes about 2,950 (FP4 at 128 rows) and 2,700 (tiered
// at 8 rows) with a CTA's start and end spread over 64 tiles, and 56% and 66% of the
// issue slots are used (16 sequences x 32k tokens: 360 and 327 us).  So the roles
// wait for one another over a tile; which for which has not been measured.
// Addresses that run along with a warp's tiles, instead of computed per tile, gave
// 1-2%.  The kernels of more than 32 rows spill up to 32 bytes (120 loaded) at the 80
// registers a thread that the launch has, those of fewer rows none.
#pragma once
#include <type_traits>

#include "kvq_decode.cuh"
#include "kvq_tc.cuh"
#include "kvq_tree.cuh"

namespace kvq {
namespace tree {

constexpr int kM = kTreeRows;
constexpr int kDequantWarps = 16;
constexpr int kThreads = 32 * (4 + kDequantWarps + 4);
// Registers a thread: the launch has 80 each; the softmax warps take what the others give up.
constexpr int kRegsLaunch = 80, kRegsSoftmax = 144, kRegsDequant = 72, kRegsRest = 48;
static_assert(4 * kRegsSoftmax + kDequantWarps * kRegsDequant + 4 * kRegsRest <= (kThreads / 32) * kRegsLaunch,
              "setmaxnreg shares exceed what the launch has");
constexpr int kMeta = 4;                // tiles whose page records are kept: K(i) is written once S(i - 2) is done, whose
                                        // MMAs were issued after the softmax of tile i - 4
constexpr float kPBias = 6.f;           // p = 2^(s f - m + kPBias): small p keep their bits; p <= 2^15 by the check on the sums

template <int FMT, int D>
struct Plan {
  using F = Fmt<FMT>;
  static constexpr bool kPair = F::kMain == kBlkInt4;        // K as an fp16 pair
  static constexpr int kTok = kPair ? 64 : 128;              // (two K tiles of 128 tokens would not fit)
  static constexpr int kPages = kTok / kPage;
  static constexpr int kTile = kTok * D * 2;                 // bytes of an fp16 tile
  static constexpr int kBuf = (kPair ? 3 : 2) * kTile;       // one buffer: K [, K low], V
  // a page's slot: its (virtual) block from offset 0 (the group format copies the group's codebook into each)
  static constexpr int kSlot = F::kGroup ? 12 * D + kOutPrefetch : half_slot_bytes<FMT, D>();
  static constexpr bool kShift = FMT == KVQ_FMT_TIERED;      // pages have a V shift
  static constexpr int misc(int depth) {
    return 8 * 14 + 2 * kMeta * kPages * 4 + 4 * kDequantWarps * depth + 8 +
           (kShift ? kMeta * kPages * 8 + 4 * kDequantWarps * depth : 0);
  }
  static constexpr int smem(int depth) {   // 1024: alignment slack
    return 1024 + 2 * kBuf + kDequantWarps * depth * kSlot + misc(depth);
  }
  static constexpr int fit() {
    int d = 6;
    while (d > 1 && smem(d) > 227 * 1024) --d;
    return d;
  }
  static constexpr int kDepth = fit();                       // slots of a warp's copy ring
  static constexpr int kSmem = smem(kDepth);
  static_assert(kDepth >= 2 && kSlot % 16 == 0 && kTile % 1024 == 0, "tree attention plan");
};

// A bounded mbarrier wait on the SM's own clock: gives up after 2e8 cycles, 100 ms.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, long long limit = 200000000ll) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_sleep(bar, parity, 20000u))
    if (clock64() - t0 > limit) return false;
  return true;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((unsigned short)v) : "memory");
}

// The four bytes of a word, each two e2m1 nibbles, as f16x2.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&x)[4]) {
  asm("{ .reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
      : "r"(w));
}
// The four bytes of a word, e4m3, as two f16x2.
__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t& x, uint32_t& y) {
  asm("{ .reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(x), "=r"(y)
      : "r"(w));
}

// The power of two b of an FP8 page's V scale that goes to P instead of the fp16
// tile: P holds p 2^b, the tile v 2^-b.  With a scale of 2^e to 2^(e+1) and codes of
// 2^-9 to 448, e - b in -5..6 keeps every element in fp16's normal range (rounded
// once, by 2^-11 at most), so b follows e outside -9..2; inside (a page's largest
// |v| between 0.9 and 3584) it stays at -4, and CB2 pages have 0.  The reference m
// of a row is of p 2^b, and the fp32 sums are of p: b is held to -48..48, which leaves
// the heaviest p above 2^-90 whatever the other pages have.  So elements of a page
// whose largest |v| is below 5e-14 are off by up to 2^-73, and one above 1.6e19 is
// infinite.  A scale of 0 has b = -4.
__device__ __forceinline__ int v_shift(float scale) {
  const int e = scale == 0.f ? 0 : (int)((__float_as_uint(scale) >> 23) & 255u) - 127;
  return max(-48, min(48, min(max(-4, e - 6), e + 5)));
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }   // |e| < 127

// Where a page's values go in a swizzled tile, as offsets from its start.  A row
// is 64 fp16 (128 bytes); 16-byte chunk k of row r lies at chunk k ^ (r % 8).
template <int D, int TOK>
struct KTile {   // rows = tokens, D / 64 row groups
  static constexpr int kStep4 = TOK * 128;   // four steps: the next row group
  int page;
  __device__ __forceinline__ uint32_t at(int t, int c) const {
    const int row = kPage * page + t;
    return (c >> 6) * (TOK * 128) + row * 128 + (((c >> 3 & 7) ^ (t & 7)) << 4) + (c & 7) * 2;
  }
  // lane's row of a group of four steps, and of its step s (matrices: tokens 0-7 / 8-15 x channels 0-7 / 8-15; the
  // swizzled chunk (2 s + half) ^ (row % 8) of a 128-byte row)
  __device__ __forceinline__ uint32_t lane_row(int lane) const {
    return (kPage * page + (lane & 15)) * 128 + (((lane & 7) ^ (lane >> 4)) << 4);
  }
  __device__ __forceinline__ uint32_t step(uint32_t row, int s) const { return row ^ (s << 5); }
};
template <int D, int TOK>
struct VTile {   // rows = channels, TOK / 64 row groups
  static constexpr int kStep4 = 4 * 2048;
  int page;
  __device__ __forceinline__ uint32_t at(int t, int c) const {
    return (page >> 2) * (D * 128) + c * 128 + ((((page & 3) * 2 + (t >> 3)) ^ (c & 7)) << 4) + (t & 7) * 2;
  }
  // (matrices: channels 0-7 / 8-15 x tokens 0-7 / 8-15)
  __device__ __forceinline__ uint32_t lane_row(int lane) const {
    return (page >> 2) * (D * 128) + (lane & 15) * 128 + ((((page & 3) * 2 + (lane >> 4)) ^ (lane & 7)) << 4);
  }
  __device__ __forceinline__ uint32_t step(uint32_t row, int s) const { return row + s * 2048; }
};

// The outliers of a side-list, stored over their slots' values: two records at
// a time, a token a lane.  The prefetched records are loaded before the codes
// are expanded (`load`) and stored after them (`store`); later ones, rare, come
// from global memory.
template <int D>
struct SidePatch {
  uint32_t head[kChunk / 2], value[kChunk / 2];
  int n;
  __device__ __forceinline__ void load(uint32_t side_s, int lane) {
    n = min((int)lds8(side_s), D);
#pragma unroll
    for (int k = 0; k < kChunk / 2; ++k) {
      const uint32_t rec = side_s + 4 + 20 * (2 * k + (lane >> 4));
      head[k] = lds32(rec);
      value[k] = lds8(rec + 4 + (lane & 15));
    }
  }
  template <class Tile, class Side>
  __device__ __forceinline__ void store(const Tile& tile, uint32_t buf, int lane, Side&& side_g) {
    const int t = lane & 15, half = lane >> 4;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kChunk / 2; ++k)
      if (2 * k + half < n && ((head[k] >> (16 + t)) & 1u))
        sts16(buf + tile.at(t, head[k] & (D - 1)), e4m3x2_to_f16x2(value[k]));
    if (__builtin_expect(n > kChunk, 0)) {
      const uint8_t* side = side_g();
      for (int i = kChunk + half; i < n; i += 2) {
        const uint8_t* rec = side + 4 + 20 * i;
        if ((*reinterpret_cast<const uint16_t*>(rec + 2) >> t) & 1u) sts16(buf + tile.at(t, rec[0] & (D - 1)), e4m3x2_to_f16x2(rec[4 + t]));
      }
    }
  }
};

// Tokens from `ntok` on as zeros in a V tile (their probability is 0, and stale bytes may stand for anything).
template <int D, class Tile>
__device__ __forceinline__ void zero_tokens(const Tile& tile, uint32_t buf, int ntok, int lane) {
  for (int c = lane; c < D; c += 32)
#pragma unroll
    for (int t = 0; t < kPage; ++t)
      if (t >= ntok) sts16(buf + tile.at(t, c), 0u);
}

// One K block (role 0) or V block (role 1) -> its place in the fp16 tile, four
// steps (64 channels) at a time: their loads overlap, and the loop is kept
// rolled -- the warps of a scheduler run three different loops (softmax, K, V),
// and unrolled ones spent half the time waiting for instructions.
//   blk    shared address of the page's slot
//   gblk   a function that gives the block in global memory (side-list records past the prefetch)
//   tier   the block is an FP8 block
//   buf    the tile (low: the second K tile of INT4)
// K of an FP8 block is left unscaled (its page's scale is applied to the scores), V is scaled by all but v_shift's power.
template <int FMT, int D, int ROLE, class Tile, class GBlk>
__device__ __forceinline__ void dequant_block(uint32_t blk, GBlk&& gblk, bool tier, const Tile& tile, uint32_t buf,
                                              uint32_t low, int lane) {
  using F = Fmt<FMT>;
  constexpr int NS = D / 16, BLK = F::kMain;
  const int g = lane >> 2, q4 = lane & 3;
  uint32_t row = buf + tile.lane_row(lane);
  if (FMT == KVQ_FMT_TIERED && tier) {
    float sc = 1.f;
    if (ROLE == 1) {
      sc = ldsf(blk + fp8_sc_off(D));
      sc *= exp2_int(-v_shift(sc));
    }
#pragma unroll 1
    for (int s0 = 0; s0 < NS; s0 += 4, row += Tile::kStep4) {
      const uint4 w0 = lds128(blk + 8 * NS * lane + 8 * s0), w1 = lds128(blk + 8 * NS * lane + 8 * s0 + 16);
      const uint2 w[4] = {{w0.x, w0.y}, {w0.z, w0.w}, {w1.x, w1.y}, {w1.z, w1.w}};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t x[4];
        e4m3x4(w[k].x, x[0], x[1]);
        e4m3x4(w[k].y, x[2], x[3]);
        if (ROLE == 1)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float2 f = __half22float2(u32_as_h2(x[r]));
            x[r] = h2_as_u32(__floats2half2_rn(f.x * sc, f.y * sc));
          }
        stmatrix4(tile.step(row, k), x);
      }
    }
    return;
  }
  if constexpr (BLK == kBlkInt4) {
    constexpr int NG = D / 32, CAP = int4_cap(D), NZ = ROLE == 0 ? 2 : 4;   // NZ: tokens whose scale and minimum the lane needs
    uint32_t lrow = low + tile.lane_row(lane);
#pragma unroll 1
    for (int s0 = 0; s0 < NS; s0 += 4, row += Tile::kStep4, lrow += Tile::kStep4) {
      const uint4 w4 = lds128(blk + 4 * NS * lane + 4 * s0);   // one u32 of nibbles per step
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      uint32_t z[2][NZ];
#pragma unroll
      for (int i = 0; i < NZ; ++i) {
        const int t = ROLE == 0 ? g + 8 * i : 2 * q4 + (i & 1) + 8 * (i >> 1);
        const uint2 zz = lds64(blk + int4_sz_off(D) + 4 * (t * NG + (s0 >> 1)));
        z[0][i] = zz.x;
        z[1][i] = zz.y;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t hi[4], lo[4];
        float S[NZ], M[NZ];
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
          S[i] = fp16_bits_to_float(z[k >> 1][i]);
          M[i] = fp16_bits_to_float(z[k >> 1][i] >> 16);
        }
        if constexpr (ROLE == 0) {
          int4_k_frag(w[k], S[0], M[0], S[1], M[1], hi, lo);
          stmatrix4(tile.step(lrow, k), lo);
        } else {
          int4_v_frag(w[k], S, M, hi, lo);
        }
        stmatrix4(tile.step(row, k), hi);
      }
    }
    __syncwarp();
    for (int e = lane; e < kPage * CAP; e += 32) {
      const int t = e / CAP;
      if (e - t * CAP < (int)lds8(blk + int4_cnt_off(D) + t)) {
        const int c = lds8(blk + int4_ch_off(D) + e) & (D - 1);
        sts16(buf + tile.at(t, c), lds16(blk + int4_val_off(D) + 2 * e));
        if (ROLE == 0) sts16(low + tile.at(t, c), 0u);
      }
    }
  } else if constexpr (BLK == kBlkE2m1) {
#pragma unroll 1
    for (int s0 = 0; s0 < NS; s0 += 4, row += Tile::kStep4) {
      const uint4 w4 = lds128(blk + 4 * NS * lane + 4 * s0);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      // scales as f16x2.  K: of tokens g (registers 0, 2) and g + 8; V: of tokens 2q, 2q + 1 (registers 0, 1) and + 8
      uint32_t sc[4][ROLE == 0 ? 1 : 2];
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const uint32_t at = blk + e2m1_sc_off(D) + 16 * (s0 + k);
        if constexpr (ROLE == 0) {
          const uint32_t lo = prmt(lds8(at + g), lds8(at + g + 8), 0x7740u), hi = prmt(lds8(at + 16 + g), lds8(at + 24 + g), 0x7740u);
          e4m3x4(prmt(lo, hi, 0x5410u), sc[k][0], sc[k + 1][0]);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            e4m3x4(prmt(lds16(at + 16 * i + 2 * q4), lds16(at + 16 * i + 2 * q4 + 8), 0x5410u), sc[k + i][0], sc[k + i][1]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t x[4];
        e2m1x8(w[k], x);
        if constexpr (ROLE == 0) {
          const __half2 sh = u32_as_h2(sc[k][0]), h0 = __low2half2(sh), h1 = __high2half2(sh);
          x[0] = h2_as_u32(__hmul2(u32_as_h2(x[0]), h0));
          x[1] = h2_as_u32(__hmul2(u32_as_h2(x[1]), h1));
          x[2] = h2_as_u32(__hmul2(u32_as_h2(x[2]), h0));
          x[3] = h2_as_u32(__hmul2(u32_as_h2(x[3]), h1));
        } else {
          x[0] = hmul2u(x[0], sc[k][0]);
          x[1] = hmul2u(x[1], sc[k][0]);
          x[2] = hmul2u(x[2], sc[k][1]);
          x[3] = hmul2u(x[3], sc[k][1]);
        }
        stmatrix4(tile.step(row, k), x);
      }
    }
  } else if constexpr (BLK == kBlkA3) {
    SidePatch<D> patch;
    patch.load(blk + a3_out_off(D), lane);
#pragma unroll 1
    for (int s0 = 0; s0 < NS; s0 += 4, row += Tile::kStep4) {
      const uint2 xw = lds64(blk + 2 * NS * lane + 2 * s0);                       // low code bits, two steps a word
      const uint32_t yw = lds32(blk + a3_hi_off(D) + NS * lane + s0);             // high code bit, four steps
      uint2 sc[4], zp[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (ROLE == 0) {   // 4 adjacent S and m: channels x, x + 1 (registers 0, 1), x + 8, x + 9
          const int at = 2 * (16 * (s0 + k) + 4 * q4);
          sc[k] = lds64(blk + a3_s_off(D) + at);
          zp[k] = lds64(blk + a3_m_off(D) + at);
        } else {                     // channels c (registers 0, 2) and c + 8, each for both tokens of a register
          const int at = 2 * (16 * (s0 + k) + 2 * g);
          const uint32_t s2 = lds32(blk + a3_s_off(D) + at), m2 = lds32(blk + a3_m_off(D) + at);
          sc[k] = {prmt(s2, s2, 0x1010u), prmt(s2, s2, 0x3232u)};
          zp[k] = {prmt(m2, m2, 0x1010u), prmt(m2, m2, 0x3232u)};
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = k < 2 ? xw.x : xw.y;
        uint32_t x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool second = ROLE == 0 ? r >= 2 : (r & 1) != 0;
          x[r] = a3_value(w, yw, k, r, second ? sc[k].y : sc[k].x, second ? zp[k].y : zp[k].x);
        }
        stmatrix4(tile.step(row, k), x);
      }
    }
    patch.store(tile, buf, lane, [&]() { return gblk() + a3_out_off(D); });
  } else {   // 2-bit codebooks
    SidePatch<D> patch;
    if constexpr (BLK != kBlkCb2s) patch.load(blk + cb2_out_off(D), lane);
    uint32_t book = blk + (F::kGroup ? 0 : cb2_cb_off(D)) + 16 * (ROLE == 0 ? q4 : g);
#pragma unroll 1
    for (int s0 = 0; s0 < NS; s0 += 4, row += Tile::kStep4, book += 512) {
      const uint2 w2 = lds64(blk + (F::kGroup ? cb2g_code_off(D) : 0) + 2 * NS * lane + 2 * s0);
      KCols kc[ROLE == 0 ? 4 : 1];
      uint4 vc[ROLE == 0 ? 1 : 4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if constexpr (ROLE == 0) kc[k] = cb2_k_cols(book, k);
        else vc[k] = cb2_v_cols(book, k);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = k < 2 ? w2.x : w2.y, w16 = (k & 1) ? w >> 16 : w;
        uint32_t x[4];
        if constexpr (ROLE == 0) cb2_k_expand(kc[k], w16, x);
        else cb2_v_expand(vc[k], w16, x);
        stmatrix4(tile.step(row, k), x);
      }
    }
    if constexpr (BLK == kBlkCb2s) {   // the static channels' fp16 values
      __syncwarp();
      const int n = min((int)lds8(blk + cb2s_hdr_off(D)), kMaxStatic), t = lane & 15;
      for (int i = lane >> 4; i < n; i += 2)
        sts16(buf + tile.at(t, lds8(blk + cb2s_hdr_off(D) + 1 + i) & (D - 1)), lds16(blk + cb2s_val_off(D) + 32 * i + 2 * t));
    } else {
      patch.store(tile, buf, lane, [&]() { return gblk() + cb2_out_off(D); });
    }
  }
}

// -inf in page_lse for pages [p_lo, p_hi) of the CTA's rows [r_lo, r_hi).
__device__ __forceinline__ void fill_page_lse(const TreeArgs& a, int b, int h, int r_lo, int r_hi, int p_lo, int p_hi) {
  const int n = p_hi - p_lo;
  if (n <= 0) return;
  for (int r = r_lo + (int)(threadIdx.x >> 5); r < r_hi; r += kThreads / 32) {
    float* row = page_lse_row(a, b, h, r);
    for (int p = p_lo + (int)(threadIdx.x & 31); p < p_hi; p += 32) row[p] = -INFINITY;
  }
}

// A softmax thread's row: m in log2 units, p = 2^(s f - m + kPBias), l the fp32 sum of p.  A page with a V shift b:
// P = p 2^b, and m is raised by what P needs.
template <int FMT, int D>
struct SoftmaxRow {
  static constexpr bool kShift = Plan<FMT, D>::kShift;
  float m = -INFINITY, l = 0.f, f;
  float* lse_row;
  bool vec;   // lse_row may be written two pages at a time

  // Columns [c_lo, c_hi) of S at ts, W (32 or 64) at a time, in one pass: p, the
  // pages' sums, P over S's columns.  No maximum is taken: a chunk whose sum
  // passes 2^15 (rare after the first; a p that fp16 could not hold is among
  // them) raises m to the row's maximum, scales what is there -- O (once o_free
  // says that the MMAs are done with it) and the tile's earlier P -- and is
  // computed again.
  template <int W, class OFree>
  __device__ __forceinline__ bool tile(uint32_t ts, uint32_t to, int c_lo, int c_hi, const int32_t* ntok, const float* ks,
                                       uint32_t vs, int pt, int p1, bool has_o, OFree&& o_free) {
    constexpr int NP = W / kPage;   // pages of a chunk
    uint32_t x[W];
    auto load = [&](int c) {
#pragma unroll
      for (int w = 0; w < W / 32; ++w) tc::ld32_issue(ts + c + 32 * w, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * w));
    };
    load(c_lo);
    bool o_ready = false;
#pragma unroll 1
    for (int c = c_lo; c < c_hi; c += W) {
      const int pg = c / kPage;
      int n[NP], total = 0;
      float fk[NP];
#pragma unroll
      for (int j = 0; j < NP; j += 2) {
        const int2 n2 = *reinterpret_cast<const int2*>(ntok + pg + j);
        n[j] = n2.x;
        n[j + 1] = n2.y;
        total += n2.x + n2.y;
        fk[j] = fk[j + 1] = f;
        if (FMT == KVQ_FMT_TIERED) {
          const float2 k2 = *reinterpret_cast<const float2*>(ks + pg + j);
          fk[j] *= k2.x;
          fk[j + 1] *= k2.y;
        }
      }
#pragma unroll
      for (int w = 0; w < W / 32; ++w) tc::wait_ld(*reinterpret_cast<uint32_t(*)[32]>(x + 32 * w));
      if (__builtin_expect(total != W, 0)) {   // absent tokens
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          if (FMT == KVQ_FMT_TIERED && fk[j] == 0.f) fk[j] = 1e-36f;   // a page of zeros: -inf stays -inf
#pragma unroll
          for (int k = 0; k < kPage; ++k) x[kPage * j + k] = k < n[j] ? x[kPage * j + k] : 0xFF800000u;
        }
      }
      uint32_t u[W / 2];
      float ps[NP], sum, mb;
#pragma unroll 1
      for (bool again = false;; again = true) {
        mb = (m == -INFINITY ? 0.f : m) - kPBias;
        const uint64_t nb0 = pack2(-mb, -mb);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const uint64_t f2 = pack2(fk[j], fk[j]);
          uint64_t nb = nb0;
          if constexpr (kShift) {
            const float b = shift(vs, pg + j) - mb;
            nb = pack2(b, b);
          }
          uint64_t acc = 0;   // {0.f, 0.f}
#pragma unroll
          for (int k = 0; k < kPage; k += 2) {
            const float2 y = unpack2(fma2(pack2u(x[kPage * j + k], x[kPage * j + k + 1]), f2, nb));
            const float e0 = ex2(y.x), e1 = ex2(y.y);
            u[(kPage * j + k) / 2] = h2_as_u32(__floats2half2_rn(e0, e1));
            acc = add2(acc, pack2(e0, e1));
          }
          const float2 y = unpack2(acc);
          ps[j] = y.x + y.y;
        }
        sum = ps[0] + ps[1];
#pragma unroll
        for (int j = 2; j < NP; j += 2) sum += ps[j] + ps[j + 1];
        const bool need = !(sum <= 32768.f) || m == -INFINITY;
        if (__builtin_expect(again || !__any_sync(0xffffffffu, need), 1)) break;
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const float top = page_max(x + kPage * j);
          mx = fmaxf(mx, kShift ? fmaf(top, fk[j], shift(vs, pg + j)) : top * fk[j]);
        }
        const bool up = need && mx > m;
        const float alpha = up ? ex2(m - mx) : 1.f;
        l *= alpha;
        m = up ? mx : m;
        if (has_o && !o_ready) {
          if (!o_free()) return false;
          tc::fence_after();
          o_ready = true;
        }
        if (o_ready)
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) scale_columns(to + 16 * k, alpha);
        tc::wait_st();   // the earlier chunks' P: a load is behind a store only if that is waited for
#pragma unroll 1
        for (int k = c_lo / 32; k < c / 32; ++k) scale_p(ts + 16 * k, alpha);
        tc::wait_st();
      }
      if constexpr (kShift) {
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < NP; j += 2) {
          const uint4 v4 = lds128(vs + 8 * (pg + j));
          sum = fmaf(ps[j + 1], __uint_as_float(v4.w), fmaf(ps[j], __uint_as_float(v4.y), sum));
        }
      }
      l += sum;
      if (lse_row) {
#pragma unroll
        for (int j = 0; j < NP; j += 2) {
          const float y0 = page_sum(x + kPage * j, n[j], fk[j], kShift ? mb - shift(vs, pg + j) : mb, ps[j]);
          const float y1 = page_sum(x + kPage * (j + 1), n[j + 1], fk[j + 1], kShift ? mb - shift(vs, pg + j + 1) : mb, ps[j + 1]);
          const int p = pt + pg + j;
          if (vec && p + 1 < p1) {
            *reinterpret_cast<float2*>(lse_row + p) = make_float2(y0, y1);
          } else {
            if (p < p1) lse_row[p] = y0;
            if (p + 1 < p1) lse_row[p + 1] = y1;
          }
        }
      }
      if (c + W < c_hi) load(c + W);
#pragma unroll
      for (int w = 0; w < W / 32; ++w) tc::st16(ts + c / 2 + 16 * w, u + 16 * w);
    }
    return true;
  }
  // A page's V shift, read from shared memory (vs: the tile's [PAGES] of b, 2^-b) wherever it is used: in registers
  // they cost the kernel of many rows 90 bytes of spills.
  static __device__ __forceinline__ float shift(uint32_t vs, int page) { return ldsf(vs + 8 * page); }
  static __device__ __forceinline__ float page_max(const uint32_t* y) {
    float m0 = __uint_as_float(y[0]), m1 = __uint_as_float(y[1]);
#pragma unroll
    for (int k = 2; k < kPage; k += 2) {
      m0 = fmaxf(m0, __uint_as_float(y[k]));
      m1 = fmaxf(m1, __uint_as_float(y[k + 1]));
    }
    return fmaxf(m0, m1);
  }

  // ln of a page's sum, given sum = sum 2^(s f - mb); where the page lies so far
  // below the row's maximum that its terms vanish, the sum relative to its own.
  __device__ __forceinline__ float page_sum(const uint32_t* x, int n, float fk, float mb, float sum) const {
    if (__builtin_expect(sum < 0x1p-80f && n > 0, 0)) {
      mb = page_max(x) * fk;
      if (mb == -INFINITY) return mb;
      sum = 0.f;
#pragma unroll
      for (int k = 0; k < kPage; ++k) sum += ex2(fmaf(__uint_as_float(x[k]), fk, -mb));
    }
    return n > 0 ? (__log2f(sum) + mb) * kLn2 : -INFINITY;
  }
  static __device__ __forceinline__ void scale_columns(uint32_t t, float alpha) {
    uint32_t o[16];
    tc::ld16(t, o);
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
    tc::st16(t, o);
  }
  static __device__ __forceinline__ void scale_p(uint32_t t, float alpha) {   // 16 columns of fp16 pairs
    uint32_t r[16];
    tc::ld16(t, r);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 v = __half22float2(u32_as_h2(r[k]));
      r[k] = h2_as_u32(__floats2half2_rn(v.x * alpha, v.y * alpha));
    }
    tc::st16(t, r);
  }
};

// A segment's partial state from shared memory (xo: [128][D + 4], xml: [128]) to the workspace, by n_sm warps; REP
// copies of a row are joined.  Rows are taken four at a time, so that their loads are in flight together (one at a
// time, 128 rows took 6.3 us).
template <int D, int REP>
__device__ __forceinline__ void store_partial(const TreeArgs& a, size_t part0, const float* xo, const float2* xml, int rows, int n_sm) {
  constexpr int XS = D + 4, PER = kM / REP, U = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
  for (int r0 = warp; r0 < rows; r0 += U * n_sm) {
    float2 ml[U][REP];
    float4 x[U][REP];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = min(r0 + u * n_sm, rows - 1);
#pragma unroll
      for (int c = 0; c < REP; ++c) {
        ml[u][c] = xml[c * PER + r];
        x[u][c] = *reinterpret_cast<const float4*>(xo + (c * PER + r) * XS + 4 * (lane & (D / 4 - 1)));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * n_sm;
      float M = ml[u][0].x, L = ml[u][0].y;
      float4 o = x[u][0];
      if (REP > 1) {
#pragma unroll
        for (int c = 1; c < REP; ++c) M = fmaxf(M, ml[u][c].x);
        L = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < REP; ++c) {
          const bool has = ml[u][c].x != -INFINITY;
          const float w = has ? ex2(ml[u][c].x - M) : 0.f;
          L = fmaf(w, ml[u][c].y, L);
          if (has) {
            o.x = fmaf(w, x[u][c].x, o.x);
            o.y = fmaf(w, x[u][c].y, o.y);
            o.z = fmaf(w, x[u][c].z, o.z);
            o.w = fmaf(w, x[u][c].w, o.w);
          }
        }
      }
      if (r < rows) {
        if (4 * lane < D) *reinterpret_cast<float4*>(a.part_o + (part0 + r) * D + 4 * lane) = o;
        if (lane == 0) a.part_ml[part0 + r] = make_float2(M, L);
      }
    }
  }
}

// Most rows of the FEW variant.
template <int FMT, int D>
constexpr int few_rows() { return kM / (Plan<FMT, D>::kTok / 32); }

// Few rows: the 128 tensor-memory lanes hold `rep` copies of them, and each
// copy's warps take their share of a tile's columns (P = 0 in the others), so
// that the softmax of a tile takes a rep-th of the time.  FEW: a share of 32
// columns, for up to few_rows(); else one copy or two, 64 columns a step.  Two
// kernels, because the code that one of them does not run still costs it
// instruction fetches (4% on 8 rows of the tiered format).
template <int FMT, int D, bool FEW>
__global__ void __launch_bounds__(kThreads, 1) tree_cache_kernel(const TreeArgs a) {
  using F = Fmt<FMT>;
  using P = Plan<FMT, D>;
  constexpr int TOK = P::kTok, PAGES = P::kPages, DEPTH = P::kDepth, SLOT = P::kSlot;
  extern __shared__ uint8_t raw_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nmt = (a.R + kM - 1) / kM;
  const int split = blockIdx.x, h = blockIdx.y / nmt, r0 = (blockIdx.y % nmt) * kM, b = blockIdx.z;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  {   // on its way to the L2 cache while the lengths are read: the split's page table and the query rows
    const int p = split * a.pps + 32 * tid, r = r0 + (tid - 32) / (D / 64);
    if (tid < 32) {
      if (p < min(split * a.pps + a.pps, a.ppsm)) prefetch_l2(a.page_table + (size_t)b * a.ppsm + p);
    } else if (r < min(r0 + kM, a.R)) {
      prefetch_l2(a.q + (((size_t)b * a.T + r / a.G) * a.Hq + (size_t)h * a.G + r % a.G) * D + (tid - 32) % (D / 64) * 64);
    }
  }
  const SeqView v = seq_view(a, b);
  const int live = min(v.nodes * a.G, a.R), rows = min(kM, live - r0), r_end = min(r0 + kM, a.R);
  if (split == 0 && blockIdx.y == 0 && tid == 0 && a.seq_lens[b] > a.max_seq_len) atomicOr(a.status, KVQ_STATUS_SEQ_TOO_LONG);
  const int p0 = split * a.pps, p1 = min(p0 + a.pps, v.blocks), pn = min(p0 + a.pps, a.P);
  const int n_tiles = rows > 0 && p1 > p0 ? (p1 - p0 + PAGES - 1) / PAGES : 0;
  if (a.page_lse) {
    fill_page_lse(a, b, h, max(r0, live), r_end, p0, pn);
    // (the staged pages of live rows are the merge kernel's)
    if (rows > 0) fill_page_lse(a, b, h, r0, r0 + rows, max(p0, v.blocks + (staged_tokens(a, v) + kPage - 1) / kPage), pn);
  }
  const size_t part0 = (((size_t)b * a.Hkv + h) * a.S + split) * a.R + r0;
  if (n_tiles == 0) {
    for (int r = tid; r < rows; r += kThreads) a.part_ml[part0 + r] = make_float2(-INFINITY, 0.f);
    return;
  }

  uint8_t* smem = raw_smem + (((smem_u32(raw_smem) + 1023u) & ~1023u) - smem_u32(raw_smem));
  uint8_t* slots = smem + 2 * P::kBuf;                                    // [kDequantWarps][DEPTH]
  float2* vshift = reinterpret_cast<float2*>(slots + kDequantWarps * DEPTH * SLOT);   // [kMeta][PAGES] b, 2^-b of an FP8 page's V (tiered only)
  uint64_t *k_full = reinterpret_cast<uint64_t*>(vshift + (P::kShift ? kMeta * PAGES : 0)), *k_empty = k_full + 2, *v_full = k_empty + 2,
           *v_empty = v_full + 2, *s_full = v_empty + 2, *p_full = s_full + 2, *done = p_full + 2, *drained = done + 1;
  int32_t* ntok = reinterpret_cast<int32_t*>(drained + 1);                // [kMeta][PAGES] tokens of a tile's pages
  float* kscale = reinterpret_cast<float*>(ntok + kMeta * PAGES);         // [kMeta][PAGES] FP8 pages' K scale, else 1
  int32_t* entries = reinterpret_cast<int32_t*>(kscale + kMeta * PAGES);  // [kDequantWarps][DEPTH] page-table entries of the slots
  float* vscales = reinterpret_cast<float*>(entries + kDequantWarps * DEPTH);   // [kDequantWarps][DEPTH] V scales of a K warp's FP8 pages (tiered only)
  uint32_t* tslot = reinterpret_cast<uint32_t*>(vscales + (P::kShift ? kDequantWarps * DEPTH : 0));
  const int rep = FEW ? TOK / 32 : TOK == 128 && rows <= 64 ? 2 : 1, row = tid % (kM / rep);
  const int n_sm = rep > 1 ? 4 : (rows + 31) / 32;   // softmax warps with rows
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], PAGES);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], PAGES);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], n_sm);
    }
    mbar_init(done, 1);
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  // Each role starts its first global loads before the barrier that publishes the mbarriers and the tensor memory.
  // tensor memory: S tiles (P over them) at columns 0 and 128, O at 256, Q at 384
  uint32_t tmem = 0, t_o = 0, t_q = 0;
  auto join = [&]() {
    tc::fence_before();
    asm volatile("bar.sync 0;" ::: "memory");
    tc::fence_after();
    tmem = *tslot;
    t_o = tmem + 256;
    t_q = tmem + 384;
  };
  bool ok = true;

  if (warp < 4) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---- each thread's query row into tensor memory, scaled by a power of two into fp16 range
    float f = 0.f, qs = 0.f;
    uint32_t q[D / 2] = {};   // bf16 pairs
    if (warp < n_sm) {
      const int r = r0 + row;
      if (row < rows) {
        const uint4* qr = reinterpret_cast<const uint4*>(a.q + (((size_t)b * a.T + r / a.G) * a.Hq + (size_t)h * a.G + r % a.G) * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint4 x = qr[i];
          q[4 * i] = x.x;
          q[4 * i + 1] = x.y;
          q[4 * i + 2] = x.z;
          q[4 * i + 3] = x.w;
        }
      }
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < D / 2; ++i)
        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(q[i] << 16)), fabsf(__uint_as_float(q[i] & 0xFFFF0000u))));
      int e = 0;
      frexpf(mx, &e);
      const int k = mx > 0.f && mx < INFINITY ? max(e - 15, -100) : 0;
      // the scale's sign goes with the query, so that the score factor f is positive
      qs = copysignf(ldexpf(1.f, -k), a.scale_log2);
      f = fmaxf(ldexpf(fabsf(a.scale_log2), k), 1e-36f);
    }
    join();
    if (warp < n_sm) {
#pragma unroll
      for (int i = 0; i < D / 2; ++i)
        q[i] = h2_as_u32(__floats2half2_rn(__uint_as_float(q[i] << 16) * qs, __uint_as_float(q[i] & 0xFFFF0000u) * qs));
#pragma unroll
      for (int c = 0; c < D / 64; ++c) tc::st32(t_q + ((uint32_t)(32 * warp) << 16) + 32 * c, q + 32 * c);
      tc::wait_st();
      tc::fence_before();
      asm volatile("bar.arrive 3, %0;" ::"r"(32 * n_sm + 32) : "memory");   // (the MMA warp waits)
    }
    if (warp < n_sm) {
      const uint32_t lanes = (uint32_t)(32 * warp) << 16;
      SoftmaxRow<FMT, D> sr;
      sr.f = f;
      const uint32_t vshift_s = smem_u32(vshift);
      sr.lse_row = a.page_lse && row < rows ? page_lse_row(a, b, h, r0 + row) : nullptr;
      sr.vec = (a.P & 1) == 0 && (reinterpret_cast<uintptr_t>(a.page_lse) & 7) == 0;
      const int chunks = TOK / 32 / rep, c0 = warp / (4 / rep) * chunks;   // this warp's 32-column chunks
      for (int i = 0; i < n_tiles; ++i) {
        ok = __all_sync(0xffffffffu, wait_bar(&s_full[i & 1], (i >> 1) & 1));
        if (!ok) break;
        tc::fence_after();
        const uint32_t ts = tmem + lanes + (i & 1) * 128;
        const int slot = (i & (kMeta - 1)) * PAGES, pt = p0 + i * PAGES;
        // PV(i - 1) has to be done before O changes; PV(i - 3), that barrier's phase before, is (S(i - 1) was committed after it)
        auto o_free = [&]() {
          return __all_sync(0xffffffffu, wait_bar(&v_empty[(i - 1) & 1], ((i - 1) >> 1) & 1));
        };
        const int lo = 32 * c0, hi = 32 * (c0 + chunks);
        ok = sr.template tile<FEW ? 32 : 64>(ts, t_o + lanes, lo, hi, ntok + slot, kscale + slot, vshift_s + 8 * slot, pt, p1, i > 0, o_free);
        if (!ok) break;
        if (rep > 1) {   // the columns of the row's other copies: P = 0
          const uint32_t z[16] = {};
          for (int c = 0; c < TOK / 32; ++c)
            if (c < c0 || c >= c0 + chunks) tc::st16(ts + 16 * c, z);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[i & 1]);
      }
      // Where any role's wait gave up, the MMA warp's did too (it waits for all of them) and `done` never comes: no softmax
      // warp stores, and the rows keep the NaN of the start.  The limit is above the four waits that the MMA warp may have left.
      ok = ok && __all_sync(0xffffffffu, wait_bar(done, 0, 1000000000ll));
      // ---- the partial state, through shared memory (the tiles are done): copies of a row are joined, rows stored whole
      constexpr int XS = D + 4;
      float* xo = reinterpret_cast<float*>(smem);                       // [128][XS], thread's row of O
      float2* xml = reinterpret_cast<float2*>(smem + kM * XS * 4);      // [128]
      static_assert(kM * XS * 4 + kM * 8 <= 2 * P::kBuf, "partial state fits over the tiles");
      const int n_thr = 32 * n_sm;
      if (ok) {
        tc::fence_after();
        xml[tid] = make_float2(sr.m == -INFINITY ? -INFINITY : sr.m - kPBias, sr.l);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc::ld32(t_o + lanes + 32 * c, o);
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<float4*>(xo + tid * XS + 32 * c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
        tc::fence_before();
      }
      asm volatile("bar.sync 1, %0;" ::"r"(n_thr) : "memory");
      if (ok) {
        if constexpr (FEW) {
          store_partial<D, TOK / 32>(a, part0, xo, xml, rows, n_sm);
        } else {
          if (rep == 1) store_partial<D, 1>(a, part0, xo, xml, rows, n_sm);
          else store_partial<D, 2>(a, part0, xo, xml, rows, n_sm);
        }
      }
    }
  } else if (warp >= 4 && warp < 4 + kDequantWarps) {
    // ------------------------------------------------------------------ dequantization
    // a warp takes one page's K or V; with 4 pages a tile (INT4) of every other tile
    constexpr int kTurns = kDequantWarps / (2 * PAGES);
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDequant));
    const int wi = warp - 4, j = wi % PAGES, role = wi / PAGES % 2, i0 = wi / (2 * PAGES);
    const int n_mine = i0 < n_tiles ? (n_tiles - i0 + kTurns - 1) / kTurns : 0;   // this warp's tiles i0, i0 + kTurns, ...
    uint8_t* ring = slots + wi * DEPTH * SLOT;
    const int32_t* pt = a.page_table + (size_t)b * a.ppsm;
    // The page's entry in this warp's k-th tile: a window of 32 in the lanes.  kNoPage: absent, or bad.
    // The group format looks at the whole of the page's group, which the bound on the length may cut.
    int32_t* ent = entries + wi * DEPTH;
    float* vsc = vscales + wi * DEPTH;
    int win_base = 0, win = kNoPage;
    auto load_window = [&](int base) {
      win_base = base;
      win = kNoPage;
      const int p = p0 + (i0 + (base + lane) * kTurns) * PAGES + j;
      if (base + lane >= n_mine || p >= p1) return;
      bool good = true;
      int32_t e = 0;
      const int lo = F::kGroup ? p / kGroupPages * kGroupPages : p, hi = F::kGroup ? min(lo + kGroupPages, a.ppsm) : p + 1;
      for (int x = lo; x < hi; ++x) {
        const int32_t ex = pt[x];
        const uint32_t phys = (uint32_t)ex & 0x7FFFFFFFu;
        good = good && (ex < 0 ? (FMT == KVQ_FMT_TIERED && phys < (uint32_t)a.num_tier_pages) : phys < (uint32_t)a.num_pages);
        e = x == p ? ex : e;
      }
      if (good) win = e;
      else if (role == 0) atomicOr(a.status, KVQ_STATUS_BAD_PAGE);
    };
    // where this warp's blocks of physical page 0 lie, and the bytes from a page to the next
    const size_t main_page = (size_t)a.Hkv * 2 * block_stride(F::kMain, D), tier_page = (size_t)a.Hkv * 2 * block_stride(kBlkFp8, D);
    const uint8_t* const main_src = a.pool + (size_t)(2 * h + role) * block_stride(F::kMain, D);
    const uint8_t* const tier_src = FMT == KVQ_FMT_TIERED ? a.tier_pool + (size_t)(2 * h + role) * block_stride(kBlkFp8, D) : nullptr;
    auto block_at = [&](int32_t e) {
      return FMT == KVQ_FMT_TIERED && e < 0 ? tier_src + ((uint32_t)e & 0x7FFFFFFFu) * tier_page : main_src + (uint32_t)e * main_page;
    };
    auto copy = [&](uint32_t dst, const uint8_t* src, int bytes, auto most) {   // 16 bytes a lane at a time; at most `most`
      const uint32_t d = dst + 16 * lane;
      const uint8_t* p = src + 16 * lane;
#pragma unroll
      for (int o = 0; o < most.value; o += 512)
        if (16 * lane + o < bytes) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + o), "l"(p + o) : "memory");
    };
    auto issue = [&](int k, int slot) {   // the copy of the warp's k-th block (past the last: an empty group)
      if (k < n_mine) {
        if (k - win_base >= 32) load_window(k);
        const int32_t e = __shfl_sync(0xffffffffu, win, k - win_base);
        if (lane == 0) ent[slot] = e;
        if (e != kNoPage) {
          const uint32_t dst = smem_u32(ring + slot * SLOT);
          if constexpr (F::kGroup) {
            const int page = p0 + (i0 + k * kTurns) * PAGES + j, first = page / kGroupPages * kGroupPages;
            copy(dst, block_at(pt[first]), 8 * D, std::integral_constant<int, 8 * D>{});
            copy(dst + 8 * D, block_at(e) + 8 * D, 4 * D + kOutPrefetch, std::integral_constant<int, 4 * D + kOutPrefetch>{});
          } else {
            copy(dst, block_at(e),
                 FMT == KVQ_FMT_TIERED && e < 0 ? fetch_bytes<D>(kBlkFp8)
                 : F::kMain == kBlkCb2s        ? 12 * D + 16 + 32 * a.n_static
                                               : fetch_bytes<D>(F::kMain),
                 std::integral_constant<int, SLOT>{});
            if (P::kShift && role == 0 && e < 0 && lane == 0)   // the V block's scale, beside the K block
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(vsc + slot)),
                           "l"(block_at(e) + block_stride(kBlkFp8, D) + fp8_sc_off(D))
                           : "memory");
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load_window(0);
    for (int k = 0; k < DEPTH; ++k) issue(k, k);
    if (warp == 4) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    join();
    uint64_t* const empty = role ? v_empty : k_empty;
    uint64_t* const filled = role ? v_full : k_full;
    const uint32_t base = smem_u32(smem) + role * P::kTile, ring_s = smem_u32(ring);
    const KTile<D, TOK> kt{j};
    const VTile<D, TOK> vt{j};
    int slot = 0, i = i0, left = v.len - kPage * (p0 + i0 * PAGES + j);   // tile; visible tokens from its page on
#pragma unroll 1
    for (int k = 0; k < n_mine; ++k) {
      asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
      if (i >= 2) ok = wait_bar(empty + (i & 1), ((i >> 1) - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      __syncwarp();   // every lane's part of the copy
      if (!ok) break;
      const int32_t e = ent[slot];
      const int n = e == kNoPage ? 0 : min(kPage, left);
      const bool tier = FMT == KVQ_FMT_TIERED && e < 0;
      const uint32_t blk = ring_s + slot * SLOT, buf = base + (i & 1) * P::kBuf;
      auto gblk = [&]() { return block_at(e); };
      if (role == 0) {
        const int at = (i & (kMeta - 1)) * PAGES + j;
        if (lane == 0) {
          ntok[at] = n;
          if (P::kShift) {
            kscale[at] = 1.f;
            vshift[at] = make_float2(0.f, 1.f);
            if (tier) {
              const int sh = v_shift(vsc[slot]);
              kscale[at] = ldsf(blk + fp8_sc_off(D));
              vshift[at] = make_float2((float)sh, exp2_int(-sh));
            }
          }
        }
        if (n > 0) dequant_block<FMT, D, 0>(blk, gblk, tier, kt, buf, buf + 2 * P::kTile, lane);
      } else {
        if (n > 0) dequant_block<FMT, D, 1>(blk, gblk, tier, vt, buf, 0u, lane);
        if (__builtin_expect(n < kPage, 0)) {
          __syncwarp();
          zero_tokens<D>(vt, buf, n, lane);
        }
      }
      fence_proxy_async();   // the tile for the MMAs
      __syncwarp();
      if (lane == 0) mbar_arrive(filled + (i & 1));
      issue(k + DEPTH, slot);
      slot = slot + 1 == DEPTH ? 0 : slot + 1;
      i += kTurns;
      left -= kPage * PAGES * kTurns;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    // Until the partial states are stored they are NaN, so that nothing that an earlier call left in the workspace is taken
    // for them.  (The merge kernel gives m = -inf the weight 0, and 0 x NaN makes the row's sum, out and lse NaN.)
    if (warp > 4 + kDequantWarps)
      for (int r = tid - 32 * (5 + kDequantWarps); r < rows; r += 96) a.part_ml[part0 + r] = make_float2(-INFINITY, NAN);
    join();
    if (warp == 4 + kDequantWarps) {
      asm volatile("bar.sync 3, %0;" ::"r"(32 * n_sm + 32) : "memory");   // the query rows
      tc::fence_after();
    }
    if (warp == 4 + kDequantWarps && lane == 0) {
      // ---------------------------------------------------------------- MMA
      constexpr uint32_t id_s = tc::idesc_f16(kM, TOK), id_o = tc::idesc_f16(kM, D);
      const uint64_t buf_desc = tc::desc_sw128(smem_u32(smem));
      auto scores = [&](int i) {
        if (!wait_bar(&k_full[i & 1], (i >> 1) & 1)) return false;
        // S(i) goes over P(i - 2), which PV(i - 2) reads: MMAs with different accumulators have no order of their own
        if (i >= 2 && !wait_bar(&v_empty[i & 1], ((i >> 1) - 1) & 1)) return false;
        tc::fence_after();
        const uint64_t kt = buf_desc + (i & 1) * (P::kBuf >> 4);
#pragma unroll
        for (int half = 0; half < (P::kPair ? 2 : 1); ++half)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma_ta(tmem + (i & 1) * 128, t_q + 8 * k,
                       kt + ((half * 2 * P::kTile + (k >> 2) * (TOK * 128) + (k & 3) * 32) >> 4), id_s, (half | k) != 0);
        tc::commit(&s_full[i & 1]);
        tc::commit(&k_empty[i & 1]);
        return true;
      };
      ok = scores(0);
      for (int i = 0; i < n_tiles && ok; ++i) {
        if (i + 1 < n_tiles) ok = scores(i + 1);
        ok = ok && wait_bar(&v_full[i & 1], (i >> 1) & 1) && wait_bar(&p_full[i & 1], (i >> 1) & 1);
        if (!ok) break;
        tc::fence_after();
        const uint64_t vt = buf_desc + (((i & 1) * P::kBuf + P::kTile) >> 4);
#pragma unroll
        for (int k = 0; k < TOK / 16; ++k)
          tc::mma_ta(t_o, tmem + (i & 1) * 128 + 8 * k, vt + (((k >> 2) * (D * 128) + (k & 3) * 32) >> 4), id_o, (i | k) != 0);
        tc::commit(&v_empty[i & 1]);
      }
      tc::commit(ok ? done : drained);
      if (!ok) wait_bar(drained, 0);   // tensor memory may be freed once what was issued is done
    }
  }
  if (!ok && lane == 0) atomicOr(a.status, KVQ_STATUS_TIMEOUT);
  __syncthreads();
  if (warp == 4) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int FMT, int D>
static TreeKernel tree_kernel_info(int R) {
  return {R <= few_rows<FMT, D>() ? reinterpret_cast<void*>(tree_cache_kernel<FMT, D, true>)
                                  : reinterpret_cast<void*>(tree_cache_kernel<FMT, D, false>),
          (size_t)Plan<FMT, D>::kSmem, kThreads};
}

}  // namespace tree
}  // namespace kvq
