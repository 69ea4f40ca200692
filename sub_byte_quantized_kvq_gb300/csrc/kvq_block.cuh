// kvq_block.cuh -- the value one element of a block stands for, read straight
// from its bytes (the debug path).
#pragma once
#include "kvq_common.cuh"

namespace kvq {

__device__ __forceinline__ float dq_e4m3(uint32_t b) {
  uint32_t d;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(d) : "r"(b & 0xFFu));
  return __half2float(__ushort_as_half((unsigned short)(d & 0xFFFFu)));
}
__device__ __forceinline__ float dq_e2m1(uint32_t nib) {
  const float mag[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
  return (nib & 8u) ? -mag[nib & 7u] : mag[nib & 7u];
}
__device__ __forceinline__ float dq_f16(uint32_t bits) {
  return __half2float(__ushort_as_half((unsigned short)(bits & 0xFFFFu)));
}

// The value an outlier side-list (CB2, ASYM3) gives (t, c), else v.
__device__ __forceinline__ float side_list_value(const uint8_t* hdr, int D, int t, int c, float v) {
  const int n_ch = min((int)hdr[0], D);  // a corrupt side-list never reads past its block
  for (int i = 0; i < n_ch; ++i) {
    const uint8_t* rec = hdr + 4 + 20 * i;
    const uint32_t tm = rec[2] | (rec[3] << 8);
    if (rec[0] == c && (tm >> t & 1u)) v = dq_e4m3(rec[4 + t]);
  }
  return v;
}

// Element (t, c) of block `blk` of block format bf (BlkFmt): exactly the value
// its code stands for (INT4: fmaf(q, S, m); E2M1: e2m1 * scale; CB2: fp16
// centroid or e4m3 outlier; FP8: e4m3 * scale in fp32).  cbk: the block holding
// the codebook (the group's first page for kBlkCb2g, else blk).
__device__ inline float block_value(int bf, const uint8_t* blk, const uint8_t* cbk, int role, int D, int t, int c) {
  const int NS = D / 16;
  const FragPos p = frag_pos(role, t, c);
  float v;
  if (bf == kBlkCb2g) {
    const uint8_t* cw = blk + cb2g_code_off(D) + 2 * NS * p.lane + 2 * p.step;
    const uint32_t q = ((cw[0] | (cw[1] << 8)) >> (4 * (p.slot & 3) + 2 * (p.slot >> 2))) & 3u;
    const uint8_t* cb = cbk + 8 * cb2_slot(role, c);
    v = dq_f16(cb[q] | (cb[4 + q] << 8));
    v = side_list_value(blk + cb2_out_off(D), D, t, c, v);
    return v;
  }
  if (bf == kBlkInt4) {
    const uint32_t q = (blk[4 * NS * p.lane + 4 * p.step + p.slot / 2] >> (4 * (p.slot & 1))) & 0xFu;
    const uint8_t* sz = blk + int4_sz_off(D) + 4 * (t * (D / 32) + c / 32);
    v = fmaf((float)q, dq_f16(sz[0] | (sz[1] << 8)), dq_f16(sz[2] | (sz[3] << 8)));
    const int cap = int4_cap(D), cnt = blk[int4_cnt_off(D) + t];
    for (int i = 0; i < cnt && i < cap; ++i)
      if (blk[int4_ch_off(D) + t * cap + i] == c) {
        const uint8_t* vp = blk + int4_val_off(D) + 2 * (t * cap + i);
        v = dq_f16(vp[0] | (vp[1] << 8));
      }
  } else if (bf == kBlkE2m1) {
    const uint32_t q = (blk[4 * NS * p.lane + 4 * p.step + p.slot / 2] >> (4 * (p.slot & 1))) & 0xFu;
    v = dq_e2m1(q) * dq_e4m3(blk[e2m1_sc_off(D) + 16 * (c / 16) + t]);
  } else if (bf == kBlkCb2 || bf == kBlkCb2s) {
    const uint32_t w = blk[2 * NS * p.lane + 2 * p.step] | (blk[2 * NS * p.lane + 2 * p.step + 1] << 8);
    const uint32_t q = (w >> (4 * (p.slot & 3) + 2 * (p.slot >> 2))) & 3u;
    const uint8_t* cb = blk + cb2_cb_off(D) + 8 * cb2_slot(role, c);
    v = dq_f16(cb[q] | (cb[4 + q] << 8));
    if (bf == kBlkCb2s) {   // static fp16 channels
      const uint8_t* hdr = blk + cb2s_hdr_off(D);
      const int n_s = min((int)hdr[0], kMaxStatic);
      for (int i = 0; i < n_s; ++i)
        if (hdr[1 + i] == c) {
          const uint8_t* vp = blk + cb2s_val_off(D) + 32 * i + 2 * t;
          v = dq_f16(vp[0] | (vp[1] << 8));
        }
    } else {
      v = side_list_value(blk + cb2_out_off(D), D, t, c, v);
    }
  } else if (bf == kBlkA3) {
    uint32_t vx, vy;
    memcpy(&vx, blk + 4 * (p.lane * (NS / 2) + p.step / 2), 4);
    memcpy(&vy, blk + a3_hi_off(D) + 4 * (p.lane * (NS / 4) + p.step / 4), 4);
    const int bx = 8 * (p.step % 2) + 16 * (p.slot % 2) + 2 * (p.slot / 2);
    const int by = 4 * (p.step % 4) + 16 * (p.slot % 2) + p.slot / 2;
    const uint32_t q = ((vx >> bx) & 3u) | (((vy >> by) & 1u) << 2);
    const int r = a3_rho(role, c);
    const uint8_t* sp = blk + a3_s_off(D) + 2 * r;
    const uint8_t* mp = blk + a3_m_off(D) + 2 * r;
    // fp16(q * S + m): one rounding of the exact value (fp16 fused multiply-add)
    v = __half2float(__hfma(__float2half_rn((float)q), __ushort_as_half((unsigned short)(sp[0] | (sp[1] << 8))),
                            __ushort_as_half((unsigned short)(mp[0] | (mp[1] << 8)))));
    v = side_list_value(blk + a3_out_off(D), D, t, c, v);
  } else {
    float s;
    memcpy(&s, blk + fp8_sc_off(D), 4);
    v = __fmul_rn(dq_e4m3(blk[8 * NS * p.lane + 8 * p.step + p.slot]), s);
  }
  return v;
}

}  // namespace kvq
