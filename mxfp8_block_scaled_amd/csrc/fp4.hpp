// Device helpers of the MXFP4 format: the block quantizer and the 4-bit
// operands of the scaled MFMA.
#pragma once

#include "common.hpp"
#include "launch_fp4.hpp"
#include "tile_core.hpp"

namespace mxfp8 {

// Scale byte of an MXFP4 block from the bf16 bits of its largest magnitude:
// shared exponent floor(log2 amax) - 2 (E2M1's largest exponent is 2), byte 0
// for a block of zeros, 0xFF (NaN) for one that holds an infinity or a NaN.
__device__ inline uint32_t fp4_scale_byte(uint32_t amax) {
  return amax >= 0x7F80u ? 0xFFu : (uint32_t)max((int)(amax >> 7) - 2, 0);
}
// Its value as the converter takes it (a block of 0xFF keeps finite codes: its
// scale makes every product NaN).
__device__ inline float fp4_scale_value(uint32_t sb) { return mx_scale_value(sb == 0xFFu ? 254u : sb); }

// Eight bf16 (16 bytes) -> eight E2M1 codes, element 2j in the low nibble of
// byte j; the converter rounds to nearest even and saturates to +-6.
__device__ inline uint32_t cvt8_fp4(const uint4& v, float scale) {
  uint32_t d = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, __builtin_bit_cast(bf16x2, v.x), scale, 0);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(d, __builtin_bit_cast(bf16x2, v.y), scale, 1);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(d, __builtin_bit_cast(bf16x2, v.z), scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(d, __builtin_bit_cast(bf16x2, v.w), scale, 3);
}

__device__ inline uint32_t fp4_absmax8(const uint4& v) {
  u16x2 m = {0, 0};
  m = absmax_pk(m, v.x);
  m = absmax_pk(m, v.y);
  m = absmax_pk(m, v.z);
  m = absmax_pk(m, v.w);
  return max((uint32_t)m[0], (uint32_t)m[1]);
}

// c += A x B on v_mfma_scale_f32_16x16x128_f8f6f4 with both operands in E2M1
// (cbsz, blgp 4): lane (i, g) holds K [32g, 32g + 32) of row i in four
// registers; scales, in-place accumulation and wait states as in
// tile::mfma16.
template <int kSelA, int kSelB>
__device__ __forceinline__ void mfma16_fp4(v4f& c, const tile::i4v& a, const tile::i4v& b, int sa, int sb) {
  asm volatile(
      "s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0] "
      "cbsz:4 blgp:4"
      : "+a"(c)
      : "v"(a), "v"(b), "v"(sa), "v"(sb), "n"(kSelA & 1), "n"(kSelB & 1), "n"(kSelA >> 1), "n"(kSelB >> 1));
}

}  // namespace mxfp8
