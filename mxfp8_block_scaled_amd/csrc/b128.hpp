// Device helpers of the 128-block format and of 8-bit activation checkpoints.
#pragma once

#include "common.hpp"
#include "launch_b128.hpp"

namespace mxfp8 {

// Scale byte of a 128-block from the bf16 bits of its largest magnitude (the
// rule is stated in quant_b128.hip).
__device__ inline uint32_t b128_scale_byte(uint32_t amax) {
  const int f = (int)(amax >> 7), up = (int)(amax & 0x7Fu) > 96 ? 1 : 0;
  return amax >= 0x7F80u ? 0xFFu : (uint32_t)max(f - 8 + up, 0);
}
// Its value, with the UE8M0 NaN as an fp32 NaN.
__device__ inline float b128_scale_value(uint32_t sb) {
  return __uint_as_float(sb == 0xFFu ? 0x7FC00000u : sb ? sb << 23 : 0x00400000u);
}

// Sixteen E4M3 bytes of one scale -> sixteen bf16, two 16-byte words.
__device__ inline void widen16(const uint4& q, float scale, uint4* out) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t d[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    d[2 * e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[e], scale, false));
    d[2 * e + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[e], scale, true));
  }
  out[0] = make_uint4(d[0], d[1], d[2], d[3]);
  out[1] = make_uint4(d[4], d[5], d[6], d[7]);
}

// Maximum over the sixteen lanes of a DPP row: quads, then half and whole
// row mirrors (VALU only).
__device__ inline uint32_t row16_max(uint32_t m) {
  m = quad_max(m);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, true));   // row_half_mirror
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x140, 0xF, 0xF, true));   // row_mirror
}

__device__ inline uint32_t absmax8(const uint4& v) {
  u16x2 m = {0, 0};
  m = absmax_pk(m, v.x);
  m = absmax_pk(m, v.y);
  m = absmax_pk(m, v.z);
  m = absmax_pk(m, v.w);
  return max((uint32_t)m[0], (uint32_t)m[1]);
}

}  // namespace mxfp8
