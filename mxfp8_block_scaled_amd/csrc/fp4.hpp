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

// Zeros in rows [from, to) of y [.., N] (bf16, row stride ldy): the rows of slots
// without an expert.  A wave takes whole rows, 16 bytes per lane (4096 tokens, 64
// experts, k 8, half of the ids none, 2048 x 768: 59 us; 120 with a division and
// two bytes per element).
__device__ inline void zero_rows(uint16_t* y, int64_t ldy, int from, int to, int N, int waves) {
  typedef uint32_t u4a2 __attribute__((ext_vector_type(4), aligned(2)));   // (the hardware serves any address)
  const int lane = threadIdx.x & 63;
  for (int64_t r = from + (int64_t)blockIdx.x * waves + (threadIdx.x >> 6); r < to; r += (int64_t)gridDim.x * waves)
    for (int n = lane * 8; n < N; n += 64 * 8) {
      uint16_t* d = y + r * ldy + n;
      if (n + 7 < N) *reinterpret_cast<u4a2*>(d) = u4a2{0u, 0u, 0u, 0u};
      else
        for (int e = 0; n + e < N; ++e) d[e] = 0;
    }
}

// c[u] += A[u] x B, u = 0 .. 3, on v_mfma_scale_f32_16x16x128_f8f6f4 with both
// operands in E2M1 (cbsz, blgp 4): lane (i, g) holds K [32g, 32g + 32) of row i
// in four registers; scales (A[u]: word u % 2, byte kSelA + u / 2), in-place
// accumulation and wait states as in tile::mfma16.  Four in one block: nothing
// can come between them, so the wait states in front of the first serve all.
// A 4-bit MFMA takes 16 cycles, in which the wave issues few other
// instructions; with kCopy a copy into LDS (16 bytes per lane from voff + soff
// of rsrc to lds + kAt + 16 lane) is issued between them, an MFMA in the place
// of the wait state between the m0 write and the copy.
template <int kSelA, int kSelB, bool kCopy, int kAt>
__device__ __forceinline__ void mfma16x4_fp4(v4f& c0, v4f& c1, v4f& c2, v4f& c3, const tile::i4v* a,
                                             const tile::i4v& b, int sa0, int sa1, int sb, uint32_t voff = 0,
                                             tile::i4v rsrc = {}, uint32_t soff = 0, uint32_t lds = 0) {
#define MXFP8_MFMA(C, A, S, LO, HI) \
  "v_mfma_scale_f32_16x16x128_f8f6f4 " C ", " A ", %8, " C ", " S ", %11 op_sel:[" LO ",%16,0] op_sel_hi:[" HI ",%17,0] cbsz:4 blgp:4\n\t"
#define MXFP8_OPERANDS                                                                                              \
  "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b), "v"(sa0), "v"(sa1), "v"(sb), "n"(kSelA & 1), "n"(kSelA >> 1), \
      "n"((kSelA + 1) & 1), "n"((kSelA + 1) >> 1), "n"(kSelB & 1), "n"(kSelB >> 1)
  if constexpr (kCopy) {
    asm volatile("s_nop 1\n\t" MXFP8_MFMA("%0", "%4", "%9", "%12", "%13")
                 "s_add_u32 m0, %21, %22\n\t" MXFP8_MFMA("%1", "%5", "%10", "%12", "%13")
                 "buffer_load_dwordx4 %18, %19, %20 offen lds\n\t" MXFP8_MFMA("%2", "%6", "%9", "%14", "%15")
                 MXFP8_MFMA("%3", "%7", "%10", "%14", "%15")
                 : "+a"(c0), "+a"(c1), "+a"(c2), "+a"(c3)
                 : MXFP8_OPERANDS, "v"(voff), "s"(rsrc), "s"(soff), "s"(lds), "n"(kAt)
                 : "memory", "m0", "scc");
  } else {
    asm volatile("s_nop 1\n\t" MXFP8_MFMA("%0", "%4", "%9", "%12", "%13") MXFP8_MFMA("%1", "%5", "%10", "%12", "%13")
                 MXFP8_MFMA("%2", "%6", "%9", "%14", "%15") MXFP8_MFMA("%3", "%7", "%10", "%14", "%15")
                 : "+a"(c0), "+a"(c1), "+a"(c2), "+a"(c3)
                 : MXFP8_OPERANDS);
  }
#undef MXFP8_MFMA
#undef MXFP8_OPERANDS
}

}  // namespace mxfp8
