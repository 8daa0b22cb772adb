// bf16 rows -> MXFP4 activations (the MX rule with E2M1 elements: shared
// exponent floor(log2 amax) - 2, round to nearest even, saturate to +-6), in
// the packed operand layout or row-major.  Bound by memory: 2 bytes read and
// 0.53 written per element (8192 x 8192 packed 28 us, 6.0 TB/s; 32768 x 768 by
// rows 13 us, 4.9 TB/s).  Four lanes share a block, 16 bytes each.
#include "fp4.hpp"

namespace mxfp8 {

namespace {

constexpr int kQuantThreads = 256;

struct Fp4Piece {
  uint32_t codes, scale;   // eight codes, and the byte of the block of four lanes
};
__device__ inline Fp4Piece quant8(const uint4& v) {
  const uint32_t sb = fp4_scale_byte(quad_max(fp4_absmax8(v)));
  return {cvt8_fp4(v, fp4_scale_value(sb)), sb};
}

}  // namespace

// One workgroup: a 16-row band, kSteps consecutive 128-K steps.  Sixteen lanes
// read the 256 bytes of a row's step and write 64.
template <int kSteps>
__global__ __launch_bounds__(kQuantThreads) void quant_packed_fp4_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                         int M, int KS4, int chunks,
                                                                         uint8_t* __restrict__ qp,
                                                                         uint8_t* __restrict__ sp) {
  const int tid = threadIdx.x;
  const int band = (int)blockIdx.x / chunks, s0 = ((int)blockIdx.x - band * chunks) * kSteps;
  const int rb = tid >> 4, l = tid & 15;
  const int m = band * 16 + rb;
  const int r = (band & 7) * 16 + rb;                      // row in its 128-row group
  const int64_t g = band >> 3;
  uint4 v[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    v[s] = m < M && s0 + s < KS4 ? *reinterpret_cast<const uint4*>(x + (int64_t)m * ldx + (int64_t)(s0 + s) * 128 + l * 8)
                                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (s0 + s >= KS4) break;
    const Fp4Piece p = quant8(v[s]);
    *reinterpret_cast<uint32_t*>(qp + g * KS4 * kTileBytes + packed_off(r, s0 + s, l >> 2, KS4) + (l & 3) * 4) = p.codes;
    if ((l & 3) == 0)   // block l / 4 of the step: block (l / 4) % 2 of scale tile 2 (s0 + s) + l / 8
      sp[(g * KS4 + s0 + s) * 2 * kTileScaleBytes + (l >> 3) * kTileScaleBytes + scale_off(r, (l >> 2) & 1)] =
          (uint8_t)p.scale;
  }
}

int launch_quantize_packed_fp4(const void* x, int64_t M, int64_t K, int64_t ldx, void* qp, void* sp,
                               hipStream_t stream) {
  const int64_t bands = (M + kGroupRows - 1) / kGroupRows * 8;
  const int KS4 = (int)(K / kFp4Step);
  auto go = [&](auto kern, int steps) {
    const int chunks = (KS4 + steps - 1) / steps;
    hipLaunchKernelGGL(kern, dim3((unsigned)(bands * chunks)), dim3(kQuantThreads), 0, stream, (const uint16_t*)x, ldx,
                       (int)M, KS4, chunks, (uint8_t*)qp, (uint8_t*)sp);
  };
  // Four steps per workgroup where that still gives the chip over a thousand.
  if (bands * ((KS4 + 3) / 4) >= 1024) go(quant_packed_fp4_kernel<4>, 4);
  else go(quant_packed_fp4_kernel<1>, 1);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

// Row-major: a thread takes kPieces pieces of eight elements, kQuantThreads
// apart.
template <int kPieces>
__global__ __launch_bounds__(kQuantThreads) void quant_rows_fp4_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                       uint32_t per_row, uint32_t total,
                                                                       uint8_t* __restrict__ q,
                                                                       uint8_t* __restrict__ s, int pitch) {
  const uint32_t base = (uint32_t)blockIdx.x * (kQuantThreads * kPieces) + threadIdx.x;
  uint4 v[kPieces];
  uint32_t row[kPieces], at[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const uint32_t i = min((uint32_t)(base + u * kQuantThreads), (uint32_t)(total - 1));
    row[u] = i / per_row;
    at[u] = i - row[u] * per_row;
    v[u] = *reinterpret_cast<const uint4*>(x + (int64_t)row[u] * ldx + (int64_t)at[u] * 8);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const Fp4Piece p = quant8(v[u]);
    if ((uint32_t)(base + u * kQuantThreads) < total) {
      reinterpret_cast<uint32_t*>(q)[base + u * kQuantThreads] = p.codes;
      if ((at[u] & 3) == 0) s[(int64_t)row[u] * pitch + (int64_t)(at[u] >> 2)] = (uint8_t)p.scale;
    }
  }
}

int launch_quantize_rows_fp4(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, void* s, hipStream_t stream) {
  const int64_t per_row = K / 8, total = M * per_row;
  auto go = [&](auto kern, int pieces) {
    const int64_t n = (int64_t)kQuantThreads * pieces;
    hipLaunchKernelGGL(kern, dim3((unsigned)((total + n - 1) / n)), dim3(kQuantThreads), 0, stream, (const uint16_t*)x,
                       ldx, (uint32_t)per_row, (uint32_t)total, (uint8_t*)q, (uint8_t*)s, (int)fp4_scale_pitch(K));
  };
  // (less than 2^30 pieces: the callers bound the M K / 2 bytes of codes to 32 bits)
  if (total >= (int64_t)kQuantThreads * 4 * 1024) go(quant_rows_fp4_kernel<4>, 4);
  else go(quant_rows_fp4_kernel<1>, 1);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace mxfp8
