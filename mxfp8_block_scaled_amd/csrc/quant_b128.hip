// Quantization with one scale for each block of 128: activations with a
// power-of-two (UE8M0) scale per 1 x 128 block, weights with one per
// 128 x 128 block (kept as fp32, the form checkpoints hold).
//
// The rule: scale = the smallest power of two s with amax / s <= 448 (the
// largest E4M3 value), so nothing saturates; elements RNE(v / s).  With
// amax = (1 + mant / 128) 2^(F - 127) (bf16 fields) that is
// 2^(F - 135) for mant <= 96 (1.75 * 256 = 448) and twice that above, i.e.
// the byte F - 8 + (mant > 96), at least 0; a block of zeros gets byte 0.  A
// block that holds an infinity or NaN gets byte 0xFF, the UE8M0 NaN, so every
// output it enters is NaN.  A power of two costs a floating-point element
// grid no precision, makes the dequantized value exact in bf16 (an E4M3 value
// has four significant bits), and lets the scaled MFMA apply it.
#include "b128.hpp"

namespace mxfp8 {

// Row-major: x [M, K] -> q [M, K], s [M, P], P = ceil(K / 128).  Sixteen
// consecutive lanes own one block, 16 bytes of bf16 each; a row takes 16 P
// lanes, those past K (K % 16 == 0) hold zeros and store nothing.  HBM-bound:
// 2 bytes read and 1 + 1/128 written per element.  8192 x 8192: 31 us (6.4 TB/s,
// part of x still cached from the call before).
__global__ __launch_bounds__(256) void quant_act_b128_kernel(const uint16_t* __restrict__ x, int64_t ldx, int64_t K,
                                                             int64_t lanes_per_row, int64_t total,
                                                             uint8_t* __restrict__ q, int64_t ldq,
                                                             uint8_t* __restrict__ s, int64_t lds) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= total) return;   // total is a multiple of 16: whole blocks leave
  const int64_t row = t / lanes_per_row, c = t - row * lanes_per_row;
  const bool in = c * 8 < K;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (in) v = *reinterpret_cast<const uint4*>(x + row * ldx + c * 8);
  const uint32_t sb = b128_scale_byte(row16_max(absmax8(v)));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t qd[2];
  cvt8s(w, mx_scale_value(sb), qd);
  if (in) *reinterpret_cast<uint2*>(q + row * ldq + c * 8) = make_uint2(qd[0], qd[1]);
  if ((c & 15) == 0) s[row * lds + (c >> 4)] = (uint8_t)sb;
}

int launch_quantize_b128(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, int64_t ldq, void* s, int64_t lds,
                         hipStream_t stream) {
  const int64_t lanes = b128_blocks(K) * 16, total = M * lanes;
  hipLaunchKernelGGL(quant_act_b128_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, stream,
                     (const uint16_t*)x, ldx, K, lanes, total, (uint8_t*)q, ldq, (uint8_t*)s, lds);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

// The packed operand layout of common.hpp (rows padded to 128, K to 128; pad
// elements zero, pad rows' scale byte 0): the byte of a 128-block is written
// four times, once for each of its 32-blocks, so the layout is the MX one and
// every reader of packed activations takes it.  A workgroup owns one 16-row
// band and SPW consecutive 64-K steps, staged in LDS and written as one
// contiguous run of SPW KiB.  HBM-bound: 8192 x 8192 47 us (4.3 TB/s).
template <int SPW>
__global__ __launch_bounds__(256) void quant_act_packed_b128_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                    int64_t M, int64_t K, int64_t KS, int64_t nsg,
                                                                    uint8_t* __restrict__ qp,
                                                                    uint8_t* __restrict__ sp) {
  constexpr int kLanesPerRow = SPW * 8;   // 8 elements per lane; a block is 16 lanes
  constexpr int kRowsPerWave = 64 / kLanesPerRow;
  __shared__ __attribute__((aligned(16))) uint8_t buf[SPW * kPieceBytes];
  const int64_t band = (int64_t)blockIdx.x / nsg;
  const int64_t s0 = ((int64_t)blockIdx.x - band * nsg) * SPW;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane % kLanesPerRow;
  const int s = l >> 3, c16 = (l & 7) >> 1, half = l & 1;
  const int64_t g = band >> 3;
  const int64_t k0 = s0 * kStepK + l * 8;
#pragma unroll
  for (int pass = 0; pass < 16 / (4 * kRowsPerWave); ++pass) {
    const int rb = (pass * 4 + wave) * kRowsPerWave + lane / kLanesPerRow;
    const int64_t row = band * 16 + rb;
    const int r = (int)(row & (kGroupRows - 1));
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (row < M && k0 < K) v = *reinterpret_cast<const uint4*>(x + row * ldx + k0);
    const uint32_t sb = b128_scale_byte(row16_max(absmax8(v)));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t qd[2];
    cvt8s(w, mx_scale_value(sb), qd);
    *reinterpret_cast<uint2*>(buf + s * kPieceBytes + rb * kStepK + ((c16 ^ swz(r)) << 4) + half * 8) =
        make_uint2(qd[0], qd[1]);
    if ((l & 3) == 0) sp[(g * KS + s0 + s) * kTileScaleBytes + scale_off(r, (l >> 2) & 1)] = (uint8_t)sb;
  }
  __syncthreads();
  uint8_t* dst = qp + g * KS * kTileBytes + ((band & 7) * KS + s0) * kPieceBytes;
#pragma unroll
  for (int o = tid * 16; o < SPW * kPieceBytes; o += 256 * 16)
    *reinterpret_cast<uint4*>(dst + o) = *reinterpret_cast<const uint4*>(buf + o);
}

int launch_quantize_packed_b128(const void* x, int64_t M, int64_t K, int64_t ldx, void* qp, void* sp,
                                hipStream_t stream) {
  const int64_t KS = b128_blocks(K) * 2, bands = b128_blocks(M) * 8;
  auto go = [&](auto kern, int spw) {
    hipLaunchKernelGGL(kern, dim3((unsigned)(bands * (KS / spw))), dim3(256), 0, stream, (const uint16_t*)x, ldx, M,
                       K, KS, KS / spw, (uint8_t*)qp, (uint8_t*)sp);
  };
  // Longer runs per workgroup where they divide K and still leave the chip
  // over a thousand workgroups (the rule of the MX quantizer).
  if (KS % 8 == 0 && bands * (KS / 8) >= 1024) go(quant_act_packed_b128_kernel<8>, 8);
  else if (KS % 4 == 0 && bands * (KS / 4) >= 1024) go(quant_act_packed_b128_kernel<4>, 4);
  else go(quant_act_packed_b128_kernel<2>, 2);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

// Packed activations (either scale block) -> bf16 [M, K]: element times its
// power of two, exact in bf16 for scale bytes 9 .. 246 (outside, a product can
// leave bf16's normal range).  One thread per 16-byte chunk of the real rows
// and columns; four consecutive lanes read one 64-byte row of a piece.
// HBM-bound: 8192 x 8192 42 us (4.9 TB/s).
__global__ __launch_bounds__(256) void dequant_packed_kernel(const uint8_t* __restrict__ qp,
                                                             const uint8_t* __restrict__ sp, int64_t K, int64_t KS,
                                                             int64_t chunks, int64_t total,
                                                             uint16_t* __restrict__ x, int64_t ldx) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= total) return;
  const int64_t row = t / chunks, k = (t - row * chunks) * 16, g = row >> 7, ks = k >> 6;
  const int r = (int)(row & 127), c = (int)(k >> 4) & 3;
  const uint4 q = *reinterpret_cast<const uint4*>(qp + g * KS * kTileBytes + packed_off(r, ks, c, KS));
  uint4 d[2];
  widen16(q, b128_scale_value(sp[(g * KS + ks) * kTileScaleBytes + scale_off(r, c >> 1)]), d);
  uint4* o = reinterpret_cast<uint4*>(x + row * ldx + k);
  o[0] = d[0];
  o[1] = d[1];
}

int launch_dequantize_packed(const void* qp, const void* sp, int64_t M, int64_t K, void* x, int64_t ldx,
                             hipStream_t stream) {
  const int64_t chunks = K / 16, total = M * chunks;
  hipLaunchKernelGGL(dequant_packed_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, stream,
                     (const uint8_t*)qp, (const uint8_t*)sp, K, 2 * b128_blocks(K), chunks, total, (uint16_t*)x, ldx);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

// ---------------------------------------------------------------------------
// Weights.  One workgroup per 128 x 128 tile: the tile's E4M3 bytes go through
// LDS (row-major, pitch 144 so that a column walk spreads over the banks), and
// from there to any of: the row-major bytes, the packed layout, and the packed
// layout of the transposed weight, with the block's scale at [nb][kb] resp.
// [kb][nb].  Pad rows and columns are zero.
// ---------------------------------------------------------------------------
namespace {

constexpr int kTilePitch = 144;

// Tile bytes in LDS -> packed chunks.  Chunk j (0..1023): row j / 8 of the
// operand's 128-row group, 16 bytes at contraction offset 16 (j % 8).  The
// operand's row is the tile's row (kT = false) or column (kT = true).
template <bool kT>
__device__ inline void store_packed_tile(const uint8_t* t, uint8_t* wp, int64_t group, int64_t block, int64_t KS) {
  uint8_t* dst = wp + group * KS * kTileBytes;
  for (int j = threadIdx.x; j < 1024; j += 256) {
    // Consecutive lanes take consecutive operand rows where that walks the
    // LDS rows' bytes in order (kT), else consecutive chunks of one row.
    const int r = kT ? j & 127 : j >> 3, c = kT ? j >> 7 : j & 7;
    uint4 v;
    if constexpr (!kT) {
      v = *reinterpret_cast<const uint4*>(t + r * kTilePitch + c * 16);
    } else {
      uint32_t d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t* p = t + (c * 16 + 4 * e) * kTilePitch + r;
        d[e] = (uint32_t)p[0] | (uint32_t)p[kTilePitch] << 8 | (uint32_t)p[2 * kTilePitch] << 16 |
               (uint32_t)p[3 * kTilePitch] << 24;
      }
      v = make_uint4(d[0], d[1], d[2], d[3]);
    }
    const int64_t ks = 2 * block + (c >> 2);
    *reinterpret_cast<uint4*>(dst + packed_off(r, ks, c & 3, KS)) = v;
  }
}

}  // namespace

// E4M3 bytes [N, K] + fp32 scales [nb, kb] -> packed (wp, sp) of W or W^T.
__global__ __launch_bounds__(256) void pack_b128_kernel(const uint8_t* __restrict__ w, int64_t ldw,
                                                        const float* __restrict__ ws, int64_t ldws, int64_t N,
                                                        int64_t K, int64_t NB, int64_t KB, int transpose,
                                                        uint8_t* __restrict__ wp, float* __restrict__ sp) {
  __shared__ __attribute__((aligned(16))) uint8_t t[128 * kTilePitch];
  const int64_t nb = (int64_t)blockIdx.x / KB, kb = (int64_t)blockIdx.x - nb * KB;
  for (int j = threadIdx.x; j < 1024; j += 256) {
    const int r = j >> 3, c = j & 7;
    const int64_t n = nb * 128 + r, k = kb * 128 + c * 16;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (n < N && k < K) v = *reinterpret_cast<const uint4*>(w + n * ldw + k);
    *reinterpret_cast<uint4*>(t + r * kTilePitch + c * 16) = v;
  }
  __syncthreads();
  const float s = ws[nb * ldws + kb];
  if (transpose) {
    store_packed_tile<true>(t, wp, kb, nb, 2 * NB);
    if (threadIdx.x == 0) sp[kb * NB + nb] = s;
  } else {
    store_packed_tile<false>(t, wp, nb, kb, 2 * KB);
    if (threadIdx.x == 0) sp[nb * KB + kb] = s;
  }
}

int launch_pack_b128(const void* w, const void* ws, int64_t N, int64_t K, int64_t ldw, int64_t ldws, int transpose,
                     void* wp, void* sp, hipStream_t stream) {
  const int64_t NB = b128_blocks(N), KB = b128_blocks(K);
  hipLaunchKernelGGL(pack_b128_kernel, dim3((unsigned)(NB * KB)), dim3(256), 0, stream, (const uint8_t*)w, ldw,
                     (const float*)ws, ldws, N, K, NB, KB, transpose, (uint8_t*)wp, (float*)sp);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

// bf16 [N, K] -> any of: row-major bytes (q) and scales (s); packed W
// (wp, sp); packed W^T (wtp, stp).  Null outputs are skipped.  One read of
// the weight serves them all.  mx: bit 0 / 1: sp / stp is in the scale tiles
// of the MX format instead of one fp32 per block: the block's two tiles hold
// its byte throughout.  HBM-bound: 4096 x 4096 to both packed forms
// 16 us (4.2 TB/s).
__global__ __launch_bounds__(256) void quant_weight_b128_kernel(const uint16_t* __restrict__ w, int64_t ldw, int64_t N,
                                                                int64_t K, int64_t NB, int64_t KB,
                                                                uint8_t* __restrict__ q, int64_t ldq,
                                                                float* __restrict__ s, int64_t lds,
                                                                uint8_t* __restrict__ wp, void* __restrict__ sp,
                                                                uint8_t* __restrict__ wtp, void* __restrict__ stp,
                                                                int mx) {
  __shared__ __attribute__((aligned(16))) uint8_t t[128 * kTilePitch];
  __shared__ uint32_t wmax[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t nb = (int64_t)blockIdx.x / KB, kb = (int64_t)blockIdx.x - nb * KB;
  const int c = tid & 15;
  const int64_t k = kb * 128 + c * 8;
  uint4 v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = nb * 128 + (tid >> 4) + 16 * i;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (n < N && k < K) v[i] = *reinterpret_cast<const uint4*>(w + n * ldw + k);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, absmax8(v[i]));
  m = row16_max(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  if (lane == 0) wmax[wave] = m;
  __syncthreads();
  m = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const uint32_t sb = b128_scale_byte(m);
  const float scale = b128_scale_value(sb);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = (tid >> 4) + 16 * i;
    const uint32_t e[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t qd[2];
    cvt8s(e, mx_scale_value(sb), qd);
    *reinterpret_cast<uint2*>(t + r * kTilePitch + c * 8) = make_uint2(qd[0], qd[1]);
    const int64_t n = nb * 128 + r;
    if (q != nullptr && n < N && k < K) *reinterpret_cast<uint2*>(q + n * ldq + k) = make_uint2(qd[0], qd[1]);
  }
  if (tid == 0) {
    if (s != nullptr) s[nb * lds + kb] = scale;
    if (wp != nullptr && !(mx & 1)) ((float*)sp)[nb * KB + kb] = scale;
    if (wtp != nullptr && !(mx & 2)) ((float*)stp)[kb * NB + nb] = scale;
  }
  if (tid < 2 * kTileScaleBytes / 4) {
    const uint32_t four = sb * 0x01010101u;
    if (wp != nullptr && (mx & 1)) ((uint32_t*)sp)[(nb * KB + kb) * (2 * kTileScaleBytes / 4) + tid] = four;
    if (wtp != nullptr && (mx & 2)) ((uint32_t*)stp)[(kb * NB + nb) * (2 * kTileScaleBytes / 4) + tid] = four;
  }
  if (wp == nullptr && wtp == nullptr) return;
  __syncthreads();
  if (wp != nullptr) store_packed_tile<false>(t, wp, nb, kb, 2 * KB);
  if (wtp != nullptr) store_packed_tile<true>(t, wtp, kb, nb, 2 * NB);
}

int launch_quantize_weight_b128(const void* w, int64_t N, int64_t K, int64_t ldw, void* q, int64_t ldq, void* s,
                                int64_t lds, void* wp, void* sp, void* wtp, void* stp, int mx, hipStream_t stream) {
  const int64_t NB = b128_blocks(N), KB = b128_blocks(K);
  hipLaunchKernelGGL(quant_weight_b128_kernel, dim3((unsigned)(NB * KB)), dim3(256), 0, stream, (const uint16_t*)w,
                     ldw, N, K, NB, KB, (uint8_t*)q, ldq, (float*)s, lds, (uint8_t*)wp, sp, (uint8_t*)wtp, stp, mx);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace mxfp8
