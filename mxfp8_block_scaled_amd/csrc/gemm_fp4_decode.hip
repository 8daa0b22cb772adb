// Few rows against a packed MXFP4 weight (the dense layer's M <= 16, and the
// experts' rows of a small batch), the rows quantized to MXFP4 inside.
//
// Bound by the weight's way from HBM, and at small weights by the launch and
// the chain of dependent loads.  One workgroup owns 16 weight rows over the
// whole K, each of its 16 waves a run of 128-K steps; the 16 partial sums are
// added through LDS in K order.  A lane of the 4-bit 16x16x128 MFMA holds K
// [32g, 32g + 32) of its row, which is one MX block: lane (i, g) loads the 64
// bytes of that block of row i, finds its largest magnitude and converts it by
// itself, with no exchange between lanes and no staging.
//
// Experts: workgroup (n, j) takes weight rows 16 n .. of the j-th expert that
// has rows, and all of those, 16 at a time, against the weight it holds.
#include <algorithm>

#include "fp4.hpp"

namespace mxfp8 {

namespace {

constexpr int kWaves = 16;
constexpr int kThreads = 64 * kWaves;

struct DecodeArgs {
  const uint16_t* x;
  int64_t ldx;
  int M, K;
  const uint8_t* wp;
  const uint8_t* wsp;
  int N;
  const uint16_t* bias;
  uint16_t* y;
  int64_t ldy;
  int vec;                 // y 8-byte aligned, ldy % 4 == 0
  // experts
  int R, E, topk, x_rows;
  const int* slots;
  const int* offsets;
};

}  // namespace

template <int kSteps, bool kExperts>
__global__ __launch_bounds__(kThreads) void gemm_fp4_decode_kernel(DecodeArgs p) {
  __shared__ v4f red[kWaves * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int KS = p.K / 128;
  const int kb = KS * wave / kWaves, nsteps = KS * (wave + 1) / kWaves - kb;

  int row0 = 0, row_end = p.M, n0;
  int64_t group = 0;
  if constexpr (kExperts) {
    const int blocks = (p.N + 15) / 16;
    const int j = (int)blockIdx.x / blocks;
    n0 = ((int)blockIdx.x - j * blocks) * 16;
    const int kept = max(p.offsets[p.E], 0);
    {
      // Rows of slots without an expert: zeros.
      const int64_t n = (int64_t)(p.R - kept) * p.N, stride = (int64_t)gridDim.x * kThreads;
      for (int64_t z = (int64_t)blockIdx.x * kThreads + tid; z < n; z += stride) {
        const int64_t r = z / p.N;
        p.y[(kept + r) * p.ldy + (z - r * p.N)] = 0;
      }
    }
    int at = j, e = -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = 64 * u + lane;
      const uint64_t m = __ballot(p.offsets[min(c + 1, p.E)] > p.offsets[min(c, p.E)]);
      const int n = __popcll(m);
      if (e < 0) {
        if (at < n) {
          const bool mine = ((m >> lane) & 1) && __popcll(m & ((1ull << lane) - 1ull)) == at;
          e = 64 * u + __ffsll((unsigned long long)__ballot(mine)) - 1;
        } else {
          at -= n;
        }
      }
    }
    e = __builtin_amdgcn_readfirstlane(e);
    if (e < 0) return;                       // (fewer experts with rows than workgroups)
    row0 = __builtin_amdgcn_readfirstlane(max(p.offsets[e], 0));
    row_end = __builtin_amdgcn_readfirstlane(min(p.offsets[e + 1], p.R));
    group = (int64_t)e * ((p.N + kGroupRows - 1) / kGroupRows);
  } else {
    // Dies take contiguous runs of 16-row blocks.
    n0 = xcd_remap((int)blockIdx.x, (int)gridDim.x) * 16;
  }
  group += n0 / kGroupRows;
  const int r = n0 % kGroupRows + i;

  // The weight: chunk g of row r and the scale of block g for each step, all
  // in flight together with the first rows.
  const uint8_t* wrow = p.wp + (size_t)group * KS * kTileBytes + packed_off(r, 0, g, KS);
  const uint8_t* srow = p.wsp + (size_t)group * KS * 2 * kTileScaleBytes + (g >> 1) * kTileScaleBytes + scale_off(r, g & 1);
  uint4 xv[kSteps][4];
  auto load_rows = [&](int m0) {
    // Lane (i, g): block g of row m0 + i.  (A step past the wave's run, and a
    // row past the last, stay zero.)
    const int m = m0 + i;
    const bool in = m < row_end;
    int64_t row = in ? m : 0;
    if constexpr (kExperts) {
      if (p.slots != nullptr && in) row = min((uint32_t)p.slots[m] / (uint32_t)p.topk, (uint32_t)p.x_rows - 1u);
    }
    const uint16_t* xr = p.x + row * p.ldx + (int64_t)kb * 128 + g * 32;
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        xv[u][c] = in && u < nsteps ? *reinterpret_cast<const uint4*>(xr + u * 128 + c * 8) : make_uint4(0u, 0u, 0u, 0u);
  };
  load_rows(row0);
  uint4 w[kSteps];
  int wsc[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int ks = min(kb + u, KS - 1);
    w[u] = *reinterpret_cast<const uint4*>(wrow + (size_t)ks * kPieceBytes);
    wsc[u] = srow[(size_t)ks * 2 * kTileScaleBytes];
  }
  const int n = n0 + 4 * g;
  float bv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.bias != nullptr && wave == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) bv[e] = __uint_as_float((uint32_t)p.bias[min(n + e, p.N - 1)] << 16);
  }
  __builtin_amdgcn_sched_barrier(0);

  for (int m0 = row0; m0 < row_end; m0 += 16) {
    if (m0 != row0) load_rows(m0);
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      uint32_t m = fp4_absmax8(xv[u][0]);
#pragma unroll
      for (int c = 1; c < 4; ++c) m = max(m, fp4_absmax8(xv[u][c]));
      const uint32_t sb = fp4_scale_byte(m);
      const float scale = fp4_scale_value(sb);
      v8i b = {(int)cvt8_fp4(xv[u][0], scale), (int)cvt8_fp4(xv[u][1], scale), (int)cvt8_fp4(xv[u][2], scale),
               (int)cvt8_fp4(xv[u][3], scale), 0, 0, 0, 0};
      v8i a = {(int)w[u].x, (int)w[u].y, (int)w[u].z, (int)w[u].w, 0, 0, 0, 0};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, 0, wsc[u], 0, (int)sb);
    }
    red[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave == 0) {
      v4f part[kWaves];
#pragma unroll
      for (int k = 0; k < kWaves; ++k) part[k] = red[k * 64 + lane];
      acc = part[0];
#pragma unroll
      for (int k = 1; k < kWaves; ++k) acc += part[k];
      // D[n = 4g + e][m = i]
      if (m0 + i < row_end && n < p.N) {
        const uint32_t lo = pack_bf16x2(acc[0] + bv[0], acc[1] + bv[1]);
        const uint32_t hi = pack_bf16x2(acc[2] + bv[2], acc[3] + bv[3]);
        uint16_t* yr = p.y + (size_t)(m0 + i) * p.ldy + n;
        if (p.vec && n + 3 < p.N) {
          *reinterpret_cast<uint2*>(yr) = make_uint2(lo, hi);
        } else {
          yr[0] = (uint16_t)lo;
          if (n + 1 < p.N) yr[1] = (uint16_t)(lo >> 16);
          if (n + 2 < p.N) yr[2] = (uint16_t)hi;
          if (n + 3 < p.N) yr[3] = (uint16_t)(hi >> 16);
        }
      }
    }
    if constexpr (kExperts) __syncthreads();   // red is written again
  }
}

namespace {
template <bool kExperts>
int decode(const DecodeArgs& p, int64_t blocks, hipStream_t stream) {
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
  };
  static_assert(kFp4DecodeMaxK == kWaves * 4 * 128, "a wave owns at most four steps");
  if (p.K <= kWaves * 128) return go(gemm_fp4_decode_kernel<1, kExperts>);
  if (p.K <= kWaves * 2 * 128) return go(gemm_fp4_decode_kernel<2, kExperts>);
  return go(gemm_fp4_decode_kernel<4, kExperts>);
}
}  // namespace

int launch_gemm_fp4_decode(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const void* wsp,
                           int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream) {
  DecodeArgs p = {};
  p.x = (const uint16_t*)x;
  p.ldx = ldx;
  p.M = (int)M;
  p.K = (int)K;
  p.wp = (const uint8_t*)wp;
  p.wsp = (const uint8_t*)wsp;
  p.N = (int)N;
  p.bias = (const uint16_t*)bias;
  p.y = (uint16_t*)y;
  p.ldy = ldy;
  p.vec = ldy % 4 == 0 && ((uintptr_t)y & 7) == 0;
  return decode<false>(p, (N + 15) / 16, stream);
}

int launch_experts_fp4_decode(const ExpertsArgs& a, hipStream_t stream) {
  DecodeArgs p = {};
  p.x = (const uint16_t*)a.x;
  p.ldx = a.ldx;
  p.K = (int)a.K;
  p.wp = (const uint8_t*)a.wp;
  p.wsp = (const uint8_t*)a.wsp;
  p.N = (int)a.N;
  p.y = (uint16_t*)a.y;
  p.ldy = a.ldy;
  p.vec = a.ldy % 4 == 0 && ((uintptr_t)a.y & 7) == 0;
  p.R = (int)a.R;
  p.E = (int)a.E;
  p.topk = (int)a.topk;
  p.x_rows = (int)a.x_rows;
  p.slots = a.slots;
  p.offsets = a.offsets;
  return decode<true>(p, (a.N + 15) / 16 * std::min(a.E, a.R), stream);
}

}  // namespace mxfp8
