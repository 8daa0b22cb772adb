// Few rows against a packed MXFP4 weight (the dense layer's M <= 128, and the
// experts' rows of a small batch), up to 32 and the experts' quantized to MXFP4
// inside.
//
// Bound by the weight's way from HBM, and at small weights by the launch and
// the chain of dependent loads.  One workgroup owns blocks of 16 weight rows over
// the whole K, each of its waves (16 where K is long) a run of 128-K steps; the
// partial sums are added through LDS in K order.  A lane of the 4-bit 16x16x128
// MFMA holds K [32g, 32g + 32) of its row, one MX block, but 64 bytes per lane
// would touch a cache line per four lanes: the rows are read and quantized
// sixteen lanes to a row's 256 bytes, and the codes, a quarter of that, change
// lanes through LDS (16 x 4096 x 4096: 6.2 us; each lane its own block 8.5; 1 row
// 4.3 and 4.5).  In a graph of such calls 1 x 4096 x 4096 takes 4.0 us, of which
// about 2.8 are the launch; 1 x 16384 x 8192 14.6, 4.9 TB/s; one token's eight
// experts, 1536 x 2048, 7.4, 1.8 TB/s.  The 16-row form below, 32 x 16384 x 8192:
// 23.8 us with the quantizer, 3.0 TB/s.
//
// Experts: the j-th run of workgroups has the j-th expert that has rows, and all
// of those, 16 at a time.
#include <algorithm>

#include "fp4.hpp"

namespace mxfp8 {

namespace {

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
  // experts
  int R, E, topk, x_rows;
  int runs;                // workgroups of an expert
  const int* slots;
  const int* offsets;
};

// The waves' partial sums of a lane, in K order; kBatch of them in flight.
template <int kWaves, int kBatch = kWaves>
__device__ inline v4f sum_waves(const v4f* red, int lane) {
  v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k0 = 0; k0 < kWaves; k0 += kBatch) {
    v4f part[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) part[k] = red[(k0 + k) * 64 + lane];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) v += part[k];
  }
  return v;
}

// Columns n .. n + 3 of output row m.
__device__ inline void store4(const DecodeArgs& p, const v4f& v, const float* bv, int m, int row_end, int n) {
  if (m >= row_end || n >= p.N) return;
  const uint32_t lo = pack_bf16x2(v[0] + bv[0], v[1] + bv[1]);
  const uint32_t hi = pack_bf16x2(v[2] + bv[2], v[3] + bv[3]);
  uint16_t* yr = p.y + (size_t)m * p.ldy + n;
  typedef uint32_t u2a2 __attribute__((ext_vector_type(2), aligned(2)));   // (the hardware serves any address)
  if (n + 3 < p.N) {
    *reinterpret_cast<u2a2*>(yr) = u2a2{lo, hi};
  } else {
    yr[0] = (uint16_t)lo;
    if (n + 1 < p.N) yr[1] = (uint16_t)(lo >> 16);
    if (n + 2 < p.N) yr[2] = (uint16_t)hi;
    if (n + 3 < p.N) yr[3] = (uint16_t)(hi >> 16);
  }
}

}  // namespace

// kSteps: the most steps a wave owns; kGroups: 16-row groups in flight together
// (experts: one).  kDepth: 1 for workgroups of one block of 16 weight rows; more
// for such with a run of blocks, that many in flight, where a turn of the chip does
// not hold all blocks: the rows are quantized once for the run, and the weight
// streams while sums are joined (16 rows, 16384 x 8192: 16.4 us, one block each
// 32.6; 1 row 14.0 and 19.4; 16 rows, 8192 x 4096 7.1 and 9.1; eight experts of 2048
// x 7168 15.1 and 22.7; but 1 row, 4096 x 4096, 5.0 and 3.8: more registers, later
// rows; near the border 1 row, 16384 x 2048, 5.3 and 4.8).
template <int kWaves, int kSteps, int kGroups, int kDepth, bool kExperts>
__global__ __launch_bounds__(64 * kWaves, kDepth > 1 || kSteps > 2 || kGroups > 1 ? 4 : 7) void gemm_fp4_decode_kernel(DecodeArgs p) {
  __shared__ v4f red[2][kGroups][kWaves * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int KS = p.K / 128;
  const int kb = KS * wave / kWaves, nsteps = KS * (wave + 1) / kWaves - kb;

  const int blocks = (p.N + 15) / 16;
  int row0 = 0, row_end = p.M, run, runs;   // this workgroup's run of so many
  int64_t group0 = 0;                       // the expert's first 128-row group
  if constexpr (kExperts) {
    runs = p.runs;
    const int j = (int)blockIdx.x / runs;
    run = (int)blockIdx.x - j * runs;
    zero_rows(p.y, p.ldy, max(p.offsets[p.E], 0), p.R, p.N, kWaves);
    int at = j, e = -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = 64 * u + lane;
      const int first = max(p.offsets[min(c, p.E)], 0), last = min(p.offsets[min(c + 1, p.E)], p.R);
      const uint64_t m = __ballot(last > first);
      const int n = __popcll(m);
      if (e < 0) {
        if (at < n) {
          const bool mine = ((m >> lane) & 1) && __popcll(m & ((1ull << lane) - 1ull)) == at;
          const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(mine)) - 1);
          e = 64 * u + l;
          row0 = __builtin_amdgcn_readlane(first, l);
          row_end = __builtin_amdgcn_readlane(last, l);
        } else {
          at -= n;
        }
      }
    }
    if (e < 0) return;                       // (fewer experts with rows than workgroups)
    group0 = (int64_t)e * ((p.N + kGroupRows - 1) / kGroupRows);
  } else {
    runs = (int)gridDim.x;
    // Dies take contiguous runs of blocks.
    run = xcd_remap((int)blockIdx.x, runs);
  }
  // (at most 2^20 blocks and 2^11 runs)
  const int b0 = kDepth == 1 ? run : (int)((uint32_t)blocks * (uint32_t)run / (uint32_t)runs);
  const int b1 = kDepth == 1 ? run + 1 : (int)((uint32_t)blocks * (uint32_t)(run + 1) / (uint32_t)runs);

  // A block's weight: chunk g of row i and the scale of MX block g for each step;
  // and the bias of columns 4 g .. 4 g + 3, by whole words (an odd N's last word
  // holds one value that is not the bias's and reaches no output).
  struct Block {
    uint4 w[kSteps];
    int s[kSteps];
    uint32_t bias[2];
  };
  auto load_block = [&](Block& f, int b) {
    const int n0 = min(b, b1 - 1) * 16, r = n0 % kGroupRows + i;
    const int64_t group = group0 + n0 / kGroupRows;
    const uint8_t* wrow = p.wp + (size_t)group * KS * kTileBytes + packed_off(r, 0, g, KS);
    const uint8_t* srow = p.wsp + (size_t)group * KS * 2 * kTileScaleBytes + (g >> 1) * kTileScaleBytes + scale_off(r, g & 1);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int ks = min(kb + u, KS - 1);
      f.w[u] = *reinterpret_cast<const uint4*>(wrow + (size_t)ks * kPieceBytes);
      f.s[u] = srow[(size_t)ks * 2 * kTileScaleBytes];
    }
    if (!kExperts && p.bias != nullptr) {
      const uint32_t* words = reinterpret_cast<const uint32_t*>(p.bias);
#pragma unroll
      for (int e = 0; e < 2; ++e) f.bias[e] = words[min(n0 / 2 + 2 * g + e, (p.N - 1) / 2)];
    } else {
      f.bias[0] = f.bias[1] = 0u;
    }
  };
  // 16 kGroups rows from m0 on, quantized: lane (i, g) ends with block g of row m0
  // + i.  Sixteen lanes read the 256 bytes of a row's step, and the codes of 16
  // rows go through this wave's part of `red` (a wave's LDS accesses run in their
  // order).  A step past the wave's run is zeros; of rows past the last, four at a
  // time, what was in LDS stays (their columns are not stored).
  int xq[kGroups][kSteps][4], xs[kGroups][kSteps];
  constexpr int kPart = kDepth > 1 && kSteps > 2 ? 2 : kSteps;   // steps at a time (registers)
  auto load_rows = [&](int m0) {
    const int l = lane & 15, rr = lane >> 4;
    int mine[kGroups];                       // the x row of sorted row m0 + 16 t + i
    if constexpr (kExperts) {
#pragma unroll
      for (int t = 0; t < kGroups; ++t)
        if (p.slots != nullptr)
          mine[t] = (int)min((uint32_t)p.slots[min(m0 + 16 * t + i, row_end - 1)] / (uint32_t)p.topk, (uint32_t)p.x_rows - 1u);
    }
    uint8_t* const stage = reinterpret_cast<uint8_t*>(&red[0][0][wave * 64]);
    uint8_t* const scales = reinterpret_cast<uint8_t*>(&red[1][0][wave * 64]);
#pragma unroll
    for (int u0 = 0; u0 < kSteps; u0 += kPart) {
      uint4 v[kGroups][kPart][4];
#pragma unroll
      for (int t = 0; t < kGroups; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (m0 + 16 * t + 4 * r >= row_end) break;
          const bool in = m0 + 16 * t + 4 * r + rr < row_end;
          const int64_t row = kExperts && p.slots != nullptr ? __shfl(mine[t], 4 * r + rr) : m0 + 16 * t + 4 * r + rr;
          const uint16_t* xr = p.x + row * p.ldx + (int64_t)(kb + u0) * 128 + l * 8;
#pragma unroll
          for (int u = 0; u < kPart; ++u)
            v[t][u][r] = in && u0 + u < nsteps ? *reinterpret_cast<const uint4*>(xr + u * 128) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
      for (int t = 0; t < kGroups; ++t)
#pragma unroll
        for (int u = 0; u < kPart; ++u) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (m0 + 16 * t + 4 * r >= row_end) break;
            const uint32_t sb = fp4_scale_byte(quad_max(fp4_absmax8(v[t][u][r])));
            reinterpret_cast<uint32_t*>(stage)[r * 64 + lane] = cvt8_fp4(v[t][u][r], fp4_scale_value(sb));
            if ((l & 3) == 0) scales[(4 * r + rr) * 4 + (l >> 2)] = (uint8_t)sb;
          }
          asm volatile("" ::: "memory");
          const uint4 q = reinterpret_cast<const uint4*>(stage)[i * 4 + g];
          xq[t][u0 + u][0] = (int)q.x;
          xq[t][u0 + u][1] = (int)q.y;
          xq[t][u0 + u][2] = (int)q.z;
          xq[t][u0 + u][3] = (int)q.w;
          xs[t][u0 + u] = scales[i * 4 + g];
          asm volatile("" ::: "memory");
        }
    }
  };

  // The weight first: with gathered rows the others wait for their indices.
  Block f[kDepth];
  if constexpr (kDepth == 1) load_block(f[0], b0);
  for (int m0 = row0; m0 < row_end; m0 += 16 * kGroups) {
#pragma unroll
    for (int d = 0; d < kDepth - 1; ++d) load_block(f[d], b0 + d);
    __builtin_amdgcn_sched_barrier(0);
    load_rows(m0);
    for (int base = b0; base < b1; base += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int b = base + d;
        if (b >= b1) break;
        if constexpr (kDepth > 1) load_block(f[(d + kDepth - 1) % kDepth], b + kDepth - 1);
        v4f(&out)[kGroups][kWaves * 64] = red[kDepth == 1 ? 0 : (b - b0) & 1];
#pragma unroll
        for (int t = 0; t < kGroups; ++t) {
          v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int u = 0; u < kSteps; ++u) {
            const v8i bx = {xq[t][u][0], xq[t][u][1], xq[t][u][2], xq[t][u][3], 0, 0, 0, 0};
            const v8i aw = {(int)f[d].w[u].x, (int)f[d].w[u].y, (int)f[d].w[u].z, (int)f[d].w[u].w, 0, 0, 0, 0};
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(aw, bx, acc, 4, 4, 0, f[d].s[u], 0, xs[t][u]);
          }
          out[t][wave * 64 + lane] = acc;
        }
        // (one barrier per block: `out` is written again two blocks on, when
        // every wave has passed the next one)
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const int who = (wave - (b - b0)) & (kWaves - 1);   // the waves take turns
        if (who < kGroups) {
          const v4f v = sum_waves<kWaves, kDepth == 1 ? kWaves : 4>(out[who], lane);
          const float bv[4] = {bf16_lo(f[d].bias[0]), bf16_hi(f[d].bias[0]), bf16_lo(f[d].bias[1]), bf16_hi(f[d].bias[1])};
          store4(p, v, bv, m0 + 16 * who + i, row_end, b * 16 + 4 * g);   // D[n = 4g + e][m = i]
        }
      }
    }
    // (the last block's sums are read before the next rows' are written)
    if (kExperts && m0 + 16 * kGroups < row_end) __syncthreads();
  }
}

// 16 < M <= 128 rows, quantized beforehand into one packed 128-row group (the
// decode kernel's waves would each convert all of them again).  Waves and
// weight as there; per step a wave reads the kGroups 1 KiB pieces of the
// activations (L2) and runs an MFMA on each, the loads of the next kBatch
// steps in flight.
template <int kWaves, int kGroups, int kBatch>
__global__ __launch_bounds__(64 * kWaves) void gemm_fp4_mid_kernel(const uint8_t* __restrict__ qp,
                                                            const uint8_t* __restrict__ sp, DecodeArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  v4f* red = reinterpret_cast<v4f*>(smem);   // [kGroups][kWaves][64]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int KS = p.K / 128;
  const int kb = KS * wave / kWaves, ke = KS * (wave + 1) / kWaves;
  const int n0 = xcd_remap((int)blockIdx.x, (int)gridDim.x) * 16;
  const int r = n0 % kGroupRows + i;
  const int64_t group = n0 / kGroupRows;
  const uint8_t* wrow = p.wp + (size_t)group * KS * kTileBytes + packed_off(r, 0, g, KS);
  const uint8_t* srow = p.wsp + (size_t)group * KS * 2 * kTileScaleBytes + (g >> 1) * kTileScaleBytes + scale_off(r, g & 1);
  const uint8_t* xrow = qp + packed_off(i, 0, g, KS);                                   // + band * KS pieces
  const uint8_t* xsrow = sp + (g >> 1) * kTileScaleBytes + scale_off(i, g & 1);         // + 128 for odd bands
  struct Batch {
    uint4 w[kBatch], x[kBatch][kGroups];
    int ws[kBatch], xs[kBatch][2];
  };
  auto load = [&](Batch& f, int k) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int ks = min(k + u, KS - 1);
      f.w[u] = *reinterpret_cast<const uint4*>(wrow + (size_t)ks * kPieceBytes);
      f.ws[u] = srow[(size_t)ks * 2 * kTileScaleBytes];
#pragma unroll
      for (int t = 0; t < kGroups; ++t)
        f.x[u][t] = *reinterpret_cast<const uint4*>(xrow + ((size_t)t * KS + ks) * kPieceBytes);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        f.xs[u][e] = *reinterpret_cast<const int*>(xsrow + (size_t)ks * 2 * kTileScaleBytes + 128 * e);
    }
  };
  v4f acc[kGroups];
#pragma unroll
  for (int t = 0; t < kGroups; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const Batch& f, int k) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (k + u >= ke) continue;
      const v8i a = {(int)f.w[u].x, (int)f.w[u].y, (int)f.w[u].z, (int)f.w[u].w, 0, 0, 0, 0};
      // band t: word t % 2 of its lane's scales, byte t / 2
      tile::static_for<0, kGroups>([&](auto T) {
        constexpr int t = decltype(T)::value;
        const uint4 x = f.x[u][t];
        const v8i b = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[t], 4, 4, 0, f.ws[u], t >> 1, f.xs[u][t & 1]);
      });
    }
  };
  Batch f0, f1;
  load(f0, kb);
  const int n = n0 + 4 * g;
  float bv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.bias != nullptr && wave < kGroups) {
#pragma unroll
    for (int e = 0; e < 4; ++e) bv[e] = __uint_as_float((uint32_t)p.bias[min(n + e, p.N - 1)] << 16);
  }
  __builtin_amdgcn_sched_barrier(0);
  for (int k = kb; k < ke; k += 2 * kBatch) {
    if (k + kBatch < ke) load(f1, k + kBatch);
    multiply(f0, k);
    if (k + kBatch >= ke) break;
    if (k + 2 * kBatch < ke) load(f0, k + 2 * kBatch);
    multiply(f1, k + kBatch);
  }
#pragma unroll
  for (int t = 0; t < kGroups; ++t) red[(t * kWaves + wave) * 64 + lane] = acc[t];
  __syncthreads();
  if (wave < kGroups) store4(p, sum_waves<kWaves>(red + wave * kWaves * 64, lane), bv, 16 * wave + i, p.M, n);
}

namespace {
// parts: 1, or the experts with rows at most.
template <bool kExperts>
int decode(DecodeArgs p, int64_t parts, hipStream_t stream) {
  const int64_t blocks = (p.N + 15) / 16, cus = device_cu_count();
  auto go = [&](auto kern, int waves, int64_t runs) {
    p.runs = (int)runs;
    hipLaunchKernelGGL(kern, dim3((unsigned)(parts * runs)), dim3(64 * waves), 0, stream, p);
    return hipGetLastError() == hipSuccess ? 0 : -7;
  };
  // Workgroups with runs have 16 waves per compute unit.
  auto pick = [&](auto one, auto many, int waves) {
    if (blocks * parts <= cus * fp4_decode_per_cu(kExperts, p.M, p.K)) return go(one, waves, blocks);
    return go(many, waves, std::min(blocks, (cus * (16 / waves) + parts - 1) / parts));
  };
  static_assert(kFp4DecodeMaxK == 16 * 4 * 128, "a wave owns at most four steps");
  const int KS = p.K / 128;
  if constexpr (!kExperts) {
    if (p.M > 16) {
      if (KS <= 16) return pick(gemm_fp4_decode_kernel<16, 1, 2, 1, false>, gemm_fp4_decode_kernel<16, 1, 2, 4, false>, 16);
      return pick(gemm_fp4_decode_kernel<16, 2, 2, 1, false>, gemm_fp4_decode_kernel<16, 2, 2, 2, false>, 16);
    }
  }
  constexpr bool X = kExperts;
  if (KS <= 8) return pick(gemm_fp4_decode_kernel<4, 2, 1, 1, X>, gemm_fp4_decode_kernel<4, 2, 1, 3, X>, 4);
  if (KS <= 16) return pick(gemm_fp4_decode_kernel<8, 2, 1, 1, X>, gemm_fp4_decode_kernel<8, 2, 1, 3, X>, 8);
  if (KS <= 32) return pick(gemm_fp4_decode_kernel<16, 2, 1, 1, X>, gemm_fp4_decode_kernel<16, 2, 1, 3, X>, 16);
  return pick(gemm_fp4_decode_kernel<16, 4, 1, 1, X>, gemm_fp4_decode_kernel<16, 4, 1, 2, X>, 16);
}
template <int kWaves, int kGroups, int kBatch>
int mid(const void* qp, const void* sp, const DecodeArgs& p, hipStream_t stream) {
  constexpr int lds = kGroups * kWaves * 64 * 16;
  auto kern = gemm_fp4_mid_kernel<kWaves, kGroups, kBatch>;
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)kern, lds, lds_set)) return -7;
  hipLaunchKernelGGL(kern, dim3((unsigned)((p.N + 15) / 16)), dim3(64 * kWaves), lds, stream, (const uint8_t*)qp,
                     (const uint8_t*)sp, p);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}
}  // namespace

int launch_gemm_fp4_mid(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const void* wsp,
                        int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream) {
  DecodeArgs p = {};
  p.M = (int)M;
  p.K = (int)K;
  p.wp = (const uint8_t*)wp;
  p.wsp = (const uint8_t*)wsp;
  p.N = (int)N;
  p.bias = (const uint16_t*)bias;
  p.y = (uint16_t*)y;
  p.ldy = ldy;
  if (M <= 32) return mid<16, 2, 2>(qp, sp, p, stream);
  if (M <= 64) return mid<16, 4, 2>(qp, sp, p, stream);
  return mid<8, 8, 2>(qp, sp, p, stream);
}

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
  return decode<false>(p, 1, stream);
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
  p.R = (int)a.R;
  p.E = (int)a.E;
  p.topk = (int)a.topk;
  p.x_rows = (int)a.x_rows;
  p.slots = a.slots;
  p.offsets = a.offsets;
  return decode<true>(p, std::min(a.E, a.R), stream);
}

}  // namespace mxfp8
