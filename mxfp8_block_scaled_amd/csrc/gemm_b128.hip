// FP8 GEMM with one scale for each block of 128:
//   y[m, n] = bf16( sum_b  W[n/128, b] * ( s[m, b] * sum_{k in b} q[m, k] w[n, k] ) + bias[n] )
// E4M3 elements; s a power of two per 1 x 128 block of the activations,
// W an fp32 scale per 128 x 128 block of the weight.
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 covers exactly one block along K, and
// the scaled MFMA applies s by itself (the packed activations carry its byte).
// W's mantissa it cannot apply, so every MFMA starts from a zero accumulator
// and its four results per lane are added with v_fma under the block's
// weight scale, which one 128-row weight group shares: the scale is a scalar
// register.  Four v_fma (16 cycles) against one MFMA (32 cycles) fit in the
// MFMA's shadow; the price is that the accumulators have to be ordinary
// vector registers, half of the register file.
//
// Precision: between blocks everything is fp32.  Inside a block the sum is the
// scaled MFMA's own, measured off by up to 2^-12 of its largest product, which
// is coarser than fp32 and finer than the E4M3 operands (2^-4) and the bf16
// output.  s times that sum is an fp32 number before W is applied: activations
// above about 2^111 can overflow there though the product with a small W would not.
#include "b128.hpp"
#include "tile_core.hpp"

namespace mxfp8 {

namespace {

constexpr int kUnitScales = 0x7F7F7F7F;   // UE8M0 1.0 in every byte

// A weight scale through the scalar cache (the scales are constant while a
// kernel runs, which the address space says).  Through the vector memory the
// compiler's wait for it would drain every copy in flight behind it.
__device__ inline float scalar_scale(const float* p, int at) {
  return ((const __attribute__((address_space(4))) float*)p)[at];
}

}  // namespace

// ---------------------------------------------------------------------------
// Decode (M <= 32): a workgroup owns 16 weight rows over the whole K, its 16
// waves one run of 128-blocks each; activations are quantized on the way in.
// Bound by the weight's bytes (N K) and how many loads are in flight; the
// waves' sums meet once, in wave order, through LDS.  One block at a time: two
// or four per turn keep half the registers of two workgroups per compute unit
// busy (16 x 2048 x 2048: 6.2 us against 4.8; 8 x 8192 x 8192: 16.5, 13.7), and
// so does loading a block ahead (15.5).
// M = 1, N = K = 4096: 4.8 us (3.5 TB/s); 13 x 4000 x 2064: 6.0 us; 32 x 4096 x
// 4096: 9.5 (traced, in steady calls).
// ---------------------------------------------------------------------------
namespace {
constexpr int kDecWaves = 16;
constexpr int kDecThreads = 64 * kDecWaves;
}  // namespace

// kMG groups of sixteen activation rows; a wave stages one at a time.
template <int kMG>
struct DecodeLds {
  static constexpr int kChunksRow = 16;             // 16-byte bf16 chunks per row of a block
  static constexpr int kPitch = 128 + 16;           // staged E4M3 row (+16: rows on distinct banks)
  static constexpr int kWave = 16 * kPitch + 16;
  static constexpr int kRed = kMG * kDecWaves * 64 * 16;
  static constexpr int kBytes = kRed + kDecWaves * kWave;
};

template <int kMG>
__global__ __launch_bounds__(kDecThreads) void gemm_b128_decode_kernel(
    const uint16_t* __restrict__ x, int64_t ldx, int M, int64_t K, const uint8_t* __restrict__ wp,
    const float* __restrict__ wsc, int N, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t ldy,
    int vec_store) {
  using L = DecodeLds<kMG>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  v4f* red = reinterpret_cast<v4f*>(smem);
  uint8_t* xq = smem + L::kRed + wave * L::kWave;
  uint8_t* xs = xq + 16 * L::kPitch;
  const int n0 = xcd_remap((int)blockIdx.x, (int)gridDim.x) * 16;
  const int grp = n0 / kGroupRows, r = (n0 % kGroupRows) + i;
  const int KB = (int)((K + 127) / 128), KS = 2 * KB;
  const int kb = (int)((int64_t)KB * wave / kDecWaves), ke = (int)((int64_t)KB * (wave + 1) / kDecWaves);

  const __amdgpu_buffer_rsrc_t brsrc = raw_rsrc(bias, (bias != nullptr && wave < kMG) ? (uint32_t)N * 2u : 0u);
  uint32_t braw[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    braw[e] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(brsrc, (uint32_t)min(n0 + 4 * g + e, N - 1) * 2u, 0, 0);

  const uint8_t* wrow = wp + (size_t)grp * KS * kTileBytes + packed_off(r, 0, g, KS);
  const float* wsg = wsc + (size_t)grp * KB;
  v4f acc[kMG];
#pragma unroll
  for (int h = 0; h < kMG; ++h) acc[h] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int u = kb; u < ke; ++u) {
    uint4 xa[4];   // a row group's block: sixteen lanes own a row of it
    auto load_x = [&](int h) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        xa[q] = make_uint4(0u, 0u, 0u, 0u);
        const int row = 16 * h + 4 * q + (lane >> 4);
        const int64_t k = (int64_t)u * 128 + (lane & 15) * 8;
        if (row < M && k < K) xa[q] = *reinterpret_cast<const uint4*>(x + (size_t)row * ldx + k);
      }
    };
    load_x(0);
    const uint8_t* wt = wrow + (size_t)(2 * u) * kPieceBytes;
    const uint4 w0 = *reinterpret_cast<const uint4*>(wt), w1 = *reinterpret_cast<const uint4*>(wt + kPieceBytes);
    const float ws = scalar_scale(wsg, u);
    __builtin_amdgcn_sched_barrier(0);   // every load above the first conversion
#pragma unroll
    for (int h = 0; h < kMG; ++h) {
      const int rows = min(M - 16 * h, 16);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (4 * q < rows) {
          const int row = 4 * q + (lane >> 4);
          const uint32_t wv[4] = {xa[q].x, xa[q].y, xa[q].z, xa[q].w};
          const uint32_t sb = b128_scale_byte(row16_max(absmax8(xa[q])));
          uint32_t qv[2];
          cvt8s(wv, mx_scale_value(sb), qv);
          *reinterpret_cast<uint2*>(xq + row * L::kPitch + (lane & 15) * 8) = make_uint2(qv[0], qv[1]);
          if ((lane & 15) == 0) xs[row] = (uint8_t)sb;
        }
      }
      if (h + 1 < kMG) load_x(h + 1);   // on its way during this group's product
      // One wave's LDS accesses execute in order; this keeps the compiler from
      // moving the reads above the writes, and the next group's writes above these.
      asm volatile("" ::: "memory");
      const int rr = min(i, rows - 1);   // lanes past M repeat the last row; their outputs are dropped
      const uint8_t* p = xq + rr * L::kPitch + 16 * g;
      const uint4 b0 = *reinterpret_cast<const uint4*>(p);
      const uint4 b1 = *reinterpret_cast<const uint4*>(p + 64);
      const int sx = xs[rr];
      const v8i xb = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
      const v8i wa = {(int)w0.x, (int)w0.y, (int)w0.z, (int)w0.w, (int)w1.x, (int)w1.y, (int)w1.z, (int)w1.w};
      const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0,
                                                                        kUnitScales, 0, sx);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[h][e] = fmaf(part[e], ws, acc[h][e]);
      asm volatile("" ::: "memory");
    }
  }

  // Lane (i, g) holds D[n = 4g + j][m = 16 h + i], j = 0..3: the waves' sums in
  // wave (K) order, bias, one rounding; wave h stores group h.
#pragma unroll
  for (int h = 0; h < kMG; ++h) red[(h * kDecWaves + wave) * 64 + lane] = acc[h];
  __syncthreads();
  if (wave >= kMG) return;
  v4f part[kDecWaves];
#pragma unroll
  for (int w = 0; w < kDecWaves; ++w) part[w] = red[(wave * kDecWaves + w) * 64 + lane];
  __builtin_amdgcn_sched_barrier(0);
  v4f sum = part[0];
#pragma unroll
  for (int w = 1; w < kDecWaves; ++w) sum += part[w];
  const int n = n0 + 4 * g, row = 16 * wave + i;
  if (row >= M || n >= N) return;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = sum[e] + __uint_as_float(braw[e] << 16);
  uint16_t* yrow = y + (size_t)row * ldy;
  const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
  if (vec_store && n + 3 < N) {
    *reinterpret_cast<uint2*>(yrow + n) = make_uint2(lo, hi);
  } else {
    yrow[n] = (uint16_t)lo;
    if (n + 1 < N) yrow[n + 1] = (uint16_t)(lo >> 16);
    if (n + 2 < N) yrow[n + 2] = (uint16_t)hi;
    if (n + 3 < N) yrow[n + 3] = (uint16_t)(hi >> 16);
  }
}

namespace {
template <int kMG>
int launch_decode_k(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const float* wsc, int64_t N,
                    const void* bias, void* y, int64_t ldy, hipStream_t stream) {
  constexpr int lds = DecodeLds<kMG>::kBytes;
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)gemm_b128_decode_kernel<kMG>, lds, lds_set)) return -7;
  const int vec = (ldy % 4 == 0) && (((uintptr_t)y & 7) == 0);
  hipLaunchKernelGGL(gemm_b128_decode_kernel<kMG>, dim3((unsigned)((N + 15) / 16)), dim3(kDecThreads), lds,
                     stream, (const uint16_t*)x, ldx, (int)M, K, (const uint8_t*)wp, wsc, (int)N,
                     (const uint16_t*)bias, (uint16_t*)y, ldy, vec);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}
}  // namespace

int launch_gemm_b128_decode(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const float* wsc,
                            int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream) {
  return M > 16 ? launch_decode_k<2>(x, ldx, M, K, wp, wsc, N, bias, y, ldy, stream)
                : launch_decode_k<1>(x, ldx, M, K, wp, wsc, N, bias, y, ldy, stream);
}

// ---------------------------------------------------------------------------
// Small tiles: one 128-row weight group x 64 activation rows per workgroup over
// a run of 128-blocks, four waves 2 x 2; wave (wn, wm) owns weight rows
// 32 a + 16 wn + i and activation rows 32 b + 16 wm + i, so the byte of a
// row's scale inside its packed word (rows r + 32 k, byte k) is b, an
// immediate op_sel.  Stages of 64 K come straight from global memory into
// LDS; a 128-block reads a pair of stages; kDepth pairs are in LDS
// (three: two workgroups share a compute unit and cover each other's waits).
// Bound by a step's copies and their latency: 1000 x 2064 x 2032 11.5 us.
// ---------------------------------------------------------------------------
namespace {
constexpr int kB128Threads = 256;

constexpr int kMT = 64;      // activation rows
constexpr int kDepth = 3;    // pairs of stages (128-blocks) in LDS

struct SmallLds {
  static constexpr int kW = kGroupRows * kStepK;
  static constexpr int kX = kMT * kStepK;
  // + the activations' 256-byte scale tile, copied by wave 0; the other
  // waves' scale copies go to slots of their own, so every wave issues the
  // same number of copies (the waits count them per wave).
  static constexpr int kStage = kW + kX + 1024;
  static constexpr int kBytes = 2 * kDepth * kStage;
  static constexpr int kCopies = 2 * (2 + kMT / 64 + 1);
  static constexpr int kPitchY = 128 * 2 + 16;
  static_assert(kMT * kPitchY <= kBytes, "the output staging fits in the stages");
};
}  // namespace

template <bool kPart>
__global__ __launch_bounds__(kB128Threads, 2) void gemm_b128_small_kernel(
    const uint8_t* __restrict__ qp, const uint8_t* __restrict__ sp, int M, int KB, const uint8_t* __restrict__ wp,
    const float* __restrict__ wsc, int N, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t ldy,
    int tiles_n, int tiles_m, int splits, int vec, float* __restrict__ part, int64_t ldp) {
  using L = SmallLds;
  constexpr int kNB = kMT / 32;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int i = lane & 15, g = lane >> 4;
  const int item = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int split = kPart ? item % splits : 0;
  const int t = kPart ? item / splits : item;
  const int tn = t / tiles_m, tm = t - tn * tiles_m;
  const int p0 = kPart ? (int)((int64_t)KB * split / splits) : 0;
  const int p1 = kPart ? (int)((int64_t)KB * (split + 1) / splits) : KB;
  const int KS = 2 * KB, n0 = tn * kGroupRows;

  uint32_t braw[4][4];
  if constexpr (!kPart) {
    const __amdgpu_buffer_rsrc_t brsrc = raw_rsrc(bias, bias != nullptr ? (uint32_t)N * 2u : 0u);
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        braw[a][j] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(
            brsrc, (uint32_t)(n0 + 32 * a + 16 * wn + 4 * g + j) * 2u, 0, 0);
  }

  // Copies: wave w takes bands w and w + 4 of the weight group and band
  // 4 h + w of the activation group, whose half h is the tile's.
  const int h = tm & 1, xg = tm >> 1;
  const uint32_t gbytes = (uint32_t)KS * kTileBytes, sbytes = (uint32_t)KS * kTileScaleBytes;
  const tile::i4v wr = tile::buffer_rsrc(wp + (size_t)tn * gbytes, gbytes);
  const tile::i4v xr = tile::buffer_rsrc(qp + (size_t)xg * gbytes, gbytes);
  const tile::i4v sr = tile::buffer_rsrc(sp + (size_t)xg * sbytes, sbytes);
  const uint32_t lo16 = (uint32_t)lane * 16u;
  const uint32_t vw0 = (uint32_t)wave * KS * kPieceBytes + lo16, vw1 = vw0 + 4u * KS * kPieceBytes;
  const uint32_t vx = (uint32_t)(4 * h + wave) * KS * kPieceBytes + lo16;
  const uint32_t vs = (uint32_t)lane * 4u;
  auto issue_stage = [&](int ks, uint8_t* st) {
    const uint32_t off = (uint32_t)ks * kPieceBytes;
    tile::b2l_16(vw0, wr, off, st + wave * 1024);
    tile::b2l_16(vw1, wr, off, st + 4096 + wave * 1024);
    tile::b2l_16(vx, xr, off, st + L::kW + wave * 1024);
    tile::b2l_4(vs, sr, (uint32_t)ks * kTileScaleBytes, st + L::kW + L::kX + wave * 256);
  };
  auto stage_ptr = [&](int s) { return smem + s * L::kStage; };

  const int offW = 16 * wn * kStepK + tile_off(i, g);
  const int offX = L::kW + 16 * wm * kStepK + tile_off(i, g);
  const int offSX = L::kW + L::kX + (16 * wm + i) * 8 + (g & 1) * 4;
  auto rd16 = [](const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); };
  auto frag = [&](const uint8_t* ev, const uint8_t* od, int off) {
    const uint4 lo = rd16(ev + off), hi = rd16(od + off);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };

  v4f acc[4][kNB];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < kNB; ++b) acc[a][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const float* wsg = wsc + (size_t)tn * KB;
  // Every step issues one block's copies, past the run's end those of its
  // last block again (into a buffer nobody reads any more), so the wait for
  // block p always leaves the copies of kDepth - 1 newer blocks in flight.
#pragma unroll
  for (int d = 0; d < kDepth; ++d) {
    const int q = min(p0 + d, p1 - 1);
    issue_stage(2 * q, stage_ptr(2 * d));
    issue_stage(2 * q + 1, stage_ptr(2 * d + 1));
  }
  int at = 0;   // the block's pair of stages
  for (int p = p0; p < p1; ++p) {
    const float ws = scalar_scale(wsg, p);
    tile::wait_vmcnt<(kDepth - 1) * L::kCopies>();
    __builtin_amdgcn_s_barrier();
    const uint8_t* ev = stage_ptr(2 * at);
    const uint8_t* od = ev + L::kStage;
    v8i wf[4], xf[kNB];
#pragma unroll
    for (int a = 0; a < 4; ++a) wf[a] = frag(ev, od, offW + 32 * kStepK * a);
#pragma unroll
    for (int b = 0; b < kNB; ++b) xf[b] = frag(ev, od, offX + 32 * kStepK * b);
    // the word's bytes are rows r + 32 k of the 128-row group: the half's are 2 h + b
    const int sx = (int)(*reinterpret_cast<const uint32_t*>(((g >> 1) ? od : ev) + offSX) >> (16 * h));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    {
      const int q = min(p + kDepth, p1 - 1);
      issue_stage(2 * q, stage_ptr(2 * at));
      issue_stage(2 * q + 1, stage_ptr(2 * at + 1));
    }
    at = at + 1 == kDepth ? 0 : at + 1;
    tile::static_for<0, 4>([&](auto A) {
      constexpr int a = decltype(A)::value;
      tile::static_for<0, kNB>([&](auto B) {
        constexpr int b = decltype(B)::value;
        const v4f d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[a], xf[b], v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0,
                                                                       0, 0, kUnitScales, b, sx);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[a][b][e] = fmaf(d[e], ws, acc[a][b][e]);
      });
    });
  }

  tile::wait_vmcnt<0>();   // the last copies, before their LDS is reused or given away

  // Lane (i, g) holds D[n = 32 a + 16 wn + 4 g + j][m = 32 b + 16 wm + i].
  const int mt0 = tm * kMT;
  if constexpr (kPart) {
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < kNB; ++b) {
        const int m = mt0 + 32 * b + 16 * wm + i, n = n0 + 32 * a + 16 * wn + 4 * g;
        // ldp is N rounded up to 4: a quad is all in or all out of the row
        if (m < M && n < ldp) *reinterpret_cast<v4f*>(part + ((size_t)split * M + m) * ldp + n) = acc[a][b];
      }
    return;
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < kNB; ++b) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = acc[a][b][j] + __uint_as_float(braw[a][j] << 16);
      const int m = 32 * b + 16 * wm + i, n = 32 * a + 16 * wn + 4 * g;
      *reinterpret_cast<uint2*>(smem + m * L::kPitchY + n * 2) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  __syncthreads();
  const int c8 = (tid & 15) * 8;
#pragma unroll
  for (int q = 0; q < kMT / 16; ++q) {
    const int r = (tid >> 4) + 16 * q;
    const int m = mt0 + r;
    if (m >= M) break;
    const int n = n0 + c8;
    if (n >= N) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(smem + r * L::kPitchY + c8 * 2);
    uint16_t* dst = y + (size_t)m * ldy + n;
    if (vec && n + 7 < N) {
      *reinterpret_cast<uint4*>(dst) = v;
    } else {
      const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < N) dst[e] = (uint16_t)(w4[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// ---------------------------------------------------------------------------
// Large tiles: kG weight groups (128 kG rows) x 128 activation rows per
// workgroup, four waves 2 x 2, each 64 kG x 64 (16 kG MFMAs per 128-block).
//  * The accumulators are 64 kG vector registers per lane; the operand
//    fragments of the current and of the next block sit in registers too
//    (96 + 96 for kG = 2; one wave per SIMD has 512), so no MFMA waits for
//    LDS.
//  * LDS holds kDepth blocks (3 x 49 or 4 x 33 KiB).  At the top of step p the
//    copies of p + 1 have landed everywhere (own vmcnt, then the one barrier
//    of the step), every wave has read p, and the copies of p + kDepth go out
//    into p's buffer: a copy has kDepth - 1 whole steps to land.
//  * The MFMAs of a step carry between them the v_fma of the results three
//    MFMAs back (nearer ones are not there yet), the LDS reads of the next
//    step's fragments and the copies.
//  * Workgroups are persistent and the pipeline runs across items (a tile, or
//    with kPart a tile's run of blocks): the last steps of an item copy and
//    read the next one's first blocks.  The epilogue issues a fixed number of
//    16-byte stores per wave (rows and columns outside are dropped by the
//    buffer bounds), left in flight into the next item.
// ---------------------------------------------------------------------------
namespace {

template <int kG>
struct BigLds {
  static constexpr int kX = 8192 * kG;               // activation pieces inside a 64-K half
  static constexpr int kHalf = kX + 8192;
  static constexpr int kScale = 2 * kHalf;           // two 256-byte scale tiles, then two unused slots
  static constexpr int kBlock = kScale + 1024;
  static constexpr int kDepth = kG == 2 ? 3 : 4;     // blocks in LDS
  static constexpr int kBytes = kDepth * kBlock;
  static constexpr int kCopies = 4 * kG + 5;         // per wave and block
};

// Tile order: bands of eight activation tiles, inside a band the weight tiles
// outermost, so the tiles a die runs together share both operands.
struct BigTile {
  int tn, tm;
};
__device__ inline BigTile big_tile(int item, int tiles_n, int tiles_m) {
  const int per = 8 * tiles_n;
  const int band = item / per, r = item - band * per;
  const int rows = min(8, tiles_m - 8 * band);
  BigTile t;
  t.tn = r / rows;
  t.tm = 8 * band + r - t.tn * rows;
  return t;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Two neighbouring 16-column tiles of a wave (lane (i, g) holds columns 4 g ..
// + 3 of row i of each) as bf16: exchanging the odd 16-lane rows of the first
// with the even ones of the second gives every lane eight consecutive columns,
// of the first tile for even g, of the second for odd g.
__device__ inline u32x4 pack_pair(const v4f& lo, const v4f& hi, const float (&bl)[4], const float (&bh)[4]) {
  const uint32_t l0 = pack_bf16x2(lo[0] + bl[0], lo[1] + bl[1]), l1 = pack_bf16x2(lo[2] + bl[2], lo[3] + bl[3]);
  const uint32_t h0 = pack_bf16x2(hi[0] + bh[0], hi[1] + bh[1]), h1 = pack_bf16x2(hi[2] + bh[2], hi[3] + bh[3]);
  const auto s0 = __builtin_amdgcn_permlane16_swap(l0, h0, false, false);
  const auto s1 = __builtin_amdgcn_permlane16_swap(l1, h1, false, false);
  return u32x4{s0[0], s1[0], s0[1], s1[1]};
}
// Stores the 64 columns of two such pairs in whole 128-byte rows: half the
// lanes of each exchange rows 8 .. 15 of the first for rows 0 .. 7 of the
// second.  Byte offsets of a lane's eight columns (past the end to drop them):
// at0 row i % 8, at1 row 8 + i % 8, in both column 32 (i / 8) +
// col_of_pair(g) from the first pair's start on.  (Rows of 64 bytes: 8192 x
// 28672 x 8192 1522 us against 1487, 16384 x 8192 x 2048 290 against 272.)
__device__ inline int col_of_pair(int g) { return 16 * (g & 1) + 8 * (g >> 1); }
__device__ inline void store_pairs(u32x4 p0, u32x4 p1, __amdgpu_buffer_rsrc_t yr, uint32_t at0, uint32_t at1) {
  u32x4 a, b;
#pragma unroll
  for (int e = 0; e < 4; ++e) {   // row_ror:8 into lanes 8 .. 15, or 0 .. 7, of each sixteen
    a[e] = (uint32_t)__builtin_amdgcn_update_dpp((int)p0[e], (int)p1[e], 0x128, 0xF, 0xC, false);
    b[e] = (uint32_t)__builtin_amdgcn_update_dpp((int)p1[e], (int)p0[e], 0x128, 0xF, 0x3, false);
  }
  __builtin_amdgcn_raw_buffer_store_b128(a, yr, at0, 0, 0);
  __builtin_amdgcn_raw_buffer_store_b128(b, yr, at1, 0, 0);
}
constexpr uint32_t kDrop = 0xFFFFFFF0u;

// Bias of columns n .. n + 3 (0 past N, and with a null bias).
__device__ inline void bias4(const uint16_t* bias, int N, int n, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = 0.0f;
  if (bias == nullptr) return;   // no load: waiting for one would drain the copies in flight
  const __amdgpu_buffer_rsrc_t r = raw_rsrc(bias, (uint32_t)N * 2u);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, (uint32_t)(n + j) * 2u, 0, 0) << 16);
}

}  // namespace

template <int kG, bool kPart>
__global__ __launch_bounds__(kB128Threads, 1) void gemm_b128_big_kernel(
    const uint8_t* __restrict__ qp, const uint8_t* __restrict__ sp, int M, int KB, const uint8_t* __restrict__ wp,
    const float* __restrict__ wsc, int N, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t ldy,
    int GN, int tiles_n, int tiles_m, int lsplits, int total, float* __restrict__ part, int64_t ldp) {
  using L = BigLds<kG>;
  constexpr int kA = 4 * kG;                          // 16-row weight fragments per wave
  constexpr int kStores = kPart ? 4 * kA : 2 * kA;    // per wave and item
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int i = lane & 15, g = lane >> 4;
  const int KS = 2 * KB;
  const uint32_t gbytes = (uint32_t)KS * kTileBytes, sbytes = (uint32_t)KS * kTileScaleBytes;

  // This workgroup's items: wg, wg + grid, ... of the die-wise order.
  const int grid = (int)gridDim.x;
  const int mine = (total - (int)blockIdx.x + grid - 1) / grid;
  struct Item {
    BigTile t;
    int split, p0, p1;
  };
  auto item_at = [&](int j) {
    const int id = xcd_remap((int)blockIdx.x + j * grid, total);
    Item r;
    r.split = kPart ? id & ((1 << lsplits) - 1) : 0;   // a power of two of them
    r.t = big_tile(kPart ? id >> lsplits : id, tiles_n, tiles_m);
    const int each = KB >> lsplits, more = KB & ((1 << lsplits) - 1);   // the first `more` runs are one longer
    r.p0 = kPart ? r.split * each + min(r.split, more) : 0;
    r.p1 = kPart ? r.p0 + each + (r.split < more ? 1 : 0) : KB;
    return r;
  };

  // Copy side: the item the next copies belong to.
  // (Carried from step to step as addresses: resources carried through the
  // loop end up in vector registers.)
  struct Src {
    const uint8_t *w0, *w1, *x, *s;
  };
  struct Rsrc {
    tile::i4v w0, w1, x, s;
  };
  auto src_of = [&](BigTile t) {
    // past the last group: any data, its columns are dropped
    const int g1 = kG == 2 ? min(2 * t.tn + 1, GN - 1) : t.tn;
    return Src{wp + (size_t)(kG * t.tn) * gbytes, wp + (size_t)g1 * gbytes, qp + (size_t)t.tm * gbytes,
               sp + (size_t)t.tm * sbytes};
  };
  auto rsrc_of = [&](const Src& r) {
    return Rsrc{tile::buffer_rsrc(r.w0, gbytes), tile::buffer_rsrc(r.w1, gbytes), tile::buffer_rsrc(r.x, gbytes),
                tile::buffer_rsrc(r.s, sbytes)};
  };
  const uint32_t v0 = (uint32_t)wave * KS * kPieceBytes + (uint32_t)lane * 16u, v1 = v0 + 4u * KS * kPieceBytes;
  const uint32_t vs = (uint32_t)lane * 4u;
  // Copy j of a block: both 64-K halves of the wave's two bands of each
  // weight group, then of the activation group, then a scale tile (waves 2
  // and 3 copy theirs to the unused slots).
  auto copy = [&](auto J, const Rsrc& r, int p, uint8_t* st) {
    constexpr int j = decltype(J)::value;
    if constexpr (j < 4 * kG + 4) {
      constexpr int half = j & 1, band = (j >> 1) & 1, op = j >> 2;   // op: weight groups, then activations
      const uint32_t off = (uint32_t)(2 * p + half) * kPieceBytes;
      uint8_t* const at = st + half * L::kHalf + op * 8192 + band * 4096 + wave * 1024;
      tile::b2l_16(band ? v1 : v0, op == kG ? r.x : op == 1 ? r.w1 : r.w0, off, at);
    } else {
      tile::b2l_4(vs, r.s, (uint32_t)(2 * p + (wave & 1)) * kTileScaleBytes, st + L::kScale + wave * 256);
    }
  };

  const int offW = wn * 4096 * kG + tile_off(i, g);
  const int offX = L::kX + 16 * wm * kStepK + tile_off(i, g);
  const int offS = L::kScale + (g >> 1) * 256 + (16 * wm + i) * 8 + (g & 1) * 4;
  struct Frags {
    v8i w[kA], x[4];
    int s;
  };
  auto rd16 = [](const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); };
  auto frag = [&](const uint8_t* st, int off) {
    const uint4 lo = rd16(st + off), hi = rd16(st + off + L::kHalf);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  // Part j of the fragment reads of a block: its scale word and activation
  // fragments first.
  auto read = [&](int j, const uint8_t* st, Frags& f) {
    if (j == 0) f.s = *reinterpret_cast<const int*>(st + offS);
    if (j < 4) f.x[j] = frag(st, offX + 32 * kStepK * j);
    else f.w[j - 4] = frag(st, offW + 16 * kStepK * (j - 4));
  };

  v4f acc[kA][4];
  auto clear = [&] {
#pragma unroll
    for (int a = 0; a < kA; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();

  // Positions in the flattened (item, block) sequence: of the copies
  // (kDepth steps ahead) and of the MFMAs.  Past the last item the copies go on with
  // its blocks again (never used), so the steps need no branch and the waits
  // no other counts.
  Item ci = item_at(0), mi = ci;
  int cj = 0, cp = ci.p0, mj = 0, mp = 0;
  Src src = src_of(ci.t);
  auto advance_copy = [&] {
    if (++cp == ci.p1) {
      cj = min(cj + 1, mine - 1);
      ci = item_at(cj);
      cp = ci.p0;
      src = src_of(ci.t);
    }
  };
  auto scales_of = [&](BigTile t) {
    return wsc + (size_t)(kG == 2 ? min(2 * t.tn + wn, GN - 1) : t.tn) * KB;
  };
  const float* wsg = scales_of(mi.t);
  auto buf = [&](int b) { return smem + b * L::kBlock; };
#pragma unroll
  for (int s = 0; s < L::kDepth; ++s) {
    const Rsrc rs = rsrc_of(src);
    tile::static_for<0, L::kCopies>([&](auto J) { copy(J, rs, cp, buf(s)); });
    advance_copy();
  }
  tile::wait_vmcnt<(L::kDepth - 1) * L::kCopies>();
  __builtin_amdgcn_s_barrier();
  Frags f0, f1;
#pragma unroll
  for (int j = 0; j < 4 + kA; ++j) read(j, buf(0), f0);
  float ws = scalar_scale(wsg, mi.p0);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");

  // Lane (i, g) holds D[n = 64 kG wn + 16 a + 4 g + j][m = 32 b + 16 wm + i].
  auto epilogue = [&](const Item& it) {
    const int n0 = (it.t.tn * 2 + wn) * 64 * kG, m0 = it.t.tm * 128;
    const int rows = min(128, M - m0);
    if constexpr (kPart) {
      const __amdgpu_buffer_rsrc_t pr = raw_rsrc(part + ((size_t)it.split * M + m0) * ldp, (uint32_t)(rows * ldp * 4));
#pragma unroll
      for (int a = 0; a < kA; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int n = n0 + 16 * a + 4 * g, m = 32 * b + 16 * wm + i;
          const uint32_t at = (n < ldp && m < rows) ? (uint32_t)((m * ldp + n) * 4) : kDrop;
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[a][b]), pr, at, 0, 0);
        }
    } else {
      const __amdgpu_buffer_rsrc_t yr =
          raw_rsrc(y + (size_t)m0 * ldy, (uint32_t)(((int64_t)(rows - 1) * ldy + N) * 2));
#pragma unroll
      for (int a = 0; a < kA; a += 4) {
        float bias_n[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) bias4(bias, N, n0 + 16 * (a + q) + 4 * g, bias_n[q]);
        const int n = n0 + 16 * a + 32 * (i >> 3) + col_of_pair(g);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int m = 32 * b + 16 * wm + (i & 7);   // N % 8 == 0: eight columns are all in or all out
          const uint32_t at = (uint32_t)(((int64_t)m * ldy + n) * 2);
          store_pairs(pack_pair(acc[a][b], acc[a + 1][b], bias_n[0], bias_n[1]),
                      pack_pair(acc[a + 2][b], acc[a + 3][b], bias_n[2], bias_n[3]), yr,
                      n < N && m < rows ? at : kDrop, n < N && m + 8 < rows ? at + (uint32_t)ldy * 16u : kDrop);
        }
      }
    }
    clear();
  };

  bool stores = false;   // the stores of the last epilogue may be outstanding
  auto step = [&](Frags& f, Frags& fn, int rb) {
    // Newer than the copies of the next block: those of the kDepth - 2 after
    // it, and in an item's first kDepth - 1 steps the last epilogue's stores.
    constexpr int kNewer = (L::kDepth - 2) * L::kCopies;
    if (stores && mp < L::kDepth - 1) tile::wait_vmcnt<kNewer + kStores>();
    else tile::wait_vmcnt<kNewer>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    uint8_t* const st_free = buf(rb);
    const uint8_t* const st_next = buf(rb == L::kDepth - 1 ? 0 : rb + 1);
    v4f d[4];
    const Rsrc rs = rsrc_of(src);
    const int p = __builtin_amdgcn_readfirstlane(cp);
    // The empty asm statements keep each MFMA and each result's v_fma in its
    // place in the stream of reads and copies: as pure operations they would
    // otherwise sink below all of them.
    tile::static_for<0, 4 * kA + 3>([&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (j < 4 * kA) {
        d[j & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f.w[j >> 2], f.x[j & 3], v4f{0, 0, 0, 0},
                                                                    0, 0, 0, kUnitScales, j & 3, f.s);
        asm volatile("" : "+v"(d[j & 3]));
      }
      // kG = 2: a read and a copy every other MFMA; kG = 1: one of each.
      constexpr int k2 = kG == 2 ? j >> 1 : j;
      if constexpr ((kG == 1 || (j & 1) == 0) && k2 < 4 + kA) read(k2, st_next, fn);
      if constexpr ((kG == 1 || (j & 1) == 1) && k2 < L::kCopies)
        copy(std::integral_constant<int, (k2 < L::kCopies ? k2 : 0)>{}, rs, p, st_free);
      if constexpr (j >= 3) {
        constexpr int k = j - 3;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k >> 2][k & 3][e] = fmaf(d[k & 3][e], ws, acc[k >> 2][k & 3][e]);
        asm volatile("" : "+v"(acc[k >> 2][k & 3]));
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    advance_copy();
    if (mi.p0 + ++mp == mi.p1) {
      epilogue(mi);
      stores = true;
      mp = 0;
      mj = mj + 1;
      mi = item_at(min(mj, mine - 1));
      wsg = scales_of(mi.t);
    }
    ws = scalar_scale(wsg, mi.p0 + mp);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  int rb = 0;
  while (mj < mine) {
    step(f0, f1, rb);
    rb = rb == L::kDepth - 1 ? 0 : rb + 1;
    if (mj >= mine) break;
    step(f1, f0, rb);
    rb = rb == L::kDepth - 1 ? 0 : rb + 1;
  }
  tile::wait_vmcnt<0>();   // no copy may land after the workgroup's LDS is given away
}

// ---------------------------------------------------------------------------
// Wide tiles: 256 x 256 per workgroup, eight waves 2 (n) x 4 (m), each 128 x 64
// as above, two waves per SIMD.  A third fewer operand bytes per product than
// the 256 x 128 tiles; 256 registers per wave leave no room for a second set
// of fragments, so weight fragments are read two ahead and the SIMD's other
// wave covers what latency is left.
//  * LDS holds two blocks (2 x 66 KiB).  After a wave's last reads of block p
//    comes the step's one barrier: then p + 1 has landed everywhere, p's
//    buffer is free, the first fragments of p + 1 are read under the last
//    MFMAs of p, and the copies of p + 2 go out with the MFMAs of p + 1.
//  * Persistent, with the same epilogue.
// 8192 x 28672 x 8192: 1571 us (2.45 PFLOP/s; 256 x 128 tiles 1805, 128 x 128
// 2302, 128 x 64 2660); 4096^3: 60, 69, 89, 102 (traced, in steady calls).  The
// MFMA pipes are busy 0.65 of the time.  Timed one by one in the 256 x 128 form:
// the MFMAs alone, without v_fma, reads and copies, 1250 us, the v_fma 250 more.
// ---------------------------------------------------------------------------
namespace {
constexpr int kWideThreads = 512;
constexpr int kWideX = 16384;                        // activation pieces inside a 64-K half
constexpr int kWideHalf = 32768;                     // (256 + 256 rows) x 64 B
constexpr int kWideScale = 2 * kWideHalf;            // eight 256-byte slots: [half][group], four unused
constexpr int kWideBlock = kWideScale + 2048;
constexpr int kWideLds = 2 * kWideBlock;             // 135168
constexpr int kWideCopies = 9;                       // per wave and block
}  // namespace

__global__ __launch_bounds__(kWideThreads, 1) void gemm_b128_wide_kernel(
    const uint8_t* __restrict__ qp, const uint8_t* __restrict__ sp, int M, int KB, const uint8_t* __restrict__ wp,
    const float* __restrict__ wsc, int N, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t ldy,
    int GN, int GM, int tiles_n, int tiles_m, int total) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = (wave >> 1) & 1, wx = wave >> 2;   // weight group, row half, activation group
  const int i = lane & 15, g = lane >> 4;
  const int KS = 2 * KB;
  const uint32_t gbytes = (uint32_t)KS * kTileBytes, sbytes = (uint32_t)KS * kTileScaleBytes;
  const int grid = (int)gridDim.x;
  const int mine = (total - (int)blockIdx.x + grid - 1) / grid;
  const int steps = mine * KB;
  auto tile_at = [&](int j) { return big_tile(xcd_remap((int)blockIdx.x + j * grid, total), tiles_n, tiles_m); };

  // Copies: wave w takes band w of both weight groups and both activation
  // groups, and one of the block's four scale tiles (waves 4 .. 7 copy them
  // again, to the unused slots).
  struct Src {
    tile::i4v w0, w1, x0, x1, s;
  };
  auto src_of = [&](BigTile t) {
    Src r;
    const int g1 = min(2 * t.tn + 1, GN - 1), m1 = min(2 * t.tm + 1, GM - 1);
    r.w0 = tile::buffer_rsrc(wp + (size_t)(2 * t.tn) * gbytes, gbytes);
    r.w1 = tile::buffer_rsrc(wp + (size_t)g1 * gbytes, gbytes);
    r.x0 = tile::buffer_rsrc(qp + (size_t)(2 * t.tm) * gbytes, gbytes);
    r.x1 = tile::buffer_rsrc(qp + (size_t)m1 * gbytes, gbytes);
    r.s = tile::buffer_rsrc(sp + (size_t)((wave & 1) ? m1 : 2 * t.tm) * sbytes, sbytes);
    return r;
  };
  const uint32_t v0 = (uint32_t)wave * KS * kPieceBytes + (uint32_t)lane * 16u;
  const uint32_t vs = (uint32_t)lane * 4u;
  auto copy = [&](int j, const Src& r, int p, uint8_t* st) {
    const uint32_t off = (uint32_t)(2 * p) * kPieceBytes;
    uint8_t* b = st + wave * 1024;
    switch (j) {
      case 0: tile::b2l_16(v0, r.w0, off, b); break;
      case 1: tile::b2l_16(v0, r.w1, off, b + 8192); break;
      case 2: tile::b2l_16(v0, r.x0, off, b + kWideX); break;
      case 3: tile::b2l_16(v0, r.x1, off, b + kWideX + 8192); break;
      case 4: tile::b2l_16(v0, r.w0, off + kPieceBytes, b + kWideHalf); break;
      case 5: tile::b2l_16(v0, r.w1, off + kPieceBytes, b + kWideHalf + 8192); break;
      case 6: tile::b2l_16(v0, r.x0, off + kPieceBytes, b + kWideHalf + kWideX); break;
      case 7: tile::b2l_16(v0, r.x1, off + kPieceBytes, b + kWideHalf + kWideX + 8192); break;
      default:
        tile::b2l_4(vs, r.s, (uint32_t)(2 * p + ((wave >> 1) & 1)) * kTileScaleBytes, st + kWideScale + wave * 256);
        break;
    }
  };

  const int offW = wn * 8192 + tile_off(i, g);
  const int offX = kWideX + wx * 8192 + 16 * wm * kStepK + tile_off(i, g);
  const int offS = kWideScale + (2 * (g >> 1) + wx) * 256 + (16 * wm + i) * 8 + (g & 1) * 4;
  auto rd16 = [](const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); };
  auto frag = [&](const uint8_t* st, int off) {
    const uint4 lo = rd16(st + off), hi = rd16(st + off + kWideHalf);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };

  v4f acc[8][4];
  auto clear = [&] {
#pragma unroll
    for (int a = 0; a < 8; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();

  int cj = 0, cp = 0, mj = 0, mp = 0;
  Src src = src_of(tile_at(0));
  auto advance_copy = [&] {
    if (++cp == KB) {
      cp = 0;
      cj = min(cj + 1, mine - 1);
      src = src_of(tile_at(cj));
    }
  };
  BigTile cur = tile_at(0);
  const float* wsg = wsc + (size_t)min(2 * cur.tn + wn, GN - 1) * KB;
  auto buf = [&](int b) { return smem + b * kWideBlock; };
  // A block's copies 0 .. 4 go out at the end of a step, the others at the
  // start of the next.
  constexpr int kEarly = 5;
#pragma unroll
  for (int j = 0; j < kWideCopies; ++j) copy(j, src, cp, buf(0));
  advance_copy();
#pragma unroll
  for (int j = 0; j < kEarly; ++j) copy(j, src, cp, buf(1));
  tile::wait_vmcnt<kEarly>();
  __builtin_amdgcn_s_barrier();
  v8i x[4], w[3];
  float ws = scalar_scale(wsg, 0);
  int sx = *reinterpret_cast<const int*>(buf(0) + offS);
#pragma unroll
  for (int b = 0; b < 4; ++b) x[b] = frag(buf(0), offX + 32 * kStepK * b);
  w[0] = frag(buf(0), offW);
  w[1] = frag(buf(0), offW + 16 * kStepK);

  auto epilogue = [&](BigTile t) {
    const int n0 = t.tn * 256 + wn * 128, m0 = t.tm * 256 + wx * 128;
    const int rows = max(0, min(128, M - m0));
    const __amdgpu_buffer_rsrc_t yr = raw_rsrc(
        y + (size_t)min(m0, M - 1) * ldy, rows > 0 ? (uint32_t)(((int64_t)(rows - 1) * ldy + N) * 2) : 0u);
#pragma unroll
    for (int a = 0; a < 8; a += 4) {
      float bias_n[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) bias4(bias, N, n0 + 16 * (a + q) + 4 * g, bias_n[q]);
      const int n = n0 + 16 * a + 32 * (i >> 3) + col_of_pair(g);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int m = 32 * b + 16 * wm + (i & 7);   // N % 8 == 0: eight columns are all in or all out
        const uint32_t at = (uint32_t)(((int64_t)m * ldy + n) * 2);
        store_pairs(pack_pair(acc[a][b], acc[a + 1][b], bias_n[0], bias_n[1]),
                    pack_pair(acc[a + 2][b], acc[a + 3][b], bias_n[2], bias_n[3]), yr,
                    n < N && m < rows ? at : kDrop, n < N && m + 8 < rows ? at + (uint32_t)ldy * 16u : kDrop);
      }
    }
    clear();
  };

  for (int s = 0; s < steps; ++s) {
    uint8_t* const st = buf(s & 1);
    uint8_t* const other = buf((s & 1) ^ 1);
    v4f d[4];
    int sxn = 0;
    tile::static_for<0, 35>([&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (j < 32) {
        d[j & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[(j >> 2) % 3], x[j & 3],
                                                                    v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, kUnitScales,
                                                                    j & 3, sx);
        asm volatile("" : "+v"(d[j & 3]));
      }
      if constexpr (j < 24 && (j & 3) == 0) w[(j / 4 + 2) % 3] = frag(st, offW + 16 * kStepK * (j / 4 + 2));
      // the rest of block s + 1 (its buffer is free since the last barrier)
      if constexpr (j < kWideCopies - kEarly) copy(kEarly + j, src, cp, other);
      if constexpr (j == kWideCopies - kEarly) advance_copy();
      if constexpr (j >= 3) {
        constexpr int k = j - 3;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k >> 2][k & 3][e] = fmaf(d[k & 3][e], ws, acc[k >> 2][k & 3][e]);
        asm volatile("" : "+v"(acc[k >> 2][k & 3]));
      }
      if constexpr (j == 25) {
        // This wave has read the block, its copies of the next have landed;
        // past the barrier both hold for all.
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
      }
      if constexpr (j >= 26 && j < 26 + kEarly) copy(j - 26, src, cp, st);
      // the next block's first fragments, each where its register is free
      if constexpr (j == 27) sxn = *reinterpret_cast<const int*>(other + offS);
      if constexpr (j == 28) w[0] = frag(other, offW);
      if constexpr (j >= 29 && j < 33) x[j - 29] = frag(other, offX + 32 * kStepK * (j - 29));
      if constexpr (j == 32) w[1] = frag(other, offW + 16 * kStepK);
      __builtin_amdgcn_sched_barrier(0);
    });
    sx = sxn;
    if (++mp == KB) {
      epilogue(cur);
      mp = 0;
      mj = min(mj + 1, mine - 1);
      cur = tile_at(mj);
      wsg = wsc + (size_t)min(2 * cur.tn + wn, GN - 1) * KB;
    }
    ws = scalar_scale(wsg, mp);
  }
  tile::wait_vmcnt<0>();   // no copy may land after the workgroup's LDS is given away
}

namespace {

int persistent_grid(int total) {
  const int cus = device_cu_count();
  return total <= cus ? total : (cus >= 8 ? cus - cus % 8 : cus);
}

template <bool kPart>
int launch_small(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const float* wsc, int64_t N,
                 const void* bias, void* y, int64_t ldy, hipStream_t stream, int splits, void* part) {
  constexpr int lds = SmallLds::kBytes;
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)gemm_b128_small_kernel<kPart>, lds, lds_set)) return -7;
  const int G = (int)b128_blocks(N), tiles_m = (int)((M + kMT - 1) / kMT);
  const int vec = (ldy % 8 == 0) && (((uintptr_t)y & 15) == 0);
  hipLaunchKernelGGL(gemm_b128_small_kernel<kPart>, dim3((unsigned)(G * tiles_m * splits)), dim3(kB128Threads), lds,
                     stream, (const uint8_t*)qp, (const uint8_t*)sp, (int)M, (int)b128_blocks(K), (const uint8_t*)wp,
                     wsc, (int)N, (const uint16_t*)bias, (uint16_t*)y, ldy, G, tiles_m, splits, vec, (float*)part,
                     (N + 3) / 4 * 4);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

template <int kG, bool kPart>
int launch_large(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const float* wsc, int64_t N,
                 const void* bias, void* y, int64_t ldy, hipStream_t stream, int splits, void* part) {
  constexpr int lds = BigLds<kG>::kBytes;
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)gemm_b128_big_kernel<kG, kPart>, lds, lds_set)) return -7;
  const int GN = (int)b128_blocks(N), tiles_n = (GN + kG - 1) / kG, tiles_m = (int)b128_blocks(M);
  const int total = tiles_n * tiles_m * splits;
  hipLaunchKernelGGL((gemm_b128_big_kernel<kG, kPart>), dim3((unsigned)persistent_grid(total)), dim3(kB128Threads), lds,
                     stream, (const uint8_t*)qp, (const uint8_t*)sp, (int)M, (int)b128_blocks(K), (const uint8_t*)wp,
                     wsc, (int)N, (const uint16_t*)bias, (uint16_t*)y, ldy, GN, tiles_n, tiles_m,
                     __builtin_ctz((unsigned)splits), total, (float*)part, (N + 3) / 4 * 4);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

int launch_wide(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const float* wsc, int64_t N,
                const void* bias, void* y, int64_t ldy, hipStream_t stream) {
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)gemm_b128_wide_kernel, kWideLds, lds_set)) return -7;
  const int GN = (int)b128_blocks(N), GM = (int)b128_blocks(M), tiles_n = (GN + 1) / 2, tiles_m = (GM + 1) / 2;
  const int total = tiles_n * tiles_m;
  hipLaunchKernelGGL(gemm_b128_wide_kernel, dim3((unsigned)persistent_grid(total)), dim3(kWideThreads), kWideLds,
                     stream, (const uint8_t*)qp, (const uint8_t*)sp, (int)M, (int)b128_blocks(K), (const uint8_t*)wp,
                     wsc, (int)N, (const uint16_t*)bias, (uint16_t*)y, ldy, GN, GM, tiles_n, tiles_m, total);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace

int launch_gemm_b128_tile(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const float* wsc,
                          int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream, B128Plan plan,
                          void* part) {
  int st;
  if (plan.splits > 1) {
    st = plan.mt == 64 ? launch_small<true>(qp, sp, M, K, wp, wsc, N, bias, y, ldy, stream, plan.splits, part)
                       : launch_large<1, true>(qp, sp, M, K, wp, wsc, N, bias, y, ldy, stream, plan.splits, part);
    return st ? st : launch_splitk_reduce((const float*)part, plan.splits, M, N, (N + 3) / 4 * 4, bias, y, ldy, stream);
  }
  // The larger forms store y in 16-byte pieces with 32-bit offsets.
  const bool whole = ldy % 8 == 0 && ((uintptr_t)y & 15) == 0 && ldy <= (1 << 23);
  if (plan.mt == 64 || !whole) return launch_small<false>(qp, sp, M, K, wp, wsc, N, bias, y, ldy, stream, 1, nullptr);
  if (plan.mt == 128) return launch_large<1, false>(qp, sp, M, K, wp, wsc, N, bias, y, ldy, stream, 1, nullptr);
  if (plan.mt == 256) return launch_large<2, false>(qp, sp, M, K, wp, wsc, N, bias, y, ldy, stream, 1, nullptr);
  return launch_wide(qp, sp, M, K, wp, wsc, N, bias, y, ldy, stream);
}

}  // namespace mxfp8
