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
#include "common.hpp"
#include "launch_b128.hpp"
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
// Decode (M <= 16): a workgroup owns 16 weight rows over the whole K, its 16
// waves one run of 128-blocks each; activations are quantized on the way in.
// Bound by the weight's bytes (N K) and how many loads are in flight.  The
// run is walked kSteps blocks at a time, all loads of a turn ahead of its
// first conversion; the waves' sums meet once, in wave order, through LDS.
// ---------------------------------------------------------------------------
namespace {
constexpr int kDecWaves = 16;
constexpr int kDecThreads = 64 * kDecWaves;
}  // namespace

template <int kSteps>
struct DecodeLds {
  static constexpr int kChunksRow = kSteps * 16;    // 16-byte bf16 chunks per row of a turn
  static constexpr int kPitch = kSteps * 128 + 16;  // staged E4M3 row (+16: rows on distinct banks)
  static constexpr int kWave = 16 * kPitch + 16 * kSteps;
  static constexpr int kRed = kDecWaves * 64 * 16;
  static constexpr int kBytes = kRed + kDecWaves * kWave;
};

template <int kSteps>
__global__ __launch_bounds__(kDecThreads) void gemm_b128_decode_kernel(
    const uint16_t* __restrict__ x, int64_t ldx, int M, int64_t K, const uint8_t* __restrict__ wp,
    const float* __restrict__ wsc, int N, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t ldy,
    int vec_store) {
  using L = DecodeLds<kSteps>;
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

  const __amdgpu_buffer_rsrc_t brsrc = raw_rsrc(bias, (bias != nullptr && wave == 0) ? (uint32_t)N * 2u : 0u);
  uint32_t braw[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    braw[e] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(brsrc, (uint32_t)min(n0 + 4 * g + e, N - 1) * 2u, 0, 0);

  const uint8_t* wrow = wp + (size_t)grp * KS * kTileBytes + packed_off(r, 0, g, KS);
  const float* wsg = wsc + (size_t)grp * KB;
  const int total = M * L::kChunksRow;   // a multiple of 16: a block's sixteen lanes are all in or all out
  const int rr = min(i, M - 1);          // lanes past M repeat the last row; their outputs are dropped
  v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int u0 = kb; u0 < ke; u0 += kSteps) {
    uint4 xa[kSteps * 4];
#pragma unroll
    for (int q = 0; q < kSteps * 4; ++q) {
      xa[q] = make_uint4(0u, 0u, 0u, 0u);
      const int c = lane + 64 * q;
      if (c < total) {
        const int row = c / L::kChunksRow, col = c % L::kChunksRow;
        const int64_t k = (int64_t)(u0 + col / 16) * 128 + (col % 16) * 8;
        if (k < K) xa[q] = *reinterpret_cast<const uint4*>(x + (size_t)row * ldx + k);
      }
    }
    uint4 w0[kSteps], w1[kSteps];
    float ws[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int b = min(u0 + u, KB - 1);   // blocks past the run reload a valid one, times zero elements
      const uint8_t* wt = wrow + (size_t)(2 * b) * kPieceBytes;
      w0[u] = *reinterpret_cast<const uint4*>(wt);
      w1[u] = *reinterpret_cast<const uint4*>(wt + kPieceBytes);
      ws[u] = scalar_scale(wsg, b);
    }
    __builtin_amdgcn_sched_barrier(0);   // every load of the turn above the first conversion
#pragma unroll
    for (int q = 0; q < kSteps * 4; ++q) {
      if (64 * q < total) {
        const int c = lane + 64 * q;
        const int row = c / L::kChunksRow, col = c % L::kChunksRow;
        const uint32_t wv[4] = {xa[q].x, xa[q].y, xa[q].z, xa[q].w};
        u16x2 m = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = absmax_pk(m, wv[e]);
        uint32_t mm = quad_max(max((uint32_t)m[0], (uint32_t)m[1]));
        mm = max(mm, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mm, 0x141, 0xF, 0xF, true));
        mm = max(mm, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mm, 0x140, 0xF, 0xF, true));
        const uint32_t sb = b128_scale_byte(mm);
        uint32_t qv[2];
        cvt8s(wv, mx_scale_value(sb), qv);
        *reinterpret_cast<uint2*>(xq + row * L::kPitch + col * 8) = make_uint2(qv[0], qv[1]);
        if ((lane & 15) == 0) xs[row * kSteps + col / 16] = (uint8_t)sb;
      }
    }
    // One wave's LDS accesses execute in order; this keeps the compiler from
    // moving the reads above the writes, and the next turn's writes above these.
    asm volatile("" ::: "memory");
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const uint8_t* p = xq + rr * L::kPitch + u * 128 + 16 * g;
      const uint4 b0 = *reinterpret_cast<const uint4*>(p);
      const uint4 b1 = *reinterpret_cast<const uint4*>(p + 64);
      int sx = xs[rr * kSteps + u];
      v8i xb = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
      if (u0 + u >= ke) {
        xb = v8i{0, 0, 0, 0, 0, 0, 0, 0};
        sx = 0;
      }
      const v8i wa = {(int)w0[u].x, (int)w0[u].y, (int)w0[u].z, (int)w0[u].w,
                      (int)w1[u].x, (int)w1[u].y, (int)w1[u].z, (int)w1[u].w};
      const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0,
                                                                        kUnitScales, 0, sx);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(part[e], ws[u], acc[e]);
    }
    asm volatile("" ::: "memory");
  }

  // Lane (i, g) holds D[n = 4g + j][m = i], j = 0..3: the waves' sums in wave
  // (K) order, bias, one rounding.
  red[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  v4f part[kDecWaves];
#pragma unroll
  for (int w = 0; w < kDecWaves; ++w) part[w] = red[w * 64 + lane];
  __builtin_amdgcn_sched_barrier(0);
  acc = part[0];
#pragma unroll
  for (int w = 1; w < kDecWaves; ++w) acc += part[w];
  const int n = n0 + 4 * g;
  if (i >= M || n >= N) return;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = acc[e] + __uint_as_float(braw[e] << 16);
  uint16_t* yrow = y + (size_t)i * ldy;
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
template <int kSteps>
int launch_decode_k(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const float* wsc, int64_t N,
                    const void* bias, void* y, int64_t ldy, hipStream_t stream) {
  constexpr int lds = DecodeLds<kSteps>::kBytes;
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)gemm_b128_decode_kernel<kSteps>, lds, lds_set)) return -7;
  const int vec = (ldy % 4 == 0) && (((uintptr_t)y & 7) == 0);
  hipLaunchKernelGGL((gemm_b128_decode_kernel<kSteps>), dim3((unsigned)((N + 15) / 16)), dim3(kDecThreads), lds,
                     stream, (const uint16_t*)x, ldx, (int)M, K, (const uint8_t*)wp, wsc, (int)N,
                     (const uint16_t*)bias, (uint16_t*)y, ldy, vec);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}
}  // namespace

int launch_gemm_b128_decode(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const float* wsc,
                            int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream) {
  // Two blocks per wave and turn up to K = 4096 (one turn), four above.
  if (K <= kDecWaves * 2 * 128) return launch_decode_k<2>(x, ldx, M, K, wp, wsc, N, bias, y, ldy, stream);
  return launch_decode_k<4>(x, ldx, M, K, wp, wsc, N, bias, y, ldy, stream);
}

// ---------------------------------------------------------------------------
// Tiles: one 128-row weight group x kMT activation rows per workgroup over a
// run of 128-blocks, four waves 2 x 2; wave (wn, wm) owns weight rows
// 32 a + 16 wn + i and activation rows 32 b + 16 wm + i, so the byte of a
// row's scale inside its packed word (rows r + 32 k, byte k) is b, an
// immediate op_sel.  Stages of 64 K come straight from global memory into
// LDS; a 128-block reads a pair of stages; two pairs are in flight.
// ---------------------------------------------------------------------------
namespace {
constexpr int kB128Threads = 256;

template <int kMT>
struct B128Lds {
  static constexpr int kW = kGroupRows * kStepK;
  static constexpr int kX = kMT * kStepK;
  // + the activations' 256-byte scale tile, copied by wave 0; the other
  // waves' scale copies go to slots of their own, so every wave issues the
  // same number of copies (the waits count them per wave).
  static constexpr int kStage = kW + kX + 1024;
  static constexpr int kBytes = 4 * kStage;
  static constexpr int kCopies = 2 * (2 + kMT / 64 + 1);
  static constexpr int kPitchY = 128 * 2 + 16;
  static_assert(kMT * kPitchY <= kBytes, "the output staging fits in the stages");
};
}  // namespace

template <int kMT, bool kPart>
__global__ __launch_bounds__(kB128Threads, 2) void gemm_b128_kernel(
    const uint8_t* __restrict__ qp, const uint8_t* __restrict__ sp, int M, int KB, const uint8_t* __restrict__ wp,
    const float* __restrict__ wsc, int N, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t ldy,
    int tiles_n, int tiles_m, int splits, int vec, float* __restrict__ part, int64_t ldp) {
  using L = B128Lds<kMT>;
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

  // Copies: wave w takes bands w and w + 4 of the weight group and of the
  // activation group (kMT = 64: band 4 h + w of half h of group tm / 2).
  const int h = kMT == 64 ? (tm & 1) : 0;
  const int xg = kMT == 64 ? (tm >> 1) : tm;
  const uint32_t gbytes = (uint32_t)KS * kTileBytes, sbytes = (uint32_t)KS * kTileScaleBytes;
  const tile::i4v wr = tile::buffer_rsrc(wp + (size_t)tn * gbytes, gbytes);
  const tile::i4v xr = tile::buffer_rsrc(qp + (size_t)xg * gbytes, gbytes);
  const tile::i4v sr = tile::buffer_rsrc(sp + (size_t)xg * sbytes, sbytes);
  const uint32_t lo16 = (uint32_t)lane * 16u;
  const uint32_t vw0 = (uint32_t)wave * KS * kPieceBytes + lo16, vw1 = vw0 + 4u * KS * kPieceBytes;
  const uint32_t vx0 = (uint32_t)(kMT == 64 ? 4 * h + wave : wave) * KS * kPieceBytes + lo16;
  const uint32_t vx1 = vx0 + 4u * KS * kPieceBytes;
  const uint32_t vs = (uint32_t)lane * 4u;
  auto issue_stage = [&](int ks, uint8_t* st) {
    const uint32_t off = (uint32_t)ks * kPieceBytes;
    tile::b2l_16(vw0, wr, off, st + wave * 1024);
    tile::b2l_16(vw1, wr, off, st + 4096 + wave * 1024);
    tile::b2l_16(vx0, xr, off, st + L::kW + wave * 1024);
    if constexpr (kMT == 128) tile::b2l_16(vx1, xr, off, st + L::kW + 4096 + wave * 1024);
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
  issue_stage(2 * p0, stage_ptr(0));
  issue_stage(2 * p0 + 1, stage_ptr(1));
  if (p0 + 1 < p1) {
    issue_stage(2 * p0 + 2, stage_ptr(2));
    issue_stage(2 * p0 + 3, stage_ptr(3));
  }
  for (int p = p0; p < p1; ++p) {
    const float ws = scalar_scale(wsg, p);
    if (p + 1 < p1)
      tile::wait_vmcnt<L::kCopies>();
    else
      tile::wait_vmcnt<0>();
    __builtin_amdgcn_s_barrier();
    const int par = (p - p0) & 1;
    const uint8_t* ev = stage_ptr(2 * par);
    const uint8_t* od = ev + L::kStage;
    v8i wf[4], xf[kNB];
#pragma unroll
    for (int a = 0; a < 4; ++a) wf[a] = frag(ev, od, offW + 32 * kStepK * a);
#pragma unroll
    for (int b = 0; b < kNB; ++b) xf[b] = frag(ev, od, offX + 32 * kStepK * b);
    int sx = *reinterpret_cast<const int*>(((g >> 1) ? od : ev) + offSX);
    if constexpr (kMT == 64) sx = (int)((uint32_t)sx >> (16 * h));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    if (p + 2 < p1) {
      issue_stage(2 * p + 4, stage_ptr(2 * par));
      issue_stage(2 * p + 5, stage_ptr(2 * par + 1));
    }
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
// Large tiles: 256 weight rows (two groups) x 128 activation rows per
// workgroup, four waves 2 x 2, each 128 x 64 (32 MFMAs per 128-block).
//  * The accumulators are 128 vector registers per lane; the operand
//    fragments of the current and of the next block sit in registers too
//    (96 + 96, one wave per SIMD has 512), so no MFMA waits for LDS.
//  * LDS holds three blocks (3 x 49 KiB).  At the top of step p the copies of
//    p + 1 have landed everywhere (own vmcnt, then the one barrier of the
//    step), every wave has read p, and the copies of p + 3 go out into p's
//    buffer: a copy has two whole steps to land.
//  * The MFMAs of a step carry between them the v_fma of the results three
//    MFMAs back (nearer ones are not there yet), the LDS reads of the next step's fragments and the copies.
//  * Workgroups are persistent and the pipeline runs across tiles: the last
//    steps of a tile copy and read the next one's first blocks.  The epilogue
//    issues a fixed sixteen 16-byte stores per wave (rows and columns outside
//    are dropped by the buffer bounds), left in flight into the next tile.
// ---------------------------------------------------------------------------
namespace {

constexpr int kBigX = 16384;                       // activation pieces inside a 64-K half
constexpr int kBigHalf = 16384 + 8192;             // 256 weight rows + 128 activation rows x 64 B
constexpr int kBigScale = 2 * kBigHalf;            // two 256-byte scale tiles, then two unused slots
constexpr int kBigBlock = 2 * kBigHalf + 1024;
constexpr int kBigLds = 3 * kBigBlock;             // 150528
constexpr int kBigCopies = 13;                     // per wave and block
constexpr int kBigStores = 16;                     // per wave and tile

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

}  // namespace

__global__ __launch_bounds__(kB128Threads, 1) void gemm_b128_big_kernel(
    const uint8_t* __restrict__ qp, const uint8_t* __restrict__ sp, int M, int KB, const uint8_t* __restrict__ wp,
    const float* __restrict__ wsc, int N, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t ldy,
    int GN, int tiles_n, int tiles_m, int total) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int i = lane & 15, g = lane >> 4;
  const int KS = 2 * KB;
  const uint32_t gbytes = (uint32_t)KS * kTileBytes, sbytes = (uint32_t)KS * kTileScaleBytes;

  // This workgroup's tiles: items wg, wg + grid, ... of the die-wise order.
  const int grid = (int)gridDim.x;
  const int mine = (total - (int)blockIdx.x + grid - 1) / grid;
  const int steps = mine * KB;
  auto tile_at = [&](int j) { return big_tile(xcd_remap((int)blockIdx.x + j * grid, total), tiles_n, tiles_m); };

  // Copy side: the tile the next copies belong to.
  struct Src {
    tile::i4v w0, w1, x, s;
  };
  auto src_of = [&](BigTile t) {
    Src r;
    const int g1 = min(2 * t.tn + 1, GN - 1);      // past the last group: any data, its columns are dropped
    r.w0 = tile::buffer_rsrc(wp + (size_t)(2 * t.tn) * gbytes, gbytes);
    r.w1 = tile::buffer_rsrc(wp + (size_t)g1 * gbytes, gbytes);
    r.x = tile::buffer_rsrc(qp + (size_t)t.tm * gbytes, gbytes);
    r.s = tile::buffer_rsrc(sp + (size_t)t.tm * sbytes, sbytes);
    return r;
  };
  const uint32_t v0 = (uint32_t)wave * KS * kPieceBytes + (uint32_t)lane * 16u, v1 = v0 + 4u * KS * kPieceBytes;
  const uint32_t vs = (uint32_t)lane * 4u;
  auto copy = [&](int j, const Src& r, int p, uint8_t* st) {
    const uint32_t off = (uint32_t)(2 * p) * kPieceBytes;
    uint8_t* b = st + wave * 1024;
    switch (j) {
      case 0: tile::b2l_16(v0, r.w0, off, b); break;
      case 1: tile::b2l_16(v1, r.w0, off, b + 4096); break;
      case 2: tile::b2l_16(v0, r.w1, off, b + 8192); break;
      case 3: tile::b2l_16(v1, r.w1, off, b + 12288); break;
      case 4: tile::b2l_16(v0, r.x, off, b + kBigX); break;
      case 5: tile::b2l_16(v1, r.x, off, b + kBigX + 4096); break;
      case 6: tile::b2l_16(v0, r.w0, off + kPieceBytes, b + kBigHalf); break;
      case 7: tile::b2l_16(v1, r.w0, off + kPieceBytes, b + kBigHalf + 4096); break;
      case 8: tile::b2l_16(v0, r.w1, off + kPieceBytes, b + kBigHalf + 8192); break;
      case 9: tile::b2l_16(v1, r.w1, off + kPieceBytes, b + kBigHalf + 12288); break;
      case 10: tile::b2l_16(v0, r.x, off + kPieceBytes, b + kBigHalf + kBigX); break;
      case 11: tile::b2l_16(v1, r.x, off + kPieceBytes, b + kBigHalf + kBigX + 4096); break;
      default:
        // waves 0 and 1 copy the block's two scale tiles, 2 and 3 copy them to the unused slots
        tile::b2l_4(vs, r.s, (uint32_t)(2 * p + (wave & 1)) * kTileScaleBytes, st + kBigScale + wave * 256);
        break;
    }
  };

  const int offW = wn * 8192 + tile_off(i, g);
  const int offX = kBigX + 16 * wm * kStepK + tile_off(i, g);
  const int offS = kBigScale + (g >> 1) * 256 + (16 * wm + i) * 8 + (g & 1) * 4;
  struct Frags {
    v8i w[8], x[4];
    int s;
  };
  auto rd16 = [](const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); };
  auto frag = [&](const uint8_t* st, int off) {
    const uint4 lo = rd16(st + off), hi = rd16(st + off + kBigHalf);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  // Part j of the fragment reads of a block: its scale word and activation
  // fragments first.
  auto read = [&](int j, const uint8_t* st, Frags& f) {
    if (j == 0) f.s = *reinterpret_cast<const int*>(st + offS);
    if (j < 4) f.x[j] = frag(st, offX + 32 * kStepK * j);
    else if (j < 12) f.w[j - 4] = frag(st, offW + 16 * kStepK * (j - 4));
  };

  v4f acc[8][4];
  auto clear = [&] {
#pragma unroll
    for (int a = 0; a < 8; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[a][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();

  // Positions in the flattened (tile, block) sequence: of the copies (three
  // steps ahead) and of the MFMAs.
  int cj = 0, cp = 0, mj = 0, mp = 0;
  Src src = src_of(tile_at(0));
  // Past the last tile the copies go on with its blocks again (never used),
  // so the steps need no branch and the waits no other counts.
  auto advance_copy = [&] {
    if (++cp == KB) {
      cp = 0;
      cj = min(cj + 1, mine - 1);
      src = src_of(tile_at(cj));
    }
  };
  BigTile cur = tile_at(0);
  const float* wsg = wsc + (size_t)min(2 * cur.tn + wn, GN - 1) * KB;
  auto buf = [&](int b) { return smem + b * kBigBlock; };
#pragma unroll
  for (int s = 0; s < 3; ++s) {   // KB >= 4: three blocks of the first tile
#pragma unroll
    for (int j = 0; j < kBigCopies; ++j) copy(j, src, cp, buf(s));
    advance_copy();
  }
  tile::wait_vmcnt<2 * kBigCopies>();
  __builtin_amdgcn_s_barrier();
  Frags f0, f1;
#pragma unroll
  for (int j = 0; j < 12; ++j) read(j, buf(0), f0);
  float ws = scalar_scale(wsg, 0);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");

  // Lane (i, g) holds D[n = 128 wn + 16 a + 4 g + j][m = 32 b + 16 wm + i].
  // Exchanging the odd 16-lane rows of tile a with the even ones of tile a + 1
  // gives every lane eight consecutive n: rows 0, 2 of tile a, rows 1, 3 of
  // tile a + 1.
  auto epilogue = [&](BigTile t) {
    const int n0 = t.tn * 256 + wn * 128, m0 = t.tm * 128;
    const int nl = 16 * (g & 1) + 8 * (g >> 1);
    const int rows = min(128, M - m0);
    const __amdgpu_buffer_rsrc_t yr =
        raw_rsrc(y + (size_t)m0 * ldy, (uint32_t)(((int64_t)(rows - 1) * ldy + N) * 2));
    const __amdgpu_buffer_rsrc_t br = raw_rsrc(bias, bias != nullptr ? (uint32_t)N * 2u : 0u);
#pragma unroll
    for (int a = 0; a < 8; a += 2) {
      const int n = n0 + 16 * a + nl;
      const int nb = n0 + 16 * a + 4 * g;
      float bv[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          bv[h][j] = __uint_as_float(
              (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(br, (uint32_t)(nb + 16 * h + j) * 2u, 0, 0) << 16);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t q[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4f v = acc[a + h][b];
          q[h][0] = pack_bf16x2(v[0] + bv[h][0], v[1] + bv[h][1]);
          q[h][1] = pack_bf16x2(v[2] + bv[h][2], v[3] + bv[h][3]);
        }
        const auto s0 = __builtin_amdgcn_permlane16_swap(q[0][0], q[1][0], false, false);
        const auto s1 = __builtin_amdgcn_permlane16_swap(q[0][1], q[1][1], false, false);
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const u32x4 o = {s0[0], s1[0], s0[1], s1[1]};
        // a column past N (N % 8 == 0: whole stores) or a row past M gets an offset past the end
        const int m = 32 * b + 16 * wm + i;
        const uint32_t at = (n < N && m < rows) ? (uint32_t)(((int64_t)m * ldy + n) * 2) : 0xFFFFFFF0u;
        __builtin_amdgcn_raw_buffer_store_b128(o, yr, at, 0, 0);
      }
    }
    clear();
  };

  int s = 0;
  bool stores = false;   // the stores of the last epilogue may be outstanding
  auto step = [&](Frags& f, Frags& fn, int rb) {
    // Newer than the copies of s + 1: those of s + 2, and in a tile's first
    // two steps the last epilogue's stores.
    if (stores && mp < 2) tile::wait_vmcnt<kBigCopies + kBigStores>();
    else tile::wait_vmcnt<kBigCopies>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    uint8_t* const st_free = buf(rb);
    const uint8_t* const st_next = buf(rb == 2 ? 0 : rb + 1);
    v4f d[4];
    // The empty asm statements keep each MFMA and each result's v_fma in its
    // place in the stream of reads and copies: as pure operations they would
    // otherwise sink below all of them.
    tile::static_for<0, 35>([&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (j < 32) {
        d[j & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f.w[j >> 2], f.x[j & 3], v4f{0.0f, 0.0f, 0.0f, 0.0f},
                                                                    0, 0, 0, kUnitScales, j & 3, f.s);
        asm volatile("" : "+v"(d[j & 3]));
      }
      if constexpr (j < 24 && (j & 1) == 0) read(j >> 1, st_next, fn);
      if constexpr (j < 26 && (j & 1) == 1) copy(j >> 1, src, cp, st_free);
      if constexpr (j >= 3) {
        constexpr int k = j - 3;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k >> 2][k & 3][e] = fmaf(d[k & 3][e], ws, acc[k >> 2][k & 3][e]);
        asm volatile("" : "+v"(acc[k >> 2][k & 3]));
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    advance_copy();
    if (++mp == KB) {
      epilogue(cur);
      stores = true;
      mp = 0;
      mj = min(mj + 1, mine - 1);
      cur = tile_at(mj);
      wsg = wsc + (size_t)min(2 * cur.tn + wn, GN - 1) * KB;
    }
    ws = scalar_scale(wsg, mp);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    ++s;
  };
  int rb = 0;
  while (s < steps) {
    step(f0, f1, rb);
    rb = rb == 2 ? 0 : rb + 1;
    if (s >= steps) break;
    step(f1, f0, rb);
    rb = rb == 2 ? 0 : rb + 1;
  }
  tile::wait_vmcnt<0>();   // no copy may land after the workgroup's LDS is given away
}

namespace {
std::atomic<int> g_force_mt{0};
}

int b128_force(int mt) { return g_force_mt.exchange(mt); }

// The form and K splits with the least estimated time.  The estimates are
// lines through measurements on MI355X (us; M 17 .. 8192, N and K 512 ..
// 28672): a start of about 5, a cost per 128-block and round of workgroups
// (two of the 64- and 128-row tiles share a compute unit; alone on it one
// walks its blocks almost twice as fast), and for K splits a second launch
// and the partials' way to memory and back at about 4 TB/s.  For example
// M = 1024, N = K = 4096: 64-row tiles 26, 128-row 33, large 32;
// M = 2048: 53, 40, 36; M = 256, N = 512, K = 8192: 13 with eight splits, 51
// with large tiles.
B128Plan b128_plan(int64_t M, int64_t N, int64_t K) {
  const int64_t G = b128_blocks(N), KB = b128_blocks(K);
  const int force = g_force_mt.load(std::memory_order_relaxed);
  B128Plan best = {128, 1};
  double best_us = 1e30;
  auto offer = [&](int mt, int splits, double us) {
    if (us < best_us) {
      best_us = us;
      best = {mt, splits};
    }
  };
  for (int mt = 64; mt <= 128; mt *= 2) {
    if (force && force != mt && !(force == 256 && mt == 128)) continue;
    const int64_t tiles = G * ((M + mt - 1) / mt);
    for (int s = 1; s <= kMaxSplitK && (s == 1 || KB / s >= 2); s *= 2) {
      const int64_t items = tiles * s, rounds = (items + 511) / 512;
      const double block = mt == 64 ? (items <= 256 ? 0.35 : 0.67 * (double)rounds)
                                    : (items <= 256 ? 0.8 : 1.1 * (double)rounds);
      const double join = s > 1 ? 3.0 + (double)s * (double)M * (double)N * 8.0 / 4e6 : 0.0;
      offer(mt, s, 4.5 + block * (double)((KB + s - 1) / s) + join);
    }
  }
  // Large tiles need a run of four blocks and whole 16-byte stores.
  if ((!force || force == 256) && KB >= 4 && N % 8 == 0) {
    const int64_t tiles = (G + 1) / 2 * ((M + 127) / 128), rounds = (tiles + 255) / 256;
    const double us = 5.0 + (tiles <= 128 ? 0.73 : 0.95 * (double)rounds) * (double)KB;
    if (force == 256) best_us = 1e30;
    offer(256, 1, us);
  }
  return best;
}

namespace {
template <int kMT, bool kPart>
int launch_b128_k(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const float* wsc, int64_t N,
                  const void* bias, void* y, int64_t ldy, hipStream_t stream, int splits, void* part) {
  constexpr int lds = B128Lds<kMT>::kBytes;
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)gemm_b128_kernel<kMT, kPart>, lds, lds_set)) return -7;
  const int G = (int)b128_blocks(N), tiles_m = (int)((M + kMT - 1) / kMT);
  const int vec = (ldy % 8 == 0) && (((uintptr_t)y & 15) == 0);
  hipLaunchKernelGGL((gemm_b128_kernel<kMT, kPart>), dim3((unsigned)(G * tiles_m * splits)), dim3(kB128Threads), lds,
                     stream, (const uint8_t*)qp, (const uint8_t*)sp, (int)M, (int)b128_blocks(K), (const uint8_t*)wp,
                     wsc, (int)N, (const uint16_t*)bias, (uint16_t*)y, ldy, G, tiles_m, splits, vec, (float*)part,
                     (N + 3) / 4 * 4);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}
}  // namespace

int launch_gemm_b128_tile(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const float* wsc,
                          int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream, B128Plan plan,
                          void* part) {
  auto go = [&](auto one, auto many) {
    return plan.splits > 1 ? many(qp, sp, M, K, wp, wsc, N, bias, y, ldy, stream, plan.splits, part)
                           : one(qp, sp, M, K, wp, wsc, N, bias, y, ldy, stream, 1, part);
  };
  if (plan.mt == 256 && ldy % 8 == 0 && ((uintptr_t)y & 15) == 0 && ldy <= (1 << 23)) {
    static std::atomic<int> lds_set[kMaxDevices];
    if (!set_lds_limit_once((const void*)gemm_b128_big_kernel, kBigLds, lds_set)) return -7;
    const int GN = (int)b128_blocks(N), tiles_n = (GN + 1) / 2, tiles_m = (int)b128_blocks(M);
    const int total = tiles_n * tiles_m, cus = device_cu_count();
    const int grid = total <= cus ? total : (cus >= 8 ? cus - cus % 8 : cus);
    hipLaunchKernelGGL(gemm_b128_big_kernel, dim3((unsigned)grid), dim3(kB128Threads), kBigLds, stream,
                       (const uint8_t*)qp, (const uint8_t*)sp, (int)M, (int)b128_blocks(K), (const uint8_t*)wp, wsc,
                       (int)N, (const uint16_t*)bias, (uint16_t*)y, ldy, GN, tiles_n, tiles_m, total);
    return hipGetLastError() == hipSuccess ? 0 : -7;
  }
  const int st = plan.mt == 64 ? go(launch_b128_k<64, false>, launch_b128_k<64, true>)
                               : go(launch_b128_k<128, false>, launch_b128_k<128, true>);
  if (st || plan.splits == 1) return st;
  return launch_splitk_reduce((const float*)part, plan.splits, M, N, (N + 3) / 4 * 4, bias, y, ldy, stream);
}

}  // namespace mxfp8
