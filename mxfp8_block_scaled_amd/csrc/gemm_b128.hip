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
      ws[u] = wsg[b];
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
    const float ws = wsg[p];
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

B128Plan b128_plan(int64_t M, int64_t N, int64_t K) {
  const int64_t G = b128_blocks(N), KB = b128_blocks(K);
  B128Plan p;
  p.mt = (M <= 64 || G * ((M + 127) / 128) < 256) ? 64 : 128;
  const int64_t tiles = G * ((M + p.mt - 1) / p.mt);
  // Runs of at least four blocks while the tiles alone do not give every
  // compute unit two workgroups.
  int64_t s = 1;
  while (s < kMaxSplitK && tiles * s < 512 && KB / (2 * s) >= 4) s *= 2;
  p.splits = (int)s;
  return p;
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
  const int st = plan.mt == 64 ? go(launch_b128_k<64, false>, launch_b128_k<64, true>)
                               : go(launch_b128_k<128, false>, launch_b128_k<128, true>);
  if (st || plan.splits == 1) return st;
  return launch_splitk_reduce((const float*)part, plan.splits, M, N, (N + 3) / 4 * 4, bias, y, ldy, stream);
}

}  // namespace mxfp8
