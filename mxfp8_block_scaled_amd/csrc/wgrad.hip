// Weight gradient of a linear layer from its 8-bit activation checkpoint:
//   dW[n, k] = sum_m dY[m, n] * deq(X)[m, k],   db[n] = sum_m dY[m, n]
// dY bf16, X the packed E4M3 activations the forward GEMM read, with a
// power-of-two scale per 32 (MX) or 128 elements of a row.
//
// The sum runs over the tokens, across the scale blocks, so the scales cannot
// ride along the scaled MFMA.  E4M3 times a power of two is exact in bf16,
// so X is widened while it is staged (v_cvt_scalef32_pk_bf16_fp8, two values
// an instruction) and the product runs on v_mfma_f32_16x16x32_bf16 with exact
// products and fp32 sums: no rounding but the fp32 additions.
//
// Both operands have the summed axis as their slow axis.  They are staged in
// LDS as they lie in memory and read with the transposing LDS load
// (ds_read_b64_tr_b16: sixteen lanes read four rows of sixteen columns and
// each gets one column's four rows).
//  * A workgroup owns kT x kT of dW and a run of 64-token steps; four waves
//    2 x 2.  X is the MFMA A operand, so a lane ends with four consecutive k
//    of one n: dW rows are written in 16-byte pieces.
//  * Stages are double-buffered: dY goes straight from global memory into
//    LDS, X through registers (loaded a step ahead, widened and written while
//    the MFMAs of the current step run).
//  * LDS rows are cut into 32-byte slots (one 16-column fragment); slot c of
//    row m sits at c ^ f(m), f = bits 0, 1, 3 of m: the four rows one
//    transposing read takes and the next lane group's four (8 further) land
//    on different banks.
//  * db costs one more MFMA per dY fragment (A = ones).  Step s of the sum is
//    done by the workgroups with tile index s % tiles_k along k, so every
//    workgroup does 1 / tiles_k of it.
// Partial sums of split runs and of db go to the workspace and are added in
// a fixed order: results do not depend on timing.
#include "common.hpp"
#include "launch_b128.hpp"
#include "tile_core.hpp"

namespace mxfp8 {

namespace {

constexpr int kWgThreads = 256;
constexpr int kWgStep = 64;   // tokens per step

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ inline int slot_xor(int m) { return (m & 3) | ((m >> 1) & 4); }

template <int kT>
struct WgLds {
  static constexpr int kPitch = kT * 2;
  static constexpr int kOp = kWgStep * kPitch;   // one operand's stage
  static constexpr int kBytes = 4 * kOp;         // two operands, two stages
};

}  // namespace

template <int kT, bool kBias>
__global__ __launch_bounds__(kWgThreads, kT == 128 ? 2 : 1) void wgrad_kernel(
    const uint16_t* __restrict__ dy, int64_t M, int N, int64_t lddy, const uint8_t* __restrict__ qp,
    const uint8_t* __restrict__ sp, int K, int KS, int tiles_n, int tiles_k, int splits, void* __restrict__ out,
    int64_t ldo, int64_t split_stride, int out_bf16, int accumulate, float* __restrict__ part_db) {
  using L = WgLds<kT>;
  constexpr int kF = kT / 32;       // 16-wide fragments per wave and axis
  constexpr int kXV = kT / 64;      // 16-byte X chunks per thread and step
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave & 1, wn = wave >> 1;
  const int i = lane & 15, g = lane >> 4;
  const int item = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int split = item % splits, t = item / splits;
  const int tn = t / tiles_k, tk = t - tn * tiles_k;
  const int n0 = tn * kT, k0 = tk * kT;
  const int64_t steps = (M + kWgStep - 1) / kWgStep;
  const int64_t s0 = steps * split / splits, s1 = steps * (split + 1) / splits;

  // dY: lane l of a copy takes LDS bytes [16 l, 16 l + 16) of its KiB, i.e.
  // half h of slot c of row m, which holds logical slot c ^ f(m).  Rows past
  // M are past the resource's end and read zero; columns past N belong to
  // outputs that are not stored.
  constexpr int kLanesRow = L::kPitch / 16, kRowsCopy = 64 / kLanesRow, kCopies = kWgStep / kRowsCopy / 4;
  uint32_t vy[kCopies];
#pragma unroll
  for (int c = 0; c < kCopies; ++c) {
    const int m = (wave * kCopies + c) * kRowsCopy + lane / kLanesRow, p = lane % kLanesRow;
    const int col = ((p >> 1) ^ slot_xor(m)) * 16 + (p & 1) * 8;
    vy[c] = (uint32_t)((int64_t)m * lddy + n0 + col) * 2u;
  }
  auto issue_dy = [&](int64_t s, uint8_t* st) {
    const int64_t m0 = s * kWgStep, rows = min(M - m0, (int64_t)kWgStep);
    const tile::i4v r = tile::buffer_rsrc(dy + m0 * lddy, (uint32_t)(((rows - 1) * lddy + N) * 2));
#pragma unroll
    for (int c = 0; c < kCopies; ++c) tile::b2l_16(vy[c], r, 0u, st + (wave * kCopies + c) * 1024);
  };
  // X: chunk j = tid + 256 v of the step's tile: piece (band, 64-K step) in
  // storage order, lane = chunk of the piece.  The group's scale byte of the
  // chunk's row and 32-block goes with it.
  struct X {
    uint4 q[kXV];
    uint32_t s[kXV];
  };
  uint32_t xoff[kXV], soff[kXV], xdst[kXV];
  bool xin[kXV];
#pragma unroll
  for (int v = 0; v < kXV; ++v) {
    const int piece = wave + 4 * v;                 // 0 .. kT/16 - 1: (band of 4) x (kT / 64 K steps)
    const int band = piece & 3, kst = piece >> 2;
    const int rr = lane >> 2, pos = lane & 3;
    const int c = pos ^ swz(rr);                    // logical 16-byte chunk
    const int m = band * 16 + rr;
    const int ks = k0 / kStepK + kst;
    xin[v] = ks < KS;
    xoff[v] = (uint32_t)((size_t)band * KS * kPieceBytes + (size_t)ks * kPieceBytes + lane * 16);
    // scale_off of row m of this half group (rows 64 .. 127: + 2)
    soff[v] = (uint32_t)(ks * kTileScaleBytes + scale_off(m, c >> 1));
    const int col16 = kst * 4 + c;                  // 32-byte slot of the bf16 row
    xdst[v] = (uint32_t)(m * L::kPitch + (col16 ^ slot_xor(m)) * 32);
  }
  auto load_x = [&](int64_t s, X& x) {
    const int64_t grp = s >> 1;
    const int half = (int)(s & 1);
    const uint8_t* q = qp + (size_t)grp * KS * kTileBytes + (size_t)half * 4 * KS * kPieceBytes;
    const uint8_t* sc = sp + (size_t)grp * KS * kTileScaleBytes + half * 2;
#pragma unroll
    for (int v = 0; v < kXV; ++v) {
      x.q[v] = make_uint4(0u, 0u, 0u, 0u);
      x.s[v] = 0;
      if (xin[v]) {
        x.q[v] = *reinterpret_cast<const uint4*>(q + xoff[v]);
        x.s[v] = sc[soff[v]];
      }
    }
  };
  auto store_x = [&](const X& x, uint8_t* st) {
#pragma unroll
    for (int v = 0; v < kXV; ++v) {
      uint4 d[2];
      widen16(x.q[v], b128_scale_value(x.s[v]), d);
      *reinterpret_cast<uint4*>(st + xdst[v]) = d[0];
      *reinterpret_cast<uint4*>(st + xdst[v] + 16) = d[1];
    }
  };

  // Fragment f (sixteen columns) and 32-token half h of a stage: lane (i, g)
  // gets tokens 32 h + 8 g .. + 7 of column i.
  const int fr = 8 * g + (i >> 2);   // first token row the lane addresses; + 4 for the second read
  auto frag = [&](const uint8_t* st, int c16, int h) {
    const int m = 32 * h + fr;
    const uint8_t* p = st + m * L::kPitch + ((c16 ^ slot_xor(m)) * 32) + (i & 3) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * L::kPitch));
    const s16x8 r = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, r);
  };

  v4f acc[kF][kF];
  v4f accb[kF];
#pragma unroll
  for (int a = 0; a < kF; ++a) {
    accb[a] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int b = 0; b < kF; ++b) acc[a][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  bf16x8 ones;
#pragma unroll
  for (int e = 0; e < 8; ++e) ones[e] = (__bf16)1.0f;

  auto sy = [&](int b) { return smem + b * L::kOp; };
  auto sx = [&](int b) { return smem + (2 + b) * L::kOp; };
  X xr;
  if (s0 < s1) {
    issue_dy(s0, sy(0));
    load_x(s0, xr);
    store_x(xr, sx(0));
    if (s0 + 1 < s1) load_x(s0 + 1, xr);
  }
  int phase = (int)(s0 % tiles_k);
  for (int64_t s = s0; s < s1; ++s) {
    const int par = (int)(s - s0) & 1;
    // This step's dY copies and X stores of every wave have landed; the
    // other buffers, read in the previous step, are free after the barrier.
    tile::wait_vmcnt<0>();
    __syncthreads();
    if (s + 1 < s1) {
      issue_dy(s + 1, sy(par ^ 1));
      store_x(xr, sx(par ^ 1));
      if (s + 2 < s1) load_x(s + 2, xr);
    }
    const bool with_bias = kBias && wk == 0 && phase == tk;
    phase = phase + 1 == tiles_k ? 0 : phase + 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 fx[kF], fy[kF];
#pragma unroll
      for (int a = 0; a < kF; ++a) fx[a] = frag(sx(par), wk * kF + a, h);
#pragma unroll
      for (int b = 0; b < kF; ++b) fy[b] = frag(sy(par), wn * kF + b, h);
#pragma unroll
      for (int a = 0; a < kF; ++a)
#pragma unroll
        for (int b = 0; b < kF; ++b) acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fx[a], fy[b], acc[a][b], 0, 0, 0);
      if (with_bias) {
#pragma unroll
        for (int b = 0; b < kF; ++b) accb[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, fy[b], accb[b], 0, 0, 0);
      }
    }
  }

  // Lane (i, g) holds D[k = 16 a + 4 g + j][n = 16 b + i] of its wave's tile.
  float* of = (float*)out + (size_t)split * split_stride;
#pragma unroll
  for (int b = 0; b < kF; ++b) {
    const int n = n0 + (wn * kF + b) * 16 + i;
    if (n >= N) continue;
#pragma unroll
    for (int a = 0; a < kF; ++a) {
      const int k = k0 + (wk * kF + a) * 16 + 4 * g;
      if (k >= K) continue;   // K % 16 == 0: a quad is all in or all out
      if (out_bf16) {
        *reinterpret_cast<uint2*>((uint16_t*)out + (size_t)n * ldo + k) =
            make_uint2(pack_bf16x2(acc[a][b][0], acc[a][b][1]), pack_bf16x2(acc[a][b][2], acc[a][b][3]));
      } else {
        v4f* d = reinterpret_cast<v4f*>(of + (size_t)n * ldo + k);
        *d = accumulate ? *d + acc[a][b] : acc[a][b];
      }
    }
    // every row of the ones product holds the column sums
    if (kBias && wk == 0 && g == 0) part_db[((size_t)split * tiles_k + tk) * N + n] = accb[b][0];
  }
}

// dw = sum of the split partials in order (+ dw), db = sum of its partials in
// order.  One thread per 4 k of dW, then one per n of db.
__global__ __launch_bounds__(256) void wgrad_reduce_kernel(const float* __restrict__ part, int splits, int64_t N,
                                                           int64_t K, void* __restrict__ dw, int64_t lddw,
                                                           int out_bf16, int accumulate, int64_t quads,
                                                           const float* __restrict__ part_db, int parts_db,
                                                           float* __restrict__ db) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t < quads) {
    const int64_t per_row = K / 4, n = t / per_row, k = (t - n * per_row) * 4;
    v4f a = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < splits; ++s) a += *reinterpret_cast<const v4f*>(part + ((size_t)s * N + n) * K + k);
    if (out_bf16) {
      *reinterpret_cast<uint2*>((uint16_t*)dw + (size_t)n * lddw + k) =
          make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
    } else {
      v4f* d = reinterpret_cast<v4f*>((float*)dw + (size_t)n * lddw + k);
      *d = accumulate ? *d + a : a;
    }
    return;
  }
  const int64_t n = t - quads;
  if (n >= N || db == nullptr) return;
  float a = 0.0f;
  for (int p = 0; p < parts_db; ++p) a += part_db[(size_t)p * N + n];
  db[n] = accumulate ? db[n] + a : a;
}

WgradPlan wgrad_plan(int64_t M, int64_t N, int64_t K) {
  WgradPlan p;
  p.tile = 128;
  const int64_t tiles = ((N + p.tile - 1) / p.tile) * ((K + p.tile - 1) / p.tile);
  const int64_t steps = (M + kWgStep - 1) / kWgStep, want = 512;   // two workgroups per compute unit
  int64_t s = 1;
  while (s < 16 && tiles * s < want && steps / (2 * s) >= 4) s *= 2;
  p.splits = (int)s;
  return p;
}

size_t wgrad_dw_bytes(int64_t N, int64_t K, WgradPlan p) {
  return p.splits > 1 ? (size_t)p.splits * (size_t)N * (size_t)K * 4 : 0;
}
size_t wgrad_db_bytes(int64_t N, int64_t K, WgradPlan p) {
  return (size_t)p.splits * (size_t)((K + p.tile - 1) / p.tile) * (size_t)N * 4;
}

namespace {
template <int kT, bool kBias>
int launch_wgrad_k(const WgradArgs& a, WgradPlan p, hipStream_t stream) {
  constexpr int lds = WgLds<kT>::kBytes;
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)wgrad_kernel<kT, kBias>, lds, lds_set)) return -7;
  const int tiles_n = (int)((a.N + kT - 1) / kT), tiles_k = (int)((a.K + kT - 1) / kT);
  const bool direct = p.splits == 1;
  hipLaunchKernelGGL((wgrad_kernel<kT, kBias>), dim3((unsigned)(tiles_n * tiles_k * p.splits)), dim3(kWgThreads), lds,
                     stream, (const uint16_t*)a.dy, a.M, (int)a.N, a.lddy, (const uint8_t*)a.qp,
                     (const uint8_t*)a.sp, (int)a.K, (int)(2 * b128_blocks(a.K)), tiles_n, tiles_k, p.splits,
                     direct ? a.dw : (void*)a.part_dw, direct ? a.lddw : a.K, a.N * a.K, direct ? a.out_bf16 : 0,
                     direct ? a.accumulate : 0, a.part_db);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}
}  // namespace

int launch_wgrad(const WgradArgs& a, WgradPlan p, hipStream_t stream) {
  const bool bias = a.db != nullptr;
  int st;
  st = bias ? launch_wgrad_k<128, true>(a, p, stream) : launch_wgrad_k<128, false>(a, p, stream);
  if (st || (p.splits == 1 && !bias)) return st;
  const int64_t quads = p.splits > 1 ? a.N * (a.K / 4) : 0, total = quads + (bias ? a.N : 0);
  const int parts_db = p.splits * (int)((a.K + p.tile - 1) / p.tile);
  hipLaunchKernelGGL(wgrad_reduce_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, stream, a.part_dw,
                     p.splits, a.N, a.K, a.dw, a.lddw, a.out_bf16, a.accumulate, quads, a.part_db, parts_db, a.db);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace mxfp8
