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
#include <algorithm>

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

__device__ inline void store_db(void* db, int bf16, int accumulate, int64_t n, float v) {
  if (bf16) ((uint16_t*)db)[n] = (uint16_t)pack_bf16x2(v, 0.0f);
  else ((float*)db)[n] = accumulate ? ((float*)db)[n] + v : v;
}

template <int kT>
struct WgLds {
  static constexpr int kPitch = kT * 2;
  static constexpr int kOp = kWgStep * kPitch;   // one operand's stage
  static constexpr int kBytes = 4 * kOp;         // two operands, two stages
};

}  // namespace

template <int kT, bool kBias>
__global__ __launch_bounds__(kWgThreads, 2) void wgrad_kernel(
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

// dw = sum of the split partials in order (+ dw): one thread per 4 k.  db =
// sum of its partials: the last workgroups, sixteen columns each, thread
// (q, c) parts q, q + 16, ... of column c, then the sixteen sums in order.
__global__ __launch_bounds__(256) void wgrad_reduce_kernel(const float* __restrict__ part, int splits, int64_t N,
                                                           int64_t K, void* __restrict__ dw, int64_t lddw,
                                                           int out_bf16, int accumulate, int64_t quads,
                                                           const float* __restrict__ part_db, int parts_db,
                                                           void* __restrict__ db, int db_bf16) {
  const int64_t dw_blocks = (quads + 255) / 256;
  if ((int64_t)blockIdx.x >= dw_blocks) {
    __shared__ float red[16][17];
    const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
    const int64_t n = ((int64_t)blockIdx.x - dw_blocks) * 16 + c;
    float v = 0.0f;
    if (n < N)
      for (int p = q; p < parts_db; p += 16) v += part_db[(size_t)p * N + n];
    red[q][c] = v;
    __syncthreads();
    if (q != 0 || n >= N) return;
    v = 0.0f;
#pragma unroll
    for (int p = 0; p < 16; ++p) v += red[p][c];
    store_db(db, db_bf16, accumulate, n, v);
    return;
  }
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
}

// ---------------------------------------------------------------------------
// Large tiles: 256 x 256 of dW per workgroup, four waves 2 x 2, each 128 x 128
// (64 MFMAs per 32 tokens and wave, accumulators in the 256 AGPRs).
//  * The (tile, step) units, tile by tile, are cut into one equal run per
//    workgroup, so the chip is full whatever the number of tiles.  A run
//    holds at most two tiles it does not own whole, its first and its last;
//    their sums go to the workgroup's two slots of the workspace in lane
//    order, and wgrad_join adds a tile's pieces in token order.
//  * A step has two 32-token halves with a fragment set each.  During half 0
//    the fragments of half 1 are read; then everything in flight has landed,
//    the step's one barrier, and during half 1 the next step's first
//    fragments are read while the step's own buffer is refilled for the step
//    after next (dY copies and the widened X) and X is loaded one step
//    further.
// ---------------------------------------------------------------------------
namespace {

constexpr int kBigT = 256;
constexpr int kBigPitch = kBigT * 2;
constexpr int kBigOp = kWgStep * kBigPitch;        // 32 KiB: one operand's stage
constexpr int kBigLds = 4 * kBigOp;                // dY x 2, X x 2
constexpr int kBigTileFloats = kBigT * kBigT;

// Runs: workgroup w of G takes units [U w / G, U (w + 1) / G) of U.
__host__ __device__ inline int64_t run_start(int64_t U, int G, int64_t w) { return U * w / G; }
__host__ __device__ inline int run_of(int64_t U, int G, int64_t unit) { return (int)(((unit + 1) * G - 1) / U); }

}  // namespace

template <bool kBias>
__global__ __launch_bounds__(kWgThreads, 1) void wgrad_big_kernel(
    const uint16_t* __restrict__ dy, int64_t M, int N, int64_t lddy, const uint8_t* __restrict__ qp,
    const uint8_t* __restrict__ sp, int K, int KS, int tiles_k, int tiles, int steps, void* __restrict__ dw,
    int64_t lddw, int out_bf16, int accumulate, float* __restrict__ part, float* __restrict__ part_db, int pieces) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave & 1, wn = wave >> 1;
  const int i = lane & 15, g = lane >> 4;
  const int G = (int)gridDim.x, w = (int)blockIdx.x;
  const int64_t U = (int64_t)tiles * steps;
  const int64_t u0 = run_start(U, G, w), u1 = run_start(U, G, w + 1);

  // Fragment addresses (see wgrad_kernel): the swizzle is the lane's own, so
  // buffer, half and row offset are immediates.
  const int fx = slot_xor(8 * g + (i >> 2));
  const uint32_t lds0 = tile::lds_addr(smem);
  uint32_t xa[8], ya[8];
#pragma unroll
  for (int a = 0; a < 8; ++a) {
    const uint32_t o = lds0 + (uint32_t)((8 * g + (i >> 2)) * kBigPitch + ((a ^ fx) * 32) + (i & 3) * 8);
    xa[a] = o + 2 * kBigOp + wk * 256;
    ya[a] = o + wn * 256;
  }
  auto sy = [&](int b) { return smem + b * kBigOp; };
  auto sx = [&](int b) { return smem + (2 + b) * kBigOp; };
  auto frag = [&](uint32_t at, int b, int h) {
    lds_s16x4* const p = (lds_s16x4*)(at + (uint32_t)(b * kBigOp + h * 32 * kBigPitch));
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + 4 * kBigPitch / 8);
    const s16x8 r = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, r);
  };

  // X: the thread's four 16-byte chunks of a step lie in one token row
  // m = 16 wave + lane / 4, one per 64-K piece.  Pieces past K and past the
  // group are other columns' data or zeros; their outputs are not stored.
  const int xm = 16 * wave + (lane >> 2), xc = (lane & 3) ^ swz(lane >> 2);
  uint32_t xdst[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) xdst[v] = (uint32_t)(xm * kBigPitch + (((v * 4 + xc) ^ slot_xor(xm)) * 32));
  const uint32_t xvoff = (uint32_t)wave * KS * kPieceBytes + (uint32_t)lane * 16u;
  const uint32_t svoff = (uint32_t)scale_off(xm, xc >> 1);
  const uint32_t gbytes = (uint32_t)KS * kTileBytes, sbytes = (uint32_t)KS * kTileScaleBytes;
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  struct X {
    u32x4 q[4];
    uint32_t s[4];
  };
  auto store_x = [&](const X& x, int v, uint8_t* st) {
    uint4 d[2];
    widen16(make_uint4(x.q[v][0], x.q[v][1], x.q[v][2], x.q[v][3]), b128_scale_value(x.s[v]), d);
    *reinterpret_cast<uint4*>(st + xdst[v]) = d[0];
    *reinterpret_cast<uint4*>(st + xdst[v] + 16) = d[1];
  };

  v4f acc[8][8];
  float accb[4];

  for (int64_t u = u0; u < u1;) {
    const int t = (int)(u / steps), sa = (int)(u - (int64_t)t * steps);
    const int sb = (int)min((int64_t)steps, sa + (u1 - u));
    const int tn = t / tiles_k, tk = t - tn * tiles_k;
    const int n0 = tn * kBigT, k0 = tk * kBigT;

    // dY: lane l of copy c takes LDS bytes [16 l, + 16) of its KiB: two token
    // rows of 512 bytes, 32-byte slot c holding logical slot c ^ f(m).
    uint32_t vy[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int m = (wave * 8 + c) * 2 + (lane >> 5), p = lane & 31;
      vy[c] = (uint32_t)((int64_t)m * lddy + n0 + ((p >> 1) ^ slot_xor(m)) * 16 + (p & 1) * 8) * 2u;
    }
    auto dy_rsrc = [&](int s) {
      const int64_t m0 = (int64_t)min(s, sb - 1) * kWgStep;
      const int64_t rows = min(M - m0, (int64_t)kWgStep);
      return tile::buffer_rsrc(dy + m0 * lddy, (uint32_t)(((rows - 1) * lddy + N) * 2));
    };
    auto copy_dy = [&](int c, tile::i4v r, uint8_t* st) { tile::b2l_16(vy[c], r, 0u, st + (wave * 8 + c) * 1024); };
    auto load_x = [&](int s, X& x) {
      const int sc = min(s, sb - 1);
      const __amdgpu_buffer_rsrc_t qr = raw_rsrc(qp + (size_t)(sc >> 1) * gbytes, gbytes);
      const __amdgpu_buffer_rsrc_t sr = raw_rsrc(sp + (size_t)(sc >> 1) * sbytes, sbytes);
      const int half = sc & 1, ks = k0 / kStepK;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        x.q[v] = __builtin_amdgcn_raw_buffer_load_b128(qr, xvoff, (uint32_t)(half * 4 * KS + ks + v) * kPieceBytes, 0);
        x.s[v] = __builtin_amdgcn_raw_buffer_load_b8(sr, svoff, (uint32_t)((ks + v) * kTileScaleBytes + half * 2), 0);
      }
    };

#pragma unroll
    for (int a = 0; a < 8; ++a) {
      if (a < 4) accb[a] = 0.0f;
#pragma unroll
      for (int b = 0; b < 8; ++b) acc[a][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // Both buffers filled, X of the third step on its way.  (The barrier:
    // the last tile's fragments have been read by every wave.)
    tile::wait_vmcnt<0>();
    __syncthreads();
    X xr;
    {
      const tile::i4v r0 = dy_rsrc(sa), r1 = dy_rsrc(sa + 1);
#pragma unroll
      for (int c = 0; c < 8; ++c) copy_dy(c, r0, sy(0));
#pragma unroll
      for (int c = 0; c < 8; ++c) copy_dy(c, r1, sy(1));
      X x1;
      load_x(sa, xr);
      load_x(sa + 1, x1);
#pragma unroll
      for (int v = 0; v < 4; ++v) store_x(xr, v, sx(0));
#pragma unroll
      for (int v = 0; v < 4; ++v) store_x(x1, v, sx(1));
      load_x(sa + 2, xr);
    }
    tile::wait_vmcnt<0>();
    __syncthreads();
    bf16x8 ax[8], ay[8], bx[8], by[8];   // fragments of half 0 and of half 1
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      ax[a] = frag(xa[a], 0, 0);
      ay[a] = frag(ya[a], 0, 0);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");

    int phase = sa % tiles_k;
    // db: the two waves that hold the same dY fragments take four each; the
    // dot product with ones adds a pair of bf16 to the fp32 sum.
    auto add_bias = [&](const bf16x8 (&fy)[8]) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const auto q = __builtin_bit_cast(u32x4, wk ? fy[b + 4] : fy[b]);
        const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          accb[b] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, (uint32_t)q[e]), one, accb[b], false);
      }
    };
    // One step on buffer b.  A fragment of X is read where its predecessor
    // has one row of MFMAs left, one of dY into the other set.  The empty asm statements keep the MFMAs in their
    // places between the reads, writes and copies.
    auto step = [&](int s, auto B) {
      constexpr int b = decltype(B)::value;
      const bool with_bias = kBias && phase == tk;
      phase = phase + 1 == tiles_k ? 0 : phase + 1;
      tile::static_for<0, 64>([&](auto J) {
        constexpr int j = decltype(J)::value, a = j >> 3, c = j & 7;
        acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ax[a], ay[c], acc[a][c], 0, 0, 0);
        asm volatile("" : "+a"(acc[a][c]));
        if constexpr (c == 1) by[a] = frag(ya[a], b, 1);
        if constexpr (c == 4) bx[a] = frag(xa[a], b, 1);
        __builtin_amdgcn_sched_barrier(0);
      });
      if (with_bias) add_bias(ay);
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
#pragma unroll
      for (int v = 0; v < 4; ++v) asm volatile("" : "+v"(xr.q[v]), "+v"(xr.s[v]));   // landed: no wait further down
      const tile::i4v r = dy_rsrc(s + 2);
      tile::static_for<0, 64>([&](auto J) {
        constexpr int j = decltype(J)::value, a = j >> 3, c = j & 7;
        acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bx[a], by[c], acc[a][c], 0, 0, 0);
        asm volatile("" : "+a"(acc[a][c]));
        if constexpr (c == 1) ay[a] = frag(ya[a], b ^ 1, 0);
        if constexpr (c == 4) ax[a] = frag(xa[a], b ^ 1, 0);
        if constexpr (j % 3 == 2 && j / 3 < 8) copy_dy(j / 3, r, sy(b));
        if constexpr (j % 8 == 6 && j / 8 < 4) store_x(xr, j / 8, sx(b));
        if constexpr (j == 38) load_x(s + 3, xr);
        __builtin_amdgcn_sched_barrier(0);
      });
      if (with_bias) add_bias(by);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
    for (int s = sa; s < sb; s += 2) {
      step(s, std::integral_constant<int, 0>{});
      if (s + 1 < sb) step(s + 1, std::integral_constant<int, 1>{});
    }

    // Lane (i, g) holds D[k = 128 wk + 16 a + 4 g + j][n = 128 wn + 16 b + i].
    const bool whole = sa == 0 && sb == steps;
    if (whole) {
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const int n = n0 + wn * 128 + b * 16 + i;
        if (n < N) {
#pragma unroll
          for (int a = 0; a < 8; ++a) {
            const int k = k0 + wk * 128 + a * 16 + 4 * g;
            if (k < K) {
              if (out_bf16) {
                *reinterpret_cast<uint2*>((uint16_t*)dw + (size_t)n * lddw + k) =
                    make_uint2(pack_bf16x2(acc[a][b][0], acc[a][b][1]), pack_bf16x2(acc[a][b][2], acc[a][b][3]));
              } else {
                v4f* d = reinterpret_cast<v4f*>((float*)dw + (size_t)n * lddw + k);
                *d = accumulate ? *d + acc[a][b] : acc[a][b];
              }
            }
          }
        }
      }
    } else {
      // slot 0: the piece at the start of the run, 1: at its end
      v4f* d = reinterpret_cast<v4f*>(part + ((size_t)w * 2 + (u == u0 ? 0 : 1)) * kBigTileFloats) + wave * 4096 + lane;
#pragma unroll
      for (int a = 0; a < 8; ++a)
#pragma unroll
        for (int b = 0; b < 8; ++b) d[(a * 8 + b) * 64] = acc[a][b];
    }
    if constexpr (kBias) {
      const int piece = w - run_of(U, G, (int64_t)t * steps);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float v = accb[b];
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if (g == 0) part_db[((size_t)t * pieces + piece) * kBigT + wn * 128 + wk * 64 + b * 16 + i] = v;
      }
    }
    u += sb - sa;
  }
  tile::wait_vmcnt<0>();   // no copy may land after the workgroup's LDS is given away
}

// Joins the large tiles that several runs share, in token order (grid: 16
// workgroups per tile; those of whole tiles leave), and the parts of db (the
// last workgroups, sixteen columns each): over the tiles of a column of tiles and their pieces.
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* __restrict__ part, int64_t U, int G, int tiles,
                                                         int tiles_k, int steps, int N, int K, void* __restrict__ dw,
                                                         int64_t lddw, int out_bf16, int accumulate,
                                                         const float* __restrict__ part_db, int pieces,
                                                         void* __restrict__ db, int db_bf16) {
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= tiles * 16) {
    // sixteen columns: thread (q, c) adds the tiles q, q + 16, ... along k
    __shared__ float red[16][17];
    const int c = tid & 15, q = tid >> 4;
    const int n = ((int)blockIdx.x - tiles * 16) * 16 + c, tn = n / kBigT;
    float v = 0.0f;
    if (n < N) {
      for (int tk = q; tk < tiles_k; tk += 16) {
        const int t = tn * tiles_k + tk;
        const int np = run_of(U, G, (int64_t)(t + 1) * steps - 1) - run_of(U, G, (int64_t)t * steps) + 1;
        for (int p = 0; p < np; ++p) v += part_db[((size_t)t * pieces + p) * kBigT + n % kBigT];
      }
    }
    red[q][c] = v;
    __syncthreads();
    if (q != 0 || n >= N) return;
    v = 0.0f;
#pragma unroll
    for (int p = 0; p < 16; ++p) v += red[p][c];
    store_db(db, db_bf16, accumulate, n, v);
    return;
  }
  const int t = (int)blockIdx.x >> 4, sub = (int)blockIdx.x & 15;
  const int w0 = run_of(U, G, (int64_t)t * steps), w1 = run_of(U, G, (int64_t)(t + 1) * steps - 1);
  if (w0 == w1) return;   // one run owns the tile (and stored it)
  const int tn = t / tiles_k, tk = t - tn * tiles_k;
  for (int c = 0; c < 4; ++c) {
    const int e = sub * 1024 + c * 256 + tid;   // v4f of the tile, lane order: wave, (a, b), lane
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = w0; w <= w1; ++w) {
      // a piece lies at the start of its run unless the run began in an earlier tile
      const int slot = run_start(U, G, w) >= (int64_t)t * steps ? 0 : 1;
      v += reinterpret_cast<const v4f*>(part + ((size_t)w * 2 + slot) * kBigTileFloats)[e];
    }
    const int wave = e >> 12, ab = (e >> 6) & 63, lane = e & 63;
    const int n = tn * kBigT + (wave >> 1) * 128 + (ab & 7) * 16 + (lane & 15);
    const int k = tk * kBigT + (wave & 1) * 128 + (ab >> 3) * 16 + 4 * (lane >> 4);
    if (n >= N || k >= K) continue;
    if (out_bf16) {
      *reinterpret_cast<uint2*>((uint16_t*)dw + (size_t)n * lddw + k) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
      v4f* d = reinterpret_cast<v4f*>((float*)dw + (size_t)n * lddw + k);
      *d = accumulate ? *d + v : v;
    }
  }
}

namespace {
std::atomic<int> g_force_wgrad{0};
constexpr int64_t kRuns = 256;   // compute units
}

int wgrad_force(int tile) { return g_force_wgrad.exchange(tile); }

WgradPlan wgrad_plan(int64_t M, int64_t N, int64_t K) {
  WgradPlan p;
  const int64_t steps = (M + kWgStep - 1) / kWgStep;
  const int64_t big = ((N + 255) / 256) * ((K + 255) / 256);
  const int force = g_force_wgrad.load(std::memory_order_relaxed);
  // Large tiles once every compute unit gets a run of sixteen steps.
  p.tile = big * steps >= kRuns * 16 ? 256 : 128;
  if (force) p.tile = force;
  if (steps == 0) p.tile = 128;
  p.splits = 1;
  p.runs = 0;
  if (p.tile == 256) {
    // One run per compute unit, of eight steps at least; as many runs as
    // tiles where that leaves few units idle, for then no tile is shared.
    p.runs = (int)std::min(kRuns, std::max<int64_t>(1, big * steps / 8));
    if (big <= kRuns && big * 8 >= kRuns * 7) p.runs = (int)big;
    return p;
  }
  const int64_t tiles = ((N + 127) / 128) * ((K + 127) / 128);
  // two workgroups per compute unit
  while (p.splits < 16 && tiles * p.splits < 512 && steps / (2 * p.splits) >= 4) p.splits *= 2;
  return p;
}

namespace {
struct BigShape {
  int64_t tiles_n, tiles_k, tiles, steps, U, pieces;
  bool shared;   // some tile belongs to several runs
};
BigShape big_shape(int64_t M, int64_t N, int64_t K, WgradPlan p) {
  BigShape b;
  b.tiles_n = (N + kBigT - 1) / kBigT;
  b.tiles_k = (K + kBigT - 1) / kBigT;
  b.tiles = b.tiles_n * b.tiles_k;
  b.steps = (M + kWgStep - 1) / kWgStep;
  b.U = b.tiles * b.steps;
  b.shared = b.tiles % p.runs != 0;
  b.pieces = b.shared ? b.steps / (b.U / p.runs) + 2 : 1;
  return b;
}
}  // namespace

size_t wgrad_dw_bytes(int64_t M, int64_t N, int64_t K, WgradPlan p) {
  if (p.tile == 256) return big_shape(M, N, K, p).shared ? (size_t)p.runs * 2 * kBigTileFloats * 4 : 0;
  return p.splits > 1 ? (size_t)p.splits * (size_t)N * (size_t)K * 4 : 0;
}
size_t wgrad_db_bytes(int64_t M, int64_t N, int64_t K, WgradPlan p) {
  if (p.tile == 256) {
    const BigShape b = big_shape(M, N, K, p);
    return (size_t)b.tiles * (size_t)b.pieces * kBigT * 4;
  }
  return (size_t)p.splits * (size_t)((K + 127) / 128) * (size_t)N * 4;
}

namespace {
template <bool kBias>
int launch_small(const WgradArgs& a, WgradPlan p, hipStream_t stream) {
  constexpr int lds = WgLds<128>::kBytes;
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)wgrad_kernel<128, kBias>, lds, lds_set)) return -7;
  const int tiles_n = (int)((a.N + 127) / 128), tiles_k = (int)((a.K + 127) / 128);
  const bool direct = p.splits == 1;
  hipLaunchKernelGGL((wgrad_kernel<128, kBias>), dim3((unsigned)(tiles_n * tiles_k * p.splits)), dim3(kWgThreads), lds,
                     stream, (const uint16_t*)a.dy, a.M, (int)a.N, a.lddy, (const uint8_t*)a.qp,
                     (const uint8_t*)a.sp, (int)a.K, (int)(2 * b128_blocks(a.K)), tiles_n, tiles_k, p.splits,
                     direct ? a.dw : (void*)a.part_dw, direct ? a.lddw : a.K, a.N * a.K, direct ? a.out_bf16 : 0,
                     direct ? a.accumulate : 0, a.part_db);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

template <bool kBias>
int launch_big(const WgradArgs& a, WgradPlan p, hipStream_t stream) {
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)wgrad_big_kernel<kBias>, kBigLds, lds_set)) return -7;
  const BigShape b = big_shape(a.M, a.N, a.K, p);
  hipLaunchKernelGGL(wgrad_big_kernel<kBias>, dim3((unsigned)p.runs), dim3(kWgThreads), kBigLds, stream,
                     (const uint16_t*)a.dy, a.M, (int)a.N, a.lddy, (const uint8_t*)a.qp, (const uint8_t*)a.sp,
                     (int)a.K, (int)(2 * b128_blocks(a.K)), (int)b.tiles_k, (int)b.tiles, (int)b.steps, a.dw, a.lddw,
                     a.out_bf16, a.accumulate, a.part_dw, a.part_db, (int)b.pieces);
  if (hipGetLastError() != hipSuccess) return -7;
  if (!b.shared && !kBias) return 0;
  const int join = b.shared ? (int)b.tiles : 0, cols = kBias ? (int)((a.N + 15) / 16) : 0;
  hipLaunchKernelGGL(wgrad_join_kernel, dim3((unsigned)(join * 16 + cols)), dim3(256), 0, stream, a.part_dw, b.U,
                     p.runs, join, (int)b.tiles_k, (int)b.steps, (int)a.N, (int)a.K, a.dw, a.lddw, a.out_bf16,
                     a.accumulate, a.part_db, (int)b.pieces, a.db, a.db_bf16);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}
}  // namespace

int launch_wgrad(const WgradArgs& a, WgradPlan p, hipStream_t stream) {
  const bool bias = a.db != nullptr;
  if (p.tile == 256) return bias ? launch_big<true>(a, p, stream) : launch_big<false>(a, p, stream);
  const int st = bias ? launch_small<true>(a, p, stream) : launch_small<false>(a, p, stream);
  if (st || (p.splits == 1 && !bias)) return st;
  const int64_t quads = p.splits > 1 ? a.N * (a.K / 4) : 0;
  const int64_t blocks = (quads + 255) / 256 + (bias ? (a.N + 15) / 16 : 0);
  const int parts_db = p.splits * (int)((a.K + 127) / 128);
  hipLaunchKernelGGL(wgrad_reduce_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a.part_dw, p.splits, a.N, a.K, a.dw,
                     a.lddw, a.out_bf16, a.accumulate, quads, a.part_db, parts_db, a.db, a.db_bf16);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace mxfp8
