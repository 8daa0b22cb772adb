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
// each gets one column's four rows).  X is the MFMA A operand, so a lane ends
// with four consecutive k of one n: dW rows are written in 16-byte pieces.
// LDS rows are cut into 32-byte slots (one 16-column fragment); slot c of row
// m sits at c ^ f(m), f = bits 0, 1, 3 of m: the four rows one transposing
// read takes and the next lane group's four (8 further) land on different
// banks.
//
// db takes the dY fragments as they come by: step s is added by the
// workgroups with tile index s % tiles_k along k, so each does 1 / tiles_k.
// The (tile, 64-token step) units, tile by tile, are cut into one run per
// workgroup, equal ones, so that the chip is full whatever the number of
// tiles, or whole tiles.  A run holds at most two tiles it does not own whole,
// its first and its last; their sums go to the workgroup's two slots of the
// workspace in lane order, and wgrad_join adds a tile's pieces in token order,
// and the partial sums of db: results do not depend on timing.
//
// This file: the large tiles; wgrad_small.hip: the small tiles.
#include "wgrad.hpp"

namespace mxfp8 {

using namespace wgrad;

// ---------------------------------------------------------------------------
// Large tiles: 256 x 256 of dW per workgroup, four waves 2 x 2, each 128 x 128
// (64 MFMAs per 32 tokens and wave, accumulators in the 256 AGPRs).
//  * A step has two 32-token halves with a fragment set each.  During half 0
//    the fragments of half 1 are read; then everything in flight has landed,
//    the step's one barrier, and during half 1 the next step's first
//    fragments are read while the step's own buffer is refilled for the step
//    after next (dY copies and the widened X) and X is loaded one step
//    further.
// 16384 x 5120 x 2048: 331 us with bf16 results (1040 TFLOP/s; a bf16 library
// product of 8192^3 reaches 1230), 318 with fp32, and 28 for the join; 4096^3:
// 132, added to what is there 154.  The MFMA pipes are busy 0.47 of the time (at
// the library product's rate they would be 0.49).  No counter tells how the rest
// divides: LDS reads, and the wait for everything in flight at half a step.
// ---------------------------------------------------------------------------
namespace {

constexpr int kBigT = 256;
constexpr int kBigPitch = kBigT * 2;
constexpr int kBigOp = kWgStep * kBigPitch;        // 32 KiB: one operand's stage
constexpr int kBigLds = 4 * kBigOp;                // dY x 2, X x 2

}  // namespace

template <bool kBias>
__global__ __launch_bounds__(kWgThreads, 1) void wgrad_big_kernel(
    const uint16_t* __restrict__ dy, int64_t M, int N, int64_t lddy, const uint8_t* __restrict__ qp,
    const uint8_t* __restrict__ sp, int K, int KS, int tiles_k, int steps, Runs runs, void* __restrict__ dw,
    int64_t lddw, int out_bf16, int accumulate, float* __restrict__ part, float* __restrict__ part_db, int pieces) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave & 1, wn = wave >> 1;
  const int i = lane & 15, g = lane >> 4;
  const int w = (int)blockIdx.x;
  const int64_t u0 = runs.start(w), u1 = runs.start(w + 1);

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
        if (out_bf16) {
#pragma unroll
          for (int a = 0; a < 8; a += 2) {
            const int k = k0 + wk * 128 + a * 16 + k_of_pair(g);
            store_pair(acc[a][b], acc[a + 1][b], n < N && k < K, (uint16_t*)dw + (size_t)n * lddw + k);
          }
        } else if (n < N) {
#pragma unroll
          for (int a = 0; a < 8; ++a) {
            const int k = k0 + wk * 128 + a * 16 + 4 * g;
            if (k >= K) continue;   // K % 16 == 0: a quad is all in or all out
            v4f* d = reinterpret_cast<v4f*>((float*)dw + (size_t)n * lddw + k);
            *d = accumulate ? *d + acc[a][b] : acc[a][b];
          }
        }
      }
    } else {
      // slot 0: the piece at the start of the run, 1: at its end
      v4f* d = reinterpret_cast<v4f*>(part + ((size_t)w * 2 + (u == u0 ? 0 : 1)) * (kBigT * kBigT));
      d += wave * 4096 + lane;
#pragma unroll
      for (int a = 0; a < 8; ++a)
#pragma unroll
        for (int b = 0; b < 8; ++b) d[(a * 8 + b) * 64] = acc[a][b];
    }
    if constexpr (kBias) {
      const int piece = w - runs.of((int64_t)t * steps);
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

// Joins the tiles that several runs share, in token order (grid: kSub
// workgroups, of 256 sums of four, per tile, or per border between two runs if
// those are fewer; the ones without work leave), and the parts of db (the last
// workgroups, sixteen columns each): over the tiles of a column of tiles and
// their pieces.
template <int kT, int kWavesN>
__global__ __launch_bounds__(256) void wgrad_join_kernel(const float* __restrict__ part, Runs runs, int parts, int by_border,
                                                         int tiles_k, int steps, int N, int K, void* __restrict__ dw,
                                                         int64_t lddw, int out_bf16, int accumulate,
                                                         const float* __restrict__ part_db, int pieces,
                                                         void* __restrict__ db, int db_bf16) {
  constexpr int kA = kT / 32, kB = kT / 16 / kWavesN;   // fragments per wave along k and n
  constexpr int kSub = kT * kT / 1024;       // workgroups per tile
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= parts * kSub) {
    // sixteen columns: thread (q, c) adds the tiles q, q + 16, ... along k
    __shared__ float red[16][17];
    const int c = tid & 15, q = tid >> 4;
    const int n = ((int)blockIdx.x - parts * kSub) * 16 + c, tn = n / kT;
    float v = 0.0f;
    if (n < N) {
      for (int tk = q; tk < tiles_k; tk += 16) {
        const int t = tn * tiles_k + tk;
        int np = 1;
        if (pieces > 1) np = runs.of((int64_t)(t + 1) * steps - 1) - runs.of((int64_t)t * steps) + 1;
        for (int p = 0; p < np; ++p) v += part_db[((size_t)t * pieces + p) * kT + n % kT];
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
  int t = (int)blockIdx.x / kSub;
  const int sub = (int)blockIdx.x % kSub;
  if (by_border) {   // the tile this border cuts, if it is the tile's first
    const int64_t u = runs.start(t + 1), before = runs.start(t);
    t = (int)(u / steps);
    if (u == (int64_t)t * steps || before > (int64_t)t * steps) return;
  }
  const int w0 = runs.of((int64_t)t * steps), w1 = runs.of((int64_t)(t + 1) * steps - 1);
  if (w0 == w1) return;   // one run owns the tile (and stored it)
  const int tn = t / tiles_k, tk = t - tn * tiles_k;
  const int e = sub * 256 + tid;   // v4f of the tile, lane order: wave, (a, b), lane
  // a piece lies at the start of its run unless the run began in an earlier tile
  const v4f* p = reinterpret_cast<const v4f*>(part) + (size_t)w0 * 2 * (kT * kT / 4) + e;
  v4f v = runs.start(w0) >= (int64_t)t * steps ? *p : p[kT * kT / 4];
  // eight loads on their way at a time; added one after the other
  for (int w = w0; w < w1;) {
    const int m = min(8, w1 - w);
    v4f x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = p[(size_t)min(j + 1, m) * 2 * (kT * kT / 4)];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < m) v += x[j];
    w += m;
    p += (size_t)m * 2 * (kT * kT / 4);
  }
  const int wave = e / (kA * kB * 64), ab = (e >> 6) % (kA * kB), lane = e & 63;
  const int n = tn * kT + (wave >> 1) * (kB * 16) + (ab % kB) * 16 + (lane & 15);
  const int k = tk * kT + (wave & 1) * (kT / 2) + (ab / kB) * 16 + 4 * (lane >> 4);
  if (n >= N || k >= K) return;
  if (out_bf16) {
    *reinterpret_cast<uint2*>((uint16_t*)dw + (size_t)n * lddw + k) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
    v4f* d = reinterpret_cast<v4f*>((float*)dw + (size_t)n * lddw + k);
    *d = accumulate ? *d + v : v;
  }
}

namespace {
template <bool kBias>
int launch_big(const WgradArgs& a, const WgradPlan& p, hipStream_t stream) {
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)wgrad_big_kernel<kBias>, kBigLds, lds_set)) return -7;
  hipLaunchKernelGGL(wgrad_big_kernel<kBias>, dim3((unsigned)p.runs.count), dim3(kWgThreads), kBigLds, stream,
                     (const uint16_t*)a.dy, a.M, (int)a.N, a.lddy, (const uint8_t*)a.qp, (const uint8_t*)a.sp,
                     (int)a.K, (int)(2 * b128_blocks(a.K)), (int)p.tiles_k, (int)p.steps, p.runs, a.dw, a.lddw,
                     a.out_bf16, a.accumulate, a.part_dw, a.part_db, (int)p.pieces);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

template <int kT, int kWavesN>
int launch_join(const WgradArgs& a, const WgradPlan& p, hipStream_t stream) {
  const int borders = p.runs.count - 1, by_border = borders < p.tiles();
  const int join = !p.shared() ? 0 : by_border ? borders : (int)p.tiles();
  const int cols = a.db && !p.db_direct() ? (int)((a.N + 15) / 16) : 0;
  if (join + cols == 0) return 0;
  hipLaunchKernelGGL((wgrad_join_kernel<kT, kWavesN>), dim3((unsigned)(join * (kT * kT / 1024) + cols)), dim3(256), 0, stream,
                     a.part_dw, p.runs, join, by_border, (int)p.tiles_k, (int)p.steps, (int)a.N, (int)a.K, a.dw, a.lddw,
                     a.out_bf16, a.accumulate, a.part_db, (int)p.pieces, a.db, a.db_bf16);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}
}  // namespace

int launch_wgrad(const WgradArgs& a, WgradPlan p, hipStream_t stream) {
  if (p.tile == 128) {
    if (int st = launch_wgrad_small(a, p, stream)) return st;
    return launch_join<128, 4>(a, p, stream);
  }
  if (int st = a.db != nullptr ? launch_big<true>(a, p, stream) : launch_big<false>(a, p, stream)) return st;
  return launch_join<256, 2>(a, p, stream);
}

}  // namespace mxfp8
