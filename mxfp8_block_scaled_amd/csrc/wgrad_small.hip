// The small-tile form of the weight gradient (see wgrad.hip for the
// mathematics, the LDS layout and the runs, which both forms share).
#include "wgrad.hpp"

namespace mxfp8 {

namespace {

using namespace wgrad;

// Small tiles (128 x 128), 1 workgroup of eight waves per compute unit.
struct WgLds {
  static constexpr int kT = 128;
  static constexpr int kThreads = 512;
  static constexpr int kPitch = kT * 2;
  static constexpr int kY = kWgStep * kPitch;        // dY of a step, bf16
  static constexpr int kRaw = kWgStep * kT;          // X of a step, E4M3: eight 1 KiB pieces [64-K half][band]
  static constexpr int kStage = kY + kRaw + 8 * 256; // + per wave a 256-byte scale tile
  static constexpr int kDepth = 4;                   // steps in LDS
  static constexpr int kX = kWgStep * kPitch;        // X widened
  static constexpr int kBytes = kDepth * kStage + 2 * kX;
  static constexpr int kCopies = 2 + 1 + 1;          // per wave and step
};
static_assert(WgLds::kBytes <= 160 * 1024, "LDS of a compute unit");

}  // namespace

// ---------------------------------------------------------------------------
// Small tiles: 128 x 128 of dW, eight waves 2 (k) x 4 (n), each 64 x 32, for the
// problems whose large tiles would leave the chip empty or idle at the end.
// There a step's time is the latency of its loads, so everything comes by
// copies into LDS, three steps ahead.  Every wave widens the sixteen token
// rows of X that it copied itself, one step ahead of their MFMAs, into one of
// two buffers: one barrier per step.  A workgroup goes through its run of
// (tile, step) units without a stop: copies and fragments of the next tile are
// on their way while a tile is stored (67 x 7640 x 5888, bf16: 72 us with one
// tile per launched workgroup, 34 now; writing dW alone takes 18).  Eight waves
// rather than four of 64 x 64, which read a third less from LDS but wait more:
// 0.87 us a step against 1.0.
// ---------------------------------------------------------------------------
template <bool kBias>
__global__ __launch_bounds__(WgLds::kThreads, 1) void wgrad_kernel(
    const uint16_t* __restrict__ dy, int64_t M, int N, int64_t lddy, const uint8_t* __restrict__ qp,
    const uint8_t* __restrict__ sp, int K, int KS, int tiles_k, int steps, Runs runs, void* __restrict__ dw,
    int64_t lddw, int out_bf16, int accumulate, float* __restrict__ part, float* __restrict__ part_db, int pieces,
    void* __restrict__ db, int db_bf16) {
  using L = WgLds;
  constexpr int kA = 4, kB = 2;     // 16-wide fragments per wave along k and n
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave & 1, wn = wave >> 1;
  const int i = lane & 15, g = lane >> 4;
  const int w = xcd_remap((int)blockIdx.x, (int)gridDim.x);
  const int64_t u0 = runs.start(w);
  const int n_units = (int)(runs.start(w + 1) - u0);
  // no tokens: one step whose reads all lie past the ends of their resources
  const uint32_t gbytes = M > 0 ? (uint32_t)KS * kTileBytes : 0, sbytes = M > 0 ? (uint32_t)KS * kTileScaleBytes : 0;

  // dY: lane l of a copy takes LDS bytes [16 l, 16 l + 16) of its KiB (four
  // token rows of 256 bytes), i.e. half h of slot c of row m, which holds
  // logical slot c ^ f(m).  Rows past M are past the resource's end and read
  // zero; columns past N belong to outputs that are not stored.
  uint32_t vy[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int m = (wave * 2 + c) * 4 + (lane >> 4), p = lane & 15;
    vy[c] = (uint32_t)((int64_t)m * lddy + ((p >> 1) ^ slot_xor(m)) * 16 + (p & 1) * 8) * 2u;
  }
  auto stage = [&](int b) { return smem + b * L::kStage; };
  auto widened = [&](int b) { return smem + L::kDepth * L::kStage + b * L::kX; };
  const int t0 = (int)(u0 / steps), sa0 = (int)(u0 - (int64_t)t0 * steps);
  // The copies of the next unit to be copied, unit by unit; past the run's
  // end those of its last unit again (never used), so the waits need no other
  // counts.  (Addresses advance: at one wave per SIMD every scalar
  // instruction counts.)
  int left = n_units, cs = sa0, ctn = t0 / tiles_k, ctk = t0 - ctn * tiles_k;
  const uint16_t* yp = dy + cs * kWgStep * lddy + ctn * L::kT;
  int64_t rows = M - (int64_t)cs * kWgStep;              // token rows from this step on
  const uint8_t* xp = qp + (size_t)(cs >> 1) * gbytes;
  const uint8_t* scp = sp + (size_t)(cs >> 1) * sbytes;
  // X: the wave's piece of the eight of a step: 64-K half, band of 16 tokens
  const int xv = wave & 1, band = wave >> 1;
  const uint32_t vx0 = (uint32_t)band * KS * kPieceBytes + (uint32_t)lane * 16u, vx1 = vx0 + 4u * KS * kPieceBytes;
  auto issue = [&](uint8_t* st) {
    const int r = rows >= kWgStep ? kWgStep : (int)rows;
    const tile::i4v ry = tile::buffer_rsrc(yp, r > 0 ? (uint32_t)((r - 1) * (int)lddy + N - ctn * L::kT) * 2u : 0u);
    const tile::i4v rx = tile::buffer_rsrc(xp, gbytes);
    const tile::i4v rs = tile::buffer_rsrc(scp, sbytes);
#pragma unroll
    for (int c = 0; c < 2; ++c) tile::b2l_16(vy[c], ry, 0u, st + (wave * 2 + c) * 1024);
    // pieces past K read other columns' data or, past the group, zeros
    tile::b2l_16((cs & 1) ? vx1 : vx0, rx, (uint32_t)(2 * ctk + xv) * kPieceBytes,
                 st + L::kY + (xv * 4 + band) * 1024);
    tile::b2l_4((uint32_t)lane * 4u, rs, (uint32_t)(2 * ctk + xv) * kTileScaleBytes,
                st + L::kY + L::kRaw + wave * 256);
    if (left > 1) {
      --left;
      if (++cs < steps) {
        yp += kWgStep * lddy;
        rows -= kWgStep;
        xp += (cs & 1) ? 0 : gbytes;
        scp += (cs & 1) ? 0 : sbytes;
      } else {
        cs = 0;
        if (++ctk == tiles_k) {
          ctk = 0;
          ++ctn;
        }
        yp = dy + ctn * L::kT;
        rows = M;
        xp = qp;
        scp = sp;
      }
    }
  };
  // Widening: the thread's chunk is in token row m = 16 band + lane / 4.
  const int xm = 16 * band + (lane >> 2), xc = (lane & 3) ^ swz(lane >> 2);
  const int xdst = xm * L::kPitch + (((xv * 4 + xc) ^ slot_xor(xm)) * 32);
  struct Raw {
    uint4 q;
    uint32_t s;
  };
  auto load_raw = [&](int s, const uint8_t* st) {
    return Raw{*reinterpret_cast<const uint4*>(st + L::kY + (xv * 4 + band) * 1024 + lane * 16),
               st[L::kY + L::kRaw + wave * 256 + scale_off(xm, xc >> 1) + 2 * (s & 1)]};
  };
  auto widen = [&](const Raw& x, uint8_t* to) {
    uint4 d[2];
    widen16(x.q, b128_scale_value(x.s), d);
    uint4* o = reinterpret_cast<uint4*>(to + xdst);
    o[0] = d[0];
    o[1] = d[1];
  };

  // Fragment f (sixteen columns) and 32-token half h of a tile: lane (i, g)
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

  v4f acc[kA][kB];
  v4f accb[kB];
  auto clear = [&] {
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      accb[b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int a = 0; a < kA; ++a) acc[a][b] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
  };
  clear();
  bf16x8 ones;
#pragma unroll
  for (int e = 0; e < 8; ++e) ones[e] = (__bf16)1.0f;

  bf16x8 ax[kA], ay[kB], bx[kA], by[kB];   // fragments of half 0 and of half 1
#pragma unroll
  for (int d = 0; d < L::kDepth - 1; ++d) issue(stage(d));
  tile::wait_vmcnt<(L::kDepth - 2) * L::kCopies>();
  widen(load_raw(sa0, stage(0)), widened(0));
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int a = 0; a < kA; ++a) ax[a] = frag(widened(0), wk * kA + a, 0);
#pragma unroll
  for (int b = 0; b < kB; ++b) ay[b] = frag(stage(0), wn * kB + b, 0);
  int t = t0, tn = t0 / tiles_k, tk = t0 - tn * tiles_k;
  int s = sa0, sa = sa0, phase = sa0 % tiles_k, at = 0;
  // Stores at the end of the last unit and of the one before it, at least, in
  // halves of a tile's kA * kB; and the last unit's alone.
  int stored = 0, stored_last = 0;
  for (int r = 0; r < n_units; ++r) {
    const int next = at + 1 == L::kDepth ? 0 : at + 1, last = at == 0 ? L::kDepth - 1 : at - 1;
    const int par = r & 1, sn = s + 1 == steps ? 0 : s + 1;
    const uint8_t *const y = stage(at), *const x = widened(par);
    const uint8_t *const yn = stage(next), *const xn = widened(par ^ 1);
    const bool with_bias = kBias && wk == 0 && (db != nullptr ? 0 : phase) == tk;
    phase = phase + 1 == tiles_k ? 0 : phase + 1;
    // Half 0, with the reads of half 1 and the widening of the next step (this
    // wave's copies of it have landed: only the copies of the step after it
    // and stores issued since are in flight).  The empty asm statements keep
    // the MFMAs in their places.
    constexpr int kNewer = (L::kDepth - 3) * L::kCopies, kHalf = kA * kB / 2;
    if (stored == 0) tile::wait_vmcnt<kNewer>();
    else if (stored == 1) tile::wait_vmcnt<kNewer + kHalf>();
    else if (stored < 4) tile::wait_vmcnt<kNewer + 2 * kHalf>();
    else tile::wait_vmcnt<kNewer + 4 * kHalf>();
    const Raw raw = load_raw(sn, yn);   // (at the run's end: a copy of the last unit)
    tile::static_for<0, 8>([&](auto J) {
      constexpr int j = decltype(J)::value, a = j >> 1, c = j & 1;
      acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ax[a], ay[c], acc[a][c], 0, 0, 0);
      asm volatile("" : "+v"(acc[a][c]));
      if constexpr (j < 2) by[j] = frag(y, wn * kB + j, 1);
      else if constexpr (j < 6) bx[j - 2] = frag(x, wk * kA + j - 2, 1);
      if constexpr (j == 5) widen(raw, widened(par ^ 1));
      __builtin_amdgcn_sched_barrier(0);
    });
    if (with_bias) {
#pragma unroll
      for (int b = 0; b < kB; ++b) accb[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, ay[b], accb[b], 0, 0, 0);
    }
    // Past this barrier the next unit has landed and is widened for all waves,
    // and nobody reads the last one from LDS any more.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    issue(stage(last));
    tile::static_for<0, 8>([&](auto J) {
      constexpr int j = decltype(J)::value, a = j >> 1, c = j & 1;
      acc[a][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bx[a], by[c], acc[a][c], 0, 0, 0);
      asm volatile("" : "+v"(acc[a][c]));
      if constexpr (j < 2) ay[j] = frag(yn, wn * kB + j, 0);
      else if constexpr (j < 6) ax[j - 2] = frag(xn, wk * kA + j - 2, 0);
      __builtin_amdgcn_sched_barrier(0);
    });
    if (with_bias) {
#pragma unroll
      for (int b = 0; b < kB; ++b) accb[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, by[b], accb[b], 0, 0, 0);
    }
    at = next;
    stored = stored_last;
    stored_last = 0;
    if (sn == 0 || r + 1 == n_units) {
      // Lane (i, g) holds D[k = 64 wk + 16 a + 4 g + j][n = 32 wn + 16 b + i].
      const int n0 = tn * L::kT, k0 = tk * L::kT;
      if (sa == 0 && sn == 0) {
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const int n = n0 + (wn * kB + b) * 16 + i;
          if (out_bf16) {
#pragma unroll
            for (int a = 0; a < kA; a += 2) {
              const int k = k0 + (wk * kA + a) * 16 + k_of_pair(g);
              store_pair(acc[a][b], acc[a + 1][b], n < N && k < K, (uint16_t*)dw + (size_t)n * lddw + k);
            }
          } else if (n < N) {
            float* const row = (float*)dw + (size_t)n * lddw;
            const int k = k0 + wk * kA * 16 + 4 * g;   // K % 16 == 0: a quad is all in or all out
            if (accumulate) {
#pragma unroll
              for (int a = 0; a < kA; ++a)
                if (k + 16 * a < K) *reinterpret_cast<v4f*>(row + k + 16 * a) += acc[a][b];
            } else {
#pragma unroll
              for (int a = 0; a < kA; ++a)
                if (k + 16 * a < K) *reinterpret_cast<v4f*>(row + k + 16 * a) = acc[a][b];
            }
          }
        }
        // at the matrix's edge a wave may have skipped some
        if (n0 + L::kT <= N && k0 + L::kT <= K) stored_last = out_bf16 ? 1 : 2;
      } else {
        // slot 0: the piece at the start of the run, 1: at its end
        v4f* d = reinterpret_cast<v4f*>(part + ((size_t)w * 2 + (t == t0 ? 0 : 1)) * (L::kT * L::kT));
        d += wave * 512 + lane;
#pragma unroll
        for (int a = 0; a < kA; ++a)
#pragma unroll
          for (int b = 0; b < kB; ++b) d[(a * kB + b) * 64] = acc[a][b];
        stored_last = 2;
      }
      // every row of the ones product holds the column sums
      if (kBias && wk == 0 && g == 0 && db != nullptr) {
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const int n = n0 + (wn * kB + b) * 16 + i;
          if (tk == 0 && n < N) store_db(db, db_bf16, accumulate, n, accb[b][0]);
        }
      } else if (kBias && wk == 0 && g == 0) {
        const int piece = w - runs.of((int64_t)t * steps);
#pragma unroll
        for (int b = 0; b < kB; ++b)
          part_db[((size_t)t * pieces + piece) * L::kT + (wn * kB + b) * 16 + i] = accb[b][0];
      }
      clear();
      ++t;
      sa = 0;
      phase = 0;
      if (++tk == tiles_k) {
        tk = 0;
        ++tn;
      }
    }
    stored += stored_last;
    s = sn;
  }
  tile::wait_vmcnt<0>();   // no copy may land after the workgroup's LDS is given away
}

namespace {
template <bool kBias>
int launch_small(const WgradArgs& a, const WgradPlan& p, hipStream_t stream) {
  constexpr int lds = WgLds::kBytes;
  static std::atomic<int> lds_set[kMaxDevices];
  if (!set_lds_limit_once((const void*)wgrad_kernel<kBias>, lds, lds_set)) return -7;
  hipLaunchKernelGGL((wgrad_kernel<kBias>), dim3((unsigned)p.runs.count), dim3(WgLds::kThreads), lds, stream,
                     (const uint16_t*)a.dy, a.M, (int)a.N, a.lddy, (const uint8_t*)a.qp, (const uint8_t*)a.sp,
                     (int)a.K, (int)(2 * b128_blocks(a.K)), (int)p.tiles_k, (int)p.steps, p.runs, a.dw, a.lddw,
                     a.out_bf16, a.accumulate, a.part_dw, a.part_db, (int)p.pieces,
                     p.db_direct() ? a.db : nullptr, a.db_bf16);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace

int launch_wgrad_small(const WgradArgs& a, const WgradPlan& p, hipStream_t stream) {
  return a.db != nullptr ? launch_small<true>(a, p, stream) : launch_small<false>(a, p, stream);
}

}  // namespace mxfp8
