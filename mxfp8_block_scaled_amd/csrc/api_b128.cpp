// C ABI (include/mxfp8.h) of the 128-block FP8 layer, the weight gradient
// from 8-bit activation checkpoints and the router's balance loss: argument
// validation on the host, device check, launches.  Nothing here allocates
// device memory or synchronizes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <numeric>

#include "launch_b128.hpp"
#include "mxfp8.h"

namespace {

using mxfp8::b128_blocks;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

constexpr int64_t kMaxRows = (int64_t)1 << 30, kMaxK = (int64_t)1 << 24;

// A blocked axis that is summed over: 16-byte chunks of E4M3 bytes, 32-bit
// offsets inside a packed 128-row group.
bool summed_ok(int64_t K) { return K >= 16 && K % 16 == 0 && K <= kMaxK; }
bool rows_ok(int64_t N) { return N >= 1 && N <= kMaxRows; }
// Workgroup count of a launch with one workgroup per 128 x 128 tile.
bool tiles_ok(int64_t N, int64_t K) { return b128_blocks(N) * b128_blocks(K) <= INT32_MAX; }
bool act_grid_ok(int64_t M, int64_t K) {
  return b128_blocks(M) * b128_blocks(K) * 8 <= INT32_MAX;   // packed quantizer: bands x 128-blocks at most
}

size_t act_bytes(int64_t M, int64_t K) { return (size_t)b128_blocks(M) * 128 * (size_t)b128_blocks(K) * 128; }
size_t act_scale_bytes(int64_t M, int64_t K) { return act_bytes(M, K) / 32; }

int check_weight(const void* wp, const void* sp, int64_t N, int64_t K) {
  if (!wp || !sp) return MXFP8_E_NULLPTR;
  if (!rows_ok(N) || !summed_ok(K)) return MXFP8_E_SHAPE;
  if (!aligned(wp, 256) || !aligned(sp, 256)) return MXFP8_E_ALIGN;
  return MXFP8_OK;
}

int check_out(const void* y, int64_t N, int64_t ldy, const void* bias) {
  if (!y) return MXFP8_E_NULLPTR;
  if (ldy < N) return MXFP8_E_LD;
  if (!aligned(y, 2) || (bias && !aligned(bias, 2))) return MXFP8_E_ALIGN;
  return MXFP8_OK;
}

// The tile GEMM's grid and the split-K reduce's (one thread per 4 outputs)
// in 32-bit range.
bool gemm_grid_ok(int64_t M, int64_t N) {
  return b128_blocks(N) * ((M + 63) / 64) * mxfp8::kMaxSplitK <= INT32_MAX && M * ((N + 3) / 4) / 256 < INT32_MAX;
}

// Test hooks: pinned forms (0: by shape).
std::atomic<int> g_force_mt{0}, g_force_wgrad{0};

// The form and K splits with the least estimated time.  The estimates are
// lines through measurements on MI355X (us; M 17 .. 8192, N and K 512 ..
// 28672): a start, a cost per 128-block and round of workgroups, and for K
// splits a second launch and the partials' way to memory and back.  For
// example, at N = K = 4096 (64-row, 128-row, 256 x 128, 256 x 256 tiles):
//   M = 256    18   22   30   43  (with K splits in the first two)
//   M = 1024   27   26   34   46
//   M = 2048   50   47   37   49
//   M = 4096  100   90   69   59
// All four forms move 10 to 20 TB/s from L2 into LDS, so the bytes a tile
// reads for its products decide, where there are tiles for all compute units.
mxfp8::B128Plan b128_plan(int64_t M, int64_t N, int64_t K, int force, double* us) {
  const int64_t G = b128_blocks(N), KB = b128_blocks(K), GM = b128_blocks(M);
  // The larger forms write whole 16-byte pieces and address a tile's rows with
  // 32 bits; any other N, and at launch a y whose rows are not 16-byte aligned,
  // takes the 64-row tiles at every size.  What that costs (us, GEMM alone, N
  // just below and at a multiple of 8): 4096 x 4095 x 4096 117, 4096^3 61 (its
  // y off by one element 120); 4096 x 9001 and 9008 x 4096 250, 153; 2048 x
  // 32001 and 32008 x 4096 453, 247; 8192 x 28671 and 28672 x 8192 2840, 1571.
  const bool whole = N % 8 == 0 && N <= ((int64_t)1 << 22);
  mxfp8::B128Plan best = {64, 1};
  double best_us = 1e30;
  auto offer = [&](int mt, int splits, double t) {
    if (t < best_us) {
      best_us = t;
      best = {mt, splits};
      if (us) *us = t;
    }
  };
  auto join = [&](int s) { return s > 1 ? 3.0 + (double)s * (double)M * (double)N * 8.0 / 4e6 : 0.0; };
  auto blocks = [&](int s) { return (double)((KB + s - 1) / s); };
  auto wanted = [&](int mt) { return !force || force == mt || !whole; };
  const int64_t small = G * ((M + 63) / 64);
  for (int s = 1; wanted(64) && s <= mxfp8::kMaxSplitK && (s == 1 || KB / s >= 2); s *= 2) {
    const int64_t items = small * s;
    offer(64, s, 4.5 + (items <= 256 ? 0.35 : 0.67 * (double)((items + 511) / 512)) * blocks(s) + join(s));
  }
  if (!whole) return best;
  for (int s = 1; wanted(128) && s <= mxfp8::kMaxSplitK && (s == 1 || KB / s >= 2); s *= 2)
    offer(128, s, 4.5 + 0.65 * (double)((G * GM * s + 255) / 256) * blocks(s) + join(s));
  const int64_t large = (G + 1) / 2 * GM, wide = (G + 1) / 2 * ((GM + 1) / 2);
  if (wanted(256)) {
    const double rounds = (double)((large + 255) / 256);
    offer(256, 1, 5.0 + (large <= 128 ? 0.75 : (rounds > 1.0 ? 1.03 : 0.95) * rounds) * blocks(1));
  }
  if (wanted(512)) offer(512, 1, 5.0 + (wide <= 128 ? 1.25 : 1.7 * (double)((wide + 255) / 256)) * blocks(1));
  return best;
}

// Few rows: one launch that quantizes inside, without a workspace, or the
// quantizer and a tile form.  Lines through measurements (us; M 1 .. 32, N 512
// .. 28672, K 2048 .. 16384): a decode workgroup (16 weight rows) converts all
// activations, a second group of 16 rows costs another pass; the tile forms
// read the weight faster but start later.  For example, decode and tiles: 16 x
// 4096 x 4096 6.2, 12; 32 x 4096 x 4096 9.3, 13; 12 x 8192 x 8192 15.3, 19; 32
// x 8192 x 8192 29, 20; 1 x 28672 x 8192 38, 38; 16 rows of it 54, 38.
bool decode_form(int64_t M, int64_t N, int64_t K) {
  if (M > mxfp8::kB128DecodeMaxM) return false;
  if (M > 16 && g_force_mt.load(std::memory_order_relaxed) != 0) return false;
  double tile = 0.0;
  b128_plan(std::max<int64_t>(M, 1), N, K, 0, &tile);
  const double weight = (double)N * (double)K, rounds = std::max(1.0, (double)((N + 15) / 16) / 256.0);
  tile = std::max(tile, 4.5 + weight / 8e6) + 3.0;
  const double convert = 256.0 * rounds * (double)K * (1.17e-6 + 1.45e-7 * (double)M + (M > 16 ? 5.5e-7 : 0.0));
  return 3.0 + std::max(weight / 6.5e6, convert + 0.5 * (rounds - 1.0)) <= tile;
}

mxfp8::B128Plan b128_plan(int64_t M, int64_t N, int64_t K) {
  return b128_plan(M, N, K, g_force_mt.load(std::memory_order_relaxed), nullptr);
}

// The training step's weights are quantized from bf16, so their scales are
// powers of two and the scaled MFMA can apply them as well.  Where its 256 x
// 256 tiles are faster than the forms above, the step's GEMMs take the MXFP8
// tile GEMM, which has no v_fma: the same kind of line, measured with them
// (8192 x 4096 x 4096: 100 us against 116; 4096^3: 52, 62; 4096 x 2048 x 2048:
// 27, 25).  By the sizes alone: the forward call lays out scales that the
// backward call reads.
bool mx_gemm(int64_t M, int64_t N, int64_t K) {
  if (M <= mxfp8::kB128DecodeMaxM || K % 256 != 0) return false;
  double us = 0.0;
  b128_plan(M, N, K, 0, &us);
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  return 5.0 + (tiles <= 128 ? 1.1 : 1.42 * (double)((tiles + 255) / 256)) * (double)b128_blocks(K) < us;
}

constexpr int64_t kRuns = 256;   // compute units

// The form and the runs with the least estimated time (us, lines through
// measurements on MI355X: N and K 160 .. 8192, M 64 .. 16384): a start, a cost
// per tile and per 64-token step of a workgroup, and where tiles are shared
// the partials' way to memory and back and the launch that joins them.  For
// example (M, N, K; small tiles whole and in equal runs, large tiles the same):
//   512 x 1024 x 1024     14   17   32   32
//   16384 x 256 x 256    226   26  454   37
//   1000 x 2064 x 2032    37   38   48   43
//   4096 x 4096 x 4096   247  243  143  151
//   16384 x 5120 x 2048  665  561  435  374
mxfp8::WgradPlan wgrad_plan(int64_t M, int64_t N, int64_t K) {
  const int64_t steps = std::max<int64_t>(1, (M + mxfp8::kWgStep - 1) / mxfp8::kWgStep);
  const int force = g_force_wgrad.load(std::memory_order_relaxed);
  mxfp8::WgradPlan best = {};
  double best_us = 1e30;
  for (int tile : {128, 256}) {
    if (M == 0 ? tile != 128 : force && force != tile) continue;   // without tokens the small form writes the zeros
    const int64_t tn = (N + tile - 1) / tile, tk = (K + tile - 1) / tile, tiles = tn * tk, units = tiles * steps;
    auto offer = [&](mxfp8::Runs runs, int64_t pieces, double us) {
      if (us >= best_us) return;
      best_us = us;
      best = {tile, runs, tn, tk, steps, pieces};
    };
    auto ceil_div = [](int64_t a, int64_t b) { return (double)((a + b - 1) / b); };
    const bool small = tile == 128;
    // Whole tiles, one run per compute unit at most.
    const int64_t whole = std::min(kRuns, tiles);
    const double per_step = small ? 0.87 : whole == kRuns ? 1.95 : 1.62, per_tile = small ? 3.3 : 23.0;
    offer({tiles, (int)steps, (int)whole}, 1,
          (small ? 5.0 : 0.0) + ceil_div(tiles, whole) * (per_tile + per_step * (double)steps));
    // Equal runs, of two or eight steps at least.
    for (int64_t r = std::min(kRuns, units / (small ? 2 : 8)); r >= 2; r /= 2) {
      // a shared tile's pieces: its steps over the shortest run, and one more at either end
      const int64_t pieces = steps / (units / r) + 2;
      const double join = small ? 0.045 * (double)r + 0.12 * (double)pieces
                                : 0.08 * (double)(r + tiles - std::gcd(r, tiles));
      const double touched = ceil_div(tiles, r) + (!small && tiles > r ? 1.0 : 0.0);
      offer({units, 1, (int)r}, pieces,
            (small ? 5.0 + 3.3 * touched : 18.0 * touched) + (small ? 0.87 : 2.0) * ceil_div(units, r) + join);
    }
  }
  return best;
}

// fp32 partials of dW, then of db.
size_t wgrad_dw_bytes(const mxfp8::WgradPlan& p) {
  return p.shared() ? (size_t)p.runs.count * 2 * p.tile * p.tile * 4 : 0;
}
size_t wgrad_db_bytes(const mxfp8::WgradPlan& p) {
  return p.db_direct() ? 0 : (size_t)p.tiles() * (size_t)p.pieces * p.tile * 4;
}

size_t part_bytes(int64_t M, int64_t N, mxfp8::B128Plan p) {
  return p.splits > 1 ? round_up((size_t)p.splits * (size_t)M * (size_t)((N + 3) / 4 * 4) * 4, 256) : 0;
}

size_t linear_ws(int64_t M, int64_t N, int64_t K) {
  if (decode_form(M, N, K)) return 0;
  return round_up(act_bytes(M, K), 256) + round_up(act_scale_bytes(M, K), 256) +
         part_bytes(M, N, b128_plan(M, N, K));
}

size_t weight_scale_bytes(int64_t N, int64_t K, bool mx) {
  return mx ? act_scale_bytes(N, K) : (size_t)b128_blocks(N) * b128_blocks(K) * 4;
}

// What the layer's forward call keeps for its backward call: the transposed
// prepared weight (MXFP8_KEEP_DX), then the packed activations (MXFP8_KEEP_DW).
struct Kept {
  uint8_t *wt, *st, *q, *s;
};
size_t kept_layout(int64_t M, int64_t N, int64_t K, int keep, uint8_t* base, Kept* k) {
  size_t off = 0;
  auto take = [&](bool want, size_t bytes) {
    uint8_t* p = want && base ? base + off : nullptr;
    if (want) off += round_up(bytes, 256);
    return p;
  };
  const bool dx = keep & MXFP8_KEEP_DX, dw = (keep & MXFP8_KEEP_DW) && M > 0;
  Kept v;
  v.wt = take(dx, act_bytes(K, N));
  v.st = take(dx, weight_scale_bytes(K, N, mx_gemm(M, K, N)));
  v.q = take(dw, act_bytes(M, K));
  v.s = take(dw, act_scale_bytes(M, K));
  if (k) *k = v;
  return off;
}

// Forward workspace: the prepared weight and its scales, then the GEMM's
// (activations that are not kept, partials).
size_t forward_weight_bytes(int64_t M, int64_t N, int64_t K) {
  return round_up(act_bytes(N, K), 256) + round_up(weight_scale_bytes(N, K, mx_gemm(M, N, K)), 256);
}

int check_layer(int64_t M, int64_t N, int64_t K, int keep) {
  if (M < 0 || M > kMaxRows || !summed_ok(N) || !summed_ok(K) || (keep & ~(MXFP8_KEEP_DX | MXFP8_KEEP_DW)))
    return MXFP8_E_SHAPE;
  return MXFP8_OK;
}

int check_logits(const void* logits, int dtype, int64_t T, int64_t E, int64_t ldl, int64_t topk) {
  if (T < 0 || T > ((int64_t)1 << 31) - 1 || E < 1 || E > mxfp8::kMoeMaxExperts || topk < 1 || topk > E ||
      topk > mxfp8::kMoeMaxTopk || (dtype != MXFP8_F32 && dtype != MXFP8_BF16))
    return MXFP8_E_SHAPE;
  if (T == 0) return MXFP8_OK;
  if (!logits) return MXFP8_E_NULLPTR;
  if (ldl < E) return MXFP8_E_LD;
  if (!aligned(logits, dtype == MXFP8_F32 ? 4 : 2)) return MXFP8_E_ALIGN;
  return MXFP8_OK;
}

}  // namespace

extern "C" {

int mxfp8_quantize_b128(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, void* q_e4m3, int64_t ldq,
                        void* s_e8m0, int64_t lds, void* stream) {
  if (M < 0 || M > kMaxRows || !summed_ok(K)) return MXFP8_E_SHAPE;
  if (M == 0) return MXFP8_OK;
  if (!x_bf16 || !q_e4m3 || !s_e8m0) return MXFP8_E_NULLPTR;
  if (ldx < K || ldx % 8 != 0 || ldq < K || ldq % 16 != 0 || lds < b128_blocks(K)) return MXFP8_E_LD;
  if (!aligned(x_bf16, 16) || !aligned(q_e4m3, 16)) return MXFP8_E_ALIGN;
  if (M * b128_blocks(K) / 16 >= INT32_MAX) return MXFP8_E_SHAPE;
  if (int st = mxfp8::check_device_current()) return st;
  return mxfp8::launch_quantize_b128(x_bf16, M, K, ldx, q_e4m3, ldq, s_e8m0, lds, (hipStream_t)stream);
}

int mxfp8_packed_act_b128_bytes(int64_t M, int64_t K, size_t* q_bytes, size_t* s_bytes) {
  if (!q_bytes || !s_bytes) return MXFP8_E_NULLPTR;
  if (!rows_ok(M) || !summed_ok(K)) return MXFP8_E_SHAPE;
  *q_bytes = act_bytes(M, K);
  *s_bytes = act_scale_bytes(M, K);
  return MXFP8_OK;
}

int mxfp8_quantize_act_packed_b128(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, void* q_packed,
                                   void* s_packed, void* stream) {
  if (M < 0 || M > kMaxRows || !summed_ok(K)) return MXFP8_E_SHAPE;
  if (M == 0) return MXFP8_OK;
  if (!x_bf16 || !q_packed || !s_packed) return MXFP8_E_NULLPTR;
  if (ldx < K || ldx % 8 != 0) return MXFP8_E_LD;
  if (!aligned(x_bf16, 16) || !aligned(q_packed, 256) || !aligned(s_packed, 256)) return MXFP8_E_ALIGN;
  if (!act_grid_ok(M, K)) return MXFP8_E_SHAPE;
  if (int st = mxfp8::check_device_current()) return st;
  return mxfp8::launch_quantize_packed_b128(x_bf16, M, K, ldx, q_packed, s_packed, (hipStream_t)stream);
}

int mxfp8_dequantize_act_packed(const void* q_packed, const void* s_packed, int64_t M, int64_t K, void* x_bf16,
                                int64_t ldx, void* stream) {
  if (M < 0 || M > kMaxRows || !summed_ok(K)) return MXFP8_E_SHAPE;
  if (M == 0) return MXFP8_OK;
  if (!q_packed || !s_packed || !x_bf16) return MXFP8_E_NULLPTR;
  if (ldx < K || ldx % 8 != 0) return MXFP8_E_LD;
  if (!aligned(x_bf16, 16) || !aligned(q_packed, 256) || !aligned(s_packed, 256)) return MXFP8_E_ALIGN;
  if (M * (K / 16) / 256 >= INT32_MAX) return MXFP8_E_SHAPE;
  if (int st = mxfp8::check_device_current()) return st;
  return mxfp8::launch_dequantize_packed(q_packed, s_packed, M, K, x_bf16, ldx, (hipStream_t)stream);
}

int mxfp8_prepared_weight_b128_bytes(int64_t N, int64_t K, size_t* w_bytes, size_t* s_bytes) {
  if (!w_bytes || !s_bytes) return MXFP8_E_NULLPTR;
  if (!rows_ok(N) || !summed_ok(K)) return MXFP8_E_SHAPE;
  *w_bytes = act_bytes(N, K);
  *s_bytes = (size_t)b128_blocks(N) * (size_t)b128_blocks(K) * 4;
  return MXFP8_OK;
}

int mxfp8_prepare_weight_b128(const void* w_e4m3, const float* w_s, int64_t N, int64_t K, int64_t ldw, int64_t lds,
                              int transpose, void* w_packed, void* s_packed, void* stream) {
  if (!summed_ok(K) || (transpose ? !summed_ok(N) : !rows_ok(N))) return MXFP8_E_SHAPE;
  if (!w_e4m3 || !w_s || !w_packed || !s_packed) return MXFP8_E_NULLPTR;
  if (ldw < K || ldw % 16 != 0 || lds < b128_blocks(K)) return MXFP8_E_LD;
  if (!aligned(w_e4m3, 16) || !aligned(w_s, 4) || !aligned(w_packed, 256) || !aligned(s_packed, 256))
    return MXFP8_E_ALIGN;
  if (!tiles_ok(N, K)) return MXFP8_E_SHAPE;
  if (int st = mxfp8::check_device_current()) return st;
  return mxfp8::launch_pack_b128(w_e4m3, w_s, N, K, ldw, lds, transpose, w_packed, s_packed, (hipStream_t)stream);
}

int mxfp8_quantize_weight_b128(const void* w_bf16, int64_t N, int64_t K, int64_t ldw, void* q_e4m3, int64_t ldq,
                               float* s, int64_t lds, void* w_packed, void* s_packed, void* wt_packed,
                               void* st_packed, void* stream) {
  if (!summed_ok(K) || (wt_packed ? !summed_ok(N) : !rows_ok(N))) return MXFP8_E_SHAPE;
  if (!w_bf16 || (!q_e4m3 != !s) || (!w_packed != !s_packed) || (!wt_packed != !st_packed)) return MXFP8_E_NULLPTR;
  if (!q_e4m3 && !w_packed && !wt_packed) return MXFP8_E_NULLPTR;
  if (ldw < K || ldw % 8 != 0) return MXFP8_E_LD;
  if (q_e4m3 && (ldq < K || ldq % 16 != 0 || lds < b128_blocks(K))) return MXFP8_E_LD;
  if (!aligned(w_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(s, 4)) return MXFP8_E_ALIGN;
  if (!aligned(w_packed, 256) || !aligned(s_packed, 256) || !aligned(wt_packed, 256) || !aligned(st_packed, 256))
    return MXFP8_E_ALIGN;
  if (!tiles_ok(N, K)) return MXFP8_E_SHAPE;
  if (int st = mxfp8::check_device_current()) return st;
  return mxfp8::launch_quantize_weight_b128(w_bf16, N, K, ldw, q_e4m3, ldq, s, lds, w_packed, s_packed, wt_packed,
                                            st_packed, 0, (hipStream_t)stream);
}

int mxfp8_linear_b128_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return MXFP8_E_NULLPTR;
  if (M < 0 || M > kMaxRows || !rows_ok(N) || !summed_ok(K)) return MXFP8_E_SHAPE;
  *bytes = linear_ws(M, N, K);
  return MXFP8_OK;
}

int mxfp8_linear_b128(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, const void* w_packed,
                      const void* s_packed, int64_t N, const void* bias_bf16, void* y_bf16, int64_t ldy,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (M < 0 || M > kMaxRows) return MXFP8_E_SHAPE;
  if (int st = check_weight(w_packed, s_packed, N, K)) return st;
  if (M == 0) return MXFP8_OK;
  if (!x_bf16) return MXFP8_E_NULLPTR;
  if (int st = check_out(y_bf16, N, ldy, bias_bf16)) return st;
  if (ldx < K || ldx % 8 != 0) return MXFP8_E_LD;
  if (!aligned(x_bf16, 16)) return MXFP8_E_ALIGN;
  if (!gemm_grid_ok(M, N) || !act_grid_ok(M, K)) return MXFP8_E_SHAPE;
  const size_t need = linear_ws(M, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXFP8_E_WORKSPACE;
  if (!aligned(workspace, 256)) return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  hipStream_t s = (hipStream_t)stream;
  const float* wsc = (const float*)s_packed;
  if (decode_form(M, N, K))
    return mxfp8::launch_gemm_b128_decode(x_bf16, ldx, M, K, w_packed, wsc, N, bias_bf16, y_bf16, ldy, s);
  uint8_t* q = (uint8_t*)workspace;
  uint8_t* sc = q + round_up(act_bytes(M, K), 256);
  uint8_t* part = sc + round_up(act_scale_bytes(M, K), 256);
  if (int st = mxfp8::launch_quantize_packed_b128(x_bf16, M, K, ldx, q, sc, s)) return st;
  return mxfp8::launch_gemm_b128_tile(q, sc, M, K, w_packed, wsc, N, bias_bf16, y_bf16, ldy, s,
                                      b128_plan(M, N, K), part);
}

int mxfp8_gemm_packed_b128_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return MXFP8_E_NULLPTR;
  if (M < 0 || M > kMaxRows || !rows_ok(N) || !summed_ok(K)) return MXFP8_E_SHAPE;
  const size_t b = M == 0 ? 0 : part_bytes(M, N, b128_plan(M, N, K));
  *bytes = b > 256 ? b : 256;
  return MXFP8_OK;
}

int mxfp8_gemm_packed_b128(const void* q_packed, const void* s_packed, int64_t M, int64_t K, const void* w_packed,
                           const void* ws_packed, int64_t N, const void* bias_bf16, void* y_bf16, int64_t ldy,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (M < 0 || M > kMaxRows) return MXFP8_E_SHAPE;
  if (int st = check_weight(w_packed, ws_packed, N, K)) return st;
  if (M == 0) return MXFP8_OK;
  if (!q_packed || !s_packed) return MXFP8_E_NULLPTR;
  if (int st = check_out(y_bf16, N, ldy, bias_bf16)) return st;
  if (!aligned(q_packed, 256) || !aligned(s_packed, 256)) return MXFP8_E_ALIGN;
  if (!gemm_grid_ok(M, N)) return MXFP8_E_SHAPE;
  size_t need = 0;
  mxfp8_gemm_packed_b128_workspace_bytes(M, N, K, &need);
  if (!workspace || workspace_bytes < need) return MXFP8_E_WORKSPACE;
  if (!aligned(workspace, 256)) return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  return mxfp8::launch_gemm_b128_tile(q_packed, s_packed, M, K, w_packed, (const float*)ws_packed, N, bias_bf16,
                                      y_bf16, ldy, (hipStream_t)stream, b128_plan(M, N, K), workspace);
}

int mxfp8_debug_force_b128(int tile) {
  if (tile != 0 && tile != 64 && tile != 128 && tile != 256 && tile != 512) return MXFP8_E_SHAPE;
  return g_force_mt.exchange(tile);
}

int mxfp8_linear_wgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return MXFP8_E_NULLPTR;
  if (M < 0 || M > kMaxRows || !rows_ok(N) || N % 8 != 0 || !summed_ok(K)) return MXFP8_E_SHAPE;
  const mxfp8::WgradPlan p = wgrad_plan(M, N, K);
  *bytes = round_up(wgrad_dw_bytes(p), 256) + round_up(wgrad_db_bytes(p), 256);
  return MXFP8_OK;
}

int mxfp8_debug_force_wgrad(int tile) {
  if (tile != 0 && tile != 128 && tile != 256) return MXFP8_E_SHAPE;
  return g_force_wgrad.exchange(tile);
}

int mxfp8_linear_wgrad(const void* dy_bf16, int64_t M, int64_t N, int64_t lddy, const void* q_packed,
                       const void* s_packed, int64_t K, void* dw, int dw_dtype, int64_t lddw, void* db,
                       int db_dtype, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (M < 0 || M > kMaxRows || !rows_ok(N) || N % 8 != 0 || !summed_ok(K)) return MXFP8_E_SHAPE;
  if (dw_dtype != MXFP8_F32 && dw_dtype != MXFP8_BF16) return MXFP8_E_SHAPE;
  if (db && db_dtype != MXFP8_F32 && db_dtype != MXFP8_BF16) return MXFP8_E_SHAPE;
  if (accumulate && (dw_dtype != MXFP8_F32 || (db && db_dtype != MXFP8_F32))) return MXFP8_E_SHAPE;
  if (!dw || (M > 0 && (!dy_bf16 || !q_packed || !s_packed))) return MXFP8_E_NULLPTR;
  if (lddw < K || lddw % 8 != 0) return MXFP8_E_LD;
  // 64 rows of dY are addressed with 32-bit byte offsets.
  if (M > 0 && (lddy < N || lddy % 8 != 0 || lddy > kMaxK)) return MXFP8_E_LD;
  if (!aligned(dw, 16) || !aligned(db, db_dtype == MXFP8_F32 ? 4 : 2)) return MXFP8_E_ALIGN;
  if (M > 0 && (!aligned(dy_bf16, 16) || !aligned(q_packed, 256) || !aligned(s_packed, 256))) return MXFP8_E_ALIGN;
  const mxfp8::WgradPlan p = wgrad_plan(M, N, K);
  // the join's grid, and a run's units in 32 bits
  if (b128_blocks(N) * b128_blocks(K) > INT32_MAX / 64 || p.tiles() * p.steps / p.runs.count >= INT32_MAX)
    return MXFP8_E_SHAPE;
  size_t need = 0;
  mxfp8_linear_wgrad_workspace_bytes(M, N, K, &need);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXFP8_E_WORKSPACE;
  if (!aligned(workspace, 256)) return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  mxfp8::WgradArgs a;
  a.dy = dy_bf16;
  a.M = M;
  a.N = N;
  a.lddy = lddy;
  a.qp = q_packed;
  a.sp = s_packed;
  a.K = K;
  a.dw = dw;
  a.lddw = lddw;
  a.out_bf16 = dw_dtype == MXFP8_BF16;
  a.accumulate = accumulate != 0;
  a.db = db;
  a.db_bf16 = db_dtype == MXFP8_BF16;
  a.part_dw = (float*)workspace;
  a.part_db = (float*)((uint8_t*)workspace + round_up(wgrad_dw_bytes(p), 256));
  return mxfp8::launch_wgrad(a, p, (hipStream_t)stream);
}

int mxfp8_linear_b128_layer_bytes(int64_t M, int64_t N, int64_t K, int keep, size_t* kept_bytes,
                                  size_t* forward_ws_bytes, size_t* backward_ws_bytes) {
  if (!kept_bytes || !forward_ws_bytes || !backward_ws_bytes) return MXFP8_E_NULLPTR;
  if (int st = check_layer(M, N, K, keep)) return st;
  *kept_bytes = kept_layout(M, N, K, keep, nullptr, nullptr);
  size_t fwd = 0;
  if (M > 0 && (keep & MXFP8_KEEP_DW)) mxfp8_gemm_packed_b128_workspace_bytes(M, N, K, &fwd);
  else if (M > 0) mxfp8_linear_b128_workspace_bytes(M, N, K, &fwd);
  *forward_ws_bytes = forward_weight_bytes(M, N, K) + fwd;
  // the two products of the backward call run one after the other
  size_t dx = 0, dw = 0;
  if (keep & MXFP8_KEEP_DX) mxfp8_linear_b128_workspace_bytes(M, K, N, &dx);
  if (keep & MXFP8_KEEP_DW) mxfp8_linear_wgrad_workspace_bytes(M, N, K, &dw);
  *backward_ws_bytes = dx > dw ? dx : dw;
  return MXFP8_OK;
}

int mxfp8_linear_b128_forward(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, const void* w_bf16, int64_t N,
                              int64_t ldw, const void* bias_bf16, void* y_bf16, int64_t ldy, int keep, void* kept,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_layer(M, N, K, keep)) return st;
  size_t kept_bytes = 0, need = 0, back = 0;
  mxfp8_linear_b128_layer_bytes(M, N, K, keep, &kept_bytes, &need, &back);
  if (!w_bf16 || (kept_bytes > 0 && !kept) || (M > 0 && !x_bf16)) return MXFP8_E_NULLPTR;
  if (ldw < K || ldw % 8 != 0 || (M > 0 && (ldx < K || ldx % 8 != 0))) return MXFP8_E_LD;
  if (M > 0)
    if (int st = check_out(y_bf16, N, ldy, bias_bf16)) return st;
  if (!aligned(w_bf16, 16) || !aligned(kept, 256) || (M > 0 && !aligned(x_bf16, 16))) return MXFP8_E_ALIGN;
  if (!tiles_ok(N, K) || !gemm_grid_ok(M, N) || !act_grid_ok(M, K)) return MXFP8_E_SHAPE;
  if (!workspace || workspace_bytes < need) return MXFP8_E_WORKSPACE;
  if (!aligned(workspace, 256)) return MXFP8_E_ALIGN;
  Kept k;
  kept_layout(M, N, K, keep, (uint8_t*)kept, &k);
  uint8_t* wp = (uint8_t*)workspace;
  uint8_t* sp = wp + round_up(act_bytes(N, K), 256);
  uint8_t* rest = wp + forward_weight_bytes(M, N, K);
  const size_t rest_bytes = workspace_bytes - forward_weight_bytes(M, N, K);
  const bool mx = mx_gemm(M, N, K), mx_dx = k.wt != nullptr && mx_gemm(M, K, N);
  if (int st = mxfp8::check_device_current()) return st;
  hipStream_t s = (hipStream_t)stream;
  if (int st = mxfp8::launch_quantize_weight_b128(w_bf16, N, K, ldw, nullptr, 0, nullptr, 0, wp, sp, k.wt, k.st,
                                                  (mx ? 1 : 0) | (mx_dx ? 2 : 0), s))
    return st;
  if (M == 0) return MXFP8_OK;
  const bool dw = keep & MXFP8_KEEP_DW;
  if (!dw && !mx)
    return mxfp8_linear_b128(x_bf16, M, K, ldx, wp, sp, N, bias_bf16, y_bf16, ldy, rest, rest_bytes, stream);
  uint8_t* q = dw ? k.q : rest;
  uint8_t* qs = dw ? k.s : rest + round_up(act_bytes(M, K), 256);
  if (int st = mxfp8_quantize_act_packed_b128(x_bf16, M, K, ldx, q, qs, stream)) return st;
  if (mx) return mxfp8::launch_gemm_tile(q, qs, M, K, wp, sp, N, bias_bf16, y_bf16, ldy, s);
  return mxfp8_gemm_packed_b128(q, qs, M, K, wp, sp, N, bias_bf16, y_bf16, ldy, rest, rest_bytes, stream);
}

int mxfp8_linear_b128_backward(const void* dy_bf16, int64_t M, int64_t N, int64_t lddy, int64_t K, int keep,
                               const void* kept, void* dx_bf16, int64_t lddx, void* dw, int dw_dtype, int64_t lddw,
                               void* db, int db_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_layer(M, N, K, keep)) return st;
  if ((dx_bf16 && !(keep & MXFP8_KEEP_DX)) || (dw && !(keep & MXFP8_KEEP_DW)) || (db && !dw)) return MXFP8_E_SHAPE;
  size_t kept_bytes = 0, fwd = 0, need = 0;
  mxfp8_linear_b128_layer_bytes(M, N, K, keep, &kept_bytes, &fwd, &need);
  if (kept_bytes > 0 && !kept) return MXFP8_E_NULLPTR;
  if (!aligned(kept, 256)) return MXFP8_E_ALIGN;
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXFP8_E_WORKSPACE;
  Kept k;
  kept_layout(M, N, K, keep, (uint8_t*)kept, &k);
  // the weight gradient's checks cover dY as well; a refusal after the first
  // product would leave half a result, so both sets come first
  if (dx_bf16 && M > 0) {
    if (!dy_bf16) return MXFP8_E_NULLPTR;
    if (int st = check_out(dx_bf16, K, lddx, nullptr)) return st;
    if (lddy < N || lddy % 8 != 0) return MXFP8_E_LD;
    if (!aligned(dy_bf16, 16) || !aligned(workspace, 256)) return MXFP8_E_ALIGN;
    if (!gemm_grid_ok(M, K) || !act_grid_ok(M, N)) return MXFP8_E_SHAPE;
  }
  if (dw) {
    if (int st = mxfp8_linear_wgrad(dy_bf16, M, N, lddy, k.q, k.s, K, dw, dw_dtype, lddw, db, db_dtype, 0, workspace,
                                    workspace_bytes, stream))
      return st;
  }
  if (!dx_bf16 || M == 0) return MXFP8_OK;
  if (mx_gemm(M, K, N)) {
    uint8_t* q = (uint8_t*)workspace;
    uint8_t* qs = q + round_up(act_bytes(M, N), 256);
    if (int st = mxfp8_quantize_act_packed_b128(dy_bf16, M, N, lddy, q, qs, stream)) return st;
    return mxfp8::launch_gemm_tile(q, qs, M, N, k.wt, k.st, K, nullptr, dx_bf16, lddx, (hipStream_t)stream);
  }
  return mxfp8_linear_b128(dy_bf16, M, N, lddy, k.wt, k.st, K, nullptr, dx_bf16, lddx, workspace, workspace_bytes,
                           stream);
}

int mxfp8_moe_balance_workspace_bytes(int64_t T, int64_t E, size_t* bytes) {
  if (!bytes) return MXFP8_E_NULLPTR;
  if (T < 0 || E < 1 || E > mxfp8::kMoeMaxExperts) return MXFP8_E_SHAPE;
  *bytes = mxfp8::balance_ws_bytes(T, E);
  return MXFP8_OK;
}

int mxfp8_moe_balance(const void* logits, int dtype, int64_t T, int64_t E, int64_t ldl, int64_t topk,
                      const uint8_t* valid, float coef, float z_coef, float* loss, int* counts, int* used,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_logits(logits, dtype, T, E, ldl, topk)) return st;
  if (!loss || !counts || !used) return MXFP8_E_NULLPTR;
  if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(used, 4)) return MXFP8_E_ALIGN;
  const size_t need = mxfp8::balance_ws_bytes(T, E);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXFP8_E_WORKSPACE;
  if (!aligned(workspace, 256)) return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  mxfp8::BalanceArgs a = {};
  a.logits = logits;
  a.bf16 = dtype == MXFP8_BF16;
  a.T = T;
  a.E = E;
  a.ldl = ldl;
  a.topk = topk;
  a.valid = valid;
  a.coef = coef;
  a.z_coef = z_coef;
  a.counts = counts;
  a.used = used;
  a.loss = loss;
  a.ws = workspace;
  return mxfp8::launch_balance(a, (hipStream_t)stream);
}

int mxfp8_moe_balance_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ldl, int64_t topk,
                               const uint8_t* valid, float coef, float z_coef, const int* counts, const int* used,
                               const float* grad_loss, void* dlogits, int64_t ldd, void* stream) {
  if (int st = check_logits(logits, dtype, T, E, ldl, topk)) return st;
  if (T == 0) return MXFP8_OK;
  if (!counts || !used || !dlogits) return MXFP8_E_NULLPTR;
  if (ldd < E) return MXFP8_E_LD;
  if (!aligned(dlogits, dtype == MXFP8_F32 ? 4 : 2) || !aligned(counts, 4) || !aligned(used, 4) ||
      !aligned(grad_loss, 4))
    return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  mxfp8::BalanceArgs a = {};
  a.logits = logits;
  a.bf16 = dtype == MXFP8_BF16;
  a.T = T;
  a.E = E;
  a.ldl = ldl;
  a.topk = topk;
  a.valid = valid;
  a.coef = coef;
  a.z_coef = z_coef;
  a.counts = const_cast<int*>(counts);
  a.used = const_cast<int*>(used);
  a.grad_loss = grad_loss;
  a.dlogits = dlogits;
  a.ldd = ldd;
  return mxfp8::launch_balance_backward(a, (hipStream_t)stream);
}

}  // extern "C"
