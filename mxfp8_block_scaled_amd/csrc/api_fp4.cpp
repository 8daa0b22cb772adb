// C ABI (include/mxfp8.h) of the MXFP4 x MXFP4 linear layer, of tokens sorted
// by expert and back, and of the experts' MXFP4 products: argument validation
// on the host, device check, launches.  Nothing here allocates device memory
// or synchronizes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "launch_fp4.hpp"
#include "mxfp8.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

constexpr int64_t kMaxRows = (int64_t)1 << 30, kMaxK = (int64_t)1 << 24, kMaxN = (int64_t)1 << 24;
constexpr int64_t kMaxTokens = (int64_t)1 << 24, kMaxSlots = (int64_t)1 << 26;

bool summed_ok(int64_t K) { return K >= 256 && K % 256 == 0 && K <= kMaxK; }
int64_t pad128(int64_t n) { return (n + 127) / 128 * 128; }

size_t act_bytes(int64_t M, int64_t K) { return (size_t)pad128(M) * (size_t)(K / 2); }
size_t act_scale_bytes(int64_t M, int64_t K) { return (size_t)pad128(M) * (size_t)(K / 32); }
// A launch has fewer than 2^32 threads: the quantizer's (256 per 16 rows and
// four 128-K steps), and the tile GEMM's list in 32-bit range.
constexpr int64_t kMaxThreads = UINT32_MAX;
bool act_grid_ok(int64_t M, int64_t K) { return pad128(M) / 16 * ((K + 511) / 512) * 256 <= kMaxThreads; }
bool gemm_grid_ok(int64_t M, int64_t N) { return (M + 63) / 64 * ((N + 127) / 128) <= INT32_MAX / 2; }
bool linear_grid_ok(int64_t M, int64_t N, int64_t K) { return act_grid_ok(M, K) && gemm_grid_ok(M, N); }
// The pack kernels' grids: one thread per 16 bytes, one per scale pair.  Experts
// of whole 128-row groups are packed at once where that fits.
bool pack_at_once(int64_t E, int64_t N, int64_t K) { return N % 128 == 0 && E * N * (K / 32) <= kMaxThreads - 255; }
bool pack_grid_ok(int64_t N, int64_t K) { return pad128(N) * (K / 32) <= kMaxThreads - 255; }

// Test hook: pinned form (0: by shape).
std::atomic<int> g_force{0};

// The forms with the least estimated time: lines through measurements on
// MI355X (us, 16 calls in a captured graph, the quantizer's launch included), K
// in thousands (1024).  They are of the whole chip, 256 units: the size queries
// run without a device.  On a part of one the launchers fit their grids to its
// units, and the choice of form, which changes no result, may not be the best.
// For example (decode; 16 weight rows on packed activations;
// 128 x 64 tiles that quantize their rows; tiles of 128 x 64, 128 x 128, 256 x
// 256), N x K = 4096 x 1024:
//   M = 1        3.0    6.8    6.6    8.0    9.0
//   M = 32       5.7    6.8    7.2    8.1    9.2
//   M = 128             7.1    8.9    8.2    9.4   16.2
//   M = 1000                  13.7   10.4   10.9   17.3
//   M = 4096                  47.7   27.8   23.4   23.7
// 4096 x 4096:
//   M = 1        4.0    7.0          11.5   13.9
//   M = 16       6.0    7.1          11.7   14.0
//   M = 32       8.9    7.2          11.7   14.2
//   M = 128            10.9          12.0   14.3   30.7
//   M = 1000                         20.1   19.0   33.7
//   M = 4096                         62.3   50.3   46.3
// and 16384 x 8192:
//   M = 1       14.6   23.9          17.6   20.9
//   M = 16      16.8   23.6          17.9   21.2
//   M = 32             23.8          17.6   21.3
//   M = 2048                        186.8  148.2  134.0
double thousands(int64_t K) { return (double)K / 1024.0; }
// One block of 16 weight rows for each decode workgroup.
bool decode_one(bool experts, int64_t parts, int64_t M, int64_t N, int64_t K) {
  return parts * ((N + 15) / 16) <= 256 * mxfp8::fp4_decode_per_cu(experts, M, K);
}
double decode_us(int64_t M, int64_t N, int64_t K) {
  const double k = thousands(K), m = (double)M, t = std::max(1.0, (double)N / 4096.0), w = k * (double)N / 16384.0;
  if (decode_one(false, 1, M, N, K))
    return M > 16 ? 3.1 + 0.058 * m + k * (0.11 + (K > 2048 ? 0.0275 : 0.0175) * m)
                  : 2.7 + 0.055 * m + k * (0.25 + 0.018 * m) + (t - 1.0) * (0.24 + 0.02 * k * m);
  return M > 16 ? 4.4 + 0.07 * m + w * (0.42 + 0.016 * m) + 0.51 * t : 3.6 + 0.13 * m + 1.54 * w - 0.31 * t;
}
double mid_us(int64_t M, int64_t N, int64_t K) {
  const double k = thousands(K), t = std::ceil((double)N / 4096.0);
  if (M <= 32) return 4.3 + t * std::max(2.5, 0.7 + 0.54 * k);
  if (M <= 64) return 4.1 + t * std::max(3.9, 1.3 + 0.77 * k);
  return 4.1 + t * std::max(3.0, 1.7 + 1.29 * k);
}
double tile_us(int nt, int mt, int64_t M, int64_t N, int64_t K) {
  const double k = thousands(K), q = k * (double)M / 1024.0;   // q: the quantizer's share
  const double r = (double)((M + mt - 1) / mt * ((N + nt - 1) / nt)) / 256.0;   // rounds of the chip
  if (nt == 256)
    return r <= 1.0 ? 11.9 + 4.48 * k + r * (1.8 + 2.28 * k) + 0.41 * q
                    : 9.2 - 0.8 * k + std::ceil(r) * (6.1 + 6.37 * k) + 0.62 * q;
  if (mt == 128)
    return r <= 1.0 ? 7.7 + 1.48 * k + r * (0.4 + 0.68 * k) + 0.5 * q : 7.1 + 0.82 * k + r * (1.3 + 1.85 * k) + 0.42 * q;
  return r <= 1.0 ? 7.1 + 1.06 * k + 0.7 * r * k + 0.36 * q : 6.7 + 0.49 * k + r * (0.85 + 1.28 * k) + 0.43 * q;
}
// (Past one round and K 1024 their LDS holds one workgroup per compute unit:
// more than twice the time of two launches.)
bool can_fuse(int64_t tiles, int64_t K) { return K <= mxfp8::kFp4FusedMaxK && (K <= 1024 || tiles <= 256); }
double fused_us(int64_t M, int64_t N, int64_t K) {
  const double k = thousands(K), r = (double)((M + 63) / 64 * ((N + 127) / 128)) / 256.0;
  return r <= 1.0 ? 4.8 + k * (1.46 + 0.038 * (double)std::min<int64_t>(64, M)) + r * (0.4 + 0.35 * k)
                  : 5.3 + r * (1.2 + 3.76 * k);
}

// The GEMM on packed activations: nt == 16 is the 16-row form.
mxfp8::Fp4Plan tile_plan(int64_t M, int64_t N, int64_t K, double* us = nullptr) {
  const int force = g_force.load(std::memory_order_relaxed);
  mxfp8::Fp4Plan best = {128, 64};
  double best_us = 1e30;
  auto offer = [&](int form, int nt, int mt, double t) {
    if (force == form) t = -1.0;
    if (t >= best_us) return;
    best_us = t;
    best = {nt, mt};
  };
  if (M <= mxfp8::kFp4MidMaxM) offer(16, 16, 128, mid_us(M, N, K));
  offer(64, 128, 64, tile_us(128, 64, M, N, K));
  offer(128, 128, 128, tile_us(128, 128, M, N, K));
  offer(256, 256, 256, tile_us(256, 256, M, N, K));
  if (us) *us = best_us;
  return best;
}

// The forms of one launch that quantizes inside, without a workspace: decode,
// and 128 x 64 tiles.  0: neither.
enum { kTwoLaunches = 0, kDecode = 1, kFusedTiles = 2 };
int one_launch(int64_t M, int64_t N, int64_t K) {
  const bool decode = M <= mxfp8::fp4_decode_max_m(K), fused = K <= mxfp8::kFp4FusedMaxK;
  const int force = g_force.load(std::memory_order_relaxed);
  if (force != 0) return force == 1 && decode ? kDecode : force == 2 && fused ? kFusedTiles : kTwoLaunches;
  double us = 0.0;
  tile_plan(M, N, K, &us);
  us += 1.0;   // (outside of a captured graph a second launch costs the host about 5 us)
  const double td = decode ? decode_us(M, N, K) : 1e30;
  const double tf = can_fuse((M + 63) / 64 * ((N + 127) / 128), K) ? fused_us(M, N, K) : 1e30;
  if (td <= std::min(tf, us)) return kDecode;
  return tf <= us ? kFusedTiles : kTwoLaunches;
}

int gemm(const void* q, const void* s, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
         const void* bias, void* y, int64_t ldy, hipStream_t stream) {
  const mxfp8::Fp4Plan plan = tile_plan(M, N, K);
  if (plan.nt == 16) return mxfp8::launch_gemm_fp4_mid(q, s, M, K, wp, wsp, N, bias, y, ldy, stream);
  return mxfp8::launch_gemm_fp4_tile(q, s, M, K, wp, wsp, N, bias, y, ldy, stream, plan);
}

int check_weight(const void* wp, const void* sp, int64_t N, int64_t K) {
  if (!wp || !sp) return MXFP8_E_NULLPTR;
  if (N < 1 || N > kMaxN || !summed_ok(K)) return MXFP8_E_SHAPE;
  if (!aligned(wp, 256) || !aligned(sp, 256)) return MXFP8_E_ALIGN;
  return MXFP8_OK;
}

int check_out(const void* y, int64_t N, int64_t ldy, const void* bias) {
  if (!y) return MXFP8_E_NULLPTR;
  if (ldy < N) return MXFP8_E_LD;
  if (!aligned(y, 2) || (bias && !aligned(bias, 4))) return MXFP8_E_ALIGN;
  return MXFP8_OK;
}

size_t linear_ws(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || one_launch(M, N, K) != kTwoLaunches) return 0;
  return round_up(act_bytes(M, K), 256) + round_up(act_scale_bytes(M, K), 256);
}

// T tokens with topk slots each over E experts.
bool slots_ok(int64_t T, int64_t topk) {
  return T >= 0 && T <= kMaxTokens && topk >= 1 && topk <= mxfp8::kMoeMaxTopk && T * topk <= kMaxSlots;
}
bool experts_ok(int64_t E) { return E >= 1 && E <= mxfp8::kMoeMaxExperts; }

int check_matrix(const void* p, int64_t H, int64_t ld, int size) {
  if (!p) return MXFP8_E_NULLPTR;
  if (ld < H) return MXFP8_E_LD;
  return aligned(p, size) ? MXFP8_OK : MXFP8_E_ALIGN;
}
int check_rows(int dtype, int64_t T, int64_t H, int64_t topk) {
  if ((dtype != MXFP8_F32 && dtype != MXFP8_BF16) || !slots_ok(T, topk) || H < 1 || H > kMaxK) return MXFP8_E_SHAPE;
  const int64_t per = dtype == MXFP8_BF16 ? 8 : 4;
  return T * ((H + per - 1) / per) <= kMaxThreads - 255 ? MXFP8_OK : MXFP8_E_SHAPE;
}

struct ExpertsForm {
  int one;               // as one_launch
  mxfp8::Fp4Plan plan;
};
// The same for the experts, whose rows' spread the host does not know, nor how
// many slots have an expert here: as if all R had one, X experts with rows at
// most, R / X rows each.  (A rank that holds an eighth of the experts plans for
// eight times its rows.)  Decode reads all their weights
// with its rows converted again for each 16 weight rows; tiles that quantize
// their rows take a longer start, a quantizer before them one more launch.  For
// example (rows per expert; decode, 128 x 64 tiles that quantize, tiles of 128 x
// 64, 128 x 128, 256 x 128), N x K = 2048 x 2048 and 2048 x 768:
//   8 experts, 1    10.6   12.0   12.1                    6.7    7.9    9.0
//   32, 1           14.1   18.5   16.2                   10.1    9.9   11.4
//   64, 2           21.8   27.7   23.2                   11.9   13.2   14.4
//   64, 6           41.3   46.4   31.7                   20.1   17.9   17.3
// and 128 experts, 1536 x 2048 and 2048 x 768:
//   64                            60     61     62                      40    42    42
//   256                          140    124    114                      98    89    84
ExpertsForm experts_form(int64_t R, int64_t N, int64_t K, int64_t E) {
  const int force = g_force.load(std::memory_order_relaxed);
  const double X = (double)std::max<int64_t>(1, std::min(E, R)), rows = (double)R / X;
  const double work = 1e-6 * X * (double)N * (double)K;
  const bool can_decode = K <= mxfp8::kFp4DecodeMaxK, fused = K <= mxfp8::kFp4FusedMaxK;
  if (force == 1 && can_decode) return {kDecode, {}};
  if (force == 2 && fused) return {kFusedTiles, {}};
  if (force == 0) {
    const double k = thousands(K);
    const int64_t cols = (N + 127) / 128, most = (R / 64 + std::min(E, R)) * cols;   // (row tiles: one per expert is partial)
    const double two = 8.1 + 2.05 * k + 0.05 * work;
    const double td = !can_decode || rows > 8.0                  ? 1e30
                      : decode_one(true, std::min(E, R), 0, N, K) ? 4.3 + 0.15 * work * (1.0 + rows / 8.0)
                                                            : 6.5 + 0.07 * work * (1.0 + rows / 7.0);
    const double tf = !can_fuse(std::min(E, R) * cols, K) ? 1e30
                      : most <= 256                       ? 6.3 + k * (2.0 + 0.037 * std::min(64.0, rows))
                                                          : 5.4 + 2.76 * k + work * (0.045 + 8.0e-3 * rows);
    if (td <= std::min(tf, two)) return {kDecode, {}};
    if (tf <= two) return {kFusedTiles, {}};
  }
  if (force == 256) return {kTwoLaunches, {256, 128}};
  if (force == 128) return {kTwoLaunches, {128, 128}};
  if (force == 64 || rows < 128.0) return {kTwoLaunches, {128, 64}};
  // Wide tiles read the least through L2, but one workgroup fills a compute
  // unit: where there are several rounds of them.
  return {kTwoLaunches, (double)R / 128.0 * ((double)N / 256.0) >= 6.0 * 256.0 ? mxfp8::Fp4Plan{256, 128}
                                                                         : mxfp8::Fp4Plan{128, 128}};
}
bool experts_shape_ok(int64_t x_rows, int64_t R, int64_t N, int64_t K, int64_t E) {
  return x_rows >= 0 && R >= 0 && R <= kMaxSlots && x_rows <= R && N >= 1 && N <= kMaxN && summed_ok(K) &&
         experts_ok(E) && x_rows * (K / 2) < ((int64_t)1 << 32) &&
         (R / 64 + std::min(E, R)) * ((N + 127) / 128) <= INT32_MAX / 2;
}
size_t experts_q_bytes(int64_t x_rows, int64_t K) { return round_up((size_t)x_rows * (size_t)(K / 2), 256); }
size_t experts_ws(int64_t x_rows, int64_t R, int64_t N, int64_t K, int64_t E) {
  if (R == 0 || experts_form(R, N, K, E).one != kTwoLaunches) return 0;
  return experts_q_bytes(x_rows, K) + round_up((size_t)x_rows * (size_t)mxfp8::fp4_scale_pitch(K), 256);
}

}  // namespace

extern "C" {

int mxfp8_packed_act_fp4_bytes(int64_t M, int64_t K, size_t* q_bytes, size_t* s_bytes) {
  if (!q_bytes || !s_bytes) return MXFP8_E_NULLPTR;
  if (M < 1 || M > kMaxRows || !summed_ok(K) || !act_grid_ok(M, K)) return MXFP8_E_SHAPE;
  *q_bytes = act_bytes(M, K);
  *s_bytes = act_scale_bytes(M, K);
  return MXFP8_OK;
}

int mxfp8_quantize_act_packed_fp4(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, void* q_packed,
                                  void* s_packed, void* stream) {
  if (M < 0 || M > kMaxRows || !summed_ok(K)) return MXFP8_E_SHAPE;
  if (M == 0) return MXFP8_OK;
  if (!x_bf16 || !q_packed || !s_packed) return MXFP8_E_NULLPTR;
  if (ldx < K || ldx % 8 != 0) return MXFP8_E_LD;
  if (!aligned(x_bf16, 16) || !aligned(q_packed, 256) || !aligned(s_packed, 256)) return MXFP8_E_ALIGN;
  if (!act_grid_ok(M, K)) return MXFP8_E_SHAPE;
  if (int st = mxfp8::check_device_current()) return st;
  return mxfp8::launch_quantize_packed_fp4(x_bf16, M, K, ldx, q_packed, s_packed, (hipStream_t)stream);
}

int mxfp8_gemm_packed_fp4(const void* q_packed, const void* s_packed, int64_t M, int64_t K, const void* w_packed,
                          const void* ws_packed, int64_t N, const void* bias_bf16, void* y_bf16, int64_t ldy,
                          void* stream) {
  if (M < 0 || M > kMaxRows) return MXFP8_E_SHAPE;
  if (int st = check_weight(w_packed, ws_packed, N, K)) return st;
  if (M == 0) return MXFP8_OK;
  if (!q_packed || !s_packed) return MXFP8_E_NULLPTR;
  if (!aligned(q_packed, 256) || !aligned(s_packed, 256)) return MXFP8_E_ALIGN;
  if (int st = check_out(y_bf16, N, ldy, bias_bf16)) return st;
  if (!gemm_grid_ok(M, N)) return MXFP8_E_SHAPE;
  if (int st = mxfp8::check_device_current()) return st;
  return gemm(q_packed, s_packed, M, K, w_packed, ws_packed, N, bias_bf16, y_bf16, ldy, (hipStream_t)stream);
}

int mxfp8_linear_w4a4_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return MXFP8_E_NULLPTR;
  if (M < 0 || M > kMaxRows || N < 1 || N > kMaxN || !summed_ok(K) || !linear_grid_ok(M, N, K)) return MXFP8_E_SHAPE;
  *bytes = linear_ws(M, N, K);
  return MXFP8_OK;
}

int mxfp8_linear_w4a4(const void* x_bf16, int64_t M, int64_t K, int64_t ldx, const void* w_packed,
                      const void* s_packed, int64_t N, const void* bias_bf16, void* y_bf16, int64_t ldy,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (M < 0 || M > kMaxRows) return MXFP8_E_SHAPE;
  if (int st = check_weight(w_packed, s_packed, N, K)) return st;
  if (M == 0) return MXFP8_OK;
  if (!x_bf16) return MXFP8_E_NULLPTR;
  if (ldx < K || ldx % 8 != 0) return MXFP8_E_LD;
  if (!aligned(x_bf16, 16)) return MXFP8_E_ALIGN;
  if (int st = check_out(y_bf16, N, ldy, bias_bf16)) return st;
  if (!linear_grid_ok(M, N, K)) return MXFP8_E_SHAPE;
  const size_t need = linear_ws(M, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXFP8_E_WORKSPACE;
  if (!aligned(workspace, 256)) return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  const int form = one_launch(M, N, K);
  if (form == kDecode)
    return mxfp8::launch_gemm_fp4_decode(x_bf16, ldx, M, K, w_packed, s_packed, N, bias_bf16, y_bf16, ldy,
                                         (hipStream_t)stream);
  if (form == kFusedTiles)
    return mxfp8::launch_gemm_fp4_fused(x_bf16, ldx, M, K, w_packed, s_packed, N, bias_bf16, y_bf16, ldy,
                                        (hipStream_t)stream);
  uint8_t* q = (uint8_t*)workspace;
  uint8_t* s = q + round_up(act_bytes(M, K), 256);
  if (int st = mxfp8::launch_quantize_packed_fp4(x_bf16, M, K, ldx, q, s, (hipStream_t)stream)) return st;
  return gemm(q, s, M, K, w_packed, s_packed, N, bias_bf16, y_bf16, ldy, (hipStream_t)stream);
}

int mxfp8_debug_force_w4a4(int form) {
  if (form != 0 && form != 1 && form != 2 && form != 16 && form != 64 && form != 128 && form != 256) return MXFP8_E_SHAPE;
  return g_force.exchange(form);
}

int mxfp8_moe_sort_workspace_bytes(int64_t slots, int64_t E, size_t* bytes) {
  if (!bytes) return MXFP8_E_NULLPTR;
  if (slots < 0 || slots > kMaxSlots || !experts_ok(E)) return MXFP8_E_SHAPE;
  *bytes = mxfp8::sort_ws_bytes(slots, E);
  return MXFP8_OK;
}

int mxfp8_moe_sort(const void* ids, int id_bytes, int64_t slots, int64_t E, int32_t* row_of_slot,
                   int32_t* slot_of_row, int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream) {
  if (slots < 0 || slots > kMaxSlots || !experts_ok(E) || (id_bytes != 4 && id_bytes != 8)) return MXFP8_E_SHAPE;
  if (!offsets || (slots > 0 && (!ids || !row_of_slot || !slot_of_row))) return MXFP8_E_NULLPTR;
  if (!aligned(ids, id_bytes) || !aligned(row_of_slot, 4) || !aligned(slot_of_row, 4) || !aligned(offsets, 4))
    return MXFP8_E_ALIGN;
  const size_t need = mxfp8::sort_ws_bytes(slots, E);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXFP8_E_WORKSPACE;
  if (!aligned(workspace, 256)) return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  mxfp8::SortArgs a = {};
  a.ids = ids;
  a.wide = id_bytes == 8;
  a.R = slots;
  a.E = E;
  a.rows = row_of_slot;
  a.slots = slot_of_row;
  a.offsets = offsets;
  a.ws = (int*)workspace;
  return mxfp8::launch_moe_sort(a, (hipStream_t)stream);
}

int mxfp8_moe_permute(const void* x, int dtype, int64_t T, int64_t H, int64_t ldx, int64_t topk,
                      const int32_t* row_of_slot, const int32_t* kept, void* xs, int64_t ldxs, void* stream) {
  if (int st = check_rows(dtype, T, H, topk)) return st;
  if (T == 0) return MXFP8_OK;
  const int size = dtype == MXFP8_BF16 ? 2 : 4;
  if (!row_of_slot || !kept) return MXFP8_E_NULLPTR;
  if (int st = check_matrix(x, H, ldx, size)) return st;
  if (int st = check_matrix(xs, H, ldxs, size)) return st;
  if (!aligned(row_of_slot, 4) || !aligned(kept, 4)) return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  mxfp8::PermuteArgs a = {};
  a.bf16 = dtype == MXFP8_BF16;
  a.T = T;
  a.H = H;
  a.topk = topk;
  a.rows = row_of_slot;
  a.kept = kept;
  a.tokens = x;
  a.ldt = ldx;
  a.out_sorted = xs;
  a.ldo = ldxs;
  return mxfp8::launch_moe_permute(a, (hipStream_t)stream);
}

int mxfp8_moe_unpermute(const void* ys, int dtype, int64_t T, int64_t H, int64_t ldys, int64_t topk,
                        const int32_t* row_of_slot, const int32_t* kept, const float* weights, void* y, int64_t ldy,
                        void* stream) {
  if (int st = check_rows(dtype, T, H, topk)) return st;
  if (T == 0) return MXFP8_OK;
  const int size = dtype == MXFP8_BF16 ? 2 : 4;
  if (!row_of_slot || !kept) return MXFP8_E_NULLPTR;
  if (int st = check_matrix(ys, H, ldys, size)) return st;
  if (int st = check_matrix(y, H, ldy, size)) return st;
  if (!aligned(row_of_slot, 4) || !aligned(kept, 4) || !aligned(weights, 4)) return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  mxfp8::PermuteArgs a = {};
  a.bf16 = dtype == MXFP8_BF16;
  a.T = T;
  a.H = H;
  a.topk = topk;
  a.rows = row_of_slot;
  a.kept = kept;
  a.sorted = ys;
  a.lds = ldys;
  a.weights = weights;
  a.out_tokens = y;
  a.ldo = ldy;
  return mxfp8::launch_moe_unpermute(a, (hipStream_t)stream);
}

int mxfp8_moe_unpermute_backward(const void* dy, int dtype, int64_t T, int64_t H, int64_t lddy, int64_t topk,
                                 const int32_t* row_of_slot, const int32_t* kept, const void* ys, int64_t ldys,
                                 const float* weights, void* dys, int64_t lddys, float* dweights, void* stream) {
  if (int st = check_rows(dtype, T, H, topk)) return st;
  if (T == 0) return MXFP8_OK;
  const int size = dtype == MXFP8_BF16 ? 2 : 4;
  if (!row_of_slot || !kept || (!dys && !dweights)) return MXFP8_E_NULLPTR;
  if (int st = check_matrix(dy, H, lddy, size)) return st;
  if (dweights)
    if (int st = check_matrix(ys, H, ldys, size)) return st;
  if (dys)
    if (int st = check_matrix(dys, H, lddys, size)) return st;
  if (!aligned(row_of_slot, 4) || !aligned(kept, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  mxfp8::PermuteArgs a = {};
  a.bf16 = dtype == MXFP8_BF16;
  a.T = T;
  a.H = H;
  a.topk = topk;
  a.rows = row_of_slot;
  a.kept = kept;
  a.tokens = dy;
  a.ldt = lddy;
  a.sorted = dweights ? ys : nullptr;
  a.lds = ldys;
  a.weights = weights;
  a.out_sorted = dys;
  a.ldo = lddys;
  a.dweights = dweights;
  return mxfp8::launch_moe_unpermute_backward(a, (hipStream_t)stream);
}

int mxfp8_moe_prepared_experts_fp4_bytes(int64_t E, int64_t N, int64_t K, size_t* w_bytes, size_t* s_bytes) {
  if (!w_bytes || !s_bytes) return MXFP8_E_NULLPTR;
  if (!experts_ok(E) || N < 1 || N > kMaxN || !summed_ok(K) || !pack_grid_ok(N, K)) return MXFP8_E_SHAPE;
  *w_bytes = (size_t)E * act_bytes(N, K);
  *s_bytes = (size_t)E * act_scale_bytes(N, K);
  return MXFP8_OK;
}

int mxfp8_moe_prepare_experts_fp4(const void* w_e2m1, const void* w_s_e8m0, int64_t E, int64_t N, int64_t K,
                                  void* w_packed, void* s_packed, void* stream) {
  if (!experts_ok(E)) return MXFP8_E_SHAPE;
  if (int st = check_weight(w_packed, s_packed, N, K)) return st;
  if (!w_e2m1 || !w_s_e8m0) return MXFP8_E_NULLPTR;
  if (!aligned(w_e2m1, 16)) return MXFP8_E_ALIGN;
  if (!pack_grid_ok(N, K)) return MXFP8_E_SHAPE;
  if (int st = mxfp8::check_device_current()) return st;
  const bool at_once = pack_at_once(E, N, K);
  const int64_t rows = at_once ? E * N : N, passes = at_once ? 1 : E;
  for (int64_t e = 0; e < passes; ++e) {
    const size_t w = (size_t)e * N * (K / 2), s = (size_t)e * N * (K / 32);
    if (int st = mxfp8::launch_pack_weight_fp4((const uint8_t*)w_e2m1 + w, (const uint8_t*)w_s_e8m0 + s, rows, K,
                                               K / 2, K / 32, (uint8_t*)w_packed + (size_t)e * act_bytes(N, K),
                                               (uint8_t*)s_packed + (size_t)e * act_scale_bytes(N, K),
                                               (hipStream_t)stream))
      return st;
  }
  return MXFP8_OK;
}

int mxfp8_moe_linear_w4a4_workspace_bytes(int64_t x_rows, int64_t R, int64_t N, int64_t K, int64_t E, size_t* bytes) {
  if (!bytes) return MXFP8_E_NULLPTR;
  if (!experts_shape_ok(x_rows, R, N, K, E)) return MXFP8_E_SHAPE;
  *bytes = experts_ws(x_rows, R, N, K, E);
  return MXFP8_OK;
}

int mxfp8_moe_linear_w4a4(const void* x_bf16, int64_t x_rows, int64_t K, int64_t ldx, const int32_t* slot_of_row,
                          int64_t topk, const int32_t* offsets, int64_t R, int64_t E, const void* w_packed,
                          const void* s_packed, int64_t N, void* y_bf16, int64_t ldy, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!experts_shape_ok(x_rows, R, N, K, E)) return MXFP8_E_SHAPE;
  if (slot_of_row ? topk < 1 || topk > mxfp8::kMoeMaxTopk || x_rows * topk != R : x_rows != R) return MXFP8_E_SHAPE;
  if (int st = check_weight(w_packed, s_packed, N, K)) return st;
  if (R == 0) return MXFP8_OK;
  if (!x_bf16 || !offsets) return MXFP8_E_NULLPTR;
  if (ldx < K || ldx % 8 != 0) return MXFP8_E_LD;
  if (!aligned(x_bf16, 16) || !aligned(offsets, 4) || !aligned(slot_of_row, 4)) return MXFP8_E_ALIGN;
  if (int st = check_out(y_bf16, N, ldy, nullptr)) return st;
  const size_t need = experts_ws(x_rows, R, N, K, E);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MXFP8_E_WORKSPACE;
  if (!aligned(workspace, 256)) return MXFP8_E_ALIGN;
  if (int st = mxfp8::check_device_current()) return st;
  mxfp8::ExpertsArgs a = {};
  a.x = x_bf16;
  a.x_rows = x_rows;
  a.ldx = ldx;
  a.R = R;
  a.K = K;
  a.N = N;
  a.E = E;
  a.slots = slot_of_row;
  a.topk = slot_of_row ? topk : 1;
  a.offsets = offsets;
  a.wp = w_packed;
  a.wsp = s_packed;
  a.y = y_bf16;
  a.ldy = ldy;
  const ExpertsForm f = experts_form(R, N, K, E);
  if (f.one == kDecode) return mxfp8::launch_experts_fp4_decode(a, (hipStream_t)stream);
  if (f.one == kFusedTiles) return mxfp8::launch_experts_fp4_fused(a, (hipStream_t)stream);
  uint8_t* q = (uint8_t*)workspace;
  uint8_t* s = q + experts_q_bytes(x_rows, K);
  if (int st = mxfp8::launch_quantize_rows_fp4(x_bf16, x_rows, K, ldx, q, s, (hipStream_t)stream)) return st;
  return mxfp8::launch_experts_fp4_tile(a, q, s, f.plan, (hipStream_t)stream);
}

}  // extern "C"
