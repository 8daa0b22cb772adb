// Internal launchers of the 128-block FP8 layer, the weight gradient from
// 8-bit activation checkpoints and the router's balance loss.  As in
// launch.hpp, arguments were validated by the C entry points (api_b128.cpp),
// and each returns 0 or -7 (launch error).
#pragma once

#include "launch.hpp"

namespace mxfp8 {

constexpr int64_t kB128 = 128;   // elements of a scale block along each blocked axis
__host__ __device__ inline int64_t b128_blocks(int64_t n) { return (n + kB128 - 1) / kB128; }

// x bf16 [M, K] (K % 16 == 0) -> E4M3 [M, K] + UE8M0 [M, ceil(K / 128)].
int launch_quantize_b128(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, int64_t ldq, void* s, int64_t lds,
                         hipStream_t stream);
// The same in the packed operand layout (rows padded to 128, K to 128).
int launch_quantize_packed_b128(const void* x, int64_t M, int64_t K, int64_t ldx, void* qp, void* sp,
                                hipStream_t stream);
// Packed activations (either scale block) -> bf16 [M, K].
int launch_dequantize_packed(const void* qp, const void* sp, int64_t M, int64_t K, void* x, int64_t ldx,
                             hipStream_t stream);
// E4M3 [N, K] + fp32 [ceil(N / 128), ceil(K / 128)] -> the packed weight (of
// its transpose if `transpose`) and its scales, one per (128-row group, block).
int launch_pack_b128(const void* w, const void* ws, int64_t N, int64_t K, int64_t ldw, int64_t ldws, int transpose,
                     void* wp, void* sp, hipStream_t stream);
// bf16 weight [N, K] -> any of row-major (q, s), packed (wp, sp) and packed
// transposed (wtp, stp); null outputs are skipped.  mx: bit 0 / 1: sp / stp in
// the MX format's scale tiles (N_pad K_pad / 32 bytes), for launch_gemm_tile.
int launch_quantize_weight_b128(const void* w, int64_t N, int64_t K, int64_t ldw, void* q, int64_t ldq, void* s,
                                int64_t lds, void* wp, void* sp, void* wtp, void* stp, int mx, hipStream_t stream);

// Decode GEMM: M <= 32 bf16 rows, quantized inside, against the packed weight.
constexpr int64_t kB128DecodeMaxM = 32;
int launch_gemm_b128_decode(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const float* wsc,
                            int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream);

// Tile GEMM on packed activations.  splits > 1 cuts K into that many runs of
// 128-blocks, whose fp32 partials go to `part` (splits * M * round_up(N, 4)
// floats) and are added in order by launch_splitk_reduce.
struct B128Plan {
  int mt;       // 64 or 128: activation rows of a 128-column tile; 256: large tiles; 512: wide tiles
  int splits;
};
int launch_gemm_b128_tile(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const float* wsc,
                          int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream, B128Plan plan,
                          void* part);

// Weight gradient dW[n, k] = sum_m dY[m, n] X[m, k] from packed 8-bit
// activations (either scale block), and db[n] = sum_m dY[m, n].
// The (tile, 64-token step) units, tile by tile, are cut into one run of
// consecutive units per workgroup, at multiples of `granule` units (one unit,
// or a tile's steps where no tile is shared).
struct Runs {
  int64_t granules;
  int granule;
  int count;
  __host__ __device__ int64_t start(int64_t w) const { return granules * w / count * granule; }
  __host__ __device__ int of(int64_t unit) const { return (int)(((unit / granule + 1) * count - 1) / granules); }
};
struct WgradPlan {
  int tile;          // edge of a dW tile: 128 or 256
  Runs runs;
  int64_t tiles_n, tiles_k;
  int64_t steps;     // 64-token steps, at least one
  int64_t pieces;    // most runs that share a tile (1: none is shared)
  int64_t tiles() const { return tiles_n * tiles_k; }
  bool shared() const { return pieces > 1; }
  // Whole small tiles: those with k = 0 add up all of db, which needs no parts
  // and no second launch (their steps have MFMAs to spare, the large form's do not).
  bool db_direct() const { return tile == 128 && !shared(); }
};
constexpr int kWgStep = 64;   // tokens per step
struct WgradArgs {
  const void* dy;       // bf16 [M, N], row stride lddy
  int64_t M, N, lddy;
  const void* qp;       // packed activations [M, K] and their scales
  const void* sp;
  int64_t K;
  void* dw;             // [N, K], row stride lddw: fp32, or bf16 if out_bf16
  int64_t lddw;
  int out_bf16;
  int accumulate;       // dw += and db += (dw fp32)
  void* db;             // [N] or null: fp32, or bf16 if db_bf16
  int db_bf16;
  float* part_dw;
  float* part_db;
};
int launch_wgrad(const WgradArgs& a, WgradPlan p, hipStream_t stream);
// Its small-tile kernel (wgrad_small.hip), without the join.
int launch_wgrad_small(const WgradArgs& a, const WgradPlan& p, hipStream_t stream);

// Load-balance and z loss of a router (balance.hip).
struct BalanceArgs {
  const void* logits;      // [T, E] fp32 or bf16, row stride ldl
  int bf16;
  int64_t T, E, ldl, topk;
  const uint8_t* valid;    // [T] or null
  float coef, z_coef;
  int* counts;             // [E]
  int* used;               // [1]
  float* loss;             // [1] (forward)
  const float* grad_loss;  // [1] or null (= 1)
  void* dlogits;           // [T, E], type of logits, row stride ldd (backward)
  int64_t ldd;
  void* ws;                // forward partials
};
constexpr int kBalMaxBlocks = 512;   // forward workgroups, each with partials in the workspace
constexpr int kBalTokens = 32;       // tokens a forward workgroup works on at a time
// [16] doubles, then per forward workgroup sums and counts of the experts, z
// and n, then the arrival count; nothing where there is one forward workgroup.
inline size_t balance_ws_bytes(int64_t T, int64_t E) {
  return T <= kBalTokens ? 0 : 16 * 8 + (size_t)kBalMaxBlocks * ((size_t)E * 8 + 8) + 8;
}
int launch_balance(const BalanceArgs& a, hipStream_t stream);
int launch_balance_backward(const BalanceArgs& a, hipStream_t stream);

}  // namespace mxfp8
