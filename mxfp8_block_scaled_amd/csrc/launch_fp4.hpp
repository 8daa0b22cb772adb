// Internal launchers of the MXFP4 x MXFP4 linear layer, of tokens sorted by
// expert and back, and of the experts' MXFP4 products.  As in launch.hpp,
// arguments were validated by the C entry points (api_fp4.cpp), and each
// returns 0 or -7 (launch error).
#pragma once

#include "launch.hpp"

namespace mxfp8 {

constexpr int64_t kFp4Step = 128;   // elements of one 4-bit K step (64 bytes of a row)

// x bf16 [M, K] -> the packed 4-bit operand (the layout of
// launch_pack_weight_fp4 with M in place of N; pad rows zero).
int launch_quantize_packed_fp4(const void* x, int64_t M, int64_t K, int64_t ldx, void* qp, void* sp,
                               hipStream_t stream);
// The same as row-major bytes: q [M, K / 2], s [M, K / 32] with rows of whole 16
// bytes (fp4_scale_pitch apart).
inline int64_t fp4_scale_pitch(int64_t K) { return (K / 32 + 15) / 16 * 16; }
int launch_quantize_rows_fp4(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, void* s, hipStream_t stream);

// Decode GEMM: M <= 16 bf16 rows (32 where K <= 4096), quantized inside,
// against a packed MXFP4 weight; K <= kFp4DecodeMaxK.
constexpr int64_t kFp4DecodeMaxK = 8192;
inline int64_t fp4_decode_max_m(int64_t K) { return K <= 4096 ? 32 : K <= kFp4DecodeMaxK ? 16 : 0; }
// Its workgroups of 16 weight rows each that a compute unit holds.  Where those
// are not enough, each takes a run of blocks.  (The experts': of their number at
// most, not all of which have rows.)
inline int64_t fp4_decode_per_cu(bool experts, int64_t M, int64_t K) {
  return M > 16 || K > 2048 ? 1 : K > 1024 ? (experts ? 4 : 3) : (experts ? 8 : 7);
}
int launch_gemm_fp4_decode(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const void* wsp,
                           int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream);

// The same on packed activations (one 128-row group), M <= kFp4MidMaxM.
constexpr int64_t kFp4MidMaxM = 128;
int launch_gemm_fp4_mid(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const void* wsp,
                        int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream);

// Tile GEMM of two packed MXFP4 operands.
struct Fp4Plan {
  int nt, mt;   // weight and activation rows of a workgroup's tile: 256 x 256, 128 x 128 or 128 x 64
};
int launch_gemm_fp4_tile(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const void* wsp,
                         int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream, Fp4Plan plan);

// The 128 x 64 tiles with the rows quantized by each workgroup: one launch, no
// workspace; K <= kFp4FusedMaxK.
constexpr int64_t kFp4FusedMaxK = 2048;
int launch_gemm_fp4_fused(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
                          const void* bias, void* y, int64_t ldy, hipStream_t stream);

// Rows by expert (moe_order.hip).  R = T topk slots; `rows` [R]: the sorted
// row of each slot, `slots` [R]: its inverse, `offsets` [E + 1]: the first row
// of each expert and the number of rows that have one (kept = offsets + E).
struct SortArgs {
  const void* ids;   // [R] int32, or int64 if wide
  int wide;
  int64_t R, E;
  int* rows;
  int* slots;
  int* offsets;
  int* ws;
};
constexpr int kSortChunk = 1024;       // least slots of a workgroup
constexpr int kSortMaxBlocks = 256;
int64_t sort_blocks(int64_t R);
inline size_t sort_ws_bytes(int64_t R, int64_t E) {
  const int64_t n = sort_blocks(R);
  return n <= 1 ? 0 : (size_t)n * (size_t)(E + 1) * 4;
}
int launch_moe_sort(const SortArgs& a, hipStream_t stream);

struct PermuteArgs {
  int bf16;                // element type of the matrices: bf16, or fp32
  int64_t T, H, topk;
  const int* rows;         // [T, topk]
  const int* kept;         // [1]
  const void* tokens;      // [T, H], row stride ldt: x (permute), dy (unpermute's gradient)
  int64_t ldt;
  const void* sorted;      // [T topk, H], row stride lds: ys
  int64_t lds;
  const float* weights;    // [T, topk] or null (all 1)
  void* out_tokens;        // [T, H], row stride ldo: y, dx
  void* out_sorted;        // [T topk, H], row stride ldo: xs, dys
  int64_t ldo;
  float* dweights;         // [T, topk] or null
};
int launch_moe_permute(const PermuteArgs& a, hipStream_t stream);             // out_sorted = tokens by row
int launch_moe_unpermute(const PermuteArgs& a, hipStream_t stream);           // out_tokens = weighted sums of sorted
int launch_moe_unpermute_backward(const PermuteArgs& a, hipStream_t stream);  // out_sorted, dweights

// The experts' products on sorted rows: y[r] = deq(q(x[r])) deq(W[e(r)])^T.
struct ExpertsArgs {
  const void* x;           // bf16 [rows, K], row stride ldx
  int64_t x_rows, ldx;
  int64_t R, K, N, E;
  const int* slots;        // [R]: row r reads x row slots[r] / topk; null: x row r
  int64_t topk;
  const int* offsets;      // [E + 1]
  const void* wp;          // packed weights, experts one after the other
  const void* wsp;
  void* y;                 // bf16 [R, N], row stride ldy
  int64_t ldy;
};
// Decode form: quantizes inside, no workspace.
int launch_experts_fp4_decode(const ExpertsArgs& a, hipStream_t stream);
// As launch_gemm_fp4_fused.
int launch_experts_fp4_fused(const ExpertsArgs& a, hipStream_t stream);
// Tile form on rows of launch_quantize_rows_fp4.
int launch_experts_fp4_tile(const ExpertsArgs& a, const void* q, const void* s, Fp4Plan plan, hipStream_t stream);

}  // namespace mxfp8
