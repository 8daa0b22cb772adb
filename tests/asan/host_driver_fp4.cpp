// Host-side check of the C ABI's MXFP4 x MXFP4 layer, tokens by expert and
// experts' products (api_fp4.cpp) under AddressSanitizer and UBSan: the host
// code built for the CPU, the kernel launchers replaced by stubs.  Each stub
// reads the first and last byte of every input and writes every byte its
// kernels write, outputs and workspace regions alike, with the extents the
// kernels use.  Buffers are allocated at exactly the sizes the library asks for.
// Prints "host driver ok" when every check passed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "launch_fp4.hpp"
#include "mxfp8.h"

namespace {
int g_fail = 0, g_launches = 0;
volatile uint8_t g_sink;
#define CHECK(cond)                                                          \
  do {                                                                       \
    if (!(cond)) {                                                           \
      std::fprintf(stderr, "check failed: %s (line %d)\n", #cond, __LINE__); \
      ++g_fail;                                                              \
    }                                                                        \
  } while (0)

constexpr uint8_t kCodes = 0x11, kScales = 0x12;
int64_t pad(int64_t n) { return (n + 127) / 128 * 128; }
void fill(void* p, size_t bytes, uint8_t v) {
  if (bytes) std::memset(p, v, bytes);
}
bool holds(const void* p, size_t bytes, uint8_t v) {
  const uint8_t* b = (const uint8_t*)p;
  return std::all_of(b, b + bytes, [v](uint8_t c) { return c == v; });
}
void write_rows(void* y, int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  for (int64_t r = 0; r < rows; ++r) std::memset((uint8_t*)y + (size_t)r * ld * elem, 0x5A, (size_t)cols * elem);
}
void read(const void* p, size_t bytes) {
  g_sink = ((const uint8_t*)p)[0];
  g_sink = ((const uint8_t*)p)[bytes - 1];
}
void read_rows(const void* x, int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  read(x, ((size_t)(rows - 1) * ld + cols) * elem);
}
void read_weight(const void* w, const void* s, int64_t N, int64_t K, int64_t E = 1) {
  read(w, (size_t)(E * pad(N) * (K / 2)));
  read(s, (size_t)(E * pad(N) * (K / 32)));
}
struct Exact {
  uint8_t* p;
  explicit Exact(size_t bytes) {
    void* q = nullptr;
    if (posix_memalign(&q, 256, bytes ? bytes : 1) != 0) std::abort();
    std::memset(q, 0, bytes);
    p = (uint8_t*)q;
  }
  ~Exact() { std::free(p); }
  Exact(const Exact&) = delete;
};
}  // namespace

namespace mxfp8 {
int check_device_current() { return 0; }
int64_t sort_blocks(int64_t R) {
  if (R <= 4096) return 1;
  const int64_t chunk = std::max<int64_t>(kSortChunk, (R + kSortMaxBlocks - 1) / kSortMaxBlocks);
  return (R + chunk - 1) / chunk;
}
int launch_quantize_packed_fp4(const void* x, int64_t M, int64_t K, int64_t ldx, void* qp, void* sp, hipStream_t) {
  ++g_launches;
  read_rows(x, M, K, ldx, 2);
  fill(qp, (size_t)(pad(M) * (K / 2)), kCodes);
  fill(sp, (size_t)(pad(M) * (K / 32)), kScales);
  return 0;
}
int launch_quantize_rows_fp4(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, void* s, hipStream_t) {
  ++g_launches;
  read_rows(x, M, K, ldx, 2);
  fill(q, (size_t)(M * (K / 2)), kCodes);
  fill(s, (size_t)(M * fp4_scale_pitch(K)), kScales);
  return 0;
}
int launch_pack_weight_fp4(const void* w, const void* ws, int64_t N, int64_t K, int64_t ldw, int64_t ldws, void* wp,
                           void* sp, hipStream_t) {
  ++g_launches;
  read_rows(w, N, K / 2, ldw, 1);
  read_rows(ws, N, K / 32, ldws, 1);
  fill(wp, (size_t)(pad(N) * (K / 2)), kCodes);
  fill(sp, (size_t)(pad(N) * (K / 32)), kScales);
  return 0;
}
namespace {
int packed(const void* q, const void* s, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
           const void* bias, void* y, int64_t ldy) {
  ++g_launches;
  CHECK(holds(q, (size_t)(pad(M) * (K / 2)), kCodes));
  CHECK(holds(s, (size_t)(pad(M) * (K / 32)), kScales));
  read_weight(wp, wsp, N, K);
  if (bias) read(bias, (size_t)N * 2);
  write_rows(y, M, N, ldy, 2);
  return 0;
}
int inside(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
           const void* bias, void* y, int64_t ldy) {
  ++g_launches;
  read_rows(x, M, K, ldx, 2);
  read_weight(wp, wsp, N, K);
  if (bias) read(bias, (size_t)N * 2);
  write_rows(y, M, N, ldy, 2);
  return 0;
}
int experts(const ExpertsArgs& a) {
  ++g_launches;
  if (a.slots) read(a.slots, (size_t)a.R * 4);
  read(a.offsets, (size_t)(a.E + 1) * 4);
  read_weight(a.wp, a.wsp, a.N, a.K, a.E);
  write_rows(a.y, a.R, a.N, a.ldy, 2);
  return 0;
}
}  // namespace
int launch_gemm_fp4_mid(const void* q, const void* s, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
                        const void* bias, void* y, int64_t ldy, hipStream_t) {
  CHECK(M <= kFp4MidMaxM);
  return packed(q, s, M, K, wp, wsp, N, bias, y, ldy);
}
int launch_gemm_fp4_tile(const void* q, const void* s, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
                         const void* bias, void* y, int64_t ldy, hipStream_t, Fp4Plan plan) {
  CHECK((plan.nt == 256 && plan.mt == 256) || (plan.nt == 128 && (plan.mt == 128 || plan.mt == 64)));
  return packed(q, s, M, K, wp, wsp, N, bias, y, ldy);
}
int launch_gemm_fp4_decode(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
                           const void* bias, void* y, int64_t ldy, hipStream_t) {
  CHECK(M <= fp4_decode_max_m(K));
  return inside(x, ldx, M, K, wp, wsp, N, bias, y, ldy);
}
int launch_gemm_fp4_fused(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
                          const void* bias, void* y, int64_t ldy, hipStream_t) {
  CHECK(K <= kFp4FusedMaxK);
  return inside(x, ldx, M, K, wp, wsp, N, bias, y, ldy);
}
int launch_experts_fp4_decode(const ExpertsArgs& a, hipStream_t) {
  CHECK(a.K <= kFp4DecodeMaxK);
  read_rows(a.x, a.x_rows, a.K, a.ldx, 2);
  return experts(a);
}
int launch_experts_fp4_fused(const ExpertsArgs& a, hipStream_t) {
  CHECK(a.K <= kFp4FusedMaxK);
  read_rows(a.x, a.x_rows, a.K, a.ldx, 2);
  return experts(a);
}
int launch_experts_fp4_tile(const ExpertsArgs& a, const void* q, const void* s, Fp4Plan plan, hipStream_t) {
  CHECK((plan.nt == 256 && plan.mt == 128) || (plan.nt == 128 && (plan.mt == 128 || plan.mt == 64)));
  CHECK(holds(q, (size_t)(a.x_rows * (a.K / 2)), kCodes));
  CHECK(holds(s, (size_t)(a.x_rows * fp4_scale_pitch(a.K)), kScales));
  return experts(a);
}
int launch_moe_sort(const SortArgs& a, hipStream_t) {
  ++g_launches;
  if (a.R > 0) read(a.ids, (size_t)a.R * (a.wide ? 8 : 4));
  fill(a.rows, (size_t)a.R * 4, 0);
  fill(a.slots, (size_t)a.R * 4, 0);
  fill(a.offsets, (size_t)(a.E + 1) * 4, 0);
  if (sort_blocks(a.R) > 1) fill(a.ws, (size_t)(sort_blocks(a.R) * (a.E + 1)) * 4, 1);
  return 0;
}
namespace {
int by_token(const PermuteArgs& a) {
  ++g_launches;
  const size_t elem = a.bf16 ? 2 : 4;
  const int64_t R = a.T * a.topk;
  read(a.rows, (size_t)R * 4);
  read(a.kept, 4);
  if (a.tokens) read_rows(a.tokens, a.T, a.H, a.ldt, elem);
  if (a.sorted) read_rows(a.sorted, R, a.H, a.lds, elem);
  if (a.weights) read(a.weights, (size_t)R * 4);
  if (a.out_tokens) write_rows(a.out_tokens, a.T, a.H, a.ldo, elem);
  if (a.out_sorted) write_rows(a.out_sorted, R, a.H, a.ldo, elem);
  if (a.dweights) fill(a.dweights, (size_t)R * 4, 0x33);
  return 0;
}
}  // namespace
int launch_moe_permute(const PermuteArgs& a, hipStream_t) { return by_token(a); }
int launch_moe_unpermute(const PermuteArgs& a, hipStream_t) { return by_token(a); }
int launch_moe_unpermute_backward(const PermuteArgs& a, hipStream_t) { return by_token(a); }
}  // namespace mxfp8

namespace {
const int kForms[] = {0, 1, 2, 16, 64, 128, 256};

void layer(int64_t M, int64_t N, int64_t K) {
  size_t wb = 0, sb = 0, qb = 0, qs = 0;
  CHECK(mxfp8_moe_prepared_experts_fp4_bytes(1, N, K, &wb, &sb) == 0);
  CHECK(mxfp8_packed_act_fp4_bytes(M, K, &qb, &qs) == 0);
  const int64_t ldx = K + 8, ldy = N + 3;
  Exact x((size_t)((M - 1) * ldx + K) * 2), w((size_t)N * (K / 2)), s((size_t)N * (K / 32)), wp(wb), sp(sb), q(qb),
      qsc(qs), y((size_t)((M - 1) * ldy + N) * 2), bias((size_t)N * 2);
  CHECK(mxfp8_moe_prepare_experts_fp4(w.p, s.p, 1, N, K, wp.p, sp.p, nullptr) == 0);
  CHECK(mxfp8_quantize_act_packed_fp4(x.p, M, K, ldx, q.p, qsc.p, nullptr) == 0);
  for (int form : kForms) {
    CHECK(mxfp8_debug_force_w4a4(form) >= 0);
    CHECK(mxfp8_gemm_packed_fp4(q.p, qsc.p, M, K, wp.p, sp.p, N, bias.p, y.p, ldy, nullptr) == 0);
    size_t need = 0;
    CHECK(mxfp8_linear_w4a4_workspace_bytes(M, N, K, &need) == 0);
    Exact ws(need);
    CHECK(mxfp8_linear_w4a4(x.p, M, K, ldx, wp.p, sp.p, N, nullptr, y.p, ldy, need ? ws.p : nullptr, need, nullptr) == 0);
    if (need)
      CHECK(mxfp8_linear_w4a4(x.p, M, K, ldx, wp.p, sp.p, N, nullptr, y.p, ldy, ws.p, need - 1, nullptr) ==
            MXFP8_E_WORKSPACE);
  }
  mxfp8_debug_force_w4a4(0);
}

void moe(int64_t T, int64_t topk, int64_t E, int64_t N, int64_t K, int dtype) {
  const int64_t R = T * topk, elem = dtype == MXFP8_BF16 ? 2 : 4;
  size_t need = 0, wb = 0, sb = 0;
  CHECK(mxfp8_moe_sort_workspace_bytes(R, E, &need) == 0);
  Exact ids((size_t)R * 8), rows((size_t)R * 4), slots((size_t)R * 4), offsets((size_t)(E + 1) * 4), sort_ws(need);
  for (int id_bytes : {4, 8})
    CHECK(mxfp8_moe_sort(ids.p, id_bytes, R, E, (int32_t*)rows.p, (int32_t*)slots.p, (int32_t*)offsets.p,
                         need ? sort_ws.p : nullptr, need, nullptr) == 0);
  const int32_t* kept = (const int32_t*)offsets.p + E;
  const int64_t H = N, ld = H + 1;
  Exact x((size_t)((T - 1) * ld + H) * elem), xs((size_t)((R - 1) * ld + H) * elem), y((size_t)((T - 1) * ld + H) * elem),
      dys((size_t)((R - 1) * ld + H) * elem), weights((size_t)R * 4), dw((size_t)R * 4);
  CHECK(mxfp8_moe_permute(x.p, dtype, T, H, ld, topk, (int32_t*)rows.p, kept, xs.p, ld, nullptr) == 0);
  CHECK(mxfp8_moe_unpermute(xs.p, dtype, T, H, ld, topk, (int32_t*)rows.p, kept, (float*)weights.p, y.p, ld, nullptr) == 0);
  CHECK(mxfp8_moe_unpermute(xs.p, dtype, T, H, ld, topk, (int32_t*)rows.p, kept, nullptr, y.p, ld, nullptr) == 0);
  CHECK(mxfp8_moe_unpermute_backward(y.p, dtype, T, H, ld, topk, (int32_t*)rows.p, kept, xs.p, ld, (float*)weights.p,
                                     dys.p, ld, (float*)dw.p, nullptr) == 0);
  CHECK(mxfp8_moe_unpermute_backward(y.p, dtype, T, H, ld, topk, (int32_t*)rows.p, kept, nullptr, 0, nullptr, dys.p, ld,
                                     nullptr, nullptr) == 0);
  CHECK(mxfp8_moe_prepared_experts_fp4_bytes(E, N, K, &wb, &sb) == 0);
  Exact w((size_t)(E * N * (K / 2))), s((size_t)(E * N * (K / 32))), wp(wb), sp(sb);
  CHECK(mxfp8_moe_prepare_experts_fp4(w.p, s.p, E, N, K, wp.p, sp.p, nullptr) == 0);
  CHECK(holds(wp.p, wb, kCodes) && holds(sp.p, sb, kScales));   // every expert has been laid out
  for (bool gather : {true, false})
    for (int form : kForms) {
      CHECK(mxfp8_debug_force_w4a4(form) >= 0);
      const int64_t x_rows = gather ? T : R, ldx = K + 8, ldy = N + 5;
      Exact xe((size_t)((x_rows - 1) * ldx + K) * 2), ye((size_t)((R - 1) * ldy + N) * 2);
      CHECK(mxfp8_moe_linear_w4a4_workspace_bytes(x_rows, R, N, K, E, &need) == 0);
      Exact ws(need);
      CHECK(mxfp8_moe_linear_w4a4(xe.p, x_rows, K, ldx, gather ? (int32_t*)slots.p : nullptr, topk, (int32_t*)offsets.p, R,
                                  E, wp.p, sp.p, N, ye.p, ldy, need ? ws.p : nullptr, need, nullptr) == 0);
    }
  mxfp8_debug_force_w4a4(0);
}
}  // namespace

int main() {
  for (int64_t M : {1, 16, 17, 33, 128, 129, 700})
    for (int64_t N : {1, 130, 1000})
      for (int64_t K : {256, 768, 2048, 4352, 8448}) layer(M, N, K);
  for (int dtype : {MXFP8_F32, MXFP8_BF16}) {
    moe(1, 1, 1, 1, 256, dtype);
    moe(3, 8, 16, 130, 512, dtype);
    moe(700, 8, 5, 256, 2304, dtype);
    moe(40, 2, 256, 40, 8448, dtype);
  }
  // The size rules over their whole range: no overflow in the host's arithmetic.
  for (int64_t a : {(int64_t)1, (int64_t)1000, (int64_t)1 << 20, (int64_t)1 << 24, (int64_t)1 << 30, INT64_MAX})
    for (int64_t b : {(int64_t)1, (int64_t)4096, (int64_t)1 << 24, INT64_MAX})
      for (int64_t k : {(int64_t)256, (int64_t)8192, (int64_t)1 << 24, INT64_MAX}) {
        size_t n = 0, m = 0;
        (void)mxfp8_linear_w4a4_workspace_bytes(a, b, k, &n);
        (void)mxfp8_packed_act_fp4_bytes(a, k, &n, &m);
        (void)mxfp8_moe_prepared_experts_fp4_bytes(256, b, k, &n, &m);
        (void)mxfp8_moe_linear_w4a4_workspace_bytes(a, a, b, k, 256, &n);
        (void)mxfp8_moe_sort_workspace_bytes(a, 256, &n);
      }
  CHECK(g_launches > 1000);
  if (g_fail == 0) std::printf("host driver ok\n");
  return g_fail != 0;
}
