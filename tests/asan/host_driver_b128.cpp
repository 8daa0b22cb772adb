// Host-side check of the C ABI's 128-block FP8 layer, weight gradient and
// balance loss (api_b128.cpp) under AddressSanitizer and UBSan: the host code
// built for the CPU, the kernel launchers replaced by stubs.  Each stub reads
// the first and last byte of every input and writes every byte its kernels
// write, outputs and workspace regions alike, with the extents the kernels
// use.  Buffers are allocated at exactly the sizes the library asks for, so a
// workspace carved too small, regions in the wrong place or an extent computed
// wrong is an ASan report; a region that overlaps another loses its mark,
// which the stubs check.  Prints "host driver ok" when every check passed.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "launch_b128.hpp"
#include "mxfp8.h"

namespace {
int g_fail = 0, g_launches = 0, g_mx = 0;
volatile uint8_t g_sink;
#define CHECK(cond)                                                          \
  do {                                                                       \
    if (!(cond)) {                                                           \
      std::fprintf(stderr, "check failed: %s (line %d)\n", #cond, __LINE__); \
      ++g_fail;                                                              \
    }                                                                        \
  } while (0)

constexpr uint8_t kAct = 0x11, kActScale = 0x12, kWeight = 0x21, kWeightScale = 0x22, kWeightT = 0x31,
                  kWeightTScale = 0x32, kPart = 0x41;

void fill(void* p, size_t bytes, uint8_t v) {
  if (bytes) std::memset(p, v, bytes);   // ASan checks every byte
}
bool holds(const void* p, size_t bytes, uint8_t v) {
  const uint8_t* b = (const uint8_t*)p;
  return std::all_of(b, b + bytes, [v](uint8_t c) { return c == v; });
}
void fill_rows(void* y, int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  for (int64_t r = 0; r < rows; ++r) std::memset((uint8_t*)y + (size_t)r * ld * elem, 0x5A, (size_t)cols * elem);
}
void read_rows(const void* x, int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  if (rows == 0) return;
  const uint8_t* b = (const uint8_t*)x;
  g_sink = b[0];
  g_sink = b[((size_t)(rows - 1) * ld + cols) * elem - 1];
}
size_t pad(int64_t n) { return (size_t)mxfp8::b128_blocks(n) * 128; }
size_t packed(int64_t r, int64_t k) { return pad(r) * pad(k); }
size_t wscales(int64_t n, int64_t k) { return (size_t)mxfp8::b128_blocks(n) * mxfp8::b128_blocks(k) * 4; }

uint8_t* alloc_exact(size_t bytes) {
  void* p = nullptr;
  if (posix_memalign(&p, 256, bytes ? bytes : 1) != 0) std::abort();
  std::memset(p, 0, bytes);
  return (uint8_t*)p;
}
struct Buffers {
  std::vector<uint8_t*> all;
  uint8_t* operator()(size_t bytes) {
    all.push_back(alloc_exact(bytes));
    return all.back();
  }
  ~Buffers() {
    for (uint8_t* p : all) std::free(p);
  }
};
}  // namespace

// ---------------------------------------------------------------- launch stubs
namespace mxfp8 {
int check_device_current() { return 0; }

int launch_quantize_b128(const void* x, int64_t M, int64_t K, int64_t ldx, void* q, int64_t ldq, void* s, int64_t lds,
                         hipStream_t) {
  ++g_launches;
  read_rows(x, M, K, ldx, 2);
  fill_rows(q, M, K, ldq, 1);
  fill_rows(s, M, b128_blocks(K), lds, 1);
  return 0;
}
int launch_quantize_packed_b128(const void* x, int64_t M, int64_t K, int64_t ldx, void* qp, void* sp, hipStream_t) {
  ++g_launches;
  read_rows(x, M, K, ldx, 2);
  fill(qp, packed(M, K), kAct);
  fill(sp, packed(M, K) / 32, kActScale);
  return 0;
}
int launch_dequantize_packed(const void* qp, const void* sp, int64_t M, int64_t K, void* x, int64_t ldx,
                             hipStream_t) {
  ++g_launches;
  CHECK(holds(qp, packed(M, K), kAct) && holds(sp, packed(M, K) / 32, kActScale));
  fill_rows(x, M, K, ldx, 2);
  return 0;
}
int launch_pack_b128(const void* w, const void* ws, int64_t N, int64_t K, int64_t ldw, int64_t ldws, int transpose,
                     void* wp, void* sp, hipStream_t) {
  ++g_launches;
  read_rows(w, N, K, ldw, 1);
  read_rows(ws, b128_blocks(N), b128_blocks(K), ldws, 4);
  fill(wp, packed(N, K), transpose ? kWeightT : kWeight);
  fill(sp, wscales(N, K), transpose ? kWeightTScale : kWeightScale);
  return 0;
}
int launch_quantize_weight_b128(const void* w, int64_t N, int64_t K, int64_t ldw, void* q, int64_t ldq, void* s,
                                int64_t lds, void* wp, void* sp, void* wtp, void* stp, int mx, hipStream_t) {
  ++g_launches;
  read_rows(w, N, K, ldw, 2);
  if (q) {
    fill_rows(q, N, K, ldq, 1);
    fill_rows(s, b128_blocks(N), b128_blocks(K), lds, 4);
  }
  if (wp) {
    fill(wp, packed(N, K), kWeight);
    fill(sp, mx & 1 ? packed(N, K) / 32 : wscales(N, K), kWeightScale);
  }
  if (wtp) {
    fill(wtp, packed(N, K), kWeightT);
    fill(stp, mx & 2 ? packed(N, K) / 32 : wscales(N, K), kWeightTScale);
  }
  return 0;
}
namespace {
bool weight_ok(const void* wp, const void* sc, int64_t N, int64_t K) {
  const size_t b = packed(N, K), s = wscales(N, K);
  return (holds(wp, b, kWeight) && holds(sc, s, kWeightScale)) ||
         (holds(wp, b, kWeightT) && holds(sc, s, kWeightTScale));
}
}  // namespace
int launch_gemm_b128_decode(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const float* wsc,
                            int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t) {
  ++g_launches;
  CHECK(M >= 1 && M <= kB128DecodeMaxM);
  CHECK(weight_ok(wp, wsc, N, K));
  read_rows(x, M, K, ldx, 2);
  if (bias) read_rows(bias, 1, N, N, 2);
  fill_rows(y, M, N, ldy, 2);
  return 0;
}
int launch_gemm_b128_tile(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const float* wsc,
                          int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t, B128Plan plan, void* part) {
  ++g_launches;
  CHECK(plan.mt == 64 || plan.mt == 128 || plan.mt == 256 || plan.mt == 512);
  CHECK(plan.splits >= 1 && plan.splits <= kMaxSplitK && (plan.mt <= 128 || plan.splits == 1));
  CHECK(plan.mt == 64 || N % 8 == 0);
  if (plan.splits > 1) fill(part, (size_t)plan.splits * M * ((N + 3) / 4 * 4) * 4, kPart);
  CHECK(holds(qp, packed(M, K), kAct) && holds(sp, packed(M, K) / 32, kActScale));
  CHECK(weight_ok(wp, wsc, N, K));
  if (bias) read_rows(bias, 1, N, N, 2);
  fill_rows(y, M, N, ldy, 2);
  return 0;
}
int launch_gemm_tile(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
                     const void* bias, void* y, int64_t ldy, hipStream_t, int splits, void*) {
  ++g_launches;
  ++g_mx;
  CHECK(K % 256 == 0 && splits == 1);
  const size_t w = packed(N, K);
  CHECK(holds(qp, packed(M, K), kAct) && holds(sp, packed(M, K) / 32, kActScale));
  CHECK((holds(wp, w, kWeight) && holds(wsp, w / 32, kWeightScale)) ||
        (holds(wp, w, kWeightT) && holds(wsp, w / 32, kWeightTScale)));
  if (bias) read_rows(bias, 1, N, N, 2);
  fill_rows(y, M, N, ldy, 2);
  return 0;
}
int launch_wgrad(const WgradArgs& a, WgradPlan p, hipStream_t) {
  ++g_launches;
  const int64_t T = p.tile;
  CHECK(T == 128 || T == 256);
  CHECK(p.tiles_n == (a.N + T - 1) / T && p.tiles_k == (a.K + T - 1) / T);
  CHECK(p.steps == std::max<int64_t>(1, (a.M + 63) / 64) && (a.M > 0 || T == 128));
  read_rows(a.dy, a.M, a.N, a.lddy, 2);
  if (a.M > 0) CHECK(holds(a.qp, packed(a.M, a.K), kAct) && holds(a.sp, packed(a.M, a.K) / 32, kActScale));
  // Runs in order: they cover every unit once, each tile's pieces fit the
  // count, and a run leaves partials of its first and its last tile at most.
  const int64_t U = p.tiles() * p.steps;
  const size_t slot_floats = (size_t)T * T;
  size_t dw_part = 0;
  std::vector<int64_t> pieces((size_t)p.tiles(), 0);
  CHECK(p.runs.count >= 1 && p.runs.count <= 256 && p.runs.start(0) == 0 && p.runs.start(p.runs.count) == U);
  for (int64_t w = 0; w < p.runs.count; ++w) {
    const int64_t u0 = p.runs.start(w), u1 = p.runs.start(w + 1);
    CHECK(u1 > u0);
    for (int64_t u = u0; u < u1;) {
      const int64_t t = u / p.steps, end = std::min(u1, (t + 1) * p.steps);
      const bool whole = u == t * p.steps && end == (t + 1) * p.steps;
      CHECK(p.shared() || whole);
      CHECK(whole || u == u0 || end == u1);
      CHECK(p.runs.of(u) == w && p.runs.of(end - 1) == w);
      CHECK(w - p.runs.of(t * p.steps) == pieces[(size_t)t]);
      if (!whole) {
        const size_t slot = (size_t)w * 2 + (u == u0 ? 0 : 1);
        fill(a.part_dw + slot * slot_floats, slot_floats * 4, kPart);
        dw_part = std::max(dw_part, (slot + 1) * slot_floats * 4);
      }
      ++pieces[(size_t)t];
      u = end;
    }
  }
  CHECK(*std::max_element(pieces.begin(), pieces.end()) <= p.pieces);
  CHECK((uint8_t*)a.part_dw + dw_part <= (uint8_t*)a.part_db);
  if (a.db && !p.db_direct()) fill(a.part_db, (size_t)(p.tiles() * p.pieces * T) * 4, kPart + 1);
  fill_rows(a.dw, a.N, a.K, a.lddw, a.out_bf16 ? 2 : 4);
  if (a.db) fill(a.db, (size_t)a.N * (a.db_bf16 ? 2 : 4), 0x5A);
  return 0;
}
int launch_balance(const BalanceArgs& a, hipStream_t) {
  ++g_launches;
  read_rows(a.logits, a.T, a.E, a.ldl, a.bf16 ? 2 : 4);
  if (a.valid) read_rows(a.valid, a.T, 1, 1, 1);
  // the totals, the most partials, the arrival count
  if (a.T > kBalTokens) fill(a.ws, 16 * 8 + (size_t)kBalMaxBlocks * (a.E * 8 + 8) + 4, kPart);
  fill(a.counts, (size_t)a.E * 4, 0x5A);
  fill(a.used, 4, 0x5A);
  fill(a.loss, 4, 0x5A);
  return 0;
}
int launch_balance_backward(const BalanceArgs& a, hipStream_t) {
  ++g_launches;
  read_rows(a.logits, a.T, a.E, a.ldl, a.bf16 ? 2 : 4);
  if (a.valid) read_rows(a.valid, a.T, 1, 1, 1);
  read_rows(a.counts, 1, a.E, a.E, 4);
  read_rows(a.used, 1, 1, 1, 4);
  if (a.grad_loss) read_rows(a.grad_loss, 1, 1, 1, 4);
  fill_rows(a.dlogits, a.T, a.E, a.ldd, a.bf16 ? 2 : 4);
  return 0;
}
}  // namespace mxfp8

// ---------------------------------------------------------------- driver
namespace {
size_t rows_bytes(int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  return rows ? ((size_t)(rows - 1) * ld + cols) * elem : 0;
}

void linear_case(int64_t M, int64_t N, int64_t K, int64_t extra) {
  Buffers buf;
  const int64_t ldx = K + extra, ldy = N + extra;
  uint8_t *x = buf(rows_bytes(M, K, ldx, 2)), *y = buf(rows_bytes(M, N, ldy, 2)), *bias = buf((size_t)N * 2);
  uint8_t *w = buf((size_t)N * K), *wsc = buf(wscales(N, K));
  size_t wb = 0, sb = 0, ws = 0;
  CHECK(mxfp8_prepared_weight_b128_bytes(N, K, &wb, &sb) == 0);
  uint8_t *wp = buf(wb), *sp = buf(sb);
  CHECK(mxfp8_prepare_weight_b128(w, (float*)wsc, N, K, K, mxfp8::b128_blocks(K), 0, wp, sp, nullptr) == 0);
  CHECK(mxfp8_linear_b128_workspace_bytes(M, N, K, &ws) == 0);
  uint8_t* work = buf(ws);
  CHECK(mxfp8_linear_b128(x, M, K, ldx, wp, sp, N, bias, y, ldy, ws ? work : nullptr, ws, nullptr) == 0);
  if (ws) {
    const int before = g_launches;
    CHECK(mxfp8_linear_b128(x, M, K, ldx, wp, sp, N, bias, y, ldy, work, ws - 1, nullptr) == MXFP8_E_WORKSPACE);
    CHECK(g_launches == before);
  }
  if (M == 0) return;
  size_t qb = 0, qs = 0, gs = 0;
  CHECK(mxfp8_packed_act_b128_bytes(M, K, &qb, &qs) == 0);
  uint8_t *q = buf(qb), *s = buf(qs);
  CHECK(mxfp8_quantize_act_packed_b128(x, M, K, ldx, q, s, nullptr) == 0);
  CHECK(mxfp8_gemm_packed_b128_workspace_bytes(M, N, K, &gs) == 0);
  uint8_t* g = buf(gs);
  CHECK(mxfp8_gemm_packed_b128(q, s, M, K, wp, sp, N, nullptr, y, ldy, g, gs, nullptr) == 0);
  CHECK(mxfp8_gemm_packed_b128(q, s, M, K, wp, sp, N, nullptr, y, ldy, g, gs - 1, nullptr) == MXFP8_E_WORKSPACE);
  CHECK(mxfp8_dequantize_act_packed(q, s, M, K, x, ldx, nullptr) == (ldx % 8 ? MXFP8_E_LD : 0));
}

void wgrad_case(int64_t M, int64_t N, int64_t K, int dtype, bool bias) {
  Buffers buf;
  const int64_t lddy = N + 8, lddw = K + 8;
  uint8_t* dy = buf(rows_bytes(M, N, lddy, 2));
  uint8_t *q = buf(packed(M, K)), *s = buf(packed(M, K) / 32);
  fill(q, packed(M, K), kAct);
  fill(s, packed(M, K) / 32, kActScale);
  const size_t elem = dtype == MXFP8_F32 ? 4 : 2;
  uint8_t* dw = buf(rows_bytes(N, K, lddw, elem));
  uint8_t* db = bias ? buf((size_t)N * elem) : nullptr;
  size_t ws = 0;
  CHECK(mxfp8_linear_wgrad_workspace_bytes(M, N, K, &ws) == 0);
  uint8_t* work = buf(ws);
  const int acc = dtype == MXFP8_F32;
  CHECK(mxfp8_linear_wgrad(dy, M, N, lddy, q, s, K, dw, dtype, lddw, db, dtype, acc, work, ws, nullptr) == 0);
  if (ws)
    CHECK(mxfp8_linear_wgrad(dy, M, N, lddy, q, s, K, dw, dtype, lddw, db, dtype, acc, work, ws - 1, nullptr) ==
          MXFP8_E_WORKSPACE);
}

void layer_case(int64_t M, int64_t N, int64_t K, int keep, int dtype) {
  Buffers buf;
  uint8_t *x = buf((size_t)M * K * 2), *w = buf((size_t)N * K * 2), *y = buf((size_t)M * N * 2);
  uint8_t *dy = buf((size_t)M * N * 2), *dx = buf((size_t)M * K * 2);
  const size_t elem = dtype == MXFP8_F32 ? 4 : 2;
  uint8_t *dw = buf((size_t)N * K * elem), *db = buf((size_t)N * elem), *bias = buf((size_t)N * 2);
  size_t kept = 0, fws = 0, bws = 0;
  CHECK(mxfp8_linear_b128_layer_bytes(M, N, K, keep, &kept, &fws, &bws) == 0);
  uint8_t *k = buf(kept), *f = buf(fws), *b = buf(bws);
  CHECK(mxfp8_linear_b128_forward(x, M, K, K, w, N, K, bias, y, N, keep, k, f, fws, nullptr) == 0);
  CHECK(mxfp8_linear_b128_forward(x, M, K, K, w, N, K, bias, y, N, keep, k, f, fws - 1, nullptr) ==
        MXFP8_E_WORKSPACE);
  const bool want_dx = keep & MXFP8_KEEP_DX, want_dw = keep & MXFP8_KEEP_DW;
  CHECK(mxfp8_linear_b128_backward(dy, M, N, N, K, keep, k, want_dx ? dx : nullptr, K, want_dw ? dw : nullptr, dtype,
                                   K, want_dw ? db : nullptr, dtype, b, bws, nullptr) == 0);
  // a gradient that nothing was kept for is refused
  if (!want_dx) CHECK(mxfp8_linear_b128_backward(dy, M, N, N, K, keep, k, dx, K, nullptr, dtype, K, nullptr, dtype, b,
                                                 bws, nullptr) == MXFP8_E_SHAPE);
  if (!want_dw) CHECK(mxfp8_linear_b128_backward(dy, M, N, N, K, keep, k, nullptr, K, dw, dtype, K, nullptr, dtype, b,
                                                 bws, nullptr) == MXFP8_E_SHAPE);
}

void balance_case(int64_t T, int64_t E, int64_t topk, int dtype, bool masked) {
  Buffers buf;
  const int64_t ldl = E + 3;
  const size_t elem = dtype == MXFP8_F32 ? 4 : 2;
  uint8_t *l = buf(rows_bytes(T, E, ldl, elem)), *d = buf(rows_bytes(T, E, ldl, elem));
  uint8_t* valid = masked ? buf((size_t)T) : nullptr;
  uint8_t *counts = buf((size_t)E * 4), *used = buf(4), *loss = buf(4), *g = buf(4);
  size_t ws = 0;
  CHECK(mxfp8_moe_balance_workspace_bytes(T, E, &ws) == 0);
  uint8_t* work = buf(ws);
  CHECK(mxfp8_moe_balance(l, dtype, T, E, ldl, topk, valid, 0.01f, 0.001f, (float*)loss, (int*)counts, (int*)used,
                          work, ws, nullptr) == 0);
  if (ws)
    CHECK(mxfp8_moe_balance(l, dtype, T, E, ldl, topk, valid, 0.01f, 0.001f, (float*)loss, (int*)counts, (int*)used,
                            work, ws - 1, nullptr) == MXFP8_E_WORKSPACE);
  CHECK(mxfp8_moe_balance_backward(l, dtype, T, E, ldl, topk, valid, 0.01f, 0.001f, (int*)counts, (int*)used,
                                   (float*)g, d, ldl, nullptr) == 0);
}
}  // namespace

int main() {
  const int64_t linear[][3] = {{0, 130, 256},   {1, 16, 16},      {13, 255, 2064}, {16, 130, 272}, {17, 1, 256},
                               {100, 384, 768}, {129, 200, 1040}, {300, 640, 512}, {64, 256, 8192}, {1031, 1000, 528}};
  for (const auto& s : linear)
    for (int64_t extra : {0, 24}) linear_case(s[0], s[1], s[2], extra);
  for (int tile : {64, 128, 256, 512}) {
    const int prev = mxfp8_debug_force_b128(tile);
    linear_case(300, 264, 2064, 8);
    linear_case(130, 130, 512, 0);
    mxfp8_debug_force_b128(prev);
  }
  const int64_t wgrad[][3] = {{0, 16, 32},      {1, 8, 16},        {63, 130 * 8, 48}, {512, 1024, 1024},
                              {700, 2064, 528}, {1000, 520, 2064}, {2048, 264, 272},  {65, 4096, 256}};
  for (int tile : {0, 128, 256}) {
    const int prev = mxfp8_debug_force_wgrad(tile);
    for (const auto& s : wgrad)
      for (int dtype : {MXFP8_F32, MXFP8_BF16})
        for (bool bias : {false, true}) wgrad_case(s[0], s[1], s[2], dtype, bias);
    mxfp8_debug_force_wgrad(prev);
  }
  const int64_t layer[][3] = {{0, 48, 80}, {1, 48, 80}, {16, 272, 528}, {17, 2064, 272}, {200, 528, 1040}};
  for (const auto& s : layer)
    for (int keep = 0; keep < 4; ++keep)
      for (int dtype : {MXFP8_F32, MXFP8_BF16}) layer_case(s[0], s[1], s[2], keep, dtype);
  // both products, one of them, on the MXFP8 GEMM, the choice not the hook's
  for (int force : {0, 64}) {
    const int prev = mxfp8_debug_force_b128(force), before = g_mx;
    for (int keep = 0; keep < 4; ++keep) layer_case(4096, 4096, 256, keep, MXFP8_BF16);
    CHECK(g_mx == before + 4);
    layer_case(8192, 2048, 2048, 3, MXFP8_BF16);
    CHECK(g_mx == before + 6);
    mxfp8_debug_force_b128(prev);
  }
  for (int64_t T : {0, 1, 16, 5000})
    for (int64_t E : {1, 8, 130, 256})
      for (int dtype : {MXFP8_F32, MXFP8_BF16})
        for (bool masked : {false, true}) balance_case(T, E, E < 8 ? E : 8, dtype, masked);
  // The row-major quantizers and every output set of the weight quantizer.
  {
    Buffers buf;
    const int64_t N = 144, K = 272, B = mxfp8::b128_blocks(K);
    uint8_t *w = buf((size_t)N * K * 2), *q = buf((size_t)N * K), *s8 = buf((size_t)N * B);
    CHECK(mxfp8_quantize_b128(w, N, K, K, q, K, s8, B, nullptr) == 0);
    uint8_t *s = buf(wscales(N, K)), *wp = buf(packed(N, K)), *sp = buf(wscales(N, K));
    uint8_t *wt = buf(packed(K, N)), *st = buf(wscales(K, N));
    for (int m = 1; m < 8; ++m)
      CHECK(mxfp8_quantize_weight_b128(w, N, K, K, m & 1 ? q : nullptr, K, m & 1 ? (float*)s : nullptr, B,
                                       m & 2 ? wp : nullptr, m & 2 ? sp : nullptr, m & 4 ? wt : nullptr,
                                       m & 4 ? st : nullptr, nullptr) == 0);
    CHECK(mxfp8_prepare_weight_b128(q, (float*)s, N, K, K, B, 1, wt, st, nullptr) == 0);
  }
  // Refusals come before any launch.
  const int before = g_launches;
  CHECK(mxfp8_linear_b128(nullptr, 4, 256, 256, nullptr, nullptr, 4, nullptr, nullptr, 4, nullptr, 0, nullptr) != 0);
  CHECK(mxfp8_linear_wgrad(nullptr, 4, 12, 16, nullptr, nullptr, 16, nullptr, 0, 16, nullptr, 0, 0, nullptr, 0,
                           nullptr) == MXFP8_E_SHAPE);
  CHECK(mxfp8_moe_balance(nullptr, 0, 4, 8, 8, 9, nullptr, 1, 1, nullptr, nullptr, nullptr, nullptr, 0, nullptr) ==
        MXFP8_E_SHAPE);
  CHECK(g_launches == before);
  if (g_fail) {
    std::fprintf(stderr, "%d checks failed\n", g_fail);
    return 1;
  }
  std::printf("host driver ok: %d launches checked\n", g_launches);
  return 0;
}
