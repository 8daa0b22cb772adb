// Load-balance loss and z loss of a top-k router, the tokens of each expert,
// and the gradient with respect to the logits.
//   p[t, e] = softmax(logits[t, :])[e],  lse[t] = log sum_e exp(logits[t, e])
//   c[e]    = tokens whose topk largest logits hold e (ties: lower e first,
//             as the routed layer selects),  n = tokens counted
//   loss    = coef E / (topk n^2) sum_e c[e] sum_t p[t, e]  +  z_coef / n sum_t lse[t]^2
//   dlogits = coef E / (topk n^2) p[t, e] (c[e] - sum_j c[j] p[t, j])
//             + 2 z_coef / n lse[t] p[t, e]                       (c is a constant)
// A token is counted if its mask byte is set and it has a logit other than
// -inf; the others add nothing and get a zero gradient.  n = 0: loss 0.
//
// Sixteen lanes (one DPP row) own a token, logit e = 16 c + lane in register
// c, so a wave works on four tokens and every reduction is four VALU lane
// exchanges.  The selection, not memory, is the cost of the forward pass:
// topk rounds of a maximum over E ordered integer keys.  bf16 logits leave
// sixteen bits of the key free for the index, so a round is one maximum and
// one compare per logit; fp32 logits need a second pass for the lowest index.
// Sums run per lane over its tokens, then over lanes, waves and workgroups in
// a fixed order, no atomics: results do not depend on timing.
#include <climits>

#include "common.hpp"
#include "launch_b128.hpp"

namespace mxfp8 {

namespace {

constexpr int kBalThreads = 1024;
constexpr int kBalTokens = kBalThreads / 16;   // tokens a workgroup works on at a time
constexpr int kBalMaxBlocks = 256;             // one workgroup per compute unit
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // key of -inf; 0 = not a candidate

template <int kCtrl>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}
template <int kCtrl>
__device__ inline float dppf(float v) {
  return __uint_as_float(dpp<kCtrl>(__float_as_uint(v)));
}
// Reductions over the sixteen lanes of a DPP row: quads, half row, row.
__device__ inline uint32_t row_max_u32(uint32_t v) {
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  return max(v, dpp<0x140>(v));
}
__device__ inline uint32_t row_min_u32(uint32_t v) {
  v = min(v, dpp<0xB1>(v));
  v = min(v, dpp<0x4E>(v));
  v = min(v, dpp<0x141>(v));
  return min(v, dpp<0x140>(v));
}
__device__ inline float row_max_f32(float v) {
  v = fmaxf(v, dppf<0xB1>(v));
  v = fmaxf(v, dppf<0x4E>(v));
  v = fmaxf(v, dppf<0x141>(v));
  return fmaxf(v, dppf<0x140>(v));
}
__device__ inline float row_sum_f32(float v) {
  v += dppf<0xB1>(v);
  v += dppf<0x4E>(v);
  v += dppf<0x141>(v);
  return v + dppf<0x140>(v);
}

// Unsigned key in the order of the values; both zeros alike, NaN as -inf (the
// rule of the routed layer: the selection stays in bounds).
__device__ inline uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t k = (b >> 31) ? ~b : b | 0x80000000u;
  return v != v ? kKeyNegInf : k;
}

// The logits of one token: v[c] = logit 16 c + l, -inf past E.
template <int kC, bool kBf16>
__device__ inline void load_row(const void* logits, int64_t off, int E, int l, float (&v)[kC]) {
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int e = 16 * c + l;
    v[c] = -INFINITY;
    if (e < E) {
      if constexpr (kBf16) v[c] = __uint_as_float((uint32_t)((const uint16_t*)logits)[off + e] << 16);
      else v[c] = ((const float*)logits)[off + e];
    }
  }
}

// p = softmax of the row and its log-sum-exp; false (p = 0, lse = 0) if every
// logit is -inf.  A NaN or +inf logit makes p and lse NaN.
template <int kC>
__device__ inline bool row_softmax(float (&v)[kC], float& lse) {
  float m = -INFINITY;
  uint32_t some = 0;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    m = fmaxf(m, v[c]);
    some |= v[c] != -INFINITY ? 1u : 0u;
  }
  m = row_max_f32(m);
  some = row_max_u32(some);
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    v[c] = some ? expf(v[c] - m) : 0.0f;
    s += v[c];
  }
  s = row_sum_f32(s);
  const float inv = some ? 1.0f / s : 0.0f;
#pragma unroll
  for (int c = 0; c < kC; ++c) v[c] *= inv;
  lse = some ? m + logf(s) : 0.0f;
  return some != 0;
}

// Partials of one workgroup in the workspace, arrays over the workgroups.
struct BalParts {
  float* p;     // [blocks][E] sums of p
  int* c;       // [blocks][E] tokens
  float* z;     // [blocks] sums of lse^2
  int* n;       // [blocks] tokens counted
};
__host__ __device__ inline BalParts bal_parts(void* ws, int64_t E) {
  BalParts b;
  b.p = (float*)ws;
  b.c = (int*)(b.p + kBalMaxBlocks * E);
  b.z = (float*)(b.c + kBalMaxBlocks * E);
  b.n = (int*)(b.z + kBalMaxBlocks);
  return b;
}

}  // namespace

template <int kC, bool kBf16>
__global__ __launch_bounds__(kBalThreads) void balance_kernel(const void* __restrict__ logits, int64_t T, int E,
                                                              int64_t ldl, int topk,
                                                              const uint8_t* __restrict__ valid, void* ws) {
  constexpr int kWaves = kBalThreads / 64;
  __shared__ float lp[kWaves][16 * kC];
  __shared__ int lc[kWaves][16 * kC];
  __shared__ float lz[kWaves];
  __shared__ int ln[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & 15;
  float ps[kC], zs = 0.0f;
  int cs[kC], ns = 0;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    ps[c] = 0.0f;
    cs[c] = 0;
  }
  for (int64_t t = (int64_t)blockIdx.x * kBalTokens + (tid >> 4); t < T; t += (int64_t)gridDim.x * kBalTokens) {
    if (valid != nullptr && valid[t] == 0) continue;   // a token's sixteen lanes agree
    float v[kC];
    load_row<kC, kBf16>(logits, t * ldl, E, l, v);
    uint32_t key[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      key[c] = 16 * c + l < E ? order_key(v[c]) : 0u;
      if constexpr (kBf16) key[c] = key[c] ? (key[c] & 0xFFFF0000u) | (0xFFFFu - (uint32_t)(16 * c + l)) : 0u;
    }
    float lse;
    if (!row_softmax<kC>(v, lse)) continue;
    for (int j = 0; j < topk; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < kC; ++c) m = max(m, key[c]);
      m = row_max_u32(m);
      if constexpr (kBf16) {
        // keys are distinct
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const bool hit = key[c] == m;
          cs[c] += hit ? 1 : 0;
          key[c] = hit ? 0u : key[c];
        }
      } else {
        uint32_t e = UINT_MAX;
#pragma unroll
        for (int c = 0; c < kC; ++c)
          if (key[c] == m) e = min(e, (uint32_t)(16 * c + l));
        e = row_min_u32(e);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const bool hit = e == (uint32_t)(16 * c + l);
          cs[c] += hit ? 1 : 0;
          key[c] = hit ? 0u : key[c];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) ps[c] += v[c];
    zs += lse * lse;
    ns += 1;
  }
  // Over the wave's four rows, then over the waves, in order.
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    ps[c] += __shfl_xor(ps[c], 16);
    ps[c] += __shfl_xor(ps[c], 32);
    cs[c] += __shfl_xor(cs[c], 16);
    cs[c] += __shfl_xor(cs[c], 32);
    if (lane < 16) {
      lp[wave][16 * c + l] = ps[c];
      lc[wave][16 * c + l] = cs[c];
    }
  }
  zs += __shfl_xor(zs, 16);
  zs += __shfl_xor(zs, 32);
  ns += __shfl_xor(ns, 16);
  ns += __shfl_xor(ns, 32);
  if (lane == 0) {
    lz[wave] = zs;
    ln[wave] = ns;
  }
  __syncthreads();
  const BalParts parts = bal_parts(ws, E);
  if (tid < E) {
    float p = 0.0f;
    int c = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      p += lp[w][tid];
      c += lc[w][tid];
    }
    parts.p[(int64_t)blockIdx.x * E + tid] = p;
    parts.c[(int64_t)blockIdx.x * E + tid] = c;
  }
  if (tid == 0) {
    float z = 0.0f;
    int n = 0;
    for (int w = 0; w < kWaves; ++w) {
      z += lz[w];
      n += ln[w];
    }
    parts.z[blockIdx.x] = z;
    parts.n[blockIdx.x] = n;
  }
}

// One workgroup: the partials of all blocks -> counts, n, loss.  Thread
// (q, e) adds blocks q, q + Q, ... of expert e; everything after that in
// 64 bits (one sum per expert, then one over the experts).
__global__ __launch_bounds__(kBalThreads) void balance_reduce_kernel(void* ws, int blocks, int E, int topk, float coef,
                                                                     float z_coef, int* __restrict__ counts,
                                                                     int* __restrict__ used, float* __restrict__ loss) {
  __shared__ float lp[kBalThreads];
  __shared__ int lc[kBalThreads];
  __shared__ double red[kBalThreads];
  __shared__ int ntot;
  const BalParts parts = bal_parts(ws, E);
  const int tid = threadIdx.x;
  const int Q = kBalThreads / E, q = tid / E, e = tid - q * E;
  float p = 0.0f;
  int c = 0;
  if (q < Q) {
    for (int b = q; b < blocks; b += Q) {
      p += parts.p[(int64_t)b * E + e];
      c += parts.c[(int64_t)b * E + e];
    }
  }
  lp[tid] = p;
  lc[tid] = c;
  double z = tid < blocks ? (double)parts.z[tid] : 0.0;
  if (tid == 0) ntot = 0;
  __syncthreads();
  if (tid < blocks) atomicAdd(&ntot, parts.n[tid]);   // integers: the order does not matter
  __syncthreads();
  const double n = ntot > 0 ? (double)ntot : 1.0;
  // no z loss: lse^2 may have left fp32 (a row of the type's lowest value)
  double mine = z_coef != 0.0f ? z * (double)z_coef / n : 0.0;
  if (tid < E) {
    double pe = 0.0;
    int ce = 0;
    for (int k = 0; k < Q; ++k) {
      pe += (double)lp[k * E + tid];
      ce += lc[k * E + tid];
    }
    counts[tid] = ce;
    mine += (double)coef * E / ((double)topk * n * n) * pe * ce;
  }
  red[tid] = mine;
  __syncthreads();
  for (int s = kBalThreads / 2; s > 0; s >>= 1) {
    if (tid < s) red[tid] += red[tid + s];
    __syncthreads();
  }
  if (tid == 0) {
    *loss = (float)red[0];
    *used = ntot;
  }
}

template <int kC, bool kBf16>
__global__ __launch_bounds__(256) void balance_backward_kernel(const void* __restrict__ logits, int64_t T, int E,
                                                               int64_t ldl, int topk,
                                                               const uint8_t* __restrict__ valid, float coef,
                                                               float z_coef, const int* __restrict__ counts,
                                                               const int* __restrict__ used,
                                                               const float* __restrict__ grad_loss,
                                                               void* __restrict__ dlogits, int64_t ldd) {
  const int tid = threadIdx.x, l = tid & 15;
  const double n = max(used[0], 1), g = grad_loss != nullptr ? (double)grad_loss[0] : 1.0;
  const float a = (float)(g * coef * E / ((double)topk * n * n)), b = (float)(g * 2.0 * z_coef / n);
  float cf[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) cf[c] = 16 * c + l < E ? (float)counts[16 * c + l] : 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * 16 + (tid >> 4); t < T; t += (int64_t)gridDim.x * 16) {
    float v[kC], lse = 0.0f;
    const bool in = valid == nullptr || valid[t] != 0;
    if (in) {
      load_row<kC, kBf16>(logits, t * ldl, E, l, v);
      row_softmax<kC>(v, lse);
      float inner = 0.0f;
#pragma unroll
      for (int c = 0; c < kC; ++c) inner += v[c] * cf[c];
      inner = row_sum_f32(inner);
#pragma unroll
      for (int c = 0; c < kC; ++c) v[c] = a * v[c] * (cf[c] - inner) + b * lse * v[c];
    } else {
#pragma unroll
      for (int c = 0; c < kC; ++c) v[c] = 0.0f;
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int e = 16 * c + l;
      if (e < E) {
        if constexpr (kBf16) ((uint16_t*)dlogits)[t * ldd + e] = (uint16_t)pack_bf16x2(v[c], 0.0f);
        else ((float*)dlogits)[t * ldd + e] = v[c];
      }
    }
  }
}

size_t balance_ws_bytes(int64_t T, int64_t E) {
  (void)T;
  return (size_t)kBalMaxBlocks * ((size_t)E * 8 + 8);
}

namespace {
// Calls f with the register count (logits per lane) that holds E.
template <typename F>
auto by_width(int64_t E, F f) {
  if (E <= 16) return f(std::integral_constant<int, 1>{});
  if (E <= 32) return f(std::integral_constant<int, 2>{});
  if (E <= 64) return f(std::integral_constant<int, 4>{});
  if (E <= 128) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}
}  // namespace

int launch_balance(const BalanceArgs& a, hipStream_t stream) {
  static_assert(kMoeMaxExperts <= 256, "sixteen lanes x sixteen registers hold a row of logits");
  const int64_t need = (a.T + kBalTokens - 1) / kBalTokens;
  const int blocks = (int)(need < kBalMaxBlocks ? need : kBalMaxBlocks);
  if (blocks > 0) {
    by_width(a.E, [&](auto C) {
      constexpr int c = decltype(C)::value;
      auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kBalThreads), 0, stream, a.logits, a.T, (int)a.E,
                           a.ldl, (int)a.topk, a.valid, a.ws);
      };
      if (a.bf16) go(balance_kernel<c, true>);
      else go(balance_kernel<c, false>);
      return 0;
    });
    if (hipGetLastError() != hipSuccess) return -7;
  }
  hipLaunchKernelGGL(balance_reduce_kernel, dim3(1), dim3(kBalThreads), 0, stream, a.ws, blocks, (int)a.E,
                     (int)a.topk, a.coef, a.z_coef, a.counts, a.used, a.loss);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

int launch_balance_backward(const BalanceArgs& a, hipStream_t stream) {
  const int64_t need = (a.T + 15) / 16;
  const int blocks = (int)(need < 2048 ? need : 2048);
  by_width(a.E, [&](auto C) {
    constexpr int c = decltype(C)::value;
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), 0, stream, a.logits, a.T, (int)a.E, a.ldl,
                         (int)a.topk, a.valid, a.coef, a.z_coef, a.counts, a.used, a.grad_loss, a.dlogits, a.ldd);
    };
    if (a.bf16) go(balance_backward_kernel<c, true>);
    else go(balance_backward_kernel<c, false>);
    return 0;
  });
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace mxfp8
