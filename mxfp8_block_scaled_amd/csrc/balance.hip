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
// Sixteen lanes (one DPP row) own a token, 1 .. 16 logits each, so a wave
// works on four tokens and every reduction is four VALU lane exchanges.
//
// The selection, not memory, is the cost of the forward pass.  Each lane
// sorts its logits once (ordered integer keys, a fixed network of min / max),
// then topk rounds take the largest head of the sixteen lanes and pop it: 13
// instructions a round, where scanning all logits of a lane takes 44 (256
// experts, topk 8).  The last head is the threshold, and one pass counts the
// logits at or above it.  bf16 logits leave sixteen bits of the key free for
// the index, so their keys are distinct; fp32 keys can tie, which shows in
// the number of logits at or above the threshold, and such a wave's tokens
// are selected again one logit at a time (lowest index among equals).
//
// Measured: 50000 x 256 bf16, topk 8: selection and sums 19 us, reduction 7, the
// gradient 12 (4.2 TB/s); 4096 x 128 fp32, topk 8: 7, 6 and 4.  Above topk 8 and
// 128 experts the selection takes 10 us a round (whole forward call at 50000 x
// 256: topk 8 24, 9 105, 16 171; at 50000 x 128: 30, 32, 46).
//
// Sums run per lane over its tokens, then over lanes, waves and workgroups in
// a fixed order, no atomics on values: results do not depend on timing.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "b128.hpp"

namespace mxfp8 {

namespace {

constexpr int kBalThreads = 512;
static_assert(kBalTokens == kBalThreads / 16, "tokens a workgroup works on at a time");
constexpr uint32_t kKeyNegInf = 0x007FFFFFu, kKeyPosInf = 0xFF800000u;   // order_key of the infinities

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

// Unsigned key in the order of the values, both zeros alike.  (NaN: positive
// ones above +inf, negative ones below -inf; see the forward kernel.)
__device__ inline uint32_t order_key(float v) {
  const int b = __float_as_int(v + 0.0f);
  return (uint32_t)(b ^ ((b >> 31) | (int)0x80000000));
}

// Which logit register c of lane l holds: runs of kV consecutive ones (one
// vector load), sixteen lanes side by side.
template <int kV>
__device__ inline int expert_of(int c, int l) {
  return (c / kV) * (16 * kV) + l * kV + c % kV;
}

// The logits of one token, -inf past E.  kV > 1: E and the row stride are
// multiples of kV and the rows are aligned to kV elements.
template <int kC, int kV, bool kBf16>
__device__ inline void load_row(const void* logits, int64_t off, int E, int l, float (&v)[kC]) {
#pragma unroll
  for (int c = 0; c < kC; c += kV) {
    // unconditional loads (clamped to the row's end), all in flight together
    const int e = min(expert_of<kV>(c, l), E - kV);
    if constexpr (kBf16) {
      typedef uint16_t vec __attribute__((ext_vector_type(kV)));
      const vec q = *reinterpret_cast<const vec*>((const uint16_t*)logits + off + e);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[c + j] = __uint_as_float((uint32_t)q[j] << 16);
    } else {
      typedef float vec __attribute__((ext_vector_type(kV)));
      const vec q = *reinterpret_cast<const vec*>((const float*)logits + off + e);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[c + j] = q[j];
    }
  }
  if (E < 16 * kC) {
#pragma unroll
    for (int c = 0; c < kC; ++c) v[c] = expert_of<kV>(c, l) < E ? v[c] : -INFINITY;
  }
}

// Sorts k descending: Batcher's odd-even merge sort (63 exchanges for 16).
template <int kC>
__device__ inline void sort_desc(uint32_t (&k)[kC]) {
#pragma unroll
  for (int p = 1; p < kC; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < kC; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < kC && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t x = k[i + j], y = k[i + j + q];
            k[i + j] = max(x, y);
            k[i + j + q] = min(x, y);
          }
}

// p = softmax of the row and its log-sum-exp; false (p = 0, lse = 0) if every
// logit is -inf.  A NaN or +inf logit makes p and lse NaN.  On the hardware's
// 2^y: y = (v - max) log2(e) rounds twice, so a term is off by |y| 2^-23 of
// itself, and what is far below the maximum is a small part of any sum.  A
// third of the instructions that expf takes.  (The difference comes first:
// v log2(e) leaves fp32 where v is the type's lowest value.)
template <int kC>
__device__ inline bool row_softmax(float (&v)[kC], float& lse) {
  float m = -INFINITY;
#pragma unroll
  for (int c = 0; c < kC; ++c) m = fmaxf(m, v[c]);
  m = row_max_f32(m);
  m = m == -INFINITY ? 0.0f : m;   // nothing left (or NaN alone): 2^-inf = 0 (NaN) below
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    v[c] = __builtin_amdgcn_exp2f((v[c] - m) * 1.44269504f);
    s += v[c];
  }
  s = row_sum_f32(s);
  const bool some = s != 0.0f;   // the largest logit's share is 1
  const float inv = some ? 1.0f / s : 0.0f;
#pragma unroll
  for (int c = 0; c < kC; ++c) v[c] *= inv;
  lse = some ? m + logf(s) : 0.0f;
  return some;
}

// Partials in the workspace, arrays over the forward workgroups, and what
// the reducing workgroups pass to the last one of them.
struct BalParts {
  float* p;       // [blocks][E] sums of p
  int* c;         // [blocks][E] tokens
  float* z;       // [blocks] sums of lse^2
  int* n;         // [blocks] tokens counted
  double* loss;   // [16] sums over each reducing workgroup's experts
  int* arrived;   // reducing workgroups that are done (cleared by the forward kernel)
};
__host__ __device__ inline BalParts bal_parts(void* ws, int64_t E) {
  BalParts b;
  b.loss = (double*)ws;
  b.p = (float*)(b.loss + 16);
  b.c = (int*)(b.p + kBalMaxBlocks * E);
  b.z = (float*)(b.c + kBalMaxBlocks * E);
  b.n = (int*)(b.z + kBalMaxBlocks);
  b.arrived = b.n + kBalMaxBlocks;
  return b;
}

}  // namespace

// kTop: an upper bound of topk (8 or 16; a lane's sorted keys past it are
// never reached).
template <int kC, int kV, int kTop, bool kBf16>
__global__ __launch_bounds__(kBalThreads) void balance_kernel(const void* __restrict__ logits, int64_t T, int E,
                                                              int64_t ldl, int topk,
                                                              const uint8_t* __restrict__ valid, void* ws, float coef,
                                                              float z_coef, int* __restrict__ counts,
                                                              int* __restrict__ used, float* __restrict__ loss) {
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
    load_row<kC, kV, kBf16>(logits, t * ldl, E, l, v);
    uint32_t key[kC], s[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      // Registers past E hold -inf and a larger index than every expert, so
      // they come after the last expert, and E >= topk.
      key[c] = order_key(v[c]);
      if constexpr (kBf16) key[c] = (key[c] & 0xFFFF0000u) | (0xFFFFu - (uint32_t)expert_of<kV>(c, l));
    }
    float lse;
    if (!row_softmax<kC>(v, lse)) continue;
    if (lse != lse) {
      // The selection reads NaN as -inf, like the routed layer's (the counts
      // stay in bounds; the loss is NaN all the same).
      constexpr uint32_t kMask = kBf16 ? 0xFFFF0000u : 0xFFFFFFFFu;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const uint32_t k = key[c] & kMask;
        if (k > (kKeyPosInf & kMask) || k < (kKeyNegInf & kMask)) key[c] = (kKeyNegInf & kMask) | (key[c] & ~kMask);
      }
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) s[c] = key[c];
    sort_desc<kC>(s);
    uint32_t m = 0;
    for (int j = 0; j < topk; ++j) {
      m = row_max_u32(s[0]);
      const bool hit = s[0] == m;
#pragma unroll
      for (int c = 0; c < kC && c < kTop; ++c) s[c] = hit ? (c + 1 < kC ? s[c + 1] : 0u) : s[c];
    }
    bool exact = true;
    if constexpr (!kBf16) {
      uint32_t n = 0;
#pragma unroll
      for (int c = 0; c < kC; ++c) n += key[c] >= m ? 1 : 0;
      n += dpp<0xB1>(n);
      n += dpp<0x4E>(n);
      n += dpp<0x141>(n);
      n += dpp<0x140>(n);
      exact = n == (uint32_t)topk;
    }
    if (exact) {
#pragma unroll
      for (int c = 0; c < kC; ++c) cs[c] += key[c] >= m ? 1 : 0;
    } else {
      for (int j = 0; j < topk; ++j) {
        uint32_t w = 0, e = UINT_MAX;
#pragma unroll
        for (int c = 0; c < kC; ++c) w = max(w, key[c]);
        w = row_max_u32(w);
#pragma unroll
        for (int c = 0; c < kC; ++c)
          if (key[c] == w) e = min(e, (uint32_t)expert_of<kV>(c, l));
        e = row_min_u32(e);
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const bool hit = e == (uint32_t)expert_of<kV>(c, l);
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
      lp[wave][expert_of<kV>(c, l)] = ps[c];
      lc[wave][expert_of<kV>(c, l)] = cs[c];
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
  float p = 0.0f, z = 0.0f;
  int k = 0, n = 0;
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      p += lp[w][tid];
      k += lc[w][tid];
    }
  }
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    z += lz[w];
    n += ln[w];
  }
  if (gridDim.x == 1) {
    // The only workgroup has all the sums and needs no second launch.
    __shared__ double ll[kWaves];
    const double d = n > 0 ? (double)n : 1.0;
    double mine = tid < E ? (double)coef * E / ((double)topk * d * d) * p * k : 0.0;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) mine += __shfl_xor(mine, o);
    if (lane == 0) ll[wave] = mine;
    if (tid < E) counts[tid] = k;
    __syncthreads();
    if (tid != 0) return;
    mine = z_coef != 0.0f ? (double)z * (double)z_coef / d : 0.0;   // as in the reduction below
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mine += ll[w];
    *used = n;
    *loss = (float)mine;
    return;
  }
  const BalParts parts = bal_parts(ws, E);
  if (tid < E) {
    parts.p[(int64_t)blockIdx.x * E + tid] = p;
    parts.c[(int64_t)blockIdx.x * E + tid] = k;
  }
  if (tid == 0) {
    parts.z[blockIdx.x] = z;
    parts.n[blockIdx.x] = n;
    if (blockIdx.x == 0) *parts.arrived = 0;
  }
}

// One workgroup per sixteen experts: thread (q, e) adds blocks q, q + 64, ...
// of its expert; from there in 64 bits.  Every workgroup adds up n itself
// (the loss needs it); the last to arrive adds the workgroups' shares of the
// loss in order, so the result does not depend on which one it is.
__global__ __launch_bounds__(1024) void balance_reduce_kernel(void* ws, int blocks, int E, int topk, float coef,
                                                              float z_coef, int* __restrict__ counts,
                                                              int* __restrict__ used, float* __restrict__ loss) {
  __shared__ double lp[16][16], lz[16];
  __shared__ int lc[16][16], ln[16];
  const BalParts parts = bal_parts(ws, E);
  const int tid = threadIdx.x, q = tid >> 4, c = tid & 15, wave = tid >> 6;
  const int e = (int)blockIdx.x * 16 + c;
  double p = 0.0;
  int k = 0;
  {
    // at most eight rows a thread, all loads in flight together
    constexpr int kRows = kBalMaxBlocks / 64;
    float pv[kRows];
    int kv[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t at = (int64_t)min(q + 64 * r, blocks - 1) * E + min(e, E - 1);
      pv[r] = parts.p[at];
      kv[r] = parts.c[at];
    }
    int n = tid < blocks ? parts.n[tid] : 0;
    double z = tid < blocks ? (double)parts.z[tid] : 0.0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      p += q + 64 * r < blocks ? (double)pv[r] : 0.0;
      k += q + 64 * r < blocks ? kv[r] : 0;
    }
    // over the wave's four rows of threads, n and z over the whole wave
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      if (o >= 16) {
        p += __shfl_xor(p, o);
        k += __shfl_xor(k, o);
      }
      n += __shfl_xor(n, o);
      z += __shfl_xor(z, o);
    }
    if ((tid & 63) < 16) {
      lp[wave][c] = p;
      lc[wave][c] = k;
    }
    if ((tid & 63) == 0) {
      ln[wave] = n;
      lz[wave] = z;
    }
  }
  __syncthreads();
  if (tid >= 16) return;
  p = 0.0;
  k = 0;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    p += lp[r][c];
    k += lc[r][c];
  }
  int n = ln[c];
  double z = lz[c];
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) {
    n += __shfl_xor(n, o);
    z += __shfl_xor(z, o);
  }
  const double d = n > 0 ? (double)n : 1.0;
  double mine = e < E ? (double)coef * E / ((double)topk * d * d) * p * k : 0.0;
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) mine += __shfl_xor(mine, o);
  if (e < E) counts[e] = k;
  if (tid != 0) return;
  if (blockIdx.x == 0) {
    // no z loss: lse^2 may have left fp32 (a row of the type's lowest value)
    if (z_coef != 0.0f) mine += z * (double)z_coef / d;
    *used = n;
  }
  if (gridDim.x == 1) {
    *loss = (float)mine;
    return;
  }
  __hip_atomic_store(&parts.loss[blockIdx.x], mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const int before = __hip_atomic_fetch_add(parts.arrived, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  if (before != (int)gridDim.x - 1) return;
  double sum = 0.0;
  for (int b = 0; b < (int)gridDim.x; ++b)
    sum += __hip_atomic_load(&parts.loss[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  *loss = (float)sum;
}

template <int kC, int kV, bool kBf16>
__global__ __launch_bounds__(256) void balance_backward_kernel(const void* __restrict__ logits, int64_t T, int E,
                                                               int64_t ldl, int topk,
                                                               const uint8_t* __restrict__ valid, float coef,
                                                               float z_coef, const int* __restrict__ counts,
                                                               const int* __restrict__ used,
                                                               const float* __restrict__ grad_loss,
                                                               void* __restrict__ dlogits, int64_t ldd) {
  const int tid = threadIdx.x, l = tid & 15;
  const float n = (float)max(used[0], 1), g = grad_loss != nullptr ? grad_loss[0] : 1.0f;
  const float a = g * (coef * (float)E / (float)topk / n / n), b = g * (2.0f * z_coef / n);
  // The counts through LDS: read by every lane straight from memory they cost
  // more than the logits (13 us of 22 at 50000 tokens, 256 experts).
  __shared__ __attribute__((aligned(16))) float lc[16 * kC];
  for (int e = tid; e < 16 * kC; e += 256) lc[e] = e < E ? (float)counts[e] : 0.0f;
  __syncthreads();
  float cf[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) cf[c] = lc[expert_of<kV>(c, l)];
  for (int64_t t = (int64_t)blockIdx.x * 16 + (tid >> 4); t < T; t += (int64_t)gridDim.x * 16) {
    float v[kC], lse = 0.0f;
    const bool in = valid == nullptr || valid[t] != 0;
    if (in) {
      load_row<kC, kV, kBf16>(logits, t * ldl, E, l, v);
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
    for (int c = 0; c < kC; c += kV) {
      const int e = expert_of<kV>(c, l);
      if (e >= E) continue;
      if constexpr (kBf16) {
        typedef uint16_t vec __attribute__((ext_vector_type(kV)));
        vec q;
#pragma unroll
        for (int j = 0; j < kV; ++j) q[j] = (uint16_t)pack_bf16x2(v[c + j], 0.0f);
        *reinterpret_cast<vec*>((uint16_t*)dlogits + t * ldd + e) = q;
      } else {
        typedef float vec __attribute__((ext_vector_type(kV)));
        vec q;
#pragma unroll
        for (int j = 0; j < kV; ++j) q[j] = v[c + j];
        *reinterpret_cast<vec*>((float*)dlogits + t * ldd + e) = q;
      }
    }
  }
}

namespace {
// Calls f(C, V) with the logits per lane that hold E and the vector width:
// 16 bytes or the lane's whole share if `aligned` allows it, else single
// elements.
template <typename F>
void by_width(int64_t E, int bf16, int64_t ld, const void* p, const void* p2, F f) {
  auto width = [&](auto C) {
    constexpr int c = decltype(C)::value;
    auto with = [&](auto V) {
      constexpr int v = decltype(V)::value;
      const uintptr_t bytes = (uintptr_t)v * (bf16 ? 2 : 4);
      if (v > 1 && (E % v != 0 || ld % v != 0 || ((uintptr_t)p | (uintptr_t)p2) % bytes != 0))
        f(C, std::integral_constant<int, 1>{});
      else
        f(C, V);
    };
    if (bf16) with(std::integral_constant<int, (c < 8 ? c : 8)>{});
    else with(std::integral_constant<int, (c < 4 ? c : 4)>{});
  };
  if (E <= 16) width(std::integral_constant<int, 1>{});
  else if (E <= 32) width(std::integral_constant<int, 2>{});
  else if (E <= 64) width(std::integral_constant<int, 4>{});
  else if (E <= 128) width(std::integral_constant<int, 8>{});
  else width(std::integral_constant<int, 16>{});
}
}  // namespace

int launch_balance(const BalanceArgs& a, hipStream_t stream) {
  static_assert(kMoeMaxExperts <= 256 && kMoeMaxTopk <= 16, "sixteen lanes x sixteen registers hold a row of logits");
  // one workgroup at least: it writes the results of no tokens
  const int64_t need = std::max<int64_t>(1, (a.T + kBalTokens - 1) / kBalTokens);
  const int blocks = (int)std::min<int64_t>(need, kBalMaxBlocks);
  by_width(a.E, a.bf16, a.ldl, a.logits, nullptr, [&](auto C, auto V) {
    constexpr int c = decltype(C)::value, v = decltype(V)::value;
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(kBalThreads), 0, stream, a.logits, a.T, (int)a.E, a.ldl,
                         (int)a.topk, a.valid, a.ws, a.coef, a.z_coef, a.counts, a.used, a.loss);
    };
    constexpr int top = c < 8 ? c : 8;
    if (a.topk <= 8) {
      if (a.bf16) go(balance_kernel<c, v, top, true>);
      else if constexpr (v <= 4) go(balance_kernel<c, v, top, false>);
    } else {
      if (a.bf16) go(balance_kernel<c, v, c, true>);
      else if constexpr (v <= 4) go(balance_kernel<c, v, c, false>);
    }
  });
  if (hipGetLastError() != hipSuccess) return -7;
  if (blocks == 1) return 0;
  hipLaunchKernelGGL(balance_reduce_kernel, dim3((unsigned)((a.E + 15) / 16)), dim3(1024), 0, stream, a.ws, blocks,
                     (int)a.E, (int)a.topk, a.coef, a.z_coef, a.counts, a.used, a.loss);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

int launch_balance_backward(const BalanceArgs& a, hipStream_t stream) {
  const int64_t need = (a.T + 15) / 16;
  const int blocks = (int)std::min<int64_t>(need, 2048);
  // one width for both arrays: the rows of each have to suit it
  const int64_t ld = a.ldl | a.ldd;
  by_width(a.E, a.bf16, ld, a.logits, a.dlogits, [&](auto C, auto V) {
    constexpr int c = decltype(C)::value, v = decltype(V)::value;
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, dim3((unsigned)blocks), dim3(256), 0, stream, a.logits, a.T, (int)a.E, a.ldl,
                         (int)a.topk, a.valid, a.coef, a.z_coef, a.counts, a.used, a.grad_loss, a.dlogits, a.ldd);
    };
    if (a.bf16) go(balance_backward_kernel<c, v, true>);
    else if constexpr (v <= 4) go(balance_backward_kernel<c, v, false>);
  });
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace mxfp8
