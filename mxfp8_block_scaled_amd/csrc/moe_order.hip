// Tokens sorted by expert and back.
//
//  sort       a stable counting sort of the R = T topk slots by their expert:
//             rows[slot] is the slot's place, slots its inverse, offsets[e]
//             the first place of expert e.  A slot whose id is no expert's
//             (padding, or an expert of another rank) comes behind all others;
//             offsets[E] places are the experts'.  So rows is a permutation,
//             and every row of a sorted matrix belongs to one slot.
//  permute    xs[rows[t, j]] = x[t]                     (0 for slots without an expert)
//  unpermute  y[t] = sum_j w[t, j] ys[rows[t, j]]       (slots with an expert; fp32, in slot order, rounded once)
//  its gradient  dys[rows[t, j]] = w[t, j] dy[t],  dw[t, j] = <dy[t], ys[rows[t, j]]>
// Permute's gradient is unpermute without weights.  No atomics across
// workgroups: results do not depend on timing.  (Rows out of range, which
// sort never makes, are skipped.)
//
// Measured, 4096 tokens, top 8 of 128, H 2048 bf16: sort 8.3 us (two launches,
// 5 of them the second's chain of LDS steps); permute 27.7 and unpermute 25.3,
// 5.4 and 6.0 TB/s of the 151 MB that they read and write; the gradient of both
// operands 50, 5.7 TB/s.  32768 tokens, top 2, H 4096: 137, 131 and 255 us (5.9,
// 6.1 and 5.3 TB/s).
#include <algorithm>

#include "common.hpp"
#include "launch_fp4.hpp"

namespace mxfp8 {

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxBins = (int)kMoeMaxExperts + 1;   // the last bin: slots without an expert

template <typename Id>
__device__ inline int bin_of(const Id* ids, int64_t i, int E) {
  const Id e = ids[i];
  return e >= 0 && e < E ? (int)e : E;
}

}  // namespace

// Slots of each bin in this workgroup's chunk.
template <typename Id>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const Id* __restrict__ ids, int64_t R, int E,
                                                                  int64_t chunk, int* __restrict__ counts) {
  __shared__ int hist[kMaxBins];
  const int tid = threadIdx.x;
  for (int b = tid; b <= E; b += kSortThreads) hist[b] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * chunk, last = min(first + chunk, R);
  for (int64_t i = first + tid; i < last; i += kSortThreads) atomicAdd(&hist[bin_of(ids, i, E)], 1);
  __syncthreads();
  for (int b = tid; b <= E; b += kSortThreads) counts[(int64_t)blockIdx.x * (E + 1) + b] = hist[b];
}

// Places of this workgroup's chunk.  Each of its sixteen waves owns one run of
// consecutive slots.  A bin's first place: the slots of lower bins, those of
// this bin in earlier workgroups (counts; one workgroup: none) and in earlier
// waves.  Within a wave the places go 64 slots at a time: lanes of the same
// bin find each other by one ballot per bit of the bin.
template <typename Id>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const Id* __restrict__ ids, int64_t R, int E,
                                                                  int64_t chunk, const int* __restrict__ counts,
                                                                  int* __restrict__ rows, int* __restrict__ slots,
                                                                  int* __restrict__ offsets) {
  __shared__ int hist[kSortWaves][kMaxBins];   // per wave: slots of a bin, then its next place
  __shared__ int before[kMaxBins], total[kMaxBins], start[kMaxBins];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int bins = E + 1;
  for (int i = tid; i < kSortWaves * kMaxBins; i += kSortThreads) (&hist[0][0])[i] = 0;
  for (int b = tid; b < kMaxBins; b += kSortThreads) before[b] = total[b] = 0;
  __syncthreads();

  const int64_t first = (int64_t)blockIdx.x * chunk, last = min(first + chunk, R);
  const int64_t per = ((last - first + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  const int64_t w0 = min(first + wave * per, last), w1 = min(w0 + per, last);
  for (int64_t i = w0 + lane; i < w1; i += 64) atomicAdd(&hist[wave][bin_of(ids, i, E)], 1);
  if (counts != nullptr) {
    // Thread (part, bin): the workgroups part, part + parts, ...  (integer
    // sums in LDS: their order does not matter)
    const int parts = kSortThreads / bins, b = tid % bins, part = tid / bins;
    if (part < parts) {
      int lower = 0, all = 0;
#pragma unroll 8
      for (int g = part; g < (int)gridDim.x; g += parts) {
        const int n = counts[(int64_t)g * bins + b];
        all += n;
        lower += g < (int)blockIdx.x ? n : 0;
      }
      atomicAdd(&before[b], lower);
      atomicAdd(&total[b], all);
    }
  }
  __syncthreads();
  if (counts == nullptr && tid < bins) {
    int n = 0;
    for (int w = 0; w < kSortWaves; ++w) n += hist[w][tid];
    total[tid] = n;
  }
  __syncthreads();
  // First place of each bin: wave 0, lane l holds bins 5 l .. 5 l + 4.
  constexpr int kPer = (kMaxBins + 63) / 64;
  if (wave == 0) {
    int v[kPer], sum = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int b = kPer * lane + u;
      v[u] = b < bins ? total[b] : 0;
      sum += v[u];
    }
    int run = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(run, off);
      if (lane >= off) run += o;
    }
    run -= sum;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int b = kPer * lane + u;
      if (b < bins) {
        start[b] = run;
        if (blockIdx.x == 0) offsets[b] = run;   // (bin E: the places of the experts)
      }
      run += v[u];
    }
  }
  __syncthreads();
  if (tid < bins) {
    int at = start[tid] + before[tid];
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = hist[w][tid];
      hist[w][tid] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int64_t base = w0; base < w1; base += 64) {
    const int64_t i = base + lane;
    const bool in = i < w1;
    const int b = in ? bin_of(ids, i, E) : kMaxBins;   // (kMaxBins: nobody's bin)
    uint64_t same = ~0ull;
#pragma unroll
    for (int bit = 0; bit < 9; ++bit) {
      const uint64_t m = __ballot((b >> bit) & 1);
      same &= ((b >> bit) & 1) ? m : ~m;
    }
    const uint64_t lower = same & ((1ull << lane) - 1ull);
    int at = 0;
    if (in) at = hist[wave][b] + __popcll(lower);
    // (one wave's LDS accesses run in their order: all have read before the
    // first lane of each bin moves its place on)
    __builtin_amdgcn_wave_barrier();
    if (in && lower == 0) hist[wave][b] = at + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (in) {
      rows[i] = at;
      slots[at] = (int)i;
    }
  }
}

int64_t sort_blocks(int64_t R) {
  if (R <= 4096) return 1;
  const int64_t chunk = std::max<int64_t>(kSortChunk, (R + kSortMaxBlocks - 1) / kSortMaxBlocks);
  return (R + chunk - 1) / chunk;
}

namespace {
template <typename Id>
int sort_go(const SortArgs& a, hipStream_t stream) {
  const int64_t n = sort_blocks(a.R);
  const int64_t chunk = n <= 1 ? std::max<int64_t>(a.R, 1)
                               : std::max<int64_t>(kSortChunk, (a.R + kSortMaxBlocks - 1) / kSortMaxBlocks);
  const Id* ids = (const Id*)a.ids;
  if (n > 1)
    hipLaunchKernelGGL(sort_count_kernel<Id>, dim3((unsigned)n), dim3(kSortThreads), 0, stream, ids, a.R, (int)a.E,
                       chunk, a.ws);
  hipLaunchKernelGGL(sort_place_kernel<Id>, dim3((unsigned)n), dim3(kSortThreads), 0, stream, ids, a.R, (int)a.E,
                     chunk, n > 1 ? a.ws : nullptr, a.rows, a.slots, a.offsets);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}
}  // namespace

int launch_moe_sort(const SortArgs& a, hipStream_t stream) {
  return a.wide ? sort_go<int64_t>(a, stream) : sort_go<int32_t>(a, stream);
}

// ------------------------------------------------------------------ rows there and back
//
// One thread takes 16 bytes of a token's row (eight bf16 or four fp32; the
// last piece of a row may be partial) for all topk slots of the token.  All of
// these are bound by memory.  Rows whose pieces are not 16-byte aligned take
// the same accesses through a type of the element's alignment, which the
// hardware serves.

namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef u4 u4_2 __attribute__((aligned(2)));
typedef u4 u4_4 __attribute__((aligned(4)));

// Element types: bf16 as raw words, fp32.
template <typename El, bool kAligned>
struct Piece {
  static constexpr int kN = 16 / (int)sizeof(El);
  using Any = typename std::conditional<sizeof(El) == 2, u4_2, u4_4>::type;
  __device__ static u4 load(const El* p, int n) {
    if (n >= kN) {
      if constexpr (kAligned) return *reinterpret_cast<const u4*>(p);
      else return *reinterpret_cast<const Any*>(p);
    }
    El v[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) v[e] = e < n ? p[e] : El(0);
    return __builtin_bit_cast(u4, v);
  }
  // kPast: around the caches (non-temporal)
  template <bool kPast>
  __device__ static void store(El* p, u4 v, int n) {
    using To = typename std::conditional<kAligned, u4, Any>::type;
    if (n >= kN) {
      if constexpr (kPast) __builtin_nontemporal_store((To)v, reinterpret_cast<To*>(p));
      else *reinterpret_cast<To*>(p) = v;
      return;
    }
    El w[kN];
    __builtin_memcpy(w, &v, 16);
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (e < n) p[e] = w[e];
  }
  __device__ static void widen(u4 v, float* f) {
    if constexpr (sizeof(El) == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = bf16_lo(v[e]);
        f[2 * e + 1] = bf16_hi(v[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(v[e]);
    }
  }
  __device__ static u4 narrow(const float* f) {
    u4 v;
    if constexpr (sizeof(El) == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(f[e]);
    }
    return v;
  }
};

constexpr int kRowThreads = 256;

// (token, piece) of this thread: T pieces fit 32 bits (a 64-bit division takes
// some hundred instructions).
struct Place {
  int64_t t;
  int piece;
  bool in;
};
__device__ inline Place place(uint32_t total, int pieces) {
  const uint32_t i = blockIdx.x * (uint32_t)kRowThreads + threadIdx.x, t = i / (uint32_t)pieces;
  return {(int64_t)t, (int)(i - t * pieces), i < total};
}

}  // namespace

template <typename El, bool kAligned, bool kPast>
__global__ __launch_bounds__(kRowThreads) void permute_kernel(const El* __restrict__ x, int64_t ldx, uint32_t total,
                                                              int H, int pieces, int topk, int R,
                                                              const int* __restrict__ rows,
                                                              const int* __restrict__ kept, El* __restrict__ xs,
                                                              int64_t lds) {
  using P = Piece<El, kAligned>;
  const Place at = place(total, pieces);
  if (!at.in) return;
  const int64_t t = at.t;
  const int c = at.piece * P::kN, n = H - c;
  const int here = *kept;
  const u4 v = P::load(x + t * ldx + c, n);
  const u4 zero = {0, 0, 0, 0};
  for (int j = 0; j < topk; ++j) {
    const int r = rows[t * topk + j];
    if ((uint32_t)r < (uint32_t)R) P::template store<kPast>(xs + (int64_t)r * lds + c, r < here ? v : zero, n);
  }
}

// kBatch: rows in flight.
template <typename El, bool kAligned, bool kPast, int kBatch>
__global__ __launch_bounds__(kRowThreads) void unpermute_kernel(const El* __restrict__ ys, int64_t lds, uint32_t total,
                                                                int H, int pieces, int topk, int R,
                                                                const int* __restrict__ rows,
                                                                const int* __restrict__ kept,
                                                                const float* __restrict__ weights,
                                                                El* __restrict__ y, int64_t ldy) {
  using P = Piece<El, kAligned>;
  const Place at = place(total, pieces);
  if (!at.in) return;
  const int64_t t = at.t;
  const int c = at.piece * P::kN, n = H - c;
  const uint32_t here = (uint32_t)min(max(*kept, 0), R);
  float acc[P::kN] = {};
  for (int j0 = 0; j0 < topk; j0 += kBatch) {
    u4 v[kBatch];
    float w[kBatch];
    bool on[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + u;
      const uint32_t r = j < topk ? (uint32_t)rows[t * topk + j] : here;
      on[u] = r < here;
      w[u] = on[u] && weights != nullptr ? weights[t * topk + j] : 1.0f;
      v[u] = on[u] ? P::load(ys + (int64_t)r * lds + c, n) : u4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float f[P::kN];
      P::widen(v[u], f);
      if (on[u]) {
#pragma unroll
        for (int e = 0; e < P::kN; ++e) acc[e] += w[u] * f[e];
      }
    }
  }
  P::template store<kPast>(y + t * ldy + c, P::narrow(acc), n);
}

// kWaves waves per token, their lanes along the row; the partial dot products
// of a token's slots are added over lanes and then over waves, in a fixed
// order.  A workgroup has four tokens with one wave each, or one with four.
template <typename El, bool kAligned, bool kPast, int kWaves>
__global__ __launch_bounds__(kRowThreads) void unpermute_backward_kernel(
    const El* __restrict__ dy, int64_t lddy, int64_t T, int H, int pieces, int topk, int R,
    const int* __restrict__ rows,
    const int* __restrict__ kept, const El* __restrict__ ys, int64_t ldys, const float* __restrict__ weights,
    El* __restrict__ dys, int64_t ldd, float* __restrict__ dw) {
  using P = Piece<El, kAligned>;
  constexpr int kTokens = kRowThreads / 64 / kWaves;   // tokens of a workgroup
  constexpr int kBatch = 4;
  __shared__ float part[kRowThreads / 64][kMoeMaxTopk];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kTokens + wave / kWaves;
  const int sub = wave % kWaves;
  const uint32_t here = (uint32_t)min(max(*kept, 0), R);
  if (t < T) {
    for (int j0 = 0; j0 < topk; j0 += kBatch) {
      uint32_t r[kBatch];
      float w[kBatch], dot[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = min(j0 + u, topk - 1);
        r[u] = (uint32_t)rows[t * topk + j];
        w[u] = weights != nullptr ? weights[t * topk + j] : 1.0f;
        dot[u] = 0.0f;
      }
      for (int p = sub * 64 + lane; p < pieces; p += 64 * kWaves) {
        const int c = p * P::kN, n = H - c;
        float g[P::kN];
        P::widen(P::load(dy + t * lddy + c, n), g);
        u4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          v[u] = dw != nullptr && r[u] < here ? P::load(ys + (int64_t)r[u] * ldys + c, n) : u4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          float f[P::kN];
          P::widen(v[u], f);
          if (r[u] < here && dw != nullptr) {
#pragma unroll
            for (int e = 0; e < P::kN; ++e) dot[u] += g[e] * f[e];   // (zeros past the row)
          }
          if (dys != nullptr && j0 + u < topk && r[u] < (uint32_t)R) {
            float d[P::kN];
#pragma unroll
            for (int e = 0; e < P::kN; ++e) d[e] = r[u] < here ? w[u] * g[e] : 0.0f;
            P::template store<kPast>(dys + (int64_t)r[u] * ldd + c, P::narrow(d), n);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) dot[u] += __shfl_xor(dot[u], off);
        if (lane == 0 && j0 + u < topk) part[wave][j0 + u] = dot[u];
      }
    }
  }
  if (dw == nullptr) return;
  __syncthreads();
  const int i = threadIdx.x;
  if (i < kTokens * topk) {
    const int k = i / topk, j = i - k * topk;
    const int64_t tt = (int64_t)blockIdx.x * kTokens + k;
    if (tt < T) {
      float sum = 0.0f;
#pragma unroll
      for (int s = 0; s < kWaves; ++s) sum += part[k * kWaves + s][j];
      dw[tt * topk + j] = sum;
    }
  }
}

namespace {
bool rows16(const void* p, int64_t ld, int64_t size) { return p == nullptr || (((uintptr_t)p | (uintptr_t)(ld * size)) & 15) == 0; }

// Matrices larger than the chip's L2s: results go around the caches.  In bf16,
// there, back and gradient, us in graphs that use the same buffers again: 32768
// tokens, top 2, H 4096 124, 135 and 280 around, 145, 139 and 276 through them;
// 4096 tokens, top 8, H 2048 26.4, 23.5 and 49.1 around, 24.6, 24.0 and 55.7
// through.  Smaller results stay for who reads them next.
bool past_caches(const PermuteArgs& a) { return a.T * a.topk * a.H * (a.bf16 ? 2 : 4) > (int64_t)32 << 20; }

// Calls go(element, aligned, past the caches) with the types as values.
template <typename Go>
void by_type(const PermuteArgs& a, bool aligned, Go&& go) {
  auto with = [&](auto el) {
    const bool past = past_caches(a);
    if (aligned && past) go(el, std::true_type{}, std::true_type{});
    else if (aligned) go(el, std::true_type{}, std::false_type{});
    else if (past) go(el, std::false_type{}, std::true_type{});
    else go(el, std::false_type{}, std::false_type{});
  };
  if (a.bf16) with(uint16_t{});
  else with(float{});
}
}  // namespace

int launch_moe_permute(const PermuteArgs& a, hipStream_t stream) {
  const int size = a.bf16 ? 2 : 4;
  const int pieces = (int)((a.H + 16 / size - 1) / (16 / size));
  const uint32_t total = (uint32_t)(a.T * pieces);
  by_type(a, rows16(a.tokens, a.ldt, size) && rows16(a.out_sorted, a.ldo, size), [&](auto el, auto al, auto past) {
    using El = decltype(el);
    hipLaunchKernelGGL((permute_kernel<El, decltype(al)::value, decltype(past)::value>), dim3((total + kRowThreads - 1) / kRowThreads),
                       dim3(kRowThreads), 0, stream, (const El*)a.tokens, a.ldt, total, (int)a.H, pieces, (int)a.topk,
                       (int)(a.T * a.topk), a.rows, a.kept, (El*)a.out_sorted, a.ldo);
  });
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

int launch_moe_unpermute(const PermuteArgs& a, hipStream_t stream) {
  const int size = a.bf16 ? 2 : 4;
  const int pieces = (int)((a.H + 16 / size - 1) / (16 / size));
  const uint32_t total = (uint32_t)(a.T * pieces);
  by_type(a, rows16(a.sorted, a.lds, size) && rows16(a.out_tokens, a.ldo, size), [&](auto el, auto al, auto past) {
    using El = decltype(el);
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, dim3((total + kRowThreads - 1) / kRowThreads), dim3(kRowThreads), 0, stream,
                         (const El*)a.sorted, a.lds, total, (int)a.H, pieces, (int)a.topk, (int)(a.T * a.topk), a.rows,
                         a.kept, a.weights, (El*)a.out_tokens, a.ldo);
    };
    if (a.topk <= 2) go(unpermute_kernel<El, decltype(al)::value, decltype(past)::value, 2>);
    else if (a.topk <= 4) go(unpermute_kernel<El, decltype(al)::value, decltype(past)::value, 4>);
    else go(unpermute_kernel<El, decltype(al)::value, decltype(past)::value, 8>);
  });
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

int launch_moe_unpermute_backward(const PermuteArgs& a, hipStream_t stream) {
  const int size = a.bf16 ? 2 : 4;
  const int pieces = (int)((a.H + 16 / size - 1) / (16 / size));
  const bool al16 = rows16(a.tokens, a.ldt, size) && rows16(a.sorted, a.lds, size) && rows16(a.out_sorted, a.ldo, size);
  by_type(a, al16, [&](auto el, auto al, auto past) {
    using El = decltype(el);
    auto go = [&](auto kern, int tokens) {
      hipLaunchKernelGGL(kern, dim3((unsigned)((a.T + tokens - 1) / tokens)), dim3(kRowThreads), 0, stream,
                         (const El*)a.tokens, a.ldt, a.T, (int)a.H, pieces, (int)a.topk, (int)(a.T * a.topk), a.rows, a.kept,
                         (const El*)a.sorted, a.lds, a.weights, (El*)a.out_sorted, a.ldo, a.dweights);
    };
    // Few tokens: four waves for each, or most of the chip would idle.
    if (a.T < 2048) go(unpermute_backward_kernel<El, decltype(al)::value, decltype(past)::value, 4>, 1);
    else go(unpermute_backward_kernel<El, decltype(al)::value, decltype(past)::value, 1>, 4);
  });
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace mxfp8
