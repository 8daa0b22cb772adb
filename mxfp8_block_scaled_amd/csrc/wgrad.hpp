// Device code that the two forms of the weight gradient share.
#pragma once

#include "b128.hpp"
#include "tile_core.hpp"

namespace mxfp8 {
namespace wgrad {

constexpr int kWgThreads = 256;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ inline int slot_xor(int m) { return (m & 3) | ((m >> 1) & 4); }

// Stores two neighbouring 16-wide fragments along k of one n (lane (i, g)
// holds k = 4 g .. + 3 of each) as bf16: exchanging the odd 16-lane rows of
// the first with the even ones of the second gives a lane eight consecutive k,
// k_of_pair(g) from the first fragment's start on.  Half the stores of 8-byte
// pieces and whole 64-byte runs: 42 -> 34 us at 67 x 7640 x 5888.
__device__ inline int k_of_pair(int g) { return 16 * (g & 1) + 8 * (g >> 1); }
__device__ inline void store_pair(const v4f& lo, const v4f& hi, bool in, uint16_t* to) {
  const auto s0 = __builtin_amdgcn_permlane16_swap(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(hi[0], hi[1]), false, false);
  const auto s1 = __builtin_amdgcn_permlane16_swap(pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[2], hi[3]), false, false);
  if (in) *reinterpret_cast<uint4*>(to) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
}

__device__ inline void store_db(void* db, int bf16, int accumulate, int64_t n, float v) {
  if (bf16) ((uint16_t*)db)[n] = (uint16_t)pack_bf16x2(v, 0.0f);
  else ((float*)db)[n] = accumulate ? ((float*)db)[n] + v : v;
}

}  // namespace wgrad
}  // namespace mxfp8
