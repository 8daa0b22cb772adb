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

__device__ inline void store_db(void* db, int bf16, int accumulate, int64_t n, float v) {
  if (bf16) ((uint16_t*)db)[n] = (uint16_t)pack_bf16x2(v, 0.0f);
  else ((float*)db)[n] = accumulate ? ((float*)db)[n] + v : v;
}

}  // namespace wgrad
}  // namespace mxfp8
