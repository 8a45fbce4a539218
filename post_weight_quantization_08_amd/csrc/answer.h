// Helpers of the kernels that read rows of logits.
#pragma once

#include "common.h"

namespace gq {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

template <int kDt>
__device__ __forceinline__ float load_el(const void* p, int64_t i) {
  if constexpr (kDt == GPTQ_F32) return static_cast<const float*>(p)[i];
  else if constexpr (kDt == GPTQ_F16) return f16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// Rounded once, to nearest even; NaN stays NaN.
template <int kDt>
__device__ __forceinline__ void store_el(void* p, int64_t i, float v) {
  if constexpr (kDt == GPTQ_F32) static_cast<float*>(p)[i] = v;
  else if constexpr (kDt == GPTQ_F16) static_cast<_Float16*>(p)[i] = (_Float16)v;
  else static_cast<__bf16*>(p)[i] = (__bf16)v;
}

// A float's place in the order of the top lists: larger value, larger number;
// -0 counts as +0, every NaN as the largest value.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t o) {
  if (o == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// Order of (value, index): ties go to the lower index.  Unique in a row.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  return (uint64_t)order_of(x) << 32 | (0xFFFFFFFFu - index);
}

__device__ __forceinline__ uint32_t index_of(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

}  // namespace gq
