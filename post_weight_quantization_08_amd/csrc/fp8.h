// Numbers in 8 bits: e4m3 codes (four significant bits, largest 448) with one
// power-of-two scale, an E8M0 byte b standing for 2^(b - 127), for each block of
// 128 along the sum of a product.  A power of two makes the scaling exact: the
// codes are one rounding of the values, they return to bf16 without another, and
// the matrix unit applies the bytes by itself.
#pragma once

#include "lora.h"

namespace gq {

constexpr int kF8Block = 128;

// The scale of a block whose largest magnitude has the fp32 bits `top` (sign
// off): the smallest power of two, at least 2^-100, that brings it to 448 =
// 1.75 * 2^8 or less; 255 (NaN) where the block holds a NaN or an infinity.
__device__ __forceinline__ uint32_t f8_scale(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  return (uint32_t)max((int)((top + 0x1FFFFFu) >> 23) - 8, 27);
}
// 2^(127 - b), what values are multiplied with before they are rounded.
__device__ __forceinline__ float f8_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Four codes; rounded to nearest even.  255: NaN.
__device__ __forceinline__ uint32_t f8_codes4(float x0, float x1, float x2, float x3, uint32_t b) {
  const float f = f8_inverse(b);
  int p = __builtin_amdgcn_cvt_pk_fp8_f32(x0 * f, x1 * f, 0, false);
  p = __builtin_amdgcn_cvt_pk_fp8_f32(x2 * f, x3 * f, p, true);
  return b == 255u ? 0x7F7F7F7Fu : (uint32_t)p;
}

// Elements k .. k + 7 of a row of n in fp32, zero behind its end.
template <int kDt>
__device__ __forceinline__ void f8_load8(const void* row, int k, int n, float (&v)[8]) {
  if constexpr (kDt == GPTQ_F32) {
    const float* p = static_cast<const float*>(row);
    if (k + 8 <= n) {
      f32x4 w[2];
      __builtin_memcpy(w, __builtin_assume_aligned(p + k, 4), 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = w[i / 4][i % 4];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k + i < n ? p[k + i] : 0.f;
    }
  } else {
    const u32x4 w = load8_end(static_cast<const uint16_t*>(row), k, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = lo16<kDt>(w[i]);
      v[2 * i + 1] = hi16<kDt>(w[i]);
    }
  }
}

// The largest magnitude's bits: as numbers they order as the magnitudes do, an
// infinity above all finite ones and NaN above it.
__device__ __forceinline__ uint32_t f8_top8(const float (&v)[8]) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return t;
}

inline size_t f8_elem(int dtype) { return dtype == GPTQ_F32 ? 4 : dtype == GPTQ_E4M3 ? 1 : 2; }

// A launch has fewer than 2^32 threads, the quantizing one 256 for every 64 blocks.
constexpr int64_t kF8MostBlocks = ((int64_t)1 << 30) - 64;

// Rows, of kF8MostBlocks blocks at most, into codes of `cols` padded to whole blocks and scales [rows][blocks];
// in fp8_quantize.hip.
void f8_quantize_rows(const void* X, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* codes,
                      int64_t ld_c, uint8_t* scales, hipStream_t st);

}  // namespace gq
