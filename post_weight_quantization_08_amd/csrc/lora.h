// What the adapters' kernels and the 4-bit projection with adapters share.
#pragma once

#include "answer.h"

namespace gq {

// Adapters as a kernel takes them; T is fp32 [M][rp], rp = the rank padded to 8.
struct LoraFew {
  const uint16_t* X;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const int32_t* adapter;
  float* T;
  int64_t ld_x, M, d_out;
  int d_in, rank, n, rp;
};

template <int kDt>
__device__ __forceinline__ float lo16(uint32_t w) {
  if constexpr (kDt == GPTQ_F16) return f16_bits_to_f32(w & 0xFFFFu);
  else return __uint_as_float(w << 16);
}
template <int kDt>
__device__ __forceinline__ float hi16(uint32_t w) {
  if constexpr (kDt == GPTQ_F16) return f16_bits_to_f32(w >> 16);
  else return __uint_as_float(w & 0xFFFF0000u);
}

template <int kDt>
__device__ __forceinline__ f32x4 mfma_16x16x32(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (kDt == GPTQ_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}

// 8 elements from any address.
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  u32x4 w;
  __builtin_memcpy(&w, __builtin_assume_aligned(p, 2), 16);
  return w;
}

// Elements k .. k + 7 of a row of n elements, zero behind its end.
__device__ __forceinline__ u32x4 load8_end(const uint16_t* row, int k, int n) {
  if (k + 8 <= n) return load8(row + k);
  u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < n) w[i / 2] |= (uint32_t)row[k + i] << (16 * (i & 1));
  return w;
}

// T[m][r] = s_a X[m] . A_a[r] for (m, r) number `at`, by one wave.
template <int kDt>
__device__ __forceinline__ void lora_down_one(const LoraFew& a, int64_t at) {
  const int lane = threadIdx.x & 63;
  if (at >= a.M * a.rank) return;
  const int64_t m = at / a.rank;
  const int r = (int)(at - m * a.rank);
  const int ad = __builtin_amdgcn_readfirstlane(a.adapter[m]);
  if (ad < 0 || ad >= a.n) return;
  const uint16_t* x = a.X + m * a.ld_x;
  const uint16_t* f = a.A + ((int64_t)ad * a.rank + r) * a.d_in;
  float s0 = 0.f, s1 = 0.f;
  auto add = [&](u32x4 u, u32x4 v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s0 = fmaf(lo16<kDt>(u[i]), lo16<kDt>(v[i]), s0);
      s1 = fmaf(hi16<kDt>(u[i]), hi16<kDt>(v[i]), s1);
    }
  };
  constexpr int kU = 4;
  int k = 0;
  for (; k + 512 * kU <= a.d_in; k += 512 * kU) {
    u32x4 u[kU], v[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      u[i] = load8(x + k + i * 512 + lane * 8);
      v[i] = load8(f + k + i * 512 + lane * 8);
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) add(u[i], v[i]);
  }
  for (; k < a.d_in; k += 512) add(load8_end(x, k + lane * 8, a.d_in), load8_end(f, k + lane * 8, a.d_in));
  const float s = wave_reduce(s0 + s1, [](float p, float q) { return p + q; });
  if (lane == 0) a.T[m * a.rp + r] = (a.scale ? a.scale[ad] : 1.f) * s;
}

// T[m] . B_a[row], 8 ranks at a time in one fixed order.
template <int kDt>
__device__ __forceinline__ float lora_up_one(const LoraFew& a, int ad, int64_t m, int64_t row) {
  const uint16_t* b = a.B + ((int64_t)ad * a.d_out + row) * a.rank;
  const float* t = a.T + m * a.rp;
  float s = 0.f;
  for (int k = 0; k < a.rank; k += 8) {
    const u32x4 w = load8_end(b, k, a.rank);
    const f32x4 t0 = *reinterpret_cast<const f32x4*>(t + k), t1 = *reinterpret_cast<const f32x4*>(t + k + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // T's padding holds whatever the workspace held
      const float u = e < 2 ? t0[2 * e] : t1[2 * e - 4], v = e < 2 ? t0[2 * e + 1] : t1[2 * e - 3];
      s = fmaf(k + 2 * e < a.rank ? u : 0.f, lo16<kDt>(w[e]), s);
      s = fmaf(k + 2 * e + 1 < a.rank ? v : 0.f, hi16<kDt>(w[e]), s);
    }
  }
  return s;
}

// y += the same for tokens m .. m + 3 of their own adapters, its loads asked
// for together: without a branch, at a token or an adapter that is there, and
// not used where none acts.
template <int kDt>
__device__ __forceinline__ void lora_up_four(const LoraFew& a, int m, int64_t row, f32x4& y) {
  const int64_t at = row < a.d_out ? row : a.d_out - 1;
  const uint16_t* b[4];
  const float* t[4];
  bool acts[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int tok = m + r < a.M ? m + r : (int)a.M - 1;
    const int ad = a.adapter[tok];
    acts[r] = ad >= 0 && ad < a.n;
    b[r] = a.B + ((int64_t)(acts[r] ? ad : 0) * a.d_out + at) * a.rank;
    t[r] = a.T + (int64_t)tok * a.rp;
  }
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < a.rank; k += 8) {
    u32x4 w[4];
    f32x4 t0[4], t1[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      w[r] = load8_end(b[r], k, a.rank);
      t0[r] = *reinterpret_cast<const f32x4*>(t[r] + k);
      t1[r] = *reinterpret_cast<const f32x4*>(t[r] + k + 4);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = e < 2 ? t0[r][2 * e] : t1[r][2 * e - 4], v = e < 2 ? t0[r][2 * e + 1] : t1[r][2 * e - 3];
        s[r] = fmaf(k + 2 * e < a.rank ? u : 0.f, lo16<kDt>(w[r][e]), s[r]);
        s[r] = fmaf(k + 2 * e + 1 < a.rank ? v : 0.f, hi16<kDt>(w[r][e]), s[r]);
      }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) y[r] = acts[r] ? y[r] + s[r] : y[r];
}

// The 4-bit projection (arguments as gptq_w4a16_matmul's), with adapters when
// `lora` is given; in w4a16.hip.
gptq_status w4a16_run(const void* X, int32_t x_dtype, int64_t M, int64_t d_in, int64_t ld_x, const uint8_t* qweight,
                      const uint16_t* scales, const uint8_t* zeros, const int32_t* perm, int64_t d_out,
                      int32_t group_size, float* Y, int64_t ld_y, void* workspace, size_t ws_bytes, const LoraFew* lora,
                      hipStream_t st);

}  // namespace gq
