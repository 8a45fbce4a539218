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

// An element's bits as they are, and their value.
template <int kDt>
__device__ __forceinline__ uint32_t load_bits(const void* p, int64_t i) {
  if constexpr (kDt == GPTQ_F32) return static_cast<const uint32_t*>(p)[i];
  else return static_cast<const uint16_t*>(p)[i];
}
template <int kDt>
__device__ __forceinline__ float bits_value(uint32_t b) {
  if constexpr (kDt == GPTQ_F32) return __uint_as_float(b);
  else if constexpr (kDt == GPTQ_BF16) return bf16_bits_to_f32(b);
  else return f16_bits_to_f32(b);
}
// A value's bits, rounded to nearest even; NaN stays NaN.
template <int kDt>
__device__ __forceinline__ uint32_t value_bits(float v) {
  if constexpr (kDt == GPTQ_F32) return __float_as_uint(v);
  else if constexpr (kDt == GPTQ_F16) return __builtin_bit_cast(uint16_t, (_Float16)v);
  else return __builtin_bit_cast(uint16_t, (__bf16)v);
}
template <int kDt>
__device__ __forceinline__ void store_bits(void* p, int64_t i, uint32_t b) {
  if constexpr (kDt == GPTQ_F32) static_cast<uint32_t*>(p)[i] = b;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)b;
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

// ---------------------------------------------------------------- rows in blocks
// A row is walked in 16-byte blocks on 16-byte addresses, wherever it starts:
// block b holds elements b E - h .. b E - h + E - 1, E elements of a block, h
// the elements between the boundary below the row's start and that start.
// Blocks that stick out of the row (at most the first and the last) are read
// element by element, so nothing outside the row is touched.
template <int kDt>
struct Blocks {
  static constexpr int E = kDt == GPTQ_F32 ? 4 : 8;
  const char* p0;   // address of block 0 (at most 15 bytes before the row)
  int h, vocab, n;  // elements before the row, elements, blocks

  __device__ __forceinline__ Blocks(const void* x, int64_t row, int64_t ld, int v) {
    constexpr int es = 16 / E;
    const char* p = static_cast<const char*>(x) + row * ld * es;
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    p0 = p - off;
    h = off / es;
    vocab = v;
    n = (h + v + E - 1) / E;
  }
  // blocks [first_whole(), end_whole()) lie inside the row
  __device__ __forceinline__ int first_whole() const { return h > 0 ? 1 : 0; }
  __device__ __forceinline__ int end_whole() const { return (h + vocab) / E; }
  __device__ __forceinline__ int element(int b, int e) const { return b * E - h + e; }

  __device__ __forceinline__ u32x4 load(int b) const {
    return *reinterpret_cast<const u32x4*>(p0 + (int64_t)b * 16);
  }
  static __device__ __forceinline__ void unpack(u32x4 w, float (&v)[E]) {
    if constexpr (kDt == GPTQ_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (kDt == GPTQ_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = f16_bits_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = f16_bits_to_f32(w[i] >> 16);
      }
    }
  }
  // any block; elements outside the row (and whole blocks outside) come as -inf
  __device__ __forceinline__ void fetch(int b, float (&v)[E]) const {
    if (b >= first_whole() && b < end_whole()) {
      unpack(load(b), v);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int j = element(b, e);
        v[e] = j >= 0 && j < vocab ? load_el<kDt>(p0, (int64_t)b * E + e) : -INFINITY;
      }
    }
  }
};

// 2^x by the hardware's instruction (one unit in the last place; results below
// the normal range are zero).
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// A barrier that waits for LDS only: loads and stores of global memory stay in
// flight across it.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 64 lanes' 16 (4) bytes each, one after the other from `to` on.
__device__ __forceinline__ void lds_load16(const void* from, char* to) {
  __builtin_amdgcn_global_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
__device__ __forceinline__ void lds_load4(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds(from, (__attribute__((address_space(3))) void*)to, 4, 0, 0);
}

// A value that is the same in every lane, kept in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}
template <int kCtrl>
__device__ __forceinline__ float dpp_move(float v) {
  return __uint_as_float(dpp_move<kCtrl>(__float_as_uint(v)));
}
template <int kCtrl>
__device__ __forceinline__ double dpp_move(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t m = (uint64_t)dpp_move<kCtrl>((uint32_t)(b >> 32)) << 32 | dpp_move<kCtrl>((uint32_t)b);
  return __builtin_bit_cast(double, m);
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t m = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  return __builtin_bit_cast(double, m);
}

// f over each 16 lanes, in all of them: exchanges within quads, then mirrored
// eights and sixteens (data-parallel moves, no LDS).  All lanes are active.
template <class T, class F>
__device__ __forceinline__ T row_reduce(T v, F f) {
  v = f(v, dpp_move<0xB1>(v));    // lanes 1 0 3 2
  v = f(v, dpp_move<0x4E>(v));    // lanes 2 3 0 1
  v = f(v, dpp_move<0x141>(v));   // eights mirrored
  return f(v, dpp_move<0x140>(v));   // sixteens mirrored
}

// f over the wave, the same value in every lane.
template <class T, class F>
__device__ __forceinline__ T wave_reduce(T v, F f) {
  v = row_reduce(v, f);
  return f(f(lane_value(v, 0), lane_value(v, 16)), f(lane_value(v, 32), lane_value(v, 48)));
}

// ---------------------------------------------------------------- running sums
// S = sum 2^((x - r) c) and U = sum 2^((x - r) c) (x - r) c over what was seen,
// r some reference near the maximum.  c = log2(e) / T.
struct Sums {
  float r, s, u;
};

// The sums moved to the reference `to` (>= r up to rounding).
__device__ __forceinline__ Sums moved(Sums a, float to, float c) {
  const float d = fmaxf((a.r - to) * c, -1e30f);   // finite, so that 0 * d is 0
  const float f = exp2_hw(d);
  return Sums{to, a.s * f, f * fmaf(d, a.s, a.u)};
}

}  // namespace gq
