// Gradients of low-rank adapters:  Y[m] = base[m] + s_a (X[m] A_a^T) B_a^T, a = adapter[m].
//   U[m] = s_a dY[m] B_a,  T[m] = s_a X[m] A_a^T           (rank numbers a token)
//   dA_a = sum_m U[m]^T X[m],  dB_a = sum_m dY[m]^T T[m],  dX[m] = base[m] + U[m] A_a
// over the tokens of adapter a.
//
// Launches: parts of U and T, with the tokens sorted by adapter beside them (project);
// U and T added up and laid out for what follows (terms); the sums over tokens (outer);
// their parts joined where an adapter has many tokens; dX.
//
// Sums are fp32 and keep 24 bits of everything in them.  Where 16-bit numbers meet,
// that is one product.  U, T and fp32 dY are three bf16 terms, fp16 beside them two,
// e4m3 with its scale one (exact); of their products those are taken whose size is
// 2^-16 of the largest or more.
//
// 8192 tokens, 11008 -> 4096, 64 ranks, codes and bf16, with dX: 235 us, of them project
// 65 (2.4 TB/s), terms 14, outer 67, join 6, dX 97 (3.7 TB/s).  2048 tokens of eight
// adapters of 16 ranks, 4096 -> 14336, fp16: 91 us (29, 8, 30, 5, 15).  96 tokens, 8 ranks:
// 17 us in three launches, each a chain of a few loads.
//
// The sums over tokens want eight consecutive tokens of a column in a lane.  Every lane
// loads eight columns of eight tokens and turns them in registers, which needs no LDS
// and works for every type.
#pragma once

#include "fp8.h"

namespace gq {

constexpr int kGradTile = 32;       // tokens of a step
constexpr int kGradMaxRank = 128;
constexpr int kGradMaxAdapters = 1024;

// A run of sorted tokens that one workgroup sums up.
struct GradChunk {
  int adapter, begin, end;          // positions
  int slot;                         // where its part goes, or -1: the only part
};

struct GradPlace {                  // what the sort writes
  int32_t* order;                   // [P]: the token at a position; ~token where it fills a run up to 32;
                                    // tokens without an adapter behind the runs
  GradChunk* chunks;
  int32_t* parts;                   // [n][2]: an adapter's first slot and its parts
  int32_t* count;                   // [3]: chunks, positions of the runs, of all
};

// One operand: rows of X with A, or rows of dY with B.
struct GradSide {
  const void* D;
  const uint8_t* scales;            // [M][nb], e4m3
  int64_t ld;
  int K, nb;
  const uint16_t* F;                // A [n][rank][K] or B [n][K][rank]
  int splits, per;                  // parts of the sum, and their blocks of 128
  float* sums;                      // [splits][M][rp]
  uint16_t* flat;                   // bf16 [3][P][rk]: U for dX, or null
  uint16_t* turned;                 // bf16 [3][r16][P]: what this side's product gives
  const uint16_t* by;               // the other side's, which its sum over tokens takes
  float* grad;                      // [n][rank * K]
  float* part;                      // [slots][rank * K]
  int blocks;                       // of 256 columns
};

struct GradArgs {
  GradSide side[2];
  GradPlace at;
  const int32_t* adapter;
  const float* scale;
  const void* base;                 // dX = base + U A
  void* dX;
  int64_t ld_b, ld_dx;
  int wide_dx;                      // dX and base are fp32
  int64_t M, P;
  int n, rank, rp, r16, rk;         // rank padded to 8, to tiles of 16, to steps of 32
  int chunk;
  int input_tokens;                 // of a workgroup, for dX
  int groups;                       // of four token tiles
  int halves;                       // of the ranks: more than 64 are taken 64 at a time
};

// Eight numbers of a row as loaded.
template <int kD>
struct Eight {
  static constexpr int kTerms = kD == GPTQ_F32 ? 3 : kD == GPTQ_F16 ? 2 : 1;   // bf16 terms
  static constexpr int kWords = kD == GPTQ_F32 ? 8 : kD == GPTQ_E4M3 ? 2 : 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* row, int k) {
    if constexpr (kD == GPTQ_E4M3) {
      __builtin_memcpy(w, __builtin_assume_aligned(static_cast<const uint8_t*>(row) + k, 8), 8);
    } else if constexpr (kD == GPTQ_F32) {
      __builtin_memcpy(w, __builtin_assume_aligned(static_cast<const float*>(row) + k, 4), 32);
    } else {
      __builtin_memcpy(w, __builtin_assume_aligned(static_cast<const uint16_t*>(row) + k, 2), 16);
    }
  }
  // zero behind the row's end.  Where a row ends inside eight its last numbers are loaded one by
  // one, and the compiler waits for each: 8192 x 11001 -> 4093, codes, 64 ranks 401 us, 11008 ->
  // 4096 236.
  __device__ __forceinline__ void load_end(const void* row, int k, int n) {
    if (k + 8 <= n) {
      load(row, k);
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (k + i >= n) continue;
      if constexpr (kD == GPTQ_E4M3) w[i / 4] |= (uint32_t) static_cast<const uint8_t*>(row)[k + i] << (8 * (i & 3));
      else if constexpr (kD == GPTQ_F32) w[i] = static_cast<const uint32_t*>(row)[k + i];
      else w[i / 2] |= (uint32_t) static_cast<const uint16_t*>(row)[k + i] << (16 * (i & 1));
    }
  }
  // numbers 2 i and 2 i + 1 as bf16, the largest term first; `s` is the scale of codes
  __device__ __forceinline__ void pair(int i, float s, uint32_t (&t)[kTerms]) const {
    if constexpr (kD == GPTQ_E4M3) {
      t[0] = i % 2 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i / 2], s, true))
                   : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i / 2], s, false));
    } else if constexpr (kD == GPTQ_BF16) {
      t[0] = w[i];
    } else {
      float x, y;
      if constexpr (kD == GPTQ_F16) {
        x = lo16<GPTQ_F16>(w[i]);
        y = hi16<GPTQ_F16>(w[i]);
      } else {
        x = __uint_as_float(w[2 * i]);
        y = __uint_as_float(w[2 * i + 1]);
      }
#pragma unroll
      for (int k = 0; k < kTerms; ++k) {
        t[k] = value_bits<GPTQ_BF16>(x) | value_bits<GPTQ_BF16>(y) << 16;
        if (k + 1 < kTerms) {
          x -= __uint_as_float(t[k] << 16);
          y -= __uint_as_float(t[k] & 0xFFFF0000u);
        }
      }
    }
  }
  __device__ __forceinline__ void terms(float s, u32x4 (&t)[kTerms]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t p[kTerms];
      pair(i, s, p);
#pragma unroll
      for (int k = 0; k < kTerms; ++k) t[k][i] = p[k];
    }
  }
  // codes as fp16, without the scale
  __device__ __forceinline__ u32x4 half() const {
    u32x4 t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      t[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.f, false));
      t[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.f, true));
    }
    return t;
  }
};

template <int kD>
__device__ __forceinline__ const char* grad_row(const GradSide& s, int64_t m) {
  return static_cast<const char*>(s.D) + m * s.ld * (kD == GPTQ_F32 ? 4 : kD == GPTQ_E4M3 ? 1 : 2);
}

__device__ __forceinline__ float grad_scale(uint32_t b) { return __uint_as_float(b << 23); }

// acc += the products of bf16 terms whose order is above 2^-24, the smallest first.
template <int kA, int kB>
__device__ __forceinline__ f32x4 grad_mfma(const u32x4 (&a)[kA], const u32x4 (&b)[kB], f32x4 acc) {
#pragma unroll
  for (int o = 2; o >= 0; --o)
#pragma unroll
    for (int i = 0; i < kA; ++i)
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (i + j == o) acc = mfma_16x16x32<GPTQ_BF16>(a[i], b[j], acc);
  return acc;
}

// The launches that depend on the types; in lora_grad_f16.hip and lora_grad_bf16.hip,
// for factors of either type.  codes: X is e4m3; wide: dY is fp32.
enum GradStage { kGradProject, kGradOuter, kGradInput };
void grad_launch_f16(const GradArgs& a, bool codes, bool wide, int64_t max_chunks, GradStage stage, hipStream_t st);
void grad_launch_bf16(const GradArgs& a, bool codes, bool wide, int64_t max_chunks, GradStage stage, hipStream_t st);

}  // namespace gq
