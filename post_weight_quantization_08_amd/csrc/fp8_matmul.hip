// Product of 8-bit operands with a power-of-two scale for each block of 128:
//   Y[m][n] = sum_b 2^(sx[m][b] - 127) 2^(sw[n / 128][b] - 127) sum_{k in b} x[m][k] w[n][k].
//
// 16-bit outputs: one instruction, 16x16x128 on e4m3 with a scale byte per lane and
// operand, does a block of 16 x 16 outputs: the scales cost nothing and the sums
// stay in its fp32 accumulators from the first block to the last.  It adds the
// products of eight consecutive codes after cutting each off at 2^-13 of the largest
// one's exponent (measured with single products; sums across eights keep 24 bits), an
// error of about 3e-5 of a result, far below half a step of a 16-bit output.
// fp32 outputs promise more than that: their codes become bf16 together with the
// scales, exactly, and go through 16x16x32 bf16 products at half the rate.
//
// A lane holds 32 codes of one row; which 32 of the block's 128 does not matter as
// long as both operands agree (here units q and q + 4 of 16 bytes, q = lane / 16).
// The weights are the rows of the result, so that a lane ends up with four
// consecutive outputs of one token.
#include "fp8.h"

namespace gq {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct F8MmArgs {
  const void* X;           // codes, or values
  const uint8_t* xs;       // [M][nb], with codes
  const uint8_t* W;
  const uint8_t* ws;       // [d_out / 128][nb]
  void* Y;
  float* part;             // [splits][M][d_out] where the sum is split
  int64_t ld_x, ld_w, ld_y, M, d_out;
  int d_in, nb;
  int splits, nb_split;    // parts of the sum, and their blocks
  int tiles_m, tiles_n;
};

__device__ __forceinline__ f32x4 f8_mfma(i32x8 w, i32x8 x, f32x4 c, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, (int)sw, 0, (int)sx);
}

__device__ __forceinline__ i32x8 f8_frag(u32x4 lo, u32x4 hi) {
  i32x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = (int)lo[i];
    r[i + 4] = (int)hi[i];
  }
  return r;
}

// Eight codes as bf16, scaled: an operand of a 16x16x32 product.  Exact: four
// significant bits and a power of two.
__device__ __forceinline__ u32x4 f8_wide(uint32_t c0, uint32_t c1, uint32_t b) {
  const float s = __uint_as_float(b << 23);
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, s, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, s, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, s, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, s, true));
  return r;
}

// acc[r][t] += one unit (16 codes a lane) of kR row tiles and kT token tiles, in bf16.
template <int kR, int kT>
__device__ __forceinline__ void f8_wide_unit(const u32x4 (&w)[kR], const u32x4 (&x)[kT], const uint32_t (&sw)[kR],
                                             const uint32_t (&sx)[kT], f32x4 (&acc)[kR][kT]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    u32x4 xw[kT];
#pragma unroll
    for (int t = 0; t < kT; ++t) xw[t] = f8_wide(x[t][2 * h], x[t][2 * h + 1], sx[t]);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const u32x4 ww = f8_wide(w[r][2 * h], w[r][2 * h + 1], sw[r]);
#pragma unroll
      for (int t = 0; t < kT; ++t) acc[r][t] = mfma_16x16x32<GPTQ_BF16>(ww, xw[t], acc[r][t]);
    }
  }
}

// Four consecutive outputs of token m from column n on.
template <int kY>
__device__ __forceinline__ void f8_store4(void* Y, int64_t at, int64_t left, f32x4 v) {
  if (left >= 4) {
    if constexpr (kY == GPTQ_F32) {
      __builtin_memcpy(__builtin_assume_aligned(static_cast<float*>(Y) + at, 4), &v, 16);
    } else {
      const uint2 w = {value_bits<kY>(v[0]) | value_bits<kY>(v[1]) << 16, value_bits<kY>(v[2]) | value_bits<kY>(v[3]) << 16};
      __builtin_memcpy(__builtin_assume_aligned(static_cast<uint16_t*>(Y) + at, 2), &w, 8);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) store_el<kY>(Y, at + i, v[i]);
  }
}

// ---------------------------------------------------------------- few tokens
// 16 kR rows of weights by 16 kT tokens; the waves take the sum's blocks in turn,
// straight from memory, and their sums meet in LDS.
template <int kX, int kY, int kT, int kR, int kU>
__global__ __launch_bounds__(512) void fp8_few_kernel(F8MmArgs a) {
  constexpr int kW = 8;
  constexpr int kPitch = kR * 16 + 4;
  __shared__ __align__(16) float red[kW][kT * 16][kPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * kR);
  const uint8_t* w[kR];
  const uint8_t* sw[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int64_t first = n0 + r * 16, row = first + c16;
    w[r] = a.W + (row < a.d_out ? row : a.d_out - 1) * a.ld_w + q * 16;
    sw[r] = a.ws + (first < a.d_out ? first : a.d_out - 1) / kF8Block * a.nb;
  }
  const char* x[kT];
  const uint8_t* sx[kT];
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    const int64_t m = t * 16 + c16 < a.M ? t * 16 + c16 : a.M - 1;
    x[t] = static_cast<const char*>(a.X) + m * a.ld_x * (kX == GPTQ_F32 ? 4 : kX == GPTQ_E4M3 ? 1 : 2);
    sx[t] = kX == GPTQ_E4M3 ? a.xs + m * a.nb : nullptr;
  }
  f32x4 acc[kR][kT];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < kT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Step {
    u32x4 w[2][kR], x[2][kT];              // [unit]
    uint32_t sw[kR], sx[kT];
    float v[kX == GPTQ_E4M3 ? 1 : kT][kX == GPTQ_E4M3 ? 1 : 4][8];
  };
  auto read = [&](int b, Step& s) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      s.w[0][r] = *reinterpret_cast<const u32x4*>(w[r] + b * kF8Block);
      s.w[1][r] = *reinterpret_cast<const u32x4*>(w[r] + b * kF8Block + 64);
      s.sw[r] = sw[r][b];
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      if constexpr (kX == GPTQ_E4M3) {
        s.x[0][t] = *reinterpret_cast<const u32x4*>(x[t] + b * kF8Block + q * 16);
        s.x[1][t] = *reinterpret_cast<const u32x4*>(x[t] + b * kF8Block + q * 16 + 64);
        s.sx[t] = sx[t][b];
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          // lanes without a token quantize nothing
          if (t * 16 + c16 < a.M) f8_load8<kX>(x[t], b * kF8Block + q * 16 + (h / 2) * 64 + (h % 2) * 8, a.d_in, s.v[t][h]);
          else
#pragma unroll
            for (int e = 0; e < 8; ++e) s.v[t][h][e] = 0.f;
        }
      }
    }
  };
  auto multiply = [&](Step& s) {
    if constexpr (kX != GPTQ_E4M3) {
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        uint32_t top = max(max(f8_top8(s.v[t][0]), f8_top8(s.v[t][1])), max(f8_top8(s.v[t][2]), f8_top8(s.v[t][3])));
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        s.sx[t] = f8_scale(top);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const auto& v = s.v[t][h];
          s.x[h / 2][t][(h % 2) * 2] = f8_codes4(v[0], v[1], v[2], v[3], s.sx[t]);
          s.x[h / 2][t][(h % 2) * 2 + 1] = f8_codes4(v[4], v[5], v[6], v[7], s.sx[t]);
        }
      }
    }
    if constexpr (kY == GPTQ_F32) {
#pragma unroll
      for (int u = 0; u < 2; ++u) f8_wide_unit<kR, kT>(s.w[u], s.x[u], s.sw, s.sx, acc);
    } else {
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int t = 0; t < kT; ++t)
          acc[r][t] = f8_mfma(f8_frag(s.w[0][r], s.w[1][r]), f8_frag(s.x[0][t], s.x[1][t]), acc[r][t], s.sw[r], s.sx[t]);
    }
  };
  // kU blocks' operands are asked for together
  int b = wave;
  for (; b + (kU - 1) * kW < a.nb; b += kU * kW) {
    Step s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) read(b + u * kW, s[u]);
#pragma unroll
    for (int u = 0; u < kU; ++u) multiply(s[u]);
  }
  for (; b < a.nb; b += kW) {
    Step s;
    read(b, s);
    multiply(s);
  }
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < kT; ++t) *reinterpret_cast<f32x4*>(&red[wave][t * 16 + c16][r * 16 + 4 * q]) = acc[r][t];
  __syncthreads();
  for (int i = threadIdx.x; i < kT * 16 * kR * 4; i += 512) {
    const int m = i / (kR * 4), n = i % (kR * 4) * 4;
    if (m >= a.M || n0 + n >= a.d_out) continue;
    f32x4 v = *reinterpret_cast<const f32x4*>(&red[0][m][n]);
#pragma unroll
    for (int u = 1; u < kW; ++u) v += *reinterpret_cast<const f32x4*>(&red[u][m][n]);
    f8_store4<kY>(a.Y, m * a.ld_y + n0 + n, a.d_out - n0 - n, v);
  }
}

// ---------------------------------------------------------------- many tokens
// Workgroup number -> (token tile, weight tile, part).  Workgroups go to the
// eight XCDs in turn; each gets a run of tiles, walked in bands of eight token
// tiles, so that what runs on it at one time reads few panels through its L2.
__device__ __forceinline__ void f8_place(const F8MmArgs& a, int& tm, int& tn, int& part) {
  const int total = a.tiles_m * a.tiles_n * a.splits;
  const int per = total / 8;
  int id = blockIdx.x;
  if (id < per * 8) id = id % 8 * per + id / 8;
  const int tiles = a.tiles_m * a.tiles_n;
  part = id / tiles;
  id -= part * tiles;
  const int band = id / (8 * a.tiles_n);
  const int height = min(8, a.tiles_m - band * 8);
  id -= band * 8 * a.tiles_n;
  tn = id / height;
  tm = band * 8 + id % height;
}

// kBM tokens by kBN rows of weights, kWM x kWN waves; a stage is one block of
// 128 of every row, straight from memory into LDS.  Unit u (16 bytes) of row r lies at
// slot u ^ (r / 2 % 8): the sixteen rows of a fragment's unit then cover all banks
// once.
template <int kY, int kBM, int kBN, int kWM, int kWN>
__global__ __launch_bounds__(64 * kWM * kWN) void fp8_tile_kernel(F8MmArgs a) {
  constexpr int kWaves = kWM * kWN;
  constexpr int kRows = kBM + kBN;
  constexpr int kStage = kRows * kF8Block;
  constexpr int kLoads = kRows / 8 / kWaves;           // direct loads of a wave per stage, eight rows each
  constexpr int kT = kBM / kWM / 16, kR = kBN / kWN / 16;
  static_assert(kRows % (8 * kWaves) == 0 && kBM % (8 * kWaves) == 0, "a load is of one operand");
  __shared__ __attribute__((aligned(1024))) char x0[kStage], x1[kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  int tm, tn, part;
  f8_place(a, tm, tn, part);
  const int64_t m0 = (int64_t)tm * kBM, n0 = (int64_t)tn * kBN;
  const int b0 = part * a.nb_split, b1 = min(b0 + a.nb_split, a.nb);
  // this lane's part of load i: row 8 (wave + i kWaves) + lane / 8 of the stage (tokens first), slot lane % 8
  const uint8_t* src[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = 8 * (wave + i * kWaves) + (lane >> 3);
    const int unit = (lane & 7) ^ ((row >> 1) & 7);
    // rows behind the end read the last one and are never stored
    if (i * kWaves * 8 < kBM) src[i] = static_cast<const uint8_t*>(a.X) + min(m0 + row, a.M - 1) * a.ld_x + unit * 16;
    else src[i] = a.W + min(n0 + row - kBM, a.d_out - 1) * a.ld_w + unit * 16;
  }
  const int wm = wave / kWN, wn = wave % kWN;          // this wave's tokens and rows
  const uint8_t* sx[kT];
#pragma unroll
  for (int t = 0; t < kT; ++t) sx[t] = a.xs + min(m0 + wm * (kT * 16) + t * 16 + c16, a.M - 1) * a.nb;
  constexpr int kWide = kR * 16 > kF8Block ? kR * 16 / kF8Block : 1;   // tiles of 128 rows that a wave's rows touch
  const uint8_t* sw[kWide];
#pragma unroll
  for (int r = 0; r < kWide; ++r) sw[r] = a.ws + min(n0 + wn * (kR * 16) + r * kF8Block, a.d_out - 1) / kF8Block * a.nb;

  uint32_t bx[2][kT], bw[2][kWide];
  auto fetch = [&](int b, char* to, uint32_t (&ux)[kT], uint32_t (&uw)[kWide]) {
    const int at = min(b, b1 - 1);
#pragma unroll
    for (int t = 0; t < kT; ++t) ux[t] = sx[t][at];
#pragma unroll
    for (int r = 0; r < kWide; ++r) uw[r] = sw[r][at];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) lds_load16(src[i] + (int64_t)at * kF8Block, to + (wave + i * kWaves) * 1024);
  };
  f32x4 acc[kR][kT];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < kT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int slot0 = (q ^ ((c16 >> 1) & 7)) * 16, slot1 = slot0 ^ 64;   // unit q + 4 = q ^ 4
  const int at_x = (wm * (kT * 16) + c16) * kF8Block, at_w = (kBM + wn * (kR * 16) + c16) * kF8Block;
  auto multiply = [&](const char* from, const uint32_t (&ux)[kT], const uint32_t (&uw)[kWide]) {
    if constexpr (kY == GPTQ_F32) {
      uint32_t us[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) us[r] = uw[r * 16 / kF8Block];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        u32x4 xf[kT], wf[kR];
#pragma unroll
        for (int t = 0; t < kT; ++t)
          xf[t] = *reinterpret_cast<const u32x4*>(from + at_x + t * 16 * kF8Block + (u ? slot1 : slot0));
#pragma unroll
        for (int r = 0; r < kR; ++r)
          wf[r] = *reinterpret_cast<const u32x4*>(from + at_w + r * 16 * kF8Block + (u ? slot1 : slot0));
        f8_wide_unit<kR, kT>(wf, xf, us, ux, acc);
      }
      return;
    }
    i32x8 xf[kT];
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      const char* p = from + at_x + t * 16 * kF8Block;
      xf[t] = f8_frag(*reinterpret_cast<const u32x4*>(p + slot0), *reinterpret_cast<const u32x4*>(p + slot1));
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const char* p = from + at_w + r * 16 * kF8Block;
      const i32x8 wf = f8_frag(*reinterpret_cast<const u32x4*>(p + slot0), *reinterpret_cast<const u32x4*>(p + slot1));
#pragma unroll
      for (int t = 0; t < kT; ++t) acc[r][t] = f8_mfma(wf, xf[t], acc[r][t], uw[r * 16 / kF8Block], ux[t]);
    }
  };
  fetch(b0, x0, bx[0], bw[0]);
#define GQ_F8_STAGE(u, CUR, NEXT)                                         \
  {                                                                       \
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); \
    fetch(b + (u) + 1, NEXT, bx[1 - (u)], bw[1 - (u)]);                   \
    if (b + (u) < b1) multiply(CUR, bx[u], bw[u]);                        \
  }
  for (int b = b0; b < b1; b += 2) {
    GQ_F8_STAGE(0, x0, x1);
    GQ_F8_STAGE(1, x1, x0);
  }
#undef GQ_F8_STAGE
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");     // no direct load ends after the workgroup
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    const int64_t m = m0 + wm * (kT * 16) + t * 16 + c16;
    if (m >= a.M) continue;
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int64_t n = n0 + wn * (kR * 16) + r * 16 + 4 * q;
      if (n >= a.d_out) continue;
      if (a.splits > 1) f8_store4<GPTQ_F32>(a.part, ((int64_t)part * a.M + m) * a.d_out + n, a.d_out - n, acc[r][t]);
      else f8_store4<kY>(a.Y, m * a.ld_y + n, a.d_out - n, acc[r][t]);
    }
  }
}

// The parts of a split sum added up in order.
template <int kY>
__global__ __launch_bounds__(256) void fp8_join_kernel(F8MmArgs a) {
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, m = blockIdx.y;
  if (n >= a.d_out) return;
  const int64_t step = a.M * a.d_out, at = m * a.d_out + n, left = a.d_out - n;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < a.splits; ++p) {
    f32x4 w = {0.f, 0.f, 0.f, 0.f};
    if (left >= 4) {
      __builtin_memcpy(&w, __builtin_assume_aligned(a.part + p * step + at, 4), 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) w[i] = a.part[p * step + at + i];
    }
    v += w;
  }
  f8_store4<kY>(a.Y, m * a.ld_y + n, left, v);
}

constexpr int kF8Few = 64;          // tokens up to which weights go straight to the matrix units
constexpr int kF8Fused = 16;        // tokens up to which values are quantized beside the product

struct F8Plan {
  bool few, fused;
  int bm, bn, splits;
  size_t off_scales, off_part, total;
};

static F8Plan f8_plan(int64_t M, int64_t d_in, int64_t d_out, bool codes) {
  F8Plan p{};
  const int64_t nb = cdiv(d_in, kF8Block);
  p.few = M <= kF8Few;
  p.fused = !codes && M <= kF8Fused;
  if (!codes && !p.fused) {
    p.off_scales = align_up((size_t)M * nb * kF8Block, 256);
    p.total = align_up(p.off_scales + (size_t)M * nb, 256);
  }
  p.splits = 1;
  if (!p.few) {
    p.bm = p.bn = cdiv(M, 256) * cdiv(d_out, 256) >= 256 ? 256 : 128;
    if (p.bm == 128) {
      const int64_t tiles = cdiv(M, 128) * cdiv(d_out, 128);
      while (p.splits < 8 && tiles * p.splits < 256 && nb / (p.splits * 2) >= 8) p.splits *= 2;
    }
  }
  p.off_part = p.total;
  if (p.splits > 1) p.total += (size_t)p.splits * M * d_out * 4;
  return p;
}

size_t fp8_matmul_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out) {
  return f8_plan(M, d_in, d_out, false).total;
}

template <int kX, int kY, int kT, int kR, int kU>
static void f8_launch_few(const F8MmArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((fp8_few_kernel<kX, kY, kT, kR, kU>), dim3((unsigned)cdiv(a.d_out, 16 * kR)), dim3(512), 0, st, a);
}

template <int kY>
static void f8_run(F8MmArgs& a, int x_dtype, const F8Plan& p, hipStream_t st) {
  if (p.few) {
    if (x_dtype == GPTQ_F32) f8_launch_few<GPTQ_F32, kY, 1, 1, 2>(a, st);
    else if (x_dtype == GPTQ_F16) f8_launch_few<GPTQ_F16, kY, 1, 1, 2>(a, st);
    else if (x_dtype == GPTQ_BF16) f8_launch_few<GPTQ_BF16, kY, 1, 1, 2>(a, st);
    else if (a.M <= 16) f8_launch_few<GPTQ_E4M3, kY, 1, 1, 4>(a, st);
    else if (a.M <= 32) f8_launch_few<GPTQ_E4M3, kY, 2, 2, 2>(a, st);
    else f8_launch_few<GPTQ_E4M3, kY, 4, 2, 2>(a, st);
    return;
  }
  a.tiles_m = (int)cdiv(a.M, p.bm);
  a.tiles_n = (int)cdiv(a.d_out, p.bn);
  a.splits = p.splits;
  a.nb_split = (int)cdiv(a.nb, p.splits);
  const dim3 grid((unsigned)((int64_t)a.tiles_m * a.tiles_n * a.splits));
  if (p.bm == 256) hipLaunchKernelGGL((fp8_tile_kernel<kY, 256, 256, 4, 2>), grid, dim3(512), 0, st, a);
  else hipLaunchKernelGGL((fp8_tile_kernel<kY, 128, 128, 2, 2>), grid, dim3(256), 0, st, a);
  if (a.splits > 1)
    hipLaunchKernelGGL((fp8_join_kernel<kY>), dim3((unsigned)cdiv(a.d_out, 1024), (unsigned)a.M), dim3(256), 0, st, a);
}

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_fp8_matmul(const void* X, int32_t x_dtype, const uint8_t* x_scales, int64_t M, int64_t d_in,
                                       int64_t ld_x, const uint8_t* W, int64_t ld_w, const uint8_t* w_scales,
                                       int64_t d_out, void* Y, int32_t y_dtype, int64_t ld_y, void* workspace,
                                       size_t ws_bytes, void* stream) {
  const bool codes = x_dtype == GPTQ_E4M3;
  GQ_CHECK_ARG(codes || x_dtype == GPTQ_F32 || x_dtype == GPTQ_F16 || x_dtype == GPTQ_BF16);
  GQ_CHECK_ARG(y_dtype == GPTQ_F32 || y_dtype == GPTQ_F16 || y_dtype == GPTQ_BF16);
  GQ_CHECK_ARG(M >= 0 && d_in >= 1 && d_out >= 1 && ld_x >= d_in && ld_x <= ((int64_t)1 << 36));
  GQ_CHECK_ARG(!codes || (d_in % kF8Block == 0 && ld_x % 16 == 0));
  GQ_CHECK_ARG(ld_w >= cdiv(d_in, kF8Block) * kF8Block && ld_w % 16 == 0 && ld_w <= ((int64_t)1 << 36));
  GQ_CHECK_ARG(ld_y >= d_out && ld_y <= ((int64_t)1 << 36));
  if (M > ((int64_t)1 << 22) || d_in > ((int64_t)1 << 22) || d_out > ((int64_t)1 << 22)) return GPTQ_EUNSUPPORTED;
  if (M == 0) return GPTQ_OK;
  GQ_CHECK_ARG(X && W && w_scales && Y && (x_scales || !codes));
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(X) % (codes ? 16 : f8_elem(x_dtype)) == 0);
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(W) % 16 == 0 && reinterpret_cast<uintptr_t>(Y) % f8_elem(y_dtype) == 0);
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(workspace) % 256 == 0);
  const F8Plan p = f8_plan(M, d_in, d_out, codes);
  if (p.total > 0 && (workspace == nullptr || ws_bytes < p.total)) return GPTQ_ENOMEM;
  F8MmArgs a{};
  a.X = X;
  a.xs = x_scales;
  a.W = W;
  a.ws = w_scales;
  a.Y = Y;
  a.ld_x = ld_x;
  a.ld_w = ld_w;
  a.ld_y = ld_y;
  a.M = M;
  a.d_out = d_out;
  a.d_in = (int)d_in;
  a.nb = (int)cdiv(d_in, kF8Block);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part = reinterpret_cast<float*>(ws + p.off_part);
  hipStream_t st = static_cast<hipStream_t>(stream);
  TimedScope ts(kTimeFp8Matmul, st);
  int kind = x_dtype;
  if (!codes && !p.fused) {
    f8_quantize_rows(X, x_dtype, M, d_in, ld_x, ws, (int64_t)a.nb * kF8Block, ws + p.off_scales, st);
    GQ_LAUNCHED();
    a.X = ws;
    a.xs = ws + p.off_scales;
    a.ld_x = (int64_t)a.nb * kF8Block;
    kind = GPTQ_E4M3;
  }
  if (y_dtype == GPTQ_F32) f8_run<GPTQ_F32>(a, kind, p, st);
  else if (y_dtype == GPTQ_F16) f8_run<GPTQ_F16>(a, kind, p, st);
  else f8_run<GPTQ_BF16>(a, kind, p, st);
  GQ_LAUNCHED();
  return GPTQ_OK;
}
