// Product of 8-bit operands with a power-of-two scale for each block of 128:
//   Y[m][n] = sum_b 2^(sx[m][b] - 127) 2^(sw[n / 128][b] - 127) sum_{k in b} x[m][k] w[n][k].
//
// Two ways to multiply a block.  The codes become bf16 together with the scales, exactly,
// and go through 16x16x32 bf16 products.  Or one instruction, 16x16x128 (32x32x64 in large
// tiles) on e4m3 with a scale byte per lane and operand, does the block: no conversions and
// twice the rate, but it adds the products of eight consecutive codes after cutting each off
// at 2^-13 of the largest one's exponent (measured with single products; sums across eights
// keep 24 bits).  That is up to 7 * 2^-13 of the largest product of each eight: 3e-5 of a
// result for random operands, a tenth of half a step of fp16, but where terms cancel (1, -1
// and six of 2^-14) they are lost.  So the second way is taken for 16-bit outputs alone, and
// there only for more than 128 tokens, which products bound; fewer wait for the weights.  The
// two ways, bf16 outputs, us: 1 x 4096 -> 4096 8.1 and 8.0, 16 x 11008 -> 4096
// 21.2 and 21.5, 48 x 8192 -> 28672 72 and 72, 128 x 4096 -> 14336 34.3 and 34.2; 300 x
// 4096 -> 14336 61.0 and 58.6, 1024 x 4096 -> 4096 44.8 and 40.8, 2048 x 4096 -> 4096 72 and 65.
//
// 8192 x 8192 -> 28672 in codes 1.68 ms, 2.3 PFLOP/s (a large product of the library
// 3.25): direct loads of a block take as long as its products, and with two buffers
// of 64 KB little of either is hidden behind the other's end.  48 x 8192 -> 28672 62 us,
// 3.8 TB/s of weights; one token 4096 -> 4096 8 us, one launch; fp32 outputs 777 x 11000
// -> 4001 98 us: 9 to quantize the tokens, the rest to turn codes into bf16 and multiply.
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
// 16 rows of weights by up to 16 tokens in one launch: the waves take the sum's blocks
// in turn, straight from memory, quantize the tokens' values as they come, and their
// sums meet in LDS.
constexpr int kF8FewWaves = 8;

template <int kX, int kY>
__global__ __launch_bounds__(64 * kF8FewWaves) void fp8_few_kernel(F8MmArgs a) {
  constexpr int kPitch = 20;
  constexpr int kU = kX == GPTQ_F32 ? 2 : 4;                             // blocks asked for together
  constexpr int kRaw = kX == GPTQ_E4M3 ? 0 : kX == GPTQ_F32 ? 32 : 16;   // words of a lane's values
  __shared__ __align__(16) float red[kF8FewWaves][16][kPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const uint8_t* w = a.W + min(n0 + c16, a.d_out - 1) * a.ld_w + q * 16;
  const uint8_t* sw = a.ws + n0 / kF8Block * a.nb;
  // lanes without a token take the last one's values; nothing of them is stored
  const int64_t m = min((int64_t)c16, a.M - 1);
  const char* x = static_cast<const char*>(a.X) + m * a.ld_x * (kX == GPTQ_F32 ? 4 : kX == GPTQ_E4M3 ? 1 : 2);
  const uint8_t* sx = kX == GPTQ_E4M3 ? a.xs + m * a.nb : nullptr;
  f32x4 acc[1][1] = {{{0.f, 0.f, 0.f, 0.f}}};
  struct Step {
    u32x4 w[2][1], x[2][1];                // [unit]
    uint32_t sw[1], sx[1];
    uint32_t raw[kRaw ? kRaw : 1];
  };
  auto read = [&](int b, Step& s) {
    s.w[0][0] = *reinterpret_cast<const u32x4*>(w + b * kF8Block);
    s.w[1][0] = *reinterpret_cast<const u32x4*>(w + b * kF8Block + 64);
    s.sw[0] = sw[b];
    if constexpr (kX == GPTQ_E4M3) {
      s.x[0][0] = *reinterpret_cast<const u32x4*>(x + b * kF8Block + q * 16);
      s.x[1][0] = *reinterpret_cast<const u32x4*>(x + b * kF8Block + q * 16 + 64);
      s.sx[0] = sx[b];
    } else {
      constexpr int kE = kX == GPTQ_F32 ? 4 : 2;
      const int k = b * kF8Block + q * 16;
      if ((b + 1) * kF8Block <= a.d_in) {
        __builtin_memcpy(s.raw, __builtin_assume_aligned(x + (int64_t)k * kE, kE), kRaw * 2);
        __builtin_memcpy(s.raw + kRaw / 2, __builtin_assume_aligned(x + (int64_t)(k + 64) * kE, kE), kRaw * 2);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int at = k + i / 16 * 64 + i % 16;
          const uint32_t v = at < a.d_in ? load_bits<kX>(x, at) : 0u;
          if constexpr (kX == GPTQ_F32) s.raw[i] = v;
          else s.raw[i / 2] = i % 2 ? s.raw[i / 2] | v << 16 : v;
        }
      }
    }
  };
  auto multiply = [&](Step& s) {
    if constexpr (kX != GPTQ_E4M3) {
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if constexpr (kX == GPTQ_F32) v[i] = __uint_as_float(s.raw[i]);
        else v[i] = i % 2 ? hi16<kX>(s.raw[i / 2]) : lo16<kX>(s.raw[i / 2]);
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      // over the four lanes of a token, 16 and 32 apart
      const auto p = __builtin_amdgcn_permlane16_swap(top, top, false, false);
      top = max(p[0], p[1]);
      const auto o = __builtin_amdgcn_permlane32_swap(top, top, false, false);
      top = max(o[0], o[1]);
      s.sx[0] = f8_scale(top);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        s.x[i / 4][0][i % 4] = f8_codes4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], s.sx[0]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) f8_wide_unit<1, 1>(s.w[u], s.x[u], s.sw, s.sx, acc);
  };
  int b = wave;
  for (; b + (kU - 1) * kF8FewWaves < a.nb; b += kU * kF8FewWaves) {
    Step s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) read(b + u * kF8FewWaves, s[u]);
#pragma unroll
    for (int u = 0; u < kU; ++u) multiply(s[u]);
  }
  for (; b < a.nb; b += kF8FewWaves) {
    Step s;
    read(b, s);
    multiply(s);
  }
  *reinterpret_cast<f32x4*>(&red[wave][c16][4 * q]) = acc[0][0];
  __syncthreads();
  const int tok = threadIdx.x >> 2, n = threadIdx.x % 4 * 4;
  if (tok >= a.M || tok >= 16 || n0 + n >= a.d_out) return;
  f32x4 v = *reinterpret_cast<const f32x4*>(&red[0][tok][n]);
#pragma unroll
  for (int u = 1; u < kF8FewWaves; ++u) v += *reinterpret_cast<const f32x4*>(&red[u][tok][n]);
  f8_store4<kY>(a.Y, tok * a.ld_y + n0 + n, a.d_out - n0 - n, v);
}

// ---------------------------------------------------------------- many tokens
// Number -> (token tile, weight tile, part).  Workgroups go to the
// eight XCDs in turn; each gets a run of tiles, walked in bands of eight token
// tiles, so that what runs on it at one time reads few panels through its L2.
__device__ __forceinline__ void f8_place(const F8MmArgs& a, int id, int& tm, int& tn, int& part) {
  const int total = a.tiles_m * a.tiles_n * a.splits;
  const int per = total / 8;
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
template <int kY, bool kExact, int kBM, int kBN, int kWM, int kWN>
__global__ __launch_bounds__(64 * kWM * kWN, 2) void fp8_tile_kernel(F8MmArgs a) {
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
  f8_place(a, blockIdx.x, tm, tn, part);
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
    if constexpr (kExact) {
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
    // the tokens' operands and two of the weights' first, then every next one's beside
    // the products of the one two before
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * kT + 4, 0);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x8, kT, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
  };
  fetch(b0, x0, bx[0], bw[0]);
#define GQ_F8_STAGE(u, CUR, NEXT)                                         \
  {                                                                       \
    __builtin_amdgcn_s_waitcnt(0x0F70);   /* vmcnt(0), known to the compiler */ \
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");       \
    fetch(b + (u) + 1, NEXT, bx[1 - (u)], bw[1 - (u)]);                   \
    __builtin_amdgcn_sched_barrier(0);                                    \
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

// Large products with 16-bit outputs: 256 tokens by 256 rows, four waves of 128 x 128
// each (one per SIMD, so that an operand read from LDS serves four products of
// 32x32x64), the sum a block of 128 at a time in two buffers, whole 128-byte lines of
// every row (half lines keep the L2s busy for twice as long).  A block's second half is
// read while its first is multiplied, then its buffer is free for the block after the
// next.  Unit u of row r lies at slot u ^ (r / 2 % 8): the sixteen rows that are read
// together cover all banks once.
constexpr int kF8Big = 256;
constexpr int kF8BigStage = 2 * kF8Big * kF8Block;
constexpr int kF8BigWords = 30;

template <int kY>
__global__ __launch_bounds__(256, 1) void fp8_big_kernel(F8MmArgs a) {
  __shared__ __attribute__((aligned(1024))) char r0[kF8BigStage], r1[kF8BigStage];
  __shared__ uint32_t scale_x[kF8BigWords][kF8Big], scale_w[kF8BigWords][2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c32 = lane & 31, h = lane >> 5;
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t w_rows = (a.d_out + kF8Block - 1) / kF8Block;
  int tm, tn, part;
  f8_place(a, blockIdx.x, tm, tn, part);
  const int64_t m0 = (int64_t)tm * kF8Big, n0 = (int64_t)tn * kF8Big;
  uint32_t src[16];
  // this lane's part of load i: row 8 (4 i + wave) + lane / 8 of the stage (tokens
  // first), slot lane % 8; rows behind the end read the last one and are never stored
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int row = 8 * (4 * (i & 7) + wave) + (lane >> 3);
    const int unit = (lane & 7) ^ ((row >> 1) & 7);
    src[i] = unit * 16 + (i < 8 ? (uint32_t)min(row, (int)min(a.M - 1 - m0, (int64_t)kF8Big)) * (uint32_t)a.ld_x
                                : (uint32_t)min(row, (int)min(a.d_out - 1 - n0, (int64_t)kF8Big)) * (uint32_t)a.ld_w);
  }
  const uint8_t* base_x = static_cast<const uint8_t*>(a.X) + m0 * a.ld_x;
  const uint8_t* base_w = a.W + n0 * a.ld_w;
  auto dma = [&](int block, char* to) {
    const int at = min(block, a.nb - 1) * kF8Block;   // blocks behind the end read the last one, which nothing uses
#pragma unroll
    for (int i = 0; i < 16; ++i) lds_load16((i < 8 ? base_x : base_w) + at + src[i], to + (4 * i + wave) * 1024);
  };
  // Scales of four blocks in a word, one byte of which an instruction picks: up to 30
  // words of every row in LDS.  Words that would end behind the array are read there
  // and moved.
  auto stage = [&](const uint8_t* array, int64_t rows, int64_t row, int b, int g0, int words, uint32_t (&v)[6]) {
    const int64_t end = rows * a.nb - 4;
    uint32_t move[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int64_t at = row * a.nb + b + 4 * min(g0 + i, words - 1);
      move[i] = at > end ? (uint32_t)min(at - end, (int64_t)3) * 8 : 0u;
      __builtin_memcpy(&v[i], array + min(at, end), 4);
    }
    __builtin_amdgcn_sched_barrier(0);   // together
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] >>= move[i];
  };
  auto stage_scales = [&](int b) {
    const int words = min((a.nb - b + 3) / 4, kF8BigWords);
    const int64_t row = min(m0 + (int)threadIdx.x, a.M - 1), w_row = min(n0 / kF8Block + (lane & 1), w_rows - 1);
#pragma unroll 1
    for (int g = 0; g < words; g += 6) {
      uint32_t v[6];
      stage(a.xs, a.M, row, b, g, words, v);
#pragma unroll
      for (int i = 0; i < 6; ++i) scale_x[g + i][threadIdx.x] = v[i];
      if (wave == 0) {
        stage(a.ws, w_rows, w_row, b, g, words, v);
        if (lane < 2) {
#pragma unroll
          for (int i = 0; i < 6; ++i) scale_w[g + i][lane] = v[i];
        }
      }
    }
  };
  struct Frags {
    i32x8 x[4], w[4];
  };
  const int swz = (c32 >> 1) & 7;
  const int at_x = (wm * 128 + c32) * kF8Block, at_w = (kF8Big + wn * 128 + c32) * kF8Block;
  auto read = [&](const char* from, int half, Frags& f) {
    const int u0 = ((4 * half + 2 * h) ^ swz) * 16, u1 = u0 ^ 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const char* p = from + at_w + i * 32 * kF8Block;
      const char* q = from + at_x + i * 32 * kF8Block;
      f.w[i] = f8_frag(*reinterpret_cast<const u32x4*>(p + u0), *reinterpret_cast<const u32x4*>(p + u1));
      f.x[i] = f8_frag(*reinterpret_cast<const u32x4*>(q + u0), *reinterpret_cast<const u32x4*>(q + u1));
    }
  };
  f32x16 acc[4][4];
  Frags fa, fb;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[r][t][i] = 0.f;
  // Block b + k: its first half is in fa.  At the barrier its second half is read by
  // every wave, so that its buffer is free, and the next block has landed.  No branch
  // between two of them: the compiler's count of what is in flight would be lost.
#define GQ_F8_MULTIPLY(F, k)                                                            \
  _Pragma("unroll") for (int r = 0; r < 4; ++r)                                         \
  _Pragma("unroll") for (int t = 0; t < 4; ++t)                                         \
    acc[r][t] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(F.w[r], F.x[t], acc[r][t], 0, 0, (k), (int)now_w, (k), \
                                                                (int)now_x[t]);
#define GQ_F8_BLOCK(k, CUR, NXT)                                                        \
  {                                                                                     \
    read(CUR, 1, fb);                                                                   \
    GQ_F8_MULTIPLY(fa, k)                                                               \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) {                                     \
      __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);                                  \
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);                                \
    }                                                                                   \
    __builtin_amdgcn_s_waitcnt(0x0070);   /* vmcnt(0) lgkmcnt(0) */                     \
    asm volatile("s_barrier" ::: "memory");                                             \
    dma(b + (k) + 2, CUR);                                                              \
    read(NXT, 0, fa);                                                                   \
    GQ_F8_MULTIPLY(fb, k)                                                               \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) {                                     \
      if (i < 4) __builtin_amdgcn_sched_group_barrier(0x20, 4, 0);                      \
      __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);                                  \
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);                                \
    }                                                                                   \
  }
  for (int first = 0; first < a.nb; first += 4 * kF8BigWords) {
    const int end = min(first + 4 * kF8BigWords, a.nb);
    // what was asked for behind the last block has landed, and every wave is done
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
    dma(first, r0);
    dma(first + 1, r1);
    stage_scales(first);
    __builtin_amdgcn_s_waitcnt(0x0070);
    asm volatile("s_barrier" ::: "memory");
    read(r0, 0, fa);
    uint32_t now_x[4], now_w;
    auto scales = [&](int b) {
      const int g = (b - first) / 4, move = b - first & 2 ? 16 : 0;
#pragma unroll
      for (int t = 0; t < 4; ++t) now_x[t] = scale_x[g][wm * 128 + t * 32 + c32] >> move;
      now_w = scale_w[g][wn] >> move;
    };
    int b = first;
    for (; b + 2 <= end; b += 2) {
      scales(b);
      GQ_F8_BLOCK(0, r0, r1)
      GQ_F8_BLOCK(1, r1, r0)
    }
    if (b < end) {
      scales(b);
      GQ_F8_BLOCK(0, r0, r1)
    }
  }
#undef GQ_F8_BLOCK
#undef GQ_F8_MULTIPLY
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no direct load ends after the workgroup
  // eight consecutive outputs a lane: half of them from the lane 32 away
  uint16_t* out = static_cast<uint16_t*>(a.Y) + (m0 + wm * 128) * a.ld_y + n0 + wn * 128;
  const int left_m = (int)min(a.M - m0 - wm * 128, (int64_t)128), left_n = (int)min(a.d_out - n0 - wn * 128, (int64_t)128);
  const bool full = left_m == 128 && left_n == 128;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t at = (uint32_t)(t * 32 + c32) * (uint32_t)a.ld_y + 8 * h;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = value_bits<kY>(acc[r][t][8 * i + 2 * j]) | value_bits<kY>(acc[r][t][8 * i + 2 * j + 1]) << 16;
        // words 0, 1: rows 16 i + 4 h .., words 2, 3: rows 16 i + 8 + 4 h ..
        const auto lo = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        const u32x4 v = {lo[0], hi[0], lo[1], hi[1]};
        const int n = r * 32 + i * 16;
        if (full) {
          __builtin_memcpy(__builtin_assume_aligned(out + at + n, 2), &v, 16);
        } else if (t * 32 + c32 < left_m) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + 8 * h + e < left_n) out[at + n + e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
        }
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

// Up to 16 tokens take one launch, whose every workgroup quantizes all tokens, where a CU
// has one workgroup (4096 rows of weights), or two with few values to quantize.  bf16 in
// one launch, or quantized apart and in tiles of 32 tokens, us:
//   4096 -> 4096     1 token 8 and 14,    16 tokens 9 and 15,    32 (by the codes) 18 and 14
//   28672 -> 4096    1 token 32 and 38,   16 tokens 42 and 41
//   4096 -> 8192     1 token 13 and 17,   16 tokens 17 and 19
//   8192 -> 8192     1 token 22 and 24,   8 tokens 24 and 26,    12 tokens 30 and 26
//   28672 -> 8192    1 token 63 and 62,   8 tokens 69 and 65,    16 tokens 82 and 66
//   4096 -> 11008    1 token 18 and 18,   8 tokens 21 and 20,    16 tokens 24 and 21
constexpr int kF8Few = 16;
constexpr int64_t kF8FewRows = 4096, kF8FewValues = 1 << 16;
// Tiles of 256 by 256 if every CU gets one and they are more than half full: 4096 ->
// 131072, bf16 (and fp32) in tiles of 256 and in the smaller ones, us: 16 tokens 153 (221)
// and 126 (129), 100 tokens 183 (231) and 155 (165), 200 tokens 185 (247) and 221 (284).
// Tiles of 128 tokens if two of them for every CU remain, else 64 (or 32), bf16, us:
// 300 x 4096 -> 14336 56 and 50, 2048 x 4096 -> 4096 61 and 69.  The sum is split until
// every CU has a workgroup, into parts of four blocks or more: 65 x 4096 -> 4096 in 1, 4
// and 8 parts 26, 16 and 20; 128 x 8192 -> 28672 in 1 and 2 parts 62 and 87.
constexpr int64_t kF8Wide = 512;
// Tokens whose 16-bit outputs are of exact products, too.
constexpr int64_t kF8Exact = 128;

struct F8Plan {
  bool few;
  int bm, bn, splits;
  size_t off_scales, off_part, total;
};

static F8Plan f8_plan(int64_t M, int64_t d_in, int64_t d_out, bool codes) {
  F8Plan p{};
  const int64_t nb = cdiv(d_in, kF8Block);
  p.few = M <= kF8Few && (d_out <= kF8FewRows || (d_out <= 2 * kF8FewRows && M * d_in <= kF8FewValues));
  if (!codes && !p.few) {
    p.off_scales = align_up((size_t)M * nb * kF8Block, 256);
    p.total = align_up(p.off_scales + (size_t)M * nb, 256);
  }
  p.splits = 1;
  if (!p.few) {
    p.bm = p.bn = M > 128 && cdiv(M, 256) * cdiv(d_out, 256) >= 256 ? 256 : 128;
    if (p.bm == 128) {
      if (M <= 32) p.bm = 32;
      else if (M <= 64 || cdiv(M, 128) * cdiv(d_out, 128) < kF8Wide) p.bm = 64;
      const int64_t tiles = cdiv(M, p.bm) * cdiv(d_out, 128);
      while (tiles * p.splits < 256 && nb / (p.splits * 2) >= 4) p.splits *= 2;
      p.splits = (int)cdiv(nb, cdiv(nb, p.splits));
    }
  }
  p.off_part = p.total;
  if (p.splits > 1) p.total += (size_t)p.splits * M * d_out * 4;
  return p;
}

size_t fp8_matmul_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out) {
  return f8_plan(M, d_in, d_out, false).total;
}

template <int kY>
static void f8_run(F8MmArgs& a, int x_dtype, const F8Plan& p, hipStream_t st) {
  if (p.few) {
    const dim3 grid((unsigned)cdiv(a.d_out, 16)), block(64 * kF8FewWaves);
    if (x_dtype == GPTQ_F32) hipLaunchKernelGGL((fp8_few_kernel<GPTQ_F32, kY>), grid, block, 0, st, a);
    else if (x_dtype == GPTQ_F16) hipLaunchKernelGGL((fp8_few_kernel<GPTQ_F16, kY>), grid, block, 0, st, a);
    else if (x_dtype == GPTQ_BF16) hipLaunchKernelGGL((fp8_few_kernel<GPTQ_BF16, kY>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((fp8_few_kernel<GPTQ_E4M3, kY>), grid, block, 0, st, a);
    return;
  }
  a.tiles_m = (int)cdiv(a.M, p.bm);
  a.tiles_n = (int)cdiv(a.d_out, p.bn);
  a.splits = p.splits;
  a.nb_split = (int)cdiv(a.nb, p.splits);
  const dim3 grid((unsigned)((int64_t)a.tiles_m * a.tiles_n * a.splits));
  if constexpr (kY != GPTQ_F32) {
    // scales are read in words, a tile's rows by 32-bit offsets
    if (p.bm == 256 && cdiv(a.d_out, kF8Block) * a.nb >= 4 && std::max(a.ld_x, a.ld_w) <= ((int64_t)1 << 23) &&
        a.ld_y <= ((int64_t)1 << 23)) {
      hipLaunchKernelGGL((fp8_big_kernel<kY>), grid, dim3(256), 0, st, a);
      return;
    }
  }
  constexpr bool kWide = kY == GPTQ_F32;
  const bool exact = kWide || a.M <= kF8Exact;
  if (p.bm == 256) hipLaunchKernelGGL((fp8_tile_kernel<kY, kWide, 256, 256, 4, 2>), grid, dim3(512), 0, st, a);
  else if (p.bm == 128 && exact) hipLaunchKernelGGL((fp8_tile_kernel<kY, true, 128, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else if (p.bm == 128) hipLaunchKernelGGL((fp8_tile_kernel<kY, kWide, 128, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else if (p.bm == 64 && exact) hipLaunchKernelGGL((fp8_tile_kernel<kY, true, 64, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else if (p.bm == 64) hipLaunchKernelGGL((fp8_tile_kernel<kY, kWide, 64, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((fp8_tile_kernel<kY, true, 32, 128, 1, 4>), grid, dim3(256), 0, st, a);
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
  if (!codes && M * cdiv(d_in, kF8Block) > kF8MostBlocks) return GPTQ_EUNSUPPORTED;
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
  if (!codes && !p.few) {
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
