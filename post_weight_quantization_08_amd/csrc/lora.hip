// Low-rank adapters of many requests beside a shared projection:
//   Y[m] = base[m] + s_a (X[m] A_a^T) B_a^T,   a = adapter[m].
//
// Two products through T = X A^T (fp32, in the workspace).  Which rows share
// an adapter is known to the GPU alone.
//
// Few tokens (decode, kLoraFew): every token has its own adapter, so each
// token's factors are read for it alone, on vector units.  T: one wave per
// (token, rank).  Y: the r / 8 lanes of a column each take 8 ranks (16 bytes of
// B), so a wave reads B in order, and exchange their sums.
//
// Many tokens (prompts): tiles of 32 tokens on MFMA (16x16x32).  A tile takes
// one pass per adapter that occurs in it; a request's tokens lie together, so
// most tiles need one.  Rows of another adapter are left out of a pass by
// selecting, never by multiplying with zero: a NaN or infinity in one adapter
// does not reach another's rows.  For the second product T is kept as three
// 16-bit terms, which hold all of an fp32: cut off after 8 bits each for bf16;
// rounded for fp16, after rows of T were scaled by a power of two, so that
// neither their size nor their smallness leaves fp16's range.  Two terms (16 and
// 22 bits) are 0 to 3 % faster.  The second product's columns are dealt to the
// MFMA tiles so that a lane ends up with four consecutive outputs and sixteen lanes
// with 64: base and Y move in pieces of 256 (fp32) or 128 bytes, at any alignment.
//
// Bound by memory: X, base and Y once, the factors from L2 (a factor's matrix
// serves every tile of its adapter).  8192 x 11008 -> 4096, rank 64, fp32 base:
// 143 us, 75 and 70 for the products, 3.2 TB/s over both.  300 x 4096 -> 14336,
// rank 32, 16-bit: 18 us, two launches that the first loads' latency fills.
#include <type_traits>

#include "lora.h"

namespace gq {

size_t w4a16_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out);

// Tokens up to which every one is taken by itself.  Which adapters they want is
// not known here.  128 tokens in runs of four adapters, or every one with its own:
//   4096 -> 4096, rank 16:    9 or 12 us by themselves, 12 or 105 in tiles
//   4096 -> 14336, rank 32:   20 or 34,                 12 or 121
//   8192 -> 28672, rank 64:   57 or 108,                20 or 225
// and 48 tokens 7 or 8, 18 or 105; 11 or 17, 17 or 119; 26 or 46, 26 or 192.  By
// themselves is never more than 2.9 times the other way, tiles up to 13 times.
constexpr int kLoraFew = 128;
constexpr int kLoraTile = 32;       // tokens of an MFMA tile
constexpr int kLoraMaxRank = 128;

struct LoraArgs {
  const uint16_t* X;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const int32_t* adapter;
  const void* base;
  void* Y;
  float* T;                // [splits][M][rank padded to 8]
  int64_t ld_x, ld_b, ld_y, M, d_out;
  int d_in, rank, n;
  int rp;                  // rank padded to 8
  int splits, k_split;     // parts of the first product's sum, and their length
  int cols;                // output columns of a workgroup
};

// ---------------------------------------------------------------- few tokens
template <int kDt>
__global__ __launch_bounds__(256) void lora_down_few_kernel(LoraFew a) {
  lora_down_one<kDt>(a, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6));
}

// Y[m][n] = base[m][n] + T[m] . B_a[n]: a wave takes 64 columns, kL lanes each
// column's ranks 8 at a time.
template <int kDt, int kY, int kL>
__global__ __launch_bounds__(256) void lora_up_few_kernel(LoraArgs a) {
  constexpr int kPer = 64 / kL;            // columns of a step
  const int lane = threadIdx.x & 63;
  const int64_t m = blockIdx.y;
  const int64_t n0 = (int64_t)blockIdx.x * 256 + (threadIdx.x & ~63);
  const int ad = __builtin_amdgcn_readfirstlane(a.adapter[m]);
  const int64_t n = n0 + lane;
  const uint32_t base = a.base && n < a.d_out ? load_bits<kY>(a.base, m * a.ld_b + n) : 0u;
  if (ad < 0 || ad >= a.n) {
    if (n < a.d_out) store_bits<kY>(a.Y, m * a.ld_y + n, base);   // the base as it is
    return;
  }
  float y = bits_value<kY>(base);
  if (n0 < a.d_out) {
    const int k = lane % kL * 8;
    u32x4 b[kL];
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      const int64_t col = n0 + i * kPer + lane / kL;
      const uint16_t* row = a.B + ((int64_t)ad * a.d_out + (col < a.d_out ? col : a.d_out - 1)) * a.rank;
      b[i] = load8_end(row, k, a.rank);
    }
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = k + i < a.rank ? a.T[m * a.rp + k + i] : 0.f;
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // beyond the rank both are zero
        s = fmaf(t[2 * e], lo16<kDt>(b[i][e]), s);
        s = fmaf(t[2 * e + 1], hi16<kDt>(b[i][e]), s);
      }
#pragma unroll
      for (int d = 1; d < kL; d <<= 1) s += __shfl_xor(s, d);
      const float got = __shfl(s, lane % kPer * kL);
      if (lane / kPer == i) mine = got;
    }
    y += mine;
  }
  if (n < a.d_out) store_el<kY>(a.Y, m * a.ld_y + n, y);
}

// ---------------------------------------------------------------- many tokens
// Calls f(adapter, lanes' match) for every adapter among the tile's 32 tokens;
// `mine` is the adapter of token lane % 32, or -1.
template <class F>
__device__ __forceinline__ void for_each_adapter(int mine, F f) {
  uint32_t left = (uint32_t)__ballot(mine >= 0);
  while (left) {
    const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(mine == a);
    f(a);
  }
}

// Tile and part of workgroup b of `parts` per tile.  Workgroups go to the eight
// XCDs in turn, each with an L2 of its own; with many tiles every XCD takes a
// run of neighbouring ones, whose tokens mostly share an adapter, so that its
// factors stay in that L2.  With fewer than 64 tiles the runs would leave XCDs
// idle.
__device__ __forceinline__ void lora_place(const LoraArgs& a, int parts, int64_t b, int64_t& tile, int& part) {
  const int64_t tiles = (a.M + kLoraTile - 1) / kLoraTile;
  if (tiles < 64) {
    tile = b / parts;
    part = (int)(b % parts);
  } else {
    const int64_t run = (tiles + 7) / 8, i = b / 8;
    tile = b % 8 * run + i / parts;
    part = (int)(i % parts);
  }
}
static int64_t lora_blocks(int64_t M, int64_t parts) {
  const int64_t tiles = cdiv(M, kLoraTile);
  return (tiles < 64 ? tiles : cdiv(tiles, 8) * 8) * parts;
}

__device__ __forceinline__ int lora_adapter(const LoraArgs& a, int64_t m) {
  const int ad = m < a.M ? a.adapter[m] : -1;
  return ad < a.n ? ad : -1;
}

// T of 32 tokens over one part of the sum: four waves take its 64-element steps
// in turn and their sums meet in LDS.  kR rank tiles of 16.  D: rows = ranks,
// columns = tokens.
template <int kDt, int kR>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs a) {
  constexpr int kStride = kR * 16 + 4;     // floats of a token in LDS
  __shared__ __align__(16) float red[4][kLoraTile][kStride];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  int64_t tile;
  int part;
  lora_place(a, a.splits, blockIdx.x, tile, part);
  const int64_t m0 = tile * kLoraTile;
  if (m0 >= a.M) return;
  const int k0 = part * a.k_split, k1 = min(k0 + a.k_split, a.d_in);
  const int mine = lora_adapter(a, m0 + (lane & 31));
  const uint16_t* x[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) x[t] = a.X + min(m0 + t * 16 + c16, a.M - 1) * a.ld_x;
  for_each_adapter(mine, [&](int ad) {
    const uint16_t* f[kR];
#pragma unroll
    for (int t = 0; t < kR; ++t) f[t] = a.A + ((int64_t)ad * a.rank + min(t * 16 + c16, a.rank - 1)) * a.d_in;
    f32x4 acc[kR][2];
#pragma unroll
    for (int t = 0; t < kR; ++t) acc[t][0] = acc[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    // a step's operands are asked for while the step before is multiplied
    struct Step {
      u32x4 x[2][2], f[2][kR];
    };
    auto read = [&](int k, Step& p) {
      if (k + 64 <= k1) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int t = 0; t < 2; ++t) p.x[j][t] = load8(x[t] + k + 32 * j + 8 * q);
#pragma unroll
          for (int t = 0; t < kR; ++t) p.f[j][t] = load8(f[t] + k + 32 * j + 8 * q);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int t = 0; t < 2; ++t) p.x[j][t] = load8_end(x[t], k + 32 * j + 8 * q, k1);
#pragma unroll
          for (int t = 0; t < kR; ++t) p.f[j][t] = load8_end(f[t], k + 32 * j + 8 * q, k1);
        }
      }
    };
    auto multiply = [&](const Step& p) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int t = 0; t < kR; ++t) {
          acc[t][0] = mfma_16x16x32<kDt>(p.f[j][t], p.x[j][0], acc[t][0]);
          acc[t][1] = mfma_16x16x32<kDt>(p.f[j][t], p.x[j][1], acc[t][1]);
        }
    };
    const int first = k0 + wave * 64;
    if (first < k1) {
      Step even, odd;
      read(first, even);
      for (int k = first; k < k1; k += 512) {
        if (k + 256 < k1) read(k + 256, odd);
        multiply(even);
        if (k + 256 < k1) {
          if (k + 512 < k1) read(k + 512, even);
          multiply(odd);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kR; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) *reinterpret_cast<f32x4*>(&red[wave][u * 16 + c16][t * 16 + 4 * q]) = acc[t][u];
    __syncthreads();
    // 8 threads per token
    const int tok = threadIdx.x >> 3;
    if (__shfl(mine, tok & 31) == ad) {
      float* out = a.T + ((int64_t)part * a.M + m0 + tok) * a.rp;
      for (int r = (threadIdx.x & 7) * 4; r < a.rp; r += 32) {
        f32x4 s = *reinterpret_cast<const f32x4*>(&red[0][tok][r]);
#pragma unroll
        for (int w = 1; w < 4; ++w) s += *reinterpret_cast<const f32x4*>(&red[w][tok][r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = r + i < a.rank ? s[i] : 0.f;
        *reinterpret_cast<f32x4*>(out + r) = s;
      }
    }
    __syncthreads();
  });
}

// The same for rows on 16 bytes: operands through LDS.  Reading them straight
// into MFMA form gives every lane of 16 another row, 64 separate accesses per
// load, and the address units are what the kernel above waits for (8192 x
// 11008, rank 64: 97 us, address units busy half of it).  Here 16 lanes load
// 256 bytes of one row, directly into LDS, two steps of 128 elements ahead; the
// unit u of row m lies at slot u ^ (m % 16), so that a fragment's 16 rows lie in
// 16 slots.  Four waves share the kR x 2 tiles of ranks and tokens.
template <int kDt, int kR>
__global__ __launch_bounds__(256) void lora_down_lds_kernel(LoraArgs a) {
  constexpr int kRows = kLoraTile + kR * 16;           // rows of a stage: tokens, then ranks
  constexpr int kStage = kRows * 256;
  constexpr int kLoads = kRows / 16;                   // direct loads of a wave per step
  constexpr int kMine = kR == 2 ? 1 : kR / 4;          // rank tiles of a wave
  constexpr int kTok = kR == 2 ? 1 : 2;                // token tiles of a wave
  constexpr int kWait = (kLoads & 0xF) | ((kLoads >> 4) << 14) | (7 << 4) | (0xF << 8);
  static_assert(kRows % 16 == 0 && kLoads < 64, "whole loads, counted in six bits");
  // one array per stage, so the compiler sees which one a read touches
  __shared__ __attribute__((aligned(1024))) char x0[kStage], x1[kStage], x2[kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  int64_t tile;
  int part;
  lora_place(a, a.splits, blockIdx.x, tile, part);
  const int64_t m0 = tile * kLoraTile;
  if (m0 >= a.M) return;
  const int k0 = part * a.k_split, k1 = min(k0 + a.k_split, a.d_in);
  const int steps = (k1 - k0 + 127) / 128;
  const int mine = lora_adapter(a, m0 + (lane & 31));
  const int rank0 = kR == 2 ? (wave & 1) * 16 : wave * kMine * 16;   // this wave's first rank and token
  const int tok0 = kR == 2 ? (wave >> 1) * 16 : 0;
  for_each_adapter(mine, [&](int ad) {
    // this lane's part of load i: row 16 i + 4 wave + lane / 16 of the stage, slot lane % 16
    const uint16_t* src[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = 16 * i + 4 * wave + (lane >> 4);
      src[i] = row < kLoraTile
                   ? a.X + min(m0 + row, a.M - 1) * a.ld_x
                   : a.A + ((int64_t)ad * a.rank + min(row - kLoraTile, a.rank - 1)) * a.d_in;
    }
    const int unit = (lane & 15) ^ ((4 * wave + (lane >> 4)) & 15);
    auto fetch = [&](int step, char* to) {
      // units behind the part's end read its last one and are never multiplied;
      // steps behind the last one are read so that every step has as many loads
      const int k = min(k0 + min(step, steps - 1) * 128 + unit * 8, k1 - 8);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) lds_load16(src[i] + k, to + (16 * i + 4 * wave) * 256);
    };
    f32x4 acc[kMine][kTok];
#pragma unroll
    for (int r = 0; r < kMine; ++r)
#pragma unroll
      for (int t = 0; t < kTok; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](int step, const char* from) {
      const int left = k1 - (k0 + step * 128);         // elements of the step
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int u = 4 * j + q;
        u32x4 xv[kTok], fv[kMine];
#pragma unroll
        for (int t = 0; t < kTok; ++t)
          xv[t] = *reinterpret_cast<const u32x4*>(from + (tok0 + t * 16 + c16) * 256 + ((u ^ c16) * 16));
#pragma unroll
        for (int r = 0; r < kMine; ++r)
          fv[r] = *reinterpret_cast<const u32x4*>(from + (kLoraTile + rank0 + r * 16 + c16) * 256 + ((u ^ c16) * 16));
        if (left < 128 && u * 8 >= left) {
#pragma unroll
          for (int t = 0; t < kTok; ++t) xv[t] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
          for (int r = 0; r < kMine; ++r) fv[r] = u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int r = 0; r < kMine; ++r)
#pragma unroll
          for (int t = 0; t < kTok; ++t) acc[r][t] = mfma_16x16x32<kDt>(fv[r], xv[t], acc[r][t]);
      }
    };
    fetch(0, x0);
    fetch(1, x1);
#define GQ_LORA_STAGE(u, CUR, NEXT)                               \
  {                                                               \
    __builtin_amdgcn_s_waitcnt(kWait);                            \
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); \
    fetch(s + (u) + 2, NEXT);                                     \
    if (s + (u) < steps) multiply(s + (u), CUR);                  \
  }
    for (int s = 0; s < steps; s += 3) {
      GQ_LORA_STAGE(0, x0, x2);
      GQ_LORA_STAGE(1, x1, x0);
      GQ_LORA_STAGE(2, x2, x1);
    }
#undef GQ_LORA_STAGE
    // the direct loads have landed, and every wave is done reading, before the
    // next adapter's (or the end)
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const int tok = tok0 + t * 16 + c16;
      if (__shfl(mine, tok) != ad) continue;
      float* out = a.T + ((int64_t)part * a.M + m0 + tok) * a.rp;
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
        const int k = rank0 + r * 16 + 4 * q;
        f32x4 v = acc[r][t];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = k + i < a.rank ? v[i] : 0.f;
        if (k < a.rp) *reinterpret_cast<f32x4*>(out + k) = v;
      }
    }
  });
}

// 16-bit terms of 8 values, the largest first, as MFMA operands.  The first
// one of an infinity is all of it.
constexpr int kTerms = 3;
template <int kDt>
__device__ __forceinline__ void lora_split(const float (&v)[8], u32x4 (&out)[kTerms]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[2] = {v[2 * i], v[2 * i + 1]};
#pragma unroll
    for (int k = 0; k < kTerms; ++k) {
      uint32_t h[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (kDt == GPTQ_F16) {
          const _Float16 p = (_Float16)x[e];
          h[e] = __builtin_bit_cast(uint16_t, p);
          x[e] = fabsf(x[e]) == INFINITY ? 0.f : x[e] - (float)p;
        } else {
          // a NaN made by arithmetic stays one: its highest mantissa bit is set
          const uint32_t p = __float_as_uint(x[e]) & 0xFFFF0000u;
          h[e] = p >> 16;
          x[e] = fabsf(x[e]) == INFINITY ? 0.f : x[e] - __uint_as_float(p);
        }
      }
      out[k][i] = h[0] | h[1] << 16;
    }
  }
}

// 32 tokens by `cols` columns (a multiple of 256); kS steps of 32 ranks.  One
// step leaves room for four waves per SIMD, two registers short of it without
// asking (8192 x 4096 -> 14336, rank 16, 16-bit: 182 us).
template <int kDt, int kY, int kS>
__global__ __launch_bounds__(256, kS == 1 ? 4 : 1) void lora_up_kernel(LoraArgs a) {
  constexpr int kPitch = kS * 32 + 4;
  __shared__ __align__(16) float tsum[kLoraTile][kPitch];
  __shared__ u32x4 terms[2][kS][kTerms][64];   // [token tile][rank step][term][lane]
  __shared__ __align__(16) float grow[kLoraTile];   // 2^e that a token's terms were divided by
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  int64_t tile;
  int part;
  lora_place(a, (int)((a.d_out + a.cols - 1) / a.cols), blockIdx.x, tile, part);
  const int64_t m0 = tile * kLoraTile;
  if (m0 >= a.M) return;
  const int mine = lora_adapter(a, m0 + (lane & 31));
  const int64_t n_first = (int64_t)part * a.cols;
  const int64_t n_end = n_first + a.cols < a.d_out ? n_first + a.cols : a.d_out;
  const uint32_t some = (uint32_t)__ballot(mine >= 0);
  const int lead = some ? __builtin_amdgcn_readlane(mine, __builtin_ctz(some)) : -1;   // the tile's first adapter

  auto read_b = [&](int64_t n, int ad, int p, u32x4 (&b)[kS]) {
    int64_t bc = n + 4 * c16 + p;
    bc = bc < a.d_out ? bc : a.d_out - 1;
    const uint16_t* row = a.B + ((int64_t)ad * a.d_out + bc) * a.rank;
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      if (a.rank == kS * 32) b[s] = load8(row + s * 32 + 8 * q);
      else b[s] = load8_end(row, s * 32 + 8 * q, a.rank);
    }
  };
  // each wave takes 64 columns in turn; the first ones' B is on its way while T
  // is made, the next ones' while these are stored
  int64_t n = n_first + wave * 64;
  u32x4 b[4][kS];
  auto read_lead = [&]() {
    if (lead >= 0 && n < n_end) {
#pragma unroll
      for (int p = 0; p < 4; ++p) read_b(n, lead, p, b[p]);
    }
  };
  read_lead();
  // T's parts added up, scaled: 8 threads per token, 4 ranks at a time
  {
    const int tok = threadIdx.x >> 3;
    const int ad = __shfl(mine, tok & 31);
    const float sc = ad >= 0 && a.scale ? a.scale[ad] : 1.f;
    for (int r = (threadIdx.x & 7) * 4; r < kS * 32; r += 32) {
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
      if (ad >= 0 && r < a.rp) {
        const float* src = a.T + (m0 + tok) * a.rp + r;
        const int64_t step = a.M * a.rp;
        int p = 0;
        for (; p + 8 <= a.splits; p += 8) {
          f32x4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const f32x4*>(src + (p + i) * step);
#pragma unroll
          for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; p < a.splits; ++p) s += *reinterpret_cast<const f32x4*>(src + p * step);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] *= sc;
      *reinterpret_cast<f32x4*>(&tsum[tok][r]) = s;
    }
  }
  __syncthreads();
  // T's terms as operands into LDS, one wave per token tile: row c16 = token
  // t 16 + c16, 8 ranks per lane
  if (wave < 2) {
    const int t = wave;
    float v[kS][8];
    float big = 0.f;
#pragma unroll
    for (int s = 0; s < kS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 u = *reinterpret_cast<const f32x4*>(&tsum[t * 16 + c16][s * 32 + 8 * q + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[s][4 * h + i] = u[i];
          big = fmaxf(big, fabsf(u[i]) < INFINITY ? fabsf(u[i]) : 0.f);
        }
      }
    float g = 1.f;
    if constexpr (kDt == GPTQ_F16) {
      big = fmaxf(big, __shfl_xor(big, 16));
      big = fmaxf(big, __shfl_xor(big, 32));
      if (big > 0.f) {
        int e;
        frexpf(big, &e);
        g = ldexpf(1.f, e - 14);   // the largest below 2^14: its third term is above 2^-24, the least fp16
#pragma unroll
        for (int s = 0; s < kS; ++s)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[s][i] = ldexpf(v[s][i], 14 - e);
      }
    }
    if (q == 0) grow[t * 16 + c16] = g;
#pragma unroll
    for (int s = 0; s < kS; ++s) {
      u32x4 term[kTerms];
      lora_split<kDt>(v[s], term);
#pragma unroll
      for (int k = 0; k < kTerms; ++k) terms[t][s][k][lane] = term[k];
    }
  }
  __syncthreads();
  // 64 columns at a time, column 4 c16 + p in MFMA tile p.
  constexpr int kYE = kY == GPTQ_F32 ? 4 : 2;
  using Four = typename std::conditional<kY == GPTQ_F32, u32x4, uint2>::type;   // four outputs
  while (n < n_end) {
    const int64_t col = n + 4 * c16;       // this lane's four columns
    const bool whole = col + 4 <= a.d_out;
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const int64_t m = m0 + t * 16 + 4 * q;   // this lane's four tokens
      Four in[4] = {};
      if (a.base && whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const char* y = static_cast<const char*>(a.base) + (min(m + i, a.M - 1) * a.ld_b + col) * kYE;
          __builtin_memcpy(&in[i], __builtin_assume_aligned(y, kYE), sizeof(Four));
        }
      }
      f32x4 acc[4];                        // [column of the four]
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
      int own[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) own[i] = __shfl(mine, t * 16 + 4 * q + i);
      auto pass = [&](int ad, int e, const u32x4 (&w)[kS]) {
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < kS; ++s)
#pragma unroll
          for (int k = kTerms - 1; k >= 0; --k) d = mfma_16x16x32<kDt>(terms[t][s][k][lane], w[s], d);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[e][i] = own[i] == ad ? d[i] : acc[e][i];
      };
      if (lead >= 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) pass(lead, e, b[e]);
      }
      for_each_adapter((lane & 31) / 16 == t && mine != lead ? mine : -1, [&](int ad) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u32x4 w[kS];
          read_b(n, ad, e, w);
          pass(ad, e, w);
          __builtin_amdgcn_sched_barrier(0);   // one column's operands at a time
        }
      });
      const f32x4 g = *reinterpret_cast<const f32x4*>(&grow[t * 16 + 4 * q]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (m + i >= a.M) continue;
        // a token without an adapter keeps the bits of its base
        const bool keeps = own[i] < 0;
        if (whole) {
          Four out;
          if constexpr (kY == GPTQ_F32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              out[e] = __float_as_uint(fmaf(acc[e][i], g[i], __uint_as_float(in[i][e])));
          } else {
            out.x = value_bits<kY>(fmaf(acc[0][i], g[i], lo16<kY>(in[i].x))) |
                    value_bits<kY>(fmaf(acc[1][i], g[i], hi16<kY>(in[i].x))) << 16;
            out.y = value_bits<kY>(fmaf(acc[2][i], g[i], lo16<kY>(in[i].y))) |
                    value_bits<kY>(fmaf(acc[3][i], g[i], hi16<kY>(in[i].y))) << 16;
          }
          if (keeps) out = in[i];
          char* o = static_cast<char*>(a.Y) + ((m + i) * a.ld_y + col) * kYE;
          __builtin_memcpy(__builtin_assume_aligned(o, kYE), &out, sizeof(Four));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (col + e >= a.d_out) continue;
            const uint32_t base = a.base ? load_bits<kY>(a.base, (m + i) * a.ld_b + col + e) : 0u;
            const uint32_t y = value_bits<kY>(fmaf(acc[e][i], g[i], bits_value<kY>(base)));
            store_bits<kY>(a.Y, (m + i) * a.ld_y + col + e, keeps ? base : y);
          }
        }
      }
    }
    n += 256;
    read_lead();
  }
}

struct LoraPlan {
  int rp, splits, k_split, cols;
  size_t total;
};

static LoraPlan lora_plan(int64_t M, int64_t d_in, int64_t d_out, int64_t rank) {
  LoraPlan p;
  p.rp = (int)(cdiv(rank, 8) * 8);
  p.splits = 1;
  if (M > kLoraFew) {
    // parts of the sum, of at least one step per wave: for two workgroups per CU,
    // and up to eight parts also for eight of them (a tile of two adapters takes
    // twice as long and must not be the last to end: 8192 x 11008 -> 4096, rank 64,
    // 143 us, and 168 with two per CU).  The second product reads every part's T
    // again: 2048 x 8192 -> 8192, rank 64, takes 68 us in 8 parts and 85 in 32.
    const int64_t tiles = cdiv(M, kLoraTile);
    const int64_t parts = std::max(cdiv(512, tiles), std::min<int64_t>(cdiv(2048, tiles), 8));
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(parts, d_in / 256));
  }
  // columns of a workgroup: as many as leave every CU eight workgroups, so that
  // T's sum is made for more of them.  Here, with 256, 512 and 1024 columns, us:
  // 300 x 4096 -> 14336, rank 32 (256) 19, 22, 33; 8192 x 11008 -> 4096, rank 64
  // (512) 143, 143, 161; 8192 x 4096 -> 14336, rank 64 (1024) 251, 233, 234.
  p.cols = 1024;
  while (p.cols > 256 && cdiv(M, kLoraTile) * cdiv(d_out, p.cols) < 2048) p.cols /= 2;
  p.k_split = (int)(cdiv(cdiv(d_in, p.splits), 128) * 128);
  p.splits = (int)cdiv(d_in, p.k_split);
  p.total = align_up((size_t)p.splits * M * p.rp * 4, 256);
  return p;
}

size_t lora_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out, int64_t rank) {
  return lora_plan(M, d_in, d_out, rank).total;
}

size_t w4a16_lora_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out, int64_t rank) {
  return align_up(w4a16_workspace_bytes(M, d_in, d_out), 256) + lora_workspace_bytes(M, d_in, d_out, rank);
}

template <int kDt, int kY>
static void lora_up_few(const LoraArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)cdiv(a.d_out, 256), (unsigned)a.M);
  if (a.rp <= 8) hipLaunchKernelGGL((lora_up_few_kernel<kDt, kY, 1>), grid, dim3(256), 0, st, a);
  else if (a.rp <= 16) hipLaunchKernelGGL((lora_up_few_kernel<kDt, kY, 2>), grid, dim3(256), 0, st, a);
  else if (a.rp <= 32) hipLaunchKernelGGL((lora_up_few_kernel<kDt, kY, 4>), grid, dim3(256), 0, st, a);
  else if (a.rp <= 64) hipLaunchKernelGGL((lora_up_few_kernel<kDt, kY, 8>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((lora_up_few_kernel<kDt, kY, 16>), grid, dim3(256), 0, st, a);
}

template <int kDt, int kY>
static void lora_up(const LoraArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)lora_blocks(a.M, cdiv(a.d_out, a.cols)));
  if (a.rp <= 32) hipLaunchKernelGGL((lora_up_kernel<kDt, kY, 1>), grid, dim3(256), 0, st, a);
  else if (a.rp <= 64) hipLaunchKernelGGL((lora_up_kernel<kDt, kY, 2>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((lora_up_kernel<kDt, kY, 4>), grid, dim3(256), 0, st, a);
}

template <int kDt>
static void lora_launch(const LoraArgs& a, int32_t y_dtype, hipStream_t st) {
  if (a.M <= kLoraFew) {
    const LoraFew f{a.X, a.A, a.B, a.scale, a.adapter, a.T, a.ld_x, a.M, a.d_out, a.d_in, a.rank, a.n, a.rp};
    hipLaunchKernelGGL(lora_down_few_kernel<kDt>, dim3((unsigned)cdiv(a.M * a.rank, 4)), dim3(256), 0, st, f);
    if (y_dtype == GPTQ_F32) lora_up_few<kDt, GPTQ_F32>(a, st);
    else lora_up_few<kDt, kDt>(a, st);
    return;
  }
  const dim3 grid((unsigned)lora_blocks(a.M, a.splits));
  const bool aligned = a.d_in % 8 == 0 && a.ld_x % 8 == 0 && reinterpret_cast<uintptr_t>(a.X) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.A) % 16 == 0;
  if (aligned) {
    if (a.rank <= 32) hipLaunchKernelGGL((lora_down_lds_kernel<kDt, 2>), grid, dim3(256), 0, st, a);
    else if (a.rank <= 64) hipLaunchKernelGGL((lora_down_lds_kernel<kDt, 4>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((lora_down_lds_kernel<kDt, 8>), grid, dim3(256), 0, st, a);
  } else {
    if (a.rank <= 16) hipLaunchKernelGGL((lora_down_kernel<kDt, 1>), grid, dim3(256), 0, st, a);
    else if (a.rank <= 32) hipLaunchKernelGGL((lora_down_kernel<kDt, 2>), grid, dim3(256), 0, st, a);
    else if (a.rank <= 64) hipLaunchKernelGGL((lora_down_kernel<kDt, 4>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((lora_down_kernel<kDt, 8>), grid, dim3(256), 0, st, a);
  }
  if (y_dtype == GPTQ_F32) lora_up<kDt, GPTQ_F32>(a, st);
  else lora_up<kDt, kDt>(a, st);
}

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_lora_add(const void* X, int32_t x_dtype, int64_t M, int64_t d_in, int64_t ld_x,
                                     const void* A, const void* B, int64_t n_adapters, int32_t rank,
                                     const float* scale, const int32_t* adapter, const void* base, int64_t ld_b,
                                     void* Y, int32_t y_dtype, int64_t d_out, int64_t ld_y, void* workspace,
                                     size_t ws_bytes, void* stream) {
  GQ_CHECK_ARG(x_dtype == GPTQ_F16 || x_dtype == GPTQ_BF16);
  GQ_CHECK_ARG(y_dtype == GPTQ_F32 || y_dtype == x_dtype);
  GQ_CHECK_ARG(M >= 0 && M <= ((int64_t)1 << 24) && d_in >= 1 && d_in <= ((int64_t)1 << 24) && d_out >= 1 &&
               d_out <= ((int64_t)1 << 24));
  GQ_CHECK_ARG(ld_x >= d_in && ld_x <= ((int64_t)1 << 32) && ld_y >= d_out && ld_y <= ((int64_t)1 << 32));
  GQ_CHECK_ARG(base == nullptr || (ld_b >= d_out && ld_b <= ((int64_t)1 << 32)));
  GQ_CHECK_ARG(base == nullptr || base != Y || ld_b == ld_y);
  GQ_CHECK_ARG(n_adapters >= 1 && n_adapters <= ((int64_t)1 << 20) && rank >= 1);
  if (rank > kLoraMaxRank) return GPTQ_EUNSUPPORTED;
  if (M == 0) return GPTQ_OK;
  const size_t ys = y_dtype == GPTQ_F32 ? 4 : 2;
  GQ_CHECK_ARG(X && A && B && adapter && Y);
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(X) % 2 == 0 && reinterpret_cast<uintptr_t>(A) % 2 == 0 &&
               reinterpret_cast<uintptr_t>(B) % 2 == 0 && reinterpret_cast<uintptr_t>(Y) % ys == 0 &&
               reinterpret_cast<uintptr_t>(base) % ys == 0);
  const LoraPlan pl = lora_plan(M, d_in, d_out, rank);
  if (workspace == nullptr || ws_bytes < pl.total) return GPTQ_ENOMEM;
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(workspace) % 256 == 0);
  LoraArgs a{};
  a.X = static_cast<const uint16_t*>(X);
  a.A = static_cast<const uint16_t*>(A);
  a.B = static_cast<const uint16_t*>(B);
  a.scale = scale;
  a.adapter = adapter;
  a.base = base;
  a.Y = Y;
  a.T = static_cast<float*>(workspace);
  a.ld_x = ld_x;
  a.ld_b = ld_b;
  a.ld_y = ld_y;
  a.M = M;
  a.d_out = d_out;
  a.d_in = (int)d_in;
  a.rank = rank;
  a.n = (int)n_adapters;
  a.rp = pl.rp;
  a.splits = pl.splits;
  a.k_split = pl.k_split;
  a.cols = pl.cols;
  hipStream_t st = static_cast<hipStream_t>(stream);
  TimedScope ts(kTimeLora, st);
  if (x_dtype == GPTQ_F16) lora_launch<GPTQ_F16>(a, y_dtype, st);
  else lora_launch<GPTQ_BF16>(a, y_dtype, st);
  GQ_LAUNCHED();
  return GPTQ_OK;
}

extern "C" gptq_status gptq_w4a16_lora_matmul(const void* X, int32_t x_dtype, int64_t M, int64_t d_in, int64_t ld_x,
                                              const uint8_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                                              const int32_t* perm, int64_t d_out, int32_t group_size, const void* A,
                                              const void* B, int64_t n_adapters, int32_t rank, const float* scale,
                                              const int32_t* adapter, float* Y, int64_t ld_y, void* workspace,
                                              size_t ws_bytes, void* stream) {
  GQ_CHECK_ARG(M >= 1 && d_in >= 1 && d_out >= 1 && rank >= 1 && n_adapters >= 1 && n_adapters <= ((int64_t)1 << 20));
  GQ_CHECK_ARG(A && B && adapter);
  GQ_CHECK_ARG(ld_x <= ((int64_t)1 << 32) && ld_y <= ((int64_t)1 << 32));
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(A) % 2 == 0 && reinterpret_cast<uintptr_t>(B) % 2 == 0);
  if (rank > kLoraMaxRank || M > 64) return GPTQ_EUNSUPPORTED;
  if (workspace != nullptr && ws_bytes < w4a16_lora_workspace_bytes(M, d_in, d_out, rank)) return GPTQ_ENOMEM;
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(workspace) % 256 == 0);
  const size_t w4 = align_up(w4a16_workspace_bytes(M, d_in, d_out), 256);
  const LoraFew f{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(A), static_cast<const uint16_t*>(B), scale,
                  adapter, reinterpret_cast<float*>(static_cast<char*>(workspace) + w4), ld_x, M, d_out, (int)d_in, rank,
                  (int)n_adapters, (int)(cdiv(rank, 8) * 8)};
  return w4a16_run(X, x_dtype, M, d_in, ld_x, qweight, scales, zeros, perm, d_out, group_size, Y, ld_y, workspace,
                   ws_bytes, &f, static_cast<hipStream_t>(stream));
}
