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
// does not reach another's rows.  For the second product T is kept as two
// 16-bit terms, whose sum carries 16 significant bits (bf16) or 22 (fp16; rows
// of T are scaled by a power of two first, so that neither their size nor
// their smallness leaves fp16's range): 16 bits alone would put an error of
// 2^-9 or 2^-12 of the adapter's part into fp32 results.  Tokens are the MFMA's
// columns and output columns its rows, dealt so that a lane ends up with eight
// consecutive outputs of one token: base and Y move 16 or 32 bytes at a time.
// Operands are read from global memory in the form that the MFMA takes (8
// consecutive elements per lane), at any alignment.
//
// Bound by memory: X, base and Y once, the factors from L2 (a factor's matrix
// serves every tile of its adapter).
#include "lora.h"

namespace gq {

size_t w4a16_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out);

constexpr int kLoraFew = 64;        // tokens up to which every one is taken by itself
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
  float y = 0.f;
  if (a.base && n < a.d_out) y = load_el<kY>(a.base, m * a.ld_b + n);
  if (ad >= 0 && ad < a.n && n0 < a.d_out) {
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
template <int kDt>
__device__ __forceinline__ f32x4 lora_mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (kDt == GPTQ_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}

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
  const int64_t m0 = (int64_t)blockIdx.x * kLoraTile;
  const int k0 = blockIdx.y * a.k_split, k1 = min(k0 + a.k_split, a.d_in);
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
          acc[t][0] = lora_mfma<kDt>(p.f[j][t], p.x[j][0], acc[t][0]);
          acc[t][1] = lora_mfma<kDt>(p.f[j][t], p.x[j][1], acc[t][1]);
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
      float* out = a.T + ((int64_t)blockIdx.y * a.M + m0 + tok) * a.rp;
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

// hi and lo terms of 8 values, as MFMA operands.
template <int kDt>
__device__ __forceinline__ void lora_split(const float (&v)[8], u32x4& hi, u32x4& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x = v[2 * i + e];
      if constexpr (kDt == GPTQ_F16) {
        const _Float16 p = (_Float16)x, r = (_Float16)(x - (float)p);
        h[e] = __builtin_bit_cast(uint16_t, p);
        l[e] = __builtin_bit_cast(uint16_t, r);
      } else {
        const __bf16 p = (__bf16)x, r = (__bf16)(x - (float)p);
        h[e] = __builtin_bit_cast(uint16_t, p);
        l[e] = __builtin_bit_cast(uint16_t, r);
      }
    }
    hi[i] = h[0] | h[1] << 16;
    lo[i] = l[0] | l[1] << 16;
  }
}

// 32 tokens by `cols` columns (a multiple of 128); kS steps of 32 ranks.
template <int kDt, int kY, int kS>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
  constexpr int kPitch = kS * 32 + 4;
  __shared__ __align__(16) float tsum[kLoraTile][kPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * kLoraTile;
  const int mine = lora_adapter(a, m0 + (lane & 31));
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
  int own[2];                              // adapters of this lane's two tokens
  float grow[2];                           // 2^e that T's terms were divided by
  u32x4 hi[2][kS], lo[2][kS];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    own[t] = __shfl(mine, t * 16 + c16);
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
          big = fmaxf(big, fabsf(u[i]));
        }
      }
    grow[t] = 1.f;
    if constexpr (kDt == GPTQ_F16) {
      big = fmaxf(big, __shfl_xor(big, 16));
      big = fmaxf(big, __shfl_xor(big, 32));
      if (big > 0.f && big < INFINITY) {
        int e;
        frexpf(big, &e);
        grow[t] = ldexpf(1.f, e - 14);   // the largest below 2^14: the second terms stay normal numbers
#pragma unroll
        for (int s = 0; s < kS; ++s)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[s][i] = ldexpf(v[s][i], 14 - e);
      }
    }
#pragma unroll
    for (int s = 0; s < kS; ++s) lora_split<kDt>(v[s], hi[t][s], lo[t][s]);
  }
  const int64_t n_first = (int64_t)blockIdx.y * a.cols;
  const int64_t n_end = n_first + a.cols < a.d_out ? n_first + a.cols : a.d_out;
  const uint32_t tile = (uint32_t)__ballot(mine >= 0);
  const int lead = tile ? __builtin_amdgcn_readlane(mine, __builtin_ctz(tile)) : -1;   // the tile's first adapter

  // A step's base and the first adapter's B, in memory's form, asked for while
  // the step before is worked on.  kYW 16-byte words hold 8 outputs.
  constexpr int kYW = kY == GPTQ_F32 ? 2 : 1;
  constexpr int kYE = kY == GPTQ_F32 ? 4 : 2;
  struct Step {
    u32x4 y[2][kYW], b[2][kS];
  };
  auto read_b = [&](int64_t n, int ad, u32x4 (&b)[2][kS]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // the MFMA's row c16 is column 8 (c16 / 4) + 4 h + c16 % 4
      int64_t bc = n + 8 * (c16 >> 2) + 4 * h + (c16 & 3);
      bc = bc < a.d_out ? bc : a.d_out - 1;
      const uint16_t* row = a.B + ((int64_t)ad * a.d_out + bc) * a.rank;
#pragma unroll
      for (int s = 0; s < kS; ++s) {
        if (a.rank == kS * 32) b[h][s] = load8(row + s * 32 + 8 * q);
        else b[h][s] = load8_end(row, s * 32 + 8 * q, a.rank);
      }
    }
  };
  auto read = [&](int64_t n, Step& p) {
    if (a.base && a.d_out >= 8) {
      const int64_t col = min(n + 8 * q, a.d_out - 8);   // lanes at the end read theirs one by one later
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const char* y = static_cast<const char*>(a.base) + (min(m0 + t * 16 + c16, a.M - 1) * a.ld_b + col) * kYE;
#pragma unroll
        for (int w = 0; w < kYW; ++w) {
          if constexpr (kY == GPTQ_F32) __builtin_memcpy(&p.y[t][w], __builtin_assume_aligned(y + 16 * w, 4), 16);
          else __builtin_memcpy(&p.y[t][w], __builtin_assume_aligned(y, 2), 16);
        }
      }
    }
    if (lead >= 0) read_b(n, lead, p.b);
  };
  auto finish = [&](int64_t n, const Step& p) {
    const int64_t col = n + 8 * q;         // this lane's eight columns
    const bool whole = col + 8 <= a.d_out;
    f32x4 acc[2][2];                       // [token tile][column half]
#pragma unroll
    for (int t = 0; t < 2; ++t) acc[t][0] = acc[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto pass = [&](int ad, const u32x4 (&b)[2][kS]) {
      f32x4 d[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) d[t][0] = d[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            d[t][h] = lora_mfma<kDt>(b[h][s], lo[t][s], d[t][h]);
            d[t][h] = lora_mfma<kDt>(b[h][s], hi[t][s], d[t][h]);
          }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][h][i] = own[t] == ad ? d[t][h][i] : acc[t][h][i];
    };
    for_each_adapter(mine, [&](int ad) {
      if (ad == lead) {
        pass(ad, p.b);
      } else {
        u32x4 b[2][kS];
        read_b(n, ad, b);
        pass(ad, b);
      }
    });
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t m = m0 + t * 16 + c16;
      if (m >= a.M) continue;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = 0.f;
      if (a.base) {
        if (whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (kY == GPTQ_F32) {
              y[i] = __uint_as_float(p.y[t][0][i]);
              y[4 + i] = __uint_as_float(p.y[t][kYW - 1][i]);
            } else {
              y[2 * i] = lo16<kY>(p.y[t][0][i]);
              y[2 * i + 1] = hi16<kY>(p.y[t][0][i]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + i < a.d_out) y[i] = load_el<kY>(a.base, m * a.ld_b + col + i);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[4 * h + i] = fmaf(acc[t][h][i], grow[t], y[4 * h + i]);
      if (whole) {
        if constexpr (kY == GPTQ_F32) {
          float* o = static_cast<float*>(a.Y) + m * a.ld_y + col;
          __builtin_memcpy(__builtin_assume_aligned(o, 4), &y[0], 16);
          __builtin_memcpy(__builtin_assume_aligned(o + 4, 4), &y[4], 16);
        } else {
          typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
          u16x8 w;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if constexpr (kY == GPTQ_F16) w[i] = __builtin_bit_cast(uint16_t, (_Float16)y[i]);
            else w[i] = __builtin_bit_cast(uint16_t, (__bf16)y[i]);
          }
          __builtin_memcpy(__builtin_assume_aligned(static_cast<uint16_t*>(a.Y) + m * a.ld_y + col, 2), &w, 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < a.d_out) store_el<kY>(a.Y, m * a.ld_y + col + i, y[i]);
      }
    }
  };
  int64_t n = n_first + wave * 32;
  if (n >= n_end) return;
  Step even, odd;
  read(n, even);
  for (; n < n_end; n += 256) {
    if (n + 128 < n_end) read(n + 128, odd);
    finish(n, even);
    if (n + 128 < n_end) {
      if (n + 256 < n_end) read(n + 256, even);
      finish(n + 128, odd);
    }
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
    // parts of the sum until every CU has two workgroups, of at least one step per wave
    const int64_t tiles = cdiv(M, kLoraTile);
    p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(cdiv(512, tiles), d_in / 256));
  }
  // columns of a workgroup: as many as leave every CU four workgroups, so that
  // T's sum is made for more of them
  p.cols = 1024;
  while (p.cols > 128 && cdiv(M, kLoraTile) * cdiv(d_out, p.cols) < 1024) p.cols /= 2;
  p.k_split = (int)(cdiv(cdiv(d_in, p.splits), 64) * 64);
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
  const dim3 grid((unsigned)cdiv(a.M, kLoraTile), (unsigned)cdiv(a.d_out, a.cols));
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
  const dim3 grid((unsigned)cdiv(a.M, kLoraTile), (unsigned)a.splits);
  if (a.rank <= 16) hipLaunchKernelGGL((lora_down_kernel<kDt, 1>), grid, dim3(256), 0, st, a);
  else if (a.rank <= 32) hipLaunchKernelGGL((lora_down_kernel<kDt, 2>), grid, dim3(256), 0, st, a);
  else if (a.rank <= 64) hipLaunchKernelGGL((lora_down_kernel<kDt, 4>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((lora_down_kernel<kDt, 8>), grid, dim3(256), 0, st, a);
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
