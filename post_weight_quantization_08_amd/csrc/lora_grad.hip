// Gradients of low-rank adapters:  Y[m] = base[m] + s_a (X[m] A_a^T) B_a^T, a = adapter[m].
//   U[m] = s_a dY[m] B_a,  T[m] = s_a X[m] A_a^T           (rank numbers a token)
//   dA_a = sum_m U[m]^T X[m],  dB_a = sum_m dY[m]^T T[m],  dX[m] = base[m] + U[m] A_a
// over the tokens of adapter a.
//
// Launches: tokens sorted by adapter and factors laid out (prep), U and T (project),
// the sums over tokens (outer), their parts joined where an adapter has many tokens,
// and dX by the adapters' own second product.
//
// X and dY enter as bf16 terms: one for bf16 and e4m3 (exact, scale included), two for
// fp16 (exact) and fp32 (2^-17 of a value or less); U and T as two, rounded: 2^-17 of
// them.  Their products with each other leave out low by low.  Sums are fp32.
//
// The sums over tokens want eight consecutive tokens of a column in a lane.  Every lane
// loads eight (four) columns of eight tokens and turns them in registers, which needs
// no LDS and works for every type.
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
  int32_t* order;                   // [P]: token at a position
  int32_t* pos;                     // [M]: position of a token, -1 without an adapter
  GradChunk* chunks;
  int32_t* parts;                   // [n][2]: an adapter's first slot and its parts
  int32_t* n_chunks;
};

// One operand: rows of X with A, or rows of dY with B^T.
struct GradSide {
  const void* D;
  const uint8_t* scales;            // [M][nb], e4m3
  int64_t ld;
  int K, nb;
  const uint16_t* F;                // bf16 [terms][n][rank][ld_f]
  int64_t f_term;
  int ld_f;
  float* full;                      // fp32 [M][rp], or null
  uint16_t* turned;                 // bf16 [2][rank tiles * 16][P]: what this side's product gives
  const uint16_t* by;               // the other side's `turned`, which its sum over tokens takes
  float* grad;                      // [n][rank * K]
  float* part;                      // [slots][rank * K]
  int rank_first;                   // the gradient's rows are ranks (dA) or columns (dB)
};

struct GradArgs {
  GradSide side;
  GradPlace at;
  const int32_t* adapter;
  const float* scale;
  int64_t M, P;
  int n, rank, rp;
  int terms;                        // of the factors
  int blocks;                       // column blocks
};

// ---------------------------------------------------------------- sorting
// Tokens into runs of one adapter, each starting at a multiple of 32, in their own
// order; by one workgroup: every wave counts a range, then places it.
struct GradSort {
  const int32_t* adapter;
  GradPlace at;
  int64_t M;
  int n, chunk;
};

__device__ void grad_sort(const GradSort& a, uint32_t (*hist)[kGradMaxAdapters], uint32_t* scan) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  for (int w = 0; w < 16; ++w) hist[w][t] = 0;
  __syncthreads();
  const int64_t per = (a.M + 1023) / 1024 * 64, first = wave * per, last = min(first + per, a.M);
  for (int64_t m = first + lane; m < last; m += 64) {
    const int ad = a.adapter[m];
    if (ad >= 0 && ad < a.n) atomicAdd(&hist[wave][ad], 1u);   // counts: their order is nothing
  }
  __syncthreads();
  // thread t is adapter t
  uint32_t count = 0;
  for (int w = 0; w < 16; ++w) count += hist[w][t];
  const uint32_t parts = t < a.n ? max(1u, (count + a.chunk - 1) / a.chunk) : 0u;
  auto before = [&](uint32_t v) {   // sum over the threads before this one
    uint32_t s = v;
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = (uint32_t)__shfl_up((int)s, d);
      if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 63) scan[wave] = s;
    __syncthreads();
    uint32_t base = 0;
    for (int w = 0; w < wave; ++w) base += scan[w];
    return base + s - v;
  };
  const uint32_t start = before((count + 31) / 32 * 32);
  const uint32_t chunk0 = before(parts), slot0 = before(parts > 1 ? parts : 0u);
  uint32_t next = start;
  for (int w = 0; w < 16; ++w) {
    const uint32_t c = hist[w][t];
    hist[w][t] = next;
    next += c;
  }
  if (t < a.n) {
    a.at.parts[2 * t] = (int)slot0;
    a.at.parts[2 * t + 1] = (int)parts;
    for (uint32_t p = 0; p < parts; ++p)
      a.at.chunks[chunk0 + p] = GradChunk{t, (int)(start + p * a.chunk), (int)min(start + (p + 1) * a.chunk, start + count),
                                          parts > 1 ? (int)(slot0 + p) : -1};
  }
  if (t == a.n - 1) *a.at.n_chunks = (int)(chunk0 + parts);
  __syncthreads();
  for (int64_t m0 = first; m0 < last; m0 += 64) {
    const int64_t m = m0 + lane;
    int ad = m < last ? a.adapter[m] : -1;
    if (ad < 0 || ad >= a.n) ad = -1;
    int mine = -1;
    uint64_t left = __ballot(ad >= 0);
    while (left) {
      const int one = __builtin_amdgcn_readlane(ad, __builtin_ctzll(left));
      const uint64_t same = __ballot(ad == one);
      left &= ~same;
      const uint32_t base = hist[wave][one];
      if (ad == one) mine = (int)(base + __popcll(same & ((1ull << lane) - 1)));
      if (lane == 0) hist[wave][one] = base + __popcll(same);
    }
    if (m < last) a.at.pos[m] = mine;
    if (mine >= 0) a.at.order[mine] = (int32_t)m;
  }
}

// Factors as the products want them: B^T in bf16 terms [terms][n][rank][ld_b], A in
// terms [2][n][rank][ld_a] if it is fp16, and A^T for dX.  Tiles of 32 x 32 of A and
// of B, one after the other.
struct GradPrep {
  GradSort sort;
  const uint16_t* A;
  const uint16_t* B;
  uint16_t* a_terms;        // or null
  uint16_t* b_terms;
  uint16_t* a_turned;       // or null
  int d_in, d_out, rank, ld_a, ld_b;
  int a_tiles, b_tiles;     // of one adapter: tiles along its length times tiles of ranks
};

// An fp16 or bf16 number's bf16 terms.
template <int kF>
__device__ __forceinline__ void grad_split1(uint32_t w, uint32_t& hi, uint32_t& lo) {
  if constexpr (kF == GPTQ_BF16) {
    hi = w;
    lo = 0;
  } else {
    const float x = f16_bits_to_f32(w);
    hi = value_bits<GPTQ_BF16>(x);
    lo = value_bits<GPTQ_BF16>(x - bf16_bits_to_f32(hi));
  }
}

template <int kF>
__global__ __launch_bounds__(1024) void lora_grad_prep_kernel(GradPrep a) {
  __shared__ union {
    struct {
      uint32_t hist[16][kGradMaxAdapters];
      uint32_t scan[16];
    } s;
    uint16_t tile[32][34];
  } u;
  if (blockIdx.x == 0) {
    grad_sort(a.sort, u.s.hist, u.s.scan);
    return;
  }
  const int per = a.a_tiles + a.b_tiles, id = blockIdx.x - 1, ad = id / per;
  int i = id % per;
  const bool is_b = i >= a.a_tiles;
  if (is_b) i -= a.a_tiles;
  const int rank_tiles = (a.rank + 31) / 32;
  const int r0 = i % rank_tiles * 32, k0 = i / rank_tiles * 32;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int K = is_b ? a.d_out : a.d_in, ld = is_b ? a.ld_b : a.ld_a;
  const int64_t plane = (int64_t)a.sort.n * a.rank * ld;
  if (is_b) {
    // rows of B are its length
    u.tile[y][x] = k0 + y < K && r0 + x < a.rank ? a.B[((int64_t)ad * K + k0 + y) * a.rank + r0 + x] : 0;
    __syncthreads();
    if (r0 + y < a.rank && k0 + x < ld) {
      uint32_t hi, lo;
      grad_split1<kF>(u.tile[x][y], hi, lo);
      uint16_t* o = a.b_terms + ((int64_t)ad * a.rank + r0 + y) * ld + k0 + x;
      o[0] = (uint16_t)hi;
      if (kF == GPTQ_F16) o[plane] = (uint16_t)lo;
    }
    return;
  }
  u.tile[y][x] = r0 + y < a.rank && k0 + x < K ? a.A[((int64_t)ad * a.rank + r0 + y) * K + k0 + x] : 0;
  __syncthreads();
  if (kF == GPTQ_F16 && r0 + y < a.rank && k0 + x < ld) {
    uint32_t hi, lo;
    grad_split1<kF>(u.tile[y][x], hi, lo);
    uint16_t* o = a.a_terms + ((int64_t)ad * a.rank + r0 + y) * ld + k0 + x;
    o[0] = (uint16_t)hi;
    o[plane] = (uint16_t)lo;
  }
  if (a.a_turned && k0 + y < K && r0 + x < a.rank)
    a.a_turned[((int64_t)ad * K + k0 + y) * a.rank + r0 + x] = u.tile[x][y];
}

// ---------------------------------------------------------------- eight numbers of a row
template <int kD>
struct Eight {
  static constexpr int kTerms = kD == GPTQ_F16 || kD == GPTQ_F32 ? 2 : 1;
  u32x4 w[kD == GPTQ_F32 ? 2 : 1];

  // elements k .. k + 7 of a row of n, zero behind its end (e4m3: the codes there are zero)
  __device__ __forceinline__ void load(const void* row, int k, int n) {
    if constexpr (kD == GPTQ_E4M3) {
      uint2 v = {0u, 0u};
      if (k < n) v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(row) + k);
      w[0] = u32x4{v.x, v.y, 0u, 0u};
    } else if constexpr (kD == GPTQ_F32) {
      const float* p = static_cast<const float*>(row);
      if (k + 8 <= n) {
        __builtin_memcpy(w, __builtin_assume_aligned(p + k, 4), 32);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i / 4][i % 4] = k + i < n ? __float_as_uint(p[k + i]) : 0u;
      }
    } else {
      w[0] = load8_end(static_cast<const uint16_t*>(row), k, n);
    }
  }
  __device__ __forceinline__ void clear() {
    w[0] = u32x4{0u, 0u, 0u, 0u};
    if constexpr (kD == GPTQ_F32) w[1] = w[0];
  }
  // as bf16; `b` is the scale's byte
  __device__ __forceinline__ void terms(uint32_t b, u32x4 (&t)[kTerms]) const {
    if constexpr (kD == GPTQ_E4M3) {
      const float s = __uint_as_float(b << 23);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        t[0][2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0][i], s, false));
        t[0][2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0][i], s, true));
      }
    } else if constexpr (kD == GPTQ_BF16) {
      t[0] = w[0];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x, y;
        if constexpr (kD == GPTQ_F16) {
          x = lo16<GPTQ_F16>(w[0][i]);
          y = hi16<GPTQ_F16>(w[0][i]);
        } else {
          x = __uint_as_float(w[i / 2][i % 2 * 2]);
          y = __uint_as_float(w[i / 2][i % 2 * 2 + 1]);
        }
        const uint32_t h = value_bits<GPTQ_BF16>(x) | value_bits<GPTQ_BF16>(y) << 16;
        t[0][i] = h;
        t[1][i] = value_bits<GPTQ_BF16>(x - __uint_as_float(h << 16)) |
                  value_bits<GPTQ_BF16>(y - __uint_as_float(h & 0xFFFF0000u)) << 16;
      }
    }
  }
};

template <int kD>
__device__ __forceinline__ const char* grad_row(const GradSide& s, int64_t m) {
  return static_cast<const char*>(s.D) + m * s.ld * (kD == GPTQ_F32 ? 4 : kD == GPTQ_E4M3 ? 1 : 2);
}

// ---------------------------------------------------------------- U and T
// 32 tokens by all ranks: the waves take the sum's 32-element steps in turn and their
// sums meet in LDS.  D: rows = ranks, columns = tokens.
constexpr int kProjWaves = 8;

template <int kD, int kR>
__global__ __launch_bounds__(64 * kProjWaves) void lora_grad_project_kernel(GradArgs a) {
  constexpr int kStride = kR * 16 + 4;
  constexpr int kT = Eight<kD>::kTerms;
  __shared__ __align__(16) float red[kProjWaves][kGradTile][kStride];
  const GradSide& s = a.side;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * kGradTile;
  const int64_t mine_at = m0 + (lane & 31);
  int mine = mine_at < a.M ? a.adapter[mine_at] : -1;
  if (mine < 0 || mine >= a.n) mine = -1;
  const char* x[2];
  const uint8_t* sc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t m = min(m0 + t * 16 + c16, a.M - 1);
    x[t] = grad_row<kD>(s, m);
    sc[t] = kD == GPTQ_E4M3 ? s.scales + m * s.nb : nullptr;
  }
  uint32_t left = (uint32_t)__ballot(mine >= 0);
  while (left) {
    const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(mine == ad);
    const uint16_t* f[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) f[r] = s.F + ((int64_t)ad * a.rank + min(r * 16 + c16, a.rank - 1)) * s.ld_f;
    f32x4 acc[kR][2];
#pragma unroll
    for (int r = 0; r < kR; ++r) acc[r][0] = acc[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = wave * 32; k < s.K; k += 32 * kProjWaves) {
      u32x4 d[2][kT], fw[kR], fl[kR];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        Eight<kD> e;
        e.load(x[t], k + 8 * q, s.K);
        e.terms(kD == GPTQ_E4M3 ? sc[t][k / kF8Block] : 0u, d[t]);
      }
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        fw[r] = load8_end(f[r], k + 8 * q, s.K);
        if (a.terms > 1) fl[r] = load8_end(f[r] + s.f_term, k + 8 * q, s.K);
      }
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if constexpr (kT > 1) acc[r][t] = mfma_16x16x32<GPTQ_BF16>(fw[r], d[t][kT - 1], acc[r][t]);
          if (a.terms > 1) acc[r][t] = mfma_16x16x32<GPTQ_BF16>(fl[r], d[t][0], acc[r][t]);
          acc[r][t] = mfma_16x16x32<GPTQ_BF16>(fw[r], d[t][0], acc[r][t]);
        }
    }
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int t = 0; t < 2; ++t) *reinterpret_cast<f32x4*>(&red[wave][t * 16 + c16][r * 16 + 4 * q]) = acc[r][t];
    __syncthreads();
    const int tok = threadIdx.x & 31;
    if (__shfl(mine, tok) == ad) {
      const int64_t m = m0 + tok;
      const float by = a.scale ? a.scale[ad] : 1.f;
      const int pos = a.at.pos[m];
      for (int r = (threadIdx.x >> 5) * 4; r < kR * 16; r += 8 * kProjWaves) {
        f32x4 v = *reinterpret_cast<const f32x4*>(&red[0][tok][r]);
#pragma unroll
        for (int w = 1; w < kProjWaves; ++w) v += *reinterpret_cast<const f32x4*>(&red[w][tok][r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = r + i < a.rank ? v[i] * by : 0.f;
          const uint32_t h = value_bits<GPTQ_BF16>(v[i]);
          uint16_t* o = s.turned + (int64_t)(r + i) * a.P + pos;
          o[0] = (uint16_t)h;
          o[(int64_t)(kR * 16) * a.P] = (uint16_t)value_bits<GPTQ_BF16>(v[i] - bf16_bits_to_f32(h));
        }
        if (s.full && r < a.rp) *reinterpret_cast<f32x4*>(s.full + m * a.rp + r) = v;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- sums over tokens
// A workgroup sums a chunk of one adapter's tokens for 16 kC columns and all ranks;
// its waves take the steps of 32 tokens in turn.  D: rows = ranks, columns = columns:
// lane c16 holds columns kC c16 .. + kC - 1, column p of them in tile p.
constexpr int kOuterWaves = 4;

template <int kD, int kR, int kC>
__global__ __launch_bounds__(64 * kOuterWaves) void lora_grad_outer_kernel(GradArgs a) {
  constexpr int kT = Eight<kD>::kTerms;
  static_assert(kC == 8, "eight columns a lane");
  __shared__ __align__(16) f32x4 red[kR * kC][64];
  const GradSide& s = a.side;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int block = blockIdx.x % a.blocks, ci = blockIdx.x / a.blocks;
  if (ci >= *a.at.n_chunks) return;
  const GradChunk ch = a.at.chunks[ci];
  const int n0 = block * (16 * kC), col = n0 + c16 * kC;
  const uint16_t* by[kR][2];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < 2; ++t) by[r][t] = s.by + (int64_t)((t * kR + r) * 16 + c16) * a.P;
  f32x4 acc[kR][kC];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int p = 0; p < kC; ++p) acc[r][p] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int pos = ch.begin + wave * kGradTile; pos < ch.end; pos += kOuterWaves * kGradTile) {
    const int first = pos + 8 * q;
    Eight<kD> e[8];
    uint32_t sb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sb[i] = 127u;
      if (first + i < ch.end) {
        const int64_t m = a.at.order[first + i];
        e[i].load(grad_row<kD>(s, m), col, kD == GPTQ_E4M3 ? s.nb * kF8Block : s.K);
        if (kD == GPTQ_E4M3 && col < s.nb * kF8Block) sb[i] = s.scales[m * s.nb + col / kF8Block];
      } else {
        e[i].clear();
      }
    }
    u32x4 u[kR][2];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u[r][t] = *reinterpret_cast<const u32x4*>(by[r][t] + first);
        if (pos + kGradTile > ch.end) {   // behind the chunk: another one's, or nothing
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (first + i >= ch.end) u[r][t][i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
        }
      }
    u32x4 x[8][kT];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i].terms(sb[i], x[i]);
#pragma unroll
    for (int p = 0; p < kC; ++p) {
      u32x4 d[kT];
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          d[t][j] = __builtin_amdgcn_perm(x[2 * j + 1][t][p / 2], x[2 * j][t][p / 2], p % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if constexpr (kT > 1) acc[r][p] = mfma_16x16x32<GPTQ_BF16>(u[r][0], d[kT - 1], acc[r][p]);
        acc[r][p] = mfma_16x16x32<GPTQ_BF16>(u[r][1], d[0], acc[r][p]);
        acc[r][p] = mfma_16x16x32<GPTQ_BF16>(u[r][0], d[0], acc[r][p]);
      }
    }
  }
  // the waves' sums one after the other
  for (int w = kOuterWaves - 1; w > 0; --w) {
    if (wave == w) {
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int p = 0; p < kC; ++p) red[r * kC + p][lane] = acc[r][p];
    }
    __syncthreads();
    if (wave == w - 1) {
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int p = 0; p < kC; ++p) acc[r][p] += red[r * kC + p][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
  const int64_t each = (int64_t)a.rank * s.K;
  float* out = ch.slot < 0 ? s.grad + ch.adapter * each : s.part + ch.slot * each;
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rank = r * 16 + 4 * q + i;
      if (rank >= a.rank) continue;
#pragma unroll
      for (int p = 0; p < kC; ++p)
        if (col + p < s.K) out[s.rank_first ? (int64_t)rank * s.K + col + p : (int64_t)(col + p) * a.rank + rank] = acc[r][p][i];
    }
}

// The parts of adapters that have several, added up in order.
__global__ __launch_bounds__(256) void lora_grad_join_kernel(GradArgs a) {
  const int ad = blockIdx.y, slot = a.at.parts[2 * ad], parts = a.at.parts[2 * ad + 1];
  if (parts < 2) return;
  const int64_t each = (int64_t)a.rank * a.side.K;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < each; i += (int64_t)gridDim.x * 256) {
    float v = 0.f;
    for (int p = 0; p < parts; ++p) v += a.side.part[(slot + p) * each + i];
    a.side.grad[ad * each + i] = v;
  }
}

// ---------------------------------------------------------------- host
struct GradPlan {
  int rp, r16, ld_a, ld_b, chunk;
  int64_t P, max_chunks, slots;
  size_t order, pos, chunks, parts, count, a_terms, b_terms, a_turned, full, turned_u, turned_t, part_a, part_b, total;
};

static GradPlan grad_plan(int64_t M, int64_t d_in, int64_t d_out, int64_t rank, int64_t n) {
  GradPlan p{};
  p.rp = (int)(cdiv(rank, 8) * 8);
  p.r16 = rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128;
  p.ld_a = (int)(cdiv(d_in, 8) * 8);
  p.ld_b = (int)(cdiv(d_out, 8) * 8);
  const int64_t blocks = cdiv(d_in, 128) + cdiv(d_out, 128);
  const int64_t want = std::max<int64_t>(1, std::min(cdiv(512, blocks), M / 128));
  p.chunk = (int)(cdiv(cdiv(M, want), 32) * 32);
  p.P = align_up(M + 32 * n + 32, 64);
  p.max_chunks = cdiv(M, p.chunk) + n;
  p.slots = M > p.chunk ? 2 * cdiv(M, p.chunk) : 0;
  Carver c(nullptr);
  auto take = [&](size_t bytes) {
    c.take<char>(bytes);
    return c.used - bytes;
  };
  p.order = take((size_t)p.P * 4);
  p.pos = take((size_t)M * 4);
  p.chunks = take((size_t)p.max_chunks * sizeof(GradChunk));
  p.parts = take((size_t)n * 8);
  p.count = take(4);
  p.a_terms = take((size_t)2 * n * rank * p.ld_a * 2);
  p.b_terms = take((size_t)2 * n * rank * p.ld_b * 2);
  p.a_turned = take((size_t)n * rank * d_in * 2);
  p.full = take((size_t)M * p.rp * 4);
  p.turned_u = take((size_t)2 * p.r16 * p.P * 2);
  p.turned_t = take((size_t)2 * p.r16 * p.P * 2);
  p.part_a = take((size_t)p.slots * rank * d_in * 4);
  p.part_b = take((size_t)p.slots * rank * d_out * 4);
  p.total = align_up(c.used, 256);
  return p;
}

template <int kD>
static void grad_project(const GradArgs& a, int r16, hipStream_t st) {
  const dim3 grid((unsigned)cdiv(a.M, kGradTile)), block(64 * kProjWaves);
  if (r16 == 16) hipLaunchKernelGGL((lora_grad_project_kernel<kD, 1>), grid, block, 0, st, a);
  else if (r16 == 32) hipLaunchKernelGGL((lora_grad_project_kernel<kD, 2>), grid, block, 0, st, a);
  else if (r16 == 64) hipLaunchKernelGGL((lora_grad_project_kernel<kD, 4>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((lora_grad_project_kernel<kD, 8>), grid, block, 0, st, a);
}

template <int kD>
static void grad_outer(const GradArgs& a, int r16, int64_t max_chunks, hipStream_t st) {
  const dim3 grid((unsigned)(a.blocks * max_chunks)), block(64 * kOuterWaves);
  if (r16 == 16) hipLaunchKernelGGL((lora_grad_outer_kernel<kD, 1, 8>), grid, block, 0, st, a);
  else if (r16 == 32) hipLaunchKernelGGL((lora_grad_outer_kernel<kD, 2, 8>), grid, block, 0, st, a);
  else if (r16 == 64) hipLaunchKernelGGL((lora_grad_outer_kernel<kD, 4, 8>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((lora_grad_outer_kernel<kD, 8, 8>), grid, block, 0, st, a);
}

template <class F>
static void grad_typed(int dtype, F f) {
  if (dtype == GPTQ_E4M3) f(std::integral_constant<int, GPTQ_E4M3>());
  else if (dtype == GPTQ_F32) f(std::integral_constant<int, GPTQ_F32>());
  else if (dtype == GPTQ_F16) f(std::integral_constant<int, GPTQ_F16>());
  else f(std::integral_constant<int, GPTQ_BF16>());
}

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_lora_grad_workspace_size(int64_t M, int64_t d_in, int64_t d_out, int32_t rank,
                                                     int64_t n_adapters, size_t* bytes_out) {
  GQ_CHECK_ARG(bytes_out && M >= 0 && d_in >= 1 && d_out >= 1 && rank >= 1 && n_adapters >= 1);
  if (rank > kGradMaxRank || n_adapters > kGradMaxAdapters || M > ((int64_t)1 << 22) || d_in > ((int64_t)1 << 22) ||
      d_out > ((int64_t)1 << 22))
    return GPTQ_EUNSUPPORTED;
  *bytes_out = grad_plan(std::max<int64_t>(M, 1), d_in, d_out, rank, n_adapters).total;
  return GPTQ_OK;
}

extern "C" gptq_status gptq_lora_grad(const void* X, int32_t x_dtype, const uint8_t* x_scales, int64_t M, int64_t d_in,
                                      int64_t ld_x, const void* dY, int32_t dy_dtype, int64_t d_out, int64_t ld_dy,
                                      const void* A, const void* B, int32_t dtype, int64_t n_adapters, int32_t rank,
                                      const float* scale, const int32_t* adapter, float* dA, float* dB, const void* base,
                                      int64_t ld_b, void* dX, int32_t dx_dtype, int64_t ld_dx, void* workspace,
                                      size_t ws_bytes, void* stream) {
  GQ_CHECK_ARG(dtype == GPTQ_F16 || dtype == GPTQ_BF16);
  GQ_CHECK_ARG(x_dtype == dtype || x_dtype == GPTQ_E4M3);
  GQ_CHECK_ARG(dy_dtype == dtype || dy_dtype == GPTQ_F32);
  GQ_CHECK_ARG(dX == nullptr || dx_dtype == dtype || dx_dtype == GPTQ_F32);
  GQ_CHECK_ARG(M >= 0 && d_in >= 1 && d_out >= 1 && rank >= 1 && n_adapters >= 1);
  GQ_CHECK_ARG(ld_x >= d_in && ld_x <= ((int64_t)1 << 32) && ld_dy >= d_out && ld_dy <= ((int64_t)1 << 32));
  GQ_CHECK_ARG(x_dtype != GPTQ_E4M3 || (ld_x % 16 == 0 && ld_x >= cdiv(d_in, kF8Block) * kF8Block));
  GQ_CHECK_ARG(dX == nullptr || (ld_dx >= d_in && ld_dx <= ((int64_t)1 << 32)));
  GQ_CHECK_ARG(base == nullptr || (dX != nullptr && ld_b >= d_in && ld_b <= ((int64_t)1 << 32)));
  GQ_CHECK_ARG(base == nullptr || base != dX || ld_b == ld_dx);
  if (rank > kGradMaxRank || n_adapters > kGradMaxAdapters || M > ((int64_t)1 << 22) || d_in > ((int64_t)1 << 22) ||
      d_out > ((int64_t)1 << 22))
    return GPTQ_EUNSUPPORTED;
  GQ_CHECK_ARG(dA && dB && A && B);
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(A) % 2 == 0 && reinterpret_cast<uintptr_t>(B) % 2 == 0 &&
               reinterpret_cast<uintptr_t>(dA) % 4 == 0 && reinterpret_cast<uintptr_t>(dB) % 4 == 0);
  GQ_CHECK_ARG(M == 0 || (X && dY && adapter && (x_scales || x_dtype != GPTQ_E4M3)));
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(X) % (x_dtype == GPTQ_E4M3 ? 16 : 2) == 0 &&
               reinterpret_cast<uintptr_t>(dY) % f8_elem(dy_dtype) == 0);
  GQ_CHECK_ARG(dX == nullptr || (reinterpret_cast<uintptr_t>(dX) % f8_elem(dx_dtype) == 0 &&
                                 reinterpret_cast<uintptr_t>(base) % f8_elem(dx_dtype) == 0));
  const int64_t rows = std::max<int64_t>(M, 1);
  const GradPlan p = grad_plan(rows, d_in, d_out, rank, n_adapters);
  if (workspace == nullptr || ws_bytes < p.total) return GPTQ_ENOMEM;
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(workspace) % 256 == 0);
  char* ws = static_cast<char*>(workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  TimedScope ts(kTimeLoraGrad, st);

  GradPrep pr{};
  pr.sort.adapter = adapter;
  pr.sort.at = GradPlace{reinterpret_cast<int32_t*>(ws + p.order), reinterpret_cast<int32_t*>(ws + p.pos),
                         reinterpret_cast<GradChunk*>(ws + p.chunks), reinterpret_cast<int32_t*>(ws + p.parts),
                         reinterpret_cast<int32_t*>(ws + p.count)};
  pr.sort.M = M;
  pr.sort.n = (int)n_adapters;
  pr.sort.chunk = p.chunk;
  pr.A = static_cast<const uint16_t*>(A);
  pr.B = static_cast<const uint16_t*>(B);
  const bool two = dtype == GPTQ_F16;
  pr.a_terms = two ? reinterpret_cast<uint16_t*>(ws + p.a_terms) : nullptr;
  pr.b_terms = reinterpret_cast<uint16_t*>(ws + p.b_terms);
  pr.a_turned = dX ? reinterpret_cast<uint16_t*>(ws + p.a_turned) : nullptr;
  pr.d_in = (int)d_in;
  pr.d_out = (int)d_out;
  pr.rank = rank;
  pr.ld_a = p.ld_a;
  pr.ld_b = p.ld_b;
  const int64_t rank_tiles = cdiv(rank, 32);
  pr.a_tiles = two || dX ? (int)(cdiv(p.ld_a, 32) * rank_tiles) : 0;
  pr.b_tiles = (int)(cdiv(p.ld_b, 32) * rank_tiles);
  const dim3 prep((unsigned)(1 + n_adapters * (pr.a_tiles + pr.b_tiles)));
  if (two) hipLaunchKernelGGL((lora_grad_prep_kernel<GPTQ_F16>), prep, dim3(1024), 0, st, pr);
  else hipLaunchKernelGGL((lora_grad_prep_kernel<GPTQ_BF16>), prep, dim3(1024), 0, st, pr);
  GQ_LAUNCHED();

  GradArgs a[2];                    // X with A, dY with B
  for (int i = 0; i < 2; ++i) {
    GradArgs& g = a[i];
    g = GradArgs{};
    g.at = pr.sort.at;
    g.adapter = adapter;
    g.scale = scale;
    g.M = M;
    g.P = p.P;
    g.n = (int)n_adapters;
    g.rank = rank;
    g.rp = p.rp;
    g.terms = two ? 2 : 1;
    GradSide& s = g.side;
    s.D = i ? dY : X;
    s.scales = i ? nullptr : x_scales;
    s.ld = i ? ld_dy : ld_x;
    s.K = (int)(i ? d_out : d_in);
    s.nb = (int)cdiv(s.K, kF8Block);
    s.F = i ? pr.b_terms : two ? pr.a_terms : pr.A;
    s.ld_f = i ? p.ld_b : two ? p.ld_a : (int)d_in;
    s.f_term = n_adapters * rank * (int64_t)s.ld_f;
    s.full = i && dX ? reinterpret_cast<float*>(ws + p.full) : nullptr;
    s.turned = reinterpret_cast<uint16_t*>(ws + (i ? p.turned_u : p.turned_t));
    s.by = reinterpret_cast<uint16_t*>(ws + (i ? p.turned_t : p.turned_u));
    s.grad = i ? dB : dA;
    s.part = reinterpret_cast<float*>(ws + (i ? p.part_b : p.part_a));
    s.rank_first = i == 0;
    g.blocks = (int)cdiv(s.K, 128);
  }
  const int types[2] = {x_dtype, dy_dtype};
  for (int i = 0; i < 2 && M > 0; ++i) {
    grad_typed(types[i], [&](auto d) { grad_project<d.value>(a[i], p.r16, st); });
    GQ_LAUNCHED();
  }
  for (int i = 0; i < 2; ++i) {
    grad_typed(types[i], [&](auto d) { grad_outer<d.value>(a[i], p.r16, p.max_chunks, st); });
    GQ_LAUNCHED();
    if (p.slots > 0) {
      const int64_t each = (int64_t)rank * a[i].side.K;
      hipLaunchKernelGGL(lora_grad_join_kernel, dim3((unsigned)std::min<int64_t>(cdiv(each, 256), 4096), (unsigned)n_adapters),
                         dim3(256), 0, st, a[i]);
      GQ_LAUNCHED();
    }
  }
  if (dX && M > 0) {
    lora_up_run(dtype, a[1].side.full, adapter, pr.a_turned, n_adapters, rank, base, ld_b, dX, dx_dtype, ld_dx, M, d_in, st);
    GQ_LAUNCHED();
  }
  return GPTQ_OK;
}
