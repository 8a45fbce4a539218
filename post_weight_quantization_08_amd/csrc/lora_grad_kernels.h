// The adapters' gradients: kernels that depend on the types, for one type of factors.
#pragma once

#include "lora_grad.h"

namespace gq {

// ---------------------------------------------------------------- sorting
// Tokens into runs of one adapter, in their own order, each run starting at a multiple
// of 32 and filled up to the next; by one workgroup of four waves: every wave counts a
// range of tokens, then places it.
struct GradSortShared {
  uint32_t hist[4][kGradMaxAdapters];
  uint32_t scan[4];
};

__device__ inline void grad_sort(const GradArgs& a, GradSortShared& sh) {
  constexpr int kE = kGradMaxAdapters / 256;   // adapters of a thread
  constexpr int kU = 8;                        // groups of 64 tokens read together
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  for (int w = 0; w < 4; ++w)
    for (int e = 0; e < kE; ++e) sh.hist[w][e * 256 + t] = 0;
  __syncthreads();
  const int64_t per = (a.M + 255) / 256 * 64, first = wave * per, last = min(first + per, a.M);
  auto read = [&](int64_t m0, int (&ad)[kU]) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t m = m0 + u * 64 + lane;
      const int v = a.adapter[m < last ? m : last - 1];
      ad[u] = m < last && v >= 0 && v < a.n ? v : -1;
    }
  };
  for (int64_t m0 = first; m0 < last; m0 += 64 * kU) {
    int ad[kU];
    read(m0, ad);
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (ad[u] >= 0) atomicAdd(&sh.hist[wave][ad[u]], 1u);   // counts: their order is nothing
  }
  __syncthreads();
  // thread t has adapters kE t .. kE t + kE - 1
  uint32_t count[kE], parts[kE], sum[3] = {0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int ad = kE * t + e;
    count[e] = sh.hist[0][ad] + sh.hist[1][ad] + sh.hist[2][ad] + sh.hist[3][ad];
    parts[e] = ad < a.n ? max(1u, (count[e] + a.chunk - 1) / a.chunk) : 0u;
    sum[0] += (count[e] + 31) / 32 * 32;
    sum[1] += parts[e];
    sum[2] += parts[e] > 1 ? parts[e] : 0u;
  }
  uint32_t base[3], total[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {   // sums over the threads before this one
    uint32_t s = sum[i];
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = (uint32_t)__shfl_up((int)s, d);
      if (lane >= d) s += o;
    }
    __syncthreads();
    if (lane == 63) sh.scan[wave] = s;
    __syncthreads();
    base[i] = s - sum[i];
    total[i] = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) base[i] += sh.scan[w];
      total[i] += sh.scan[w];
    }
  }
  uint32_t start[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int ad = kE * t + e;
    start[e] = base[0];
    uint32_t next = base[0];
    for (int w = 0; w < 4; ++w) {
      const uint32_t c = sh.hist[w][ad];
      sh.hist[w][ad] = next;
      next += c;
    }
    if (ad < a.n) {
      a.at.parts[2 * ad] = (int)base[2];
      a.at.parts[2 * ad + 1] = (int)parts[e];
      for (uint32_t p = 0; p < parts[e]; ++p)
        a.at.chunks[base[1] + p] =
            GradChunk{ad, (int)(start[e] + p * a.chunk), (int)min(start[e] + (p + 1) * a.chunk, start[e] + count[e]),
                      parts[e] > 1 ? (int)(base[2] + p) : -1};
    }
    base[0] += (count[e] + 31) / 32 * 32;
    base[1] += parts[e];
    base[2] += parts[e] > 1 ? parts[e] : 0u;
  }
  if (t == 0) {
    a.at.count[0] = (int)total[1];
    a.at.count[1] = (int)total[0];
  }
  __syncthreads();
  for (int64_t m0 = first; m0 < last; m0 += 64 * kU) {
    int ad[kU];
    read(m0, ad);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      int mine = -1;
      uint64_t left = __ballot(ad[u] >= 0);
      while (left) {
        const int one = __builtin_amdgcn_readlane(ad[u], __builtin_ctzll(left));
        const uint64_t same = __ballot(ad[u] == one);
        left &= ~same;
        const uint32_t at = sh.hist[wave][one];
        if (ad[u] == one) mine = (int)(at + __popcll(same & ((1ull << lane) - 1)));
        if (lane == 0) sh.hist[wave][one] = at + __popcll(same);
      }
      if (mine >= 0) a.at.order[mine] = (int32_t)(m0 + u * 64 + lane);
    }
  }
  __syncthreads();
  // the runs' ends, with their last tokens: any token of the adapter would do
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const uint32_t end = start[e] + count[e];
    if (count[e] % 32) {
      const int32_t fill = ~a.at.order[end - 1];
      for (uint32_t p = end; p < start[e] + (count[e] + 31) / 32 * 32; ++p) a.at.order[p] = fill;
    }
  }
}

// ---------------------------------------------------------------- U and T
// A wave takes 32 tokens, all ranks and one part of the sum, a block of 128 at a time.
// Of a block lane (c16, q) has elements 64 u + 16 q + 8 h + 0..7 of its row in step
// 2 u + h, so that codes come 16 bytes at a time.  D: rows = ranks, columns = tokens.
//   kRows false: F is [rank][K]; D's row i of tile p is rank 16 p + i.
//   kRows true: F is [K][rank]; a lane loads kR ranks of eight rows and turns them;
//   row i of tile p is rank kR i + p.
template <int kD, int kF, bool kRows, int kR>
__device__ __forceinline__ void grad_project(const GradArgs& a, const GradSide& s, int id) {
  const int group = id % a.groups, rank0 = id / a.groups % a.halves * 64, part = id / (a.groups * a.halves);
  const int rank = a.halves > 1 ? min(a.rank - rank0, 64) : a.rank;   // of this half
  constexpr int kT = Eight<kD>::kTerms;
  // one product of 16-bit numbers: codes with fp16 factors are scaled behind a block's sum
  constexpr bool kHalf = kF == GPTQ_F16 && kD != GPTQ_F32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int64_t m0 = ((int64_t)group * 4 + wave) * kGradTile;
  if (m0 >= a.M) return;
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
  const int b0 = part * s.per, b1 = min(b0 + s.per, s.nb);
  const bool even = a.rank % kR == 0;   // then a lane's ranks are there together, or none of them
  uint32_t left = (uint32_t)__ballot(mine >= 0);
  while (left) {
    const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(mine == ad);
    const uint16_t* f = s.F + (int64_t)ad * a.rank * s.K + (kRows ? rank0 : (int64_t)rank0 * s.K);
    f32x4 acc[kR][2];
#pragma unroll
    for (int r = 0; r < kR; ++r) acc[r][0] = acc[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Block {
      Eight<kD> d[4][2];
      uint32_t sb[2];
    };
    auto read = [&](int b, Block& k) {
      const bool whole = (b + 1) * kF8Block <= s.K;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        k.sb[t] = 127u;
        if constexpr (kD == GPTQ_E4M3) k.sb[t] = sc[t][b];
        if (whole || kD == GPTQ_E4M3) {   // codes are there up to the block's end
#pragma unroll
          for (int j = 0; j < 4; ++j) k.d[j][t].load(x[t], b * kF8Block + j / 2 * 64 + q * 16 + j % 2 * 8);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) k.d[j][t].load_end(x[t], b * kF8Block + j / 2 * 64 + q * 16 + j % 2 * 8, s.K);
        }
      }
    };
    // the factors' operand of step j
    auto factor = [&](int b, int j, u32x4 (&w)[kR]) {
      const int k = b * kF8Block + j / 2 * 64 + q * 16 + j % 2 * 8;
      if constexpr (!kRows) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const uint16_t* row = f + (int64_t)min(r * 16 + c16, rank - 1) * s.K;
          if ((b + 1) * kF8Block <= s.K) w[r] = load8(row + k);
          else w[r] = load8_end(row, k, s.K);
        }
      } else {
        uint16_t v[8][kR];
        if (even) {
          const int r0 = c16 * kR < rank ? c16 * kR : 0;   // rows of D behind the rank are not stored
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __builtin_memcpy(v[i], __builtin_assume_aligned(f + (int64_t)min(k + i, s.K - 1) * a.rank + r0, 2), 2 * kR);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int p = 0; p < kR; ++p) v[i][p] = f[(int64_t)min(k + i, s.K - 1) * a.rank + min(c16 * kR + p, rank - 1)];
        }
#pragma unroll
        for (int p = 0; p < kR; ++p)
#pragma unroll
          for (int i = 0; i < 4; ++i) w[p][i] = v[2 * i][p] | (uint32_t)v[2 * i + 1][p] << 16;
      }
    };
    auto multiply = [&](int b, const Block& k) {
      f32x4 one[kHalf && kD == GPTQ_E4M3 ? kR : 1][2];
      if constexpr (kHalf && kD == GPTQ_E4M3) {
#pragma unroll
        for (int r = 0; r < kR; ++r) one[r][0] = one[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 w[kR];
        factor(b, j, w);
        if constexpr (kHalf) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            u32x4 d;
            if constexpr (kD == GPTQ_E4M3) {
              d = k.d[j][t].half();
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) d[i] = k.d[j][t].w[i];
            }
#pragma unroll
            for (int r = 0; r < kR; ++r) {
              if constexpr (kD == GPTQ_E4M3) one[r][t] = mfma_16x16x32<GPTQ_F16>(w[r], d, one[r][t]);
              else acc[r][t] = mfma_16x16x32<GPTQ_F16>(w[r], d, acc[r][t]);
            }
          }
        } else {
          u32x4 d[2][kT];
#pragma unroll
          for (int t = 0; t < 2; ++t) k.d[j][t].terms(grad_scale(k.sb[t]), d[t]);
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            u32x4 wt[kF == GPTQ_F16 ? 2 : 1];
            Eight<kF> e;
#pragma unroll
            for (int i = 0; i < 4; ++i) e.w[i] = w[r][i];
            e.terms(1.f, wt);
#pragma unroll
            for (int t = 0; t < 2; ++t) acc[r][t] = grad_mfma(wt, d[t], acc[r][t]);
          }
        }
      }
      if constexpr (kHalf && kD == GPTQ_E4M3) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float by = grad_scale(k.sb[t]);
#pragma unroll
          for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][t][i] = fmaf(one[r][t][i], by, acc[r][t][i]);
        }
      }
    };
    if constexpr (kD == GPTQ_F32) {
      for (int b = b0; b < b1; ++b) {
        Block k;
        read(b, k);
        multiply(b, k);
      }
    } else {
      // a block's rows are asked for while the one before is multiplied
      Block even_block, odd_block;
      read(b0, even_block);
      for (int b = b0; b < b1; b += 2) {
        read(min(b + 1, b1 - 1), odd_block);
        multiply(b, even_block);
        if (b + 1 < b1) {
          read(min(b + 2, b1 - 1), even_block);
          multiply(b + 1, odd_block);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (__shfl(mine, t * 16 + c16) != ad) continue;
      float* out = s.sums + ((int64_t)part * a.M + m0 + t * 16 + c16) * a.rp + rank0;
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        // four ranks of one tile, or of the tiles that lie next to each other
        f32x4 v;
        const int first = kRows ? 4 * kR * q + 4 * r : r * 16 + 4 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = kRows ? acc[(4 * r + i) % kR][t][(4 * r + i) / kR] : acc[r][t][i];
          v[i] = first + i < rank ? v[i] : 0.f;
        }
        if (rank0 + first < a.rp) *reinterpret_cast<f32x4*>(out + first) = v;
      }
    }
  }
}

// Workgroups: the sort, then X's parts, dY's parts, and tiles of 32 x 32 of A to turn.
template <int kX, int kY, int kF, int kR>
__global__ __launch_bounds__(256) void lora_grad_project_kernel(GradArgs a) {
  __shared__ union {
    GradSortShared sort;
    uint16_t tile[32][34];
  } sh;
  int id = blockIdx.x;
  if (id == 0) {
    grad_sort(a, sh.sort);
    return;
  }
  id -= 1;
  const int wgs = a.groups * a.halves;
  if (id < wgs * a.side[0].splits) {
    grad_project<kX, kF, false, kR>(a, a.side[0], id);
    return;
  }
  id -= wgs * a.side[0].splits;
  if (id < wgs * a.side[1].splits) {
    grad_project<kY, kF, true, kR>(a, a.side[1], id);
    return;
  }
  id -= wgs * a.side[1].splits;
  const int ad = id / a.a_tiles, i = id % a.a_tiles, K = a.side[0].K;
  const int rank_tiles = (a.rank + 31) / 32, r0 = i % rank_tiles * 32, k0 = i / rank_tiles * 32;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < 32; j += 8)
    sh.tile[y + j][x] = r0 + y + j < a.rank && k0 + x < K ? a.A[((int64_t)ad * a.rank + r0 + y + j) * K + k0 + x] : 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 32; j += 8)
    if (k0 + y + j < K && r0 + x < a.rank) a.a_turned[((int64_t)ad * K + k0 + y + j) * a.rank + r0 + x] = sh.tile[x][y + j];
}

// ---------------------------------------------------------------- sums over tokens
// A workgroup sums a chunk of one adapter's tokens for 128 columns and all ranks; its
// waves take the steps of 32 tokens in turn.  D: rows = ranks, columns = columns: lane
// c16 holds columns 8 c16 .. 8 c16 + 7, column p of them in tile p.
constexpr int kOuterWaves = 4;

template <int kD, int kR, bool kRankFirst>
__device__ __forceinline__ void grad_outer(const GradArgs& a, const GradSide& s, int block, int rank0,
                                           const GradChunk& ch, f32x4 (*red)[64]) {
  constexpr int kT = Eight<kD>::kTerms;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int col = block * kF8Block + c16 * 8;
  const bool whole = (block + 1) * kF8Block <= s.K || kD == GPTQ_E4M3;
  const uint16_t* by = s.by + (int64_t)(rank0 + c16) * a.P + 8 * q;
  f32x4 acc[kR][8];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int p = 0; p < 8; ++p) acc[r][p] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Step {
    Eight<kD> e[8];
    uint32_t sb[8];
  };
  // a run is filled up to the step's end with tokens that U and T have zeros for
  auto tokens = [&](int pos, int4 (&v)[2]) {
    const int4* p = reinterpret_cast<const int4*>(a.at.order + pos + 8 * q);
    v[0] = p[0];
    v[1] = p[1];
  };
  auto read = [&](const int4 (&v)[2], Step& d) {
    const int m[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t tok = m[i] ^ (m[i] >> 31);
      if (whole) d.e[i].load(grad_row<kD>(s, tok), col);
      else d.e[i].load_end(grad_row<kD>(s, tok), col, s.K);
      d.sb[i] = 127u;
      if constexpr (kD == GPTQ_E4M3) d.sb[i] = s.scales[tok * s.nb + block];
    }
  };
  constexpr int kStep = kOuterWaves * kGradTile;
  const int first = ch.begin + wave * kGradTile;
  if (first < ch.end) {
    // rows are asked for a step ahead, as soon as the ones before are turned; their
    // numbers two steps ahead
    int4 next[2];
    Step d;
    auto clamp = [&](int pos) { return pos < ch.end ? pos : first; };
    tokens(first, next);
    read(next, d);
    tokens(clamp(first + kStep), next);
    for (int pos = first; pos < ch.end; pos += kStep) {
      u32x4 c[8][kT];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x[8][kT];
#pragma unroll
        for (int j = 0; j < 8; ++j) d.e[j].pair(i, grad_scale(d.sb[j]), x[j]);
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            c[2 * i][t][j] = __builtin_amdgcn_perm(x[2 * j + 1][t], x[2 * j][t], 0x05040100u);
            c[2 * i + 1][t][j] = __builtin_amdgcn_perm(x[2 * j + 1][t], x[2 * j][t], 0x07060302u);
          }
      }
      read(next, d);
      tokens(clamp(pos + 2 * kStep), next);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        u32x4 u[3];
#pragma unroll
        for (int t = 0; t < 3; ++t) u[t] = *reinterpret_cast<const u32x4*>(by + (int64_t)(t * a.r16 + r * 16) * a.P + pos);
#pragma unroll
        for (int p = 0; p < 8; ++p) acc[r][p] = grad_mfma(u, c[p], acc[r][p]);
      }
    }
  }
  // the waves' sums one after the other
  for (int w = kOuterWaves - 1; w > 0; --w) {
    if (wave == w) {
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int p = 0; p < 8; ++p) red[r * 8 + p][lane] = acc[r][p];
    }
    __syncthreads();
    if (wave == w - 1) {
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int p = 0; p < 8; ++p) acc[r][p] += red[r * 8 + p][lane];
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
      const int rank = rank0 + r * 16 + 4 * q + i;
      if (rank >= a.rank) continue;
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (col + p < s.K) out[kRankFirst ? (int64_t)rank * s.K + col + p : (int64_t)(col + p) * a.rank + rank] = acc[r][p][i];
    }
}

template <int kX, int kY, int kR>
__global__ __launch_bounds__(64 * kOuterWaves) void lora_grad_outer_kernel(GradArgs a) {
  __shared__ __align__(16) f32x4 red[kR * 8][64];
  const int blocks = a.side[0].blocks + a.side[1].blocks;
  const int block = blockIdx.x % blocks, rank0 = blockIdx.x / blocks % a.halves * 64, ci = blockIdx.x / (blocks * a.halves);
  if (ci >= a.at.count[0]) return;
  const GradChunk ch = a.at.chunks[ci];
  if (block < a.side[0].blocks) grad_outer<kX, kR, true>(a, a.side[0], block, rank0, ch, red);
  else grad_outer<kY, kR, false>(a, a.side[1], block - a.side[0].blocks, rank0, ch, red);
}

template <int kX, int kY, int kF, int kR>
static void grad_launch_rank(const GradArgs& a, int64_t max_chunks, bool outer, hipStream_t st) {
  if (!outer) {
    const int64_t wgs = 1 + (int64_t)a.groups * a.halves * (a.side[0].splits + a.side[1].splits) + (int64_t)a.n * a.a_tiles;
    hipLaunchKernelGGL((lora_grad_project_kernel<kX, kY, kF, kR>), dim3((unsigned)wgs), dim3(256), 0, st, a);
  } else {
    const int64_t wgs = (a.side[0].blocks + a.side[1].blocks) * a.halves * max_chunks;
    hipLaunchKernelGGL((lora_grad_outer_kernel<kX, kY, kR>), dim3((unsigned)wgs), dim3(64 * kOuterWaves), 0, st, a);
  }
}

template <int kX, int kY, int kF>
static void grad_launch_types(const GradArgs& a, int64_t max_chunks, bool outer, hipStream_t st) {
  if (a.r16 == 16) grad_launch_rank<kX, kY, kF, 1>(a, max_chunks, outer, st);
  else if (a.r16 == 32) grad_launch_rank<kX, kY, kF, 2>(a, max_chunks, outer, st);
  else grad_launch_rank<kX, kY, kF, 4>(a, max_chunks, outer, st);
}

template <int kF>
static void grad_launch(const GradArgs& a, bool codes, bool wide, int64_t max_chunks, bool outer, hipStream_t st) {
  if (codes && wide) grad_launch_types<GPTQ_E4M3, GPTQ_F32, kF>(a, max_chunks, outer, st);
  else if (codes) grad_launch_types<GPTQ_E4M3, kF, kF>(a, max_chunks, outer, st);
  else if (wide) grad_launch_types<kF, GPTQ_F32, kF>(a, max_chunks, outer, st);
  else grad_launch_types<kF, kF, kF>(a, max_chunks, outer, st);
}

}  // namespace gq
