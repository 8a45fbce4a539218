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
  uint32_t scan[4], none[4];
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
  uint32_t none = 0;
  for (int64_t m0 = first; m0 < last; m0 += 64 * kU) {
    int ad[kU];
    read(m0, ad);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (ad[u] >= 0) atomicAdd(&sh.hist[wave][ad[u]], 1u);   // counts: their order is nothing
      none += __popcll(__ballot(ad[u] < 0 && m0 + u * 64 + lane < last));
    }
  }
  if (lane == 0) sh.none[wave] = none;
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
  uint32_t outside = total[0];   // where this wave's tokens without an adapter go
  for (int w = 0; w < wave; ++w) outside += sh.none[w];
  if (t == 0) {
    a.at.count[0] = (int)total[1];
    a.at.count[1] = (int)total[0];
    a.at.count[2] = (int)(total[0] + sh.none[0] + sh.none[1] + sh.none[2] + sh.none[3]);
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
      const bool lone = ad[u] < 0 && m0 + u * 64 + lane < last;
      const uint64_t others = __ballot(lone);
      if (lone) mine = (int)(outside + __popcll(others & ((1ull << lane) - 1)));
      outside += __popcll(others);
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
// A workgroup takes 128 tokens, 32 a wave, up to 64 ranks and one part of the sum, a block
// of 128 at a time; the factors' block is laid out in LDS as operands for all four waves
// while the one before is multiplied.  Of a block lane (c16, q) has elements 64 u + 16 q +
// 8 h + 0..7 of its row in step j = 2 u + h, so that codes come 16 bytes at a time.
// D: rows = ranks, columns = tokens.  (8192 tokens, 64 ranks: every wave loading the
// factors for itself 91 us, through LDS 76, and without a condition between loads 64; the parts
// taking the blocks in turn the same.)
//   kRows false: F is [rank][K]; D's row i of tile p is rank 16 p + i.
//   kRows true: F is [K][rank]; a lane loads kR ranks of eight rows and turns them;
//   row i of tile p is rank kR i + p.
template <int kR>
struct GradProjectShared {
  u32x4 f[2][4 * kR][64];           // [buffer][step, rank tile][lane]
  int adapter[128];
};

template <int kD, int kF, bool kRows, int kR>
__device__ __forceinline__ void grad_project(const GradArgs& a, const GradSide& s, int id, GradProjectShared<kR>& sh) {
  const int group = id % a.groups, rank0 = id / a.groups % a.halves * 64, part = id / (a.groups * a.halves);
  const int rank = a.halves > 1 ? min(a.rank - rank0, 64) : a.rank;   // of this half
  constexpr int kT = Eight<kD>::kTerms;
  // one product of 16-bit numbers: codes with fp16 factors are scaled behind a block's sum
  constexpr bool kHalf = kF == GPTQ_F16 && kD != GPTQ_F32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int64_t g0 = (int64_t)group * 128, m0 = g0 + wave * kGradTile;
  if (threadIdx.x < 128) {
    const int v = g0 + threadIdx.x < a.M ? a.adapter[g0 + threadIdx.x] : -1;
    sh.adapter[threadIdx.x] = v >= 0 && v < a.n ? v : -1;
  }
  __syncthreads();
  const int mine = sh.adapter[wave * kGradTile + (lane & 31)];
  const char* x[2];
  const uint8_t* sc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t m = min(m0 + t * 16 + c16, a.M - 1);
    x[t] = grad_row<kD>(s, m);
    sc[t] = kD == GPTQ_E4M3 ? s.scales + m * s.nb : nullptr;
  }
  const int b0 = part * s.per, b1 = min(b0 + s.per, s.nb);
  int ad = -1;
  for (;;) {
    // the next adapter among the 128 tokens, the same for all waves
    const int v0 = sh.adapter[lane], v1 = sh.adapter[lane + 64];
    constexpr float kNone = kGradMaxAdapters;
    const float next = wave_reduce(min(v0 > ad ? (float)v0 : kNone, v1 > ad ? (float)v1 : kNone),
                                   [](float p, float r) { return min(p, r); });
    if (next == kNone) break;
    ad = __builtin_amdgcn_readfirstlane((int)next);
    const bool here = __ballot(mine == ad) != 0;
    const uint16_t* f = s.F + (int64_t)ad * a.rank * s.K + (kRows ? rank0 : (int64_t)rank0 * s.K);
    // this wave's kR operands of a block: step `wave` of all rank tiles; rows of B are
    // turned when they are there
    struct Factor {
      u32x4 w[kRows ? 1 : kR];
      uint16_t v[kRows ? 8 : 1][kR];
    };
    auto read_factor = [&](int b, Factor& w, auto even, auto whole) {
      const int k = b * kF8Block + wave / 2 * 64 + wave % 2 * 8, kq = q * 16;   // the wave's, the lane's
      if constexpr (!kRows) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const uint32_t row = (uint32_t)min(r * 16 + c16, rank - 1) * (uint32_t)s.K;
          if constexpr (whole) w.w[r] = load8(f + k + (row + kq));
          else w.w[r] = load8_end(f + row, k + kq, s.K);
        }
      } else {
        const uint32_t r0 = c16 * kR < rank ? c16 * kR : 0;   // rows of D behind the rank are not stored
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint16_t* row = whole ? f + (int64_t)(k + i) * a.rank + (uint32_t)(kq * a.rank + (even ? r0 : 0))
                                      : f + (int64_t)min(k + kq + i, s.K - 1) * a.rank + (even ? r0 : 0);
          if constexpr (even) {
            __builtin_memcpy(w.v[i], __builtin_assume_aligned(row, 2), 2 * kR);
          } else {
#pragma unroll
            for (int p = 0; p < kR; ++p) w.v[i][p] = row[min(c16 * kR + p, rank - 1)];
          }
          // zeros behind the last row: its infinity times the zeros of D would be a NaN
          if constexpr (!whole) {
#pragma unroll
            for (int p = 0; p < kR; ++p) w.v[i][p] = k + kq + i < s.K ? w.v[i][p] : (uint16_t)0;
          }
        }
      }
    };
    auto write_factor = [&](int buffer, const Factor& w) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if constexpr (kRows) {
          u32x4 t;
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = w.v[2 * i][r] | (uint32_t)w.v[2 * i + 1][r] << 16;
          sh.f[buffer][wave * kR + r][lane] = t;
        } else {
          sh.f[buffer][wave * kR + r][lane] = w.w[r];
        }
      }
    };
    struct Block {
      Eight<kD> d[4][2];
      uint32_t sb[2];
    };
    auto read = [&](int b, Block& k, auto whole) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        k.sb[t] = 127u;
        if constexpr (kD == GPTQ_E4M3) k.sb[t] = sc[t][b];
        if constexpr (whole || kD == GPTQ_E4M3) {   // codes are there up to the block's end
#pragma unroll
          for (int j = 0; j < 4; ++j) k.d[j][t].load(x[t], b * kF8Block + j / 2 * 64 + q * 16 + j % 2 * 8);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) k.d[j][t].load_end(x[t], b * kF8Block + j / 2 * 64 + q * 16 + j % 2 * 8, s.K);
        }
      }
    };
    f32x4 acc[kR][2];
#pragma unroll
    for (int r = 0; r < kR; ++r) acc[r][0] = acc[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](int buffer, const Block& k) {
      f32x4 one[kHalf && kD == GPTQ_E4M3 ? kR : 1][2];
      if constexpr (kHalf && kD == GPTQ_E4M3) {
#pragma unroll
        for (int r = 0; r < kR; ++r) one[r][0] = one[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 w[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) w[r] = sh.f[buffer][j * kR + r][lane];
        if constexpr (kR == 4) __builtin_amdgcn_sched_barrier(0);   // or all steps' operands are held at once
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
    // A block's rows and factors are asked for while the one before is multiplied (rows
    // of fp32 behind it: they are too many registers).  Nothing in the loop is asked for
    // on a condition: where paths with and without loads meet, the compiler waits for all.
    const int bw = min(b1, s.K / kF8Block);   // behind the whole blocks
    constexpr std::true_type kWhole{};
    constexpr bool kAhead = kD != GPTQ_F32;
    constexpr int kDeep = 2;   // blocks of rows in registers (three of codes: 67 us for 65)
    // take: whether this wave has tokens of the adapter
    auto sum = [&](auto take, auto even) {
      Factor w;
      Block k[kDeep];
      if (b0 < bw) {
        read_factor(b0, w, even, kWhole);
        if constexpr (take) {
#pragma unroll
          for (int i = 0; i + 1 < kDeep; ++i) read(min(b0 + i, bw - 1), k[i], kWhole);
        }
        write_factor(0, w);
        lds_barrier();
        for (int b = b0; b < bw;) {
#pragma unroll
          for (int i = 0; i < kDeep; ++i) {
            constexpr int kLast = kDeep - 1;
            Block& then = k[(i + kLast) % kDeep];
            const int ahead = min(b + kLast, bw - 1);
            read_factor(min(b + 1, bw - 1), w, even, kWhole);
            if constexpr (take && kAhead) read(ahead, then, kWhole);
            if constexpr (take) multiply(i, k[i]);
            write_factor((i + 1) % kDeep, w);
            if constexpr (take && !kAhead) read(ahead, then, kWhole);
            lds_barrier();
            if (++b >= bw) break;
          }
        }
      }
      if (bw < b1) {   // nobody multiplies from the first buffer any more
        read_factor(bw, w, even, std::false_type{});
        write_factor(0, w);
        if constexpr (take) read(bw, k[0], std::false_type{});
        lds_barrier();
        if constexpr (take) multiply(0, k[0]);
        lds_barrier();
      }
    };
    // Waves without tokens of the adapter go another way round the same blocks.  The barriers
    // above are the instruction itself, not __syncthreads(), which a whole workgroup has to meet
    // at one place: s_barrier counts waves, wherever each of them meets it, and both ways have
    // as many.  (All waves multiplying, whether they have tokens or not, 2048 tokens of eight
    // adapters in turns of 32: 114 us for 85.)
    auto any = [&](auto even) {
      if (here) sum(std::true_type{}, even);
      else sum(std::false_type{}, even);
    };
    if (!kRows || a.rank % kR == 0) any(std::true_type{});   // a lane's ranks are there together, or none of them
    else any(std::false_type{});
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (sh.adapter[wave * kGradTile + t * 16 + c16] != ad) continue;
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

// Workgroups: the sort, then X's parts and dY's parts.
template <int kX, int kY, int kF, int kR>
__global__ __launch_bounds__(256, kY == GPTQ_F32 ? 1 : 2) void lora_grad_project_kernel(GradArgs a) {
  __shared__ union {
    GradSortShared sort;
    GradProjectShared<kR> project;
  } sh;
  int id = blockIdx.x;
  if (id == 0) {
    grad_sort(a, sh.sort);
    return;
  }
  id -= 1;
  const int x_parts = a.groups * a.halves * a.side[0].splits;
  if (id < x_parts) grad_project<kX, kF, false, kR>(a, a.side[0], id, sh.project);
  else grad_project<kY, kF, true, kR>(a, a.side[1], id - x_parts, sh.project);
}

// ---------------------------------------------------------------- sums over tokens
// A workgroup sums a chunk of one adapter's tokens for 256 columns and up to 64 ranks: two
// waves side by side, four taking the steps of 32 tokens in turn.  U (or T) comes into
// LDS by direct loads, as operands, a step ahead (8192 tokens, 64 ranks 67 us; loaded by
// every wave when it needs it 163).  D: rows = ranks, columns = columns:
// lane c16 holds columns 8 c16 .. 8 c16 + 7, column p of them in tile p.
constexpr int kOuterSplit = 4;
constexpr int kOuterWaves = 2 * kOuterSplit;

template <int kR>
struct GradOuterShared {
  u32x4 u[kOuterSplit][3 * kR][64];   // [wave's tokens][term, rank tile][lane]
};

template <int kD, int kR, bool kRankFirst>
__device__ __forceinline__ void grad_outer(const GradArgs& a, const GradSide& s, int block, int rank0,
                                           const GradChunk& ch, GradOuterShared<kR>& u0, GradOuterShared<kR>& u1) {
  constexpr int kT = Eight<kD>::kTerms;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4, beside = wave & 1, split = wave >> 1;
  const int block128 = block * 2 + beside, col = block128 * kF8Block + c16 * 8;
  // an odd number of 128s leaves a wave without columns, and an adapter may have no
  // tokens: nothing need stand in the order at its place then
  const bool some = block128 * kF8Block < s.K && ch.begin < ch.end;
  const bool whole = (block128 + 1) * kF8Block <= s.K || kD == GPTQ_E4M3;
  const uint16_t* by = s.by + (int64_t)(rank0 + c16) * a.P + 8 * q;
  f32x4 acc[kR][8];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int p = 0; p < 8; ++p) acc[r][p] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int kStep = kOuterSplit * kGradTile;
  const int first = ch.begin + split * kGradTile, steps = (ch.end - ch.begin + kStep - 1) / kStep;
  auto clamp = [&](int pos) { return pos < ch.end ? pos : ch.begin; };
  struct Step {
    Eight<kD> e[8];
    uint32_t sb[8];
  };
  // a run is filled up to the step's end with tokens that U and T have zeros for
  auto tokens = [&](int pos, int4 (&v)[2]) {
    const int4* p = reinterpret_cast<const int4*>(a.at.order + clamp(pos) + 8 * q);
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
      if constexpr (kD == GPTQ_E4M3) d.sb[i] = s.scales[tok * s.nb + block128];
    }
  };
  // a wave loads every other operand of its tokens
  auto fetch = [&](int pos, GradOuterShared<kR>& to) {
    const uint16_t* from = by + clamp(pos);
#pragma unroll
    for (int i = 0; i < 3 * kR; i += 2) {
      const int o = min(i + beside, 3 * kR - 1);
      lds_load16(from + (int64_t)(o / kR * a.r16 + o % kR * 16) * a.P, reinterpret_cast<char*>(to.u[split][o]));
    }
  };
  // columns 2 i and 2 i + 1 of eight tokens as operands
  auto turn = [&](const Step& d, int i, u32x4 (&c)[2][kT]) {
    uint32_t x[8][kT];
#pragma unroll
    for (int j = 0; j < 8; ++j) d.e[j].pair(i, grad_scale(d.sb[j]), x[j]);
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[0][t][j] = __builtin_amdgcn_perm(x[2 * j + 1][t], x[2 * j][t], 0x05040100u);
        c[1][t][j] = __builtin_amdgcn_perm(x[2 * j + 1][t], x[2 * j][t], 0x07060302u);
      }
  };
  auto operand = [&](const GradOuterShared<kR>& from, int r, u32x4 (&u)[3]) {
#pragma unroll
    for (int t = 0; t < 3; ++t) u[t] = from.u[split][t * kR + r][lane];
  };
  int4 next[2];
  Step d;
  if (some) {
    tokens(first, next);
    read(next, d);
    tokens(first + kStep, next);
  }
  fetch(first, u0);
#define GQ_GRAD_STEP(i, CUR, NXT)                                                       \
  {                                                                                     \
    const int pos = first + (i) * kStep;                                                \
    __builtin_amdgcn_s_waitcnt(0x0070);   /* vmcnt(0) lgkmcnt(0) */                     \
    asm volatile("s_barrier" ::: "memory");                                             \
    fetch(pos + kStep, NXT);                                                            \
    if (some && pos < ch.end) {                                                         \
      if constexpr (kT == 1) {                                                          \
        /* all turned, so that the next rows can be asked for */                        \
        u32x4 c[4][2][kT];                                                              \
        _Pragma("unroll") for (int p = 0; p < 4; ++p) turn(d, p, c[p]);                 \
        read(next, d);                                                                  \
        tokens(pos + 2 * kStep, next);                                                  \
        _Pragma("unroll") for (int r = 0; r < kR; ++r) {                                \
          u32x4 u[3];                                                                   \
          operand(CUR, r, u);                                                           \
          _Pragma("unroll") for (int p = 0; p < 8; ++p) acc[r][p] = grad_mfma(u, c[p / 2][p % 2], acc[r][p]); \
        }                                                                               \
      } else {                                                                          \
        _Pragma("unroll") for (int p = 0; p < 8; p += 2) {                              \
          u32x4 c[2][kT];                                                               \
          turn(d, p / 2, c);                                                            \
          _Pragma("unroll") for (int r = 0; r < kR; ++r) {                              \
            u32x4 u[3];                                                                 \
            operand(CUR, r, u);                                                         \
            acc[r][p] = grad_mfma(u, c[0], acc[r][p]);                                  \
            acc[r][p + 1] = grad_mfma(u, c[1], acc[r][p + 1]);                          \
          }                                                                             \
          __builtin_amdgcn_sched_barrier(0);                                            \
        }                                                                               \
        read(next, d);                                                                  \
        tokens(pos + 2 * kStep, next);                                                  \
      }                                                                                 \
    }                                                                                   \
  }
  for (int i = 0; i < steps; i += 2) {
    GQ_GRAD_STEP(i, u0, u1)
    GQ_GRAD_STEP(i + 1, u1, u0)
  }
#undef GQ_GRAD_STEP
  // no direct load is in flight, and nobody reads, when the sums use the same memory:
  // four columns of a lane at a time, the last waves' in what two buffers leave
  __builtin_amdgcn_s_waitcnt(0x0070);
  __syncthreads();
  static_assert(kOuterSplit == 4 && sizeof(u0) == 12 * kR * 64 * sizeof(f32x4));
  f32x4(*red0)[64] = reinterpret_cast<f32x4(*)[64]>(u0.u);
  f32x4(*red1)[64] = reinterpret_cast<f32x4(*)[64]>(u1.u);
  auto place = [&](int w, int r, int p) -> f32x4& {
    if (w == 1) return red0[(r * 4 + p) * 2 + beside][lane];
    if (w == 2) return red1[(r * 4 + p) * 2 + beside][lane];
    return (p < 2 ? red0 : red1)[8 * kR + (r * 2 + p % 2) * 2 + beside][lane];
  };
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half) __syncthreads();
#pragma unroll
    for (int w = 1; w < 4; ++w)
      if (split == w) {
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
          for (int p = 0; p < 4; ++p) place(w, r, p) = acc[r][half * 4 + p];
      }
    __syncthreads();
    if (split == 0) {
#pragma unroll
      for (int w = 1; w < 4; ++w)
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
          for (int p = 0; p < 4; ++p) acc[r][half * 4 + p] += place(w, r, p);
    }
  }
  if (split != 0) return;
  const int64_t each = (int64_t)a.rank * s.K;
  float* out = ch.slot < 0 ? s.grad + ch.adapter * each : s.part + ch.slot * each;
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int rank = rank0 + r * 16 + 4 * q;
    if (rank + 4 <= a.rank && col + 8 <= s.K) {
      if constexpr (kRankFirst) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[8];
#pragma unroll
          for (int p = 0; p < 8; ++p) v[p] = acc[r][p][i];
          __builtin_memcpy(__builtin_assume_aligned(out + (int64_t)(rank + i) * s.K + col, 4), v, 32);
        }
      } else {
#pragma unroll
        for (int p = 0; p < 8; ++p)
          __builtin_memcpy(__builtin_assume_aligned(out + (int64_t)(col + p) * a.rank + rank, 4), &acc[r][p], 16);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int p = 0; p < 8; ++p)
        if (rank + i < a.rank && col + p < s.K)
          out[kRankFirst ? (int64_t)(rank + i) * s.K + col + p : (int64_t)(col + p) * a.rank + rank + i] = acc[r][p][i];
  }
}

template <int kX, int kY, int kR>
__global__ __launch_bounds__(64 * kOuterWaves) void lora_grad_outer_kernel(GradArgs a) {
  __shared__ GradOuterShared<kR> u0, u1;
  const int blocks = a.side[0].blocks + a.side[1].blocks;
  const int block = blockIdx.x % blocks, rank0 = blockIdx.x / blocks % a.halves * 64, ci = blockIdx.x / (blocks * a.halves);
  if (ci >= a.at.count[0]) return;
  const GradChunk ch = a.at.chunks[ci];
  if (block < a.side[0].blocks) grad_outer<kX, kR, true>(a, a.side[0], block, rank0, ch, u0, u1);
  else grad_outer<kY, kR, false>(a, a.side[1], block - a.side[0].blocks, rank0, ch, u0, u1);
}

// ---------------------------------------------------------------- dX
// A wave keeps A of 16 kC columns as operands (turned in registers) and takes 16 sorted
// tokens at a time, which share an adapter.  D: rows = tokens, columns = columns: a lane
// has kC consecutive columns of four tokens, so that base and dX move 16 bytes a lane.
// base is asked for three tiles before its turn and U one, whether they are wanted or
// not: a load on a condition would have the compiler wait for all that are in flight.
// 8192 x 11008 in 97 us, of which three fifths are waits for memory; one tile ahead 100,
// none 158.
template <int kF, int kOut, bool kBase, int kS, int kC>
__global__ __launch_bounds__(256, 2) void lora_grad_input_kernel(GradArgs a) {
  constexpr int kA = kF == GPTQ_F16 ? 2 : 1;
  constexpr int kE = kOut == GPTQ_F32 ? 4 : 2;
  constexpr int kWords = kC * kE / 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int K = a.side[0].K, wide = 64 * kC, blocks = (K + wide - 1) / wide;
  const int col = blockIdx.x % blocks * wide + wave * 16 * kC + c16 * kC;
  const int first = blockIdx.x / blocks * a.input_tokens, end = min(first + a.input_tokens, a.at.count[2]);
  const int runs = min(end, a.at.count[1]);
  if (first >= end) return;
  const bool whole = col + kC <= K;
  u32x4 f[kC][kS][kA];
  int held = -1;
  struct Place {
    int tok[4], lead;
  };
  struct Tile {
    int tok[4];                       // ~token: not stored
    uint32_t in[4][kBase ? kWords : 1];
  };
  auto tokens = [&](int pos, Place& t) {
    const int at = min(pos, end - 1) & ~15;
    const int4 v = *reinterpret_cast<const int4*>(a.at.order + at + 4 * q);   // [P], a multiple of 64
    const int lead = a.at.order[at], one = lead ^ (lead >> 31), left = end - pos - 4 * q;
    t.tok[0] = left > 0 ? v.x : ~one;
    t.tok[1] = left > 1 ? v.y : ~one;
    t.tok[2] = left > 2 ? v.z : ~one;
    t.tok[3] = left > 3 ? v.w : ~one;
    t.lead = one;
  };
  auto read = [&](const Place& p, Tile& t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.tok[i] = p.tok[i];
      if constexpr (kBase) {
        const int64_t tok = p.tok[i] ^ (p.tok[i] >> 31);
        const char* row = static_cast<const char*>(a.base) + tok * a.ld_b * kE;
        if (whole) {
          __builtin_memcpy(t.in[i], __builtin_assume_aligned(row + (int64_t)col * kE, kE), kC * kE);
        } else {
#pragma unroll
          for (int w = 0; w < kWords; ++w) t.in[i][w] = 0;
#pragma unroll
          for (int c = 0; c < kC; ++c)
            if (col + c < K) {
              if constexpr (kE == 4) t.in[i][c] = load_bits<kOut>(row, col + c);
              else t.in[i][c / 2] |= load_bits<kOut>(row, col + c) << (16 * (c & 1));
            }
        }
      }
    }
  };
  u32x4 u[kS][3];
  auto read_u = [&](int pos) {
    const int at = min(pos, end - 1) & ~15;
#pragma unroll
    for (int k = 0; k < kS; ++k)
#pragma unroll
      for (int i = 0; i < 3; ++i)
        u[k][i] = *reinterpret_cast<const u32x4*>(a.side[1].flat + ((int64_t)i * a.P + at + c16) * a.rk + k * 32 + 8 * q);
  };
  auto hold = [&](int ad) {
    held = ad;
#pragma unroll
    for (int k = 0; k < kS; ++k) {
      Eight<kF> e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rank = k * 32 + 8 * q + i;
#pragma unroll
        for (int w = 0; w < 4; ++w) e[i].w[w] = 0;
        if (rank < a.rank) {
          const uint16_t* row = a.side[0].F + ((int64_t)ad * a.rank + rank) * K;
          if (whole) {
            __builtin_memcpy(e[i].w, __builtin_assume_aligned(row + col, 2), 2 * kC);
          } else {
#pragma unroll
            for (int c = 0; c < kC; ++c)
              if (col + c < K) e[i].w[c / 2] |= (uint32_t)row[col + c] << (16 * (c & 1));
          }
        }
      }
#pragma unroll
      for (int c = 0; c < kC; c += 2) {
        uint32_t x[8][kA];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i].pair(c / 2, 1.f, x[i]);
#pragma unroll
        for (int t = 0; t < kA; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[c][k][t][j] = __builtin_amdgcn_perm(x[2 * j + 1][t], x[2 * j][t], 0x05040100u);
            f[c + 1][k][t][j] = __builtin_amdgcn_perm(x[2 * j + 1][t], x[2 * j][t], 0x07060302u);
          }
      }
    }
  };
  auto add = [&](int pos, int lead, const Tile& t) {
    const bool some = pos < runs;   // else the base's bits stay
    f32x4 acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (some) {
      const int ad = __builtin_amdgcn_readfirstlane(a.adapter[lead]);
      if (ad != held) hold(ad);
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int k = 0; k < kS; ++k) acc[c] = grad_mfma(u[k], f[c][k], acc[c]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t out[kWords];
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const uint32_t in = kBase ? t.in[i][w] : 0u;
        if constexpr (kE == 4) {
          out[w] = __float_as_uint(__uint_as_float(in) + acc[w][i]);
        } else {
          out[w] = value_bits<kOut>(lo16<kOut>(in) + acc[2 * w][i]) | value_bits<kOut>(hi16<kOut>(in) + acc[2 * w + 1][i]) << 16;
        }
        if (!some) out[w] = in;
      }
      if (t.tok[i] < 0) continue;
      char* row = static_cast<char*>(a.dX) + (int64_t)t.tok[i] * a.ld_dx * kE;
      if (whole) {
        __builtin_memcpy(__builtin_assume_aligned(row + (int64_t)col * kE, kE), out, kC * kE);
      } else {
#pragma unroll
        for (int c = 0; c < kC; ++c)
          if (col + c < K) store_bits<kOut>(row, col + c, kE == 4 ? out[c * kE / 4] : out[c / 2] >> (16 * (c & 1)) & 0xFFFFu);
      }
    }
  };
  Place p[3];
  Tile t[3];
  int leads[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) tokens(first + 16 * i, p[i]);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    read(p[i], t[i]);
    leads[i] = p[i].lead;
  }
  Place next;
  tokens(first + 48, next);
  read_u(first);
  for (int pos = first; pos < end;) {
#pragma unroll
    for (int i = 0; i < 3; ++i, pos += 16) {
      // behind the end nothing is stored
      add(pos, leads[i], t[i]);
      read_u(pos + 16);
      read(next, t[i]);
      leads[i] = next.lead;
      tokens(pos + 64, next);
    }
  }
}

// ---------------------------------------------------------------- launches
template <int kX, int kY, int kF, int kR>
static void grad_launch_rank(const GradArgs& a, int64_t max_chunks, GradStage stage, hipStream_t st) {
  if (stage == kGradProject) {
    const int64_t wgs = 1 + (int64_t)a.groups * a.halves * (a.side[0].splits + a.side[1].splits);
    hipLaunchKernelGGL((lora_grad_project_kernel<kX, kY, kF, kR>), dim3((unsigned)wgs), dim3(256), 0, st, a);
  } else {
    const int64_t wgs = (a.side[0].blocks + a.side[1].blocks) * a.halves * max_chunks;
    hipLaunchKernelGGL((lora_grad_outer_kernel<kX, kY, kR>), dim3((unsigned)wgs), dim3(64 * kOuterWaves), 0, st, a);
  }
}

template <int kX, int kY, int kF>
static void grad_launch_types(const GradArgs& a, int64_t max_chunks, GradStage stage, hipStream_t st) {
  if (a.r16 == 16) grad_launch_rank<kX, kY, kF, 1>(a, max_chunks, stage, st);
  else if (a.r16 == 32) grad_launch_rank<kX, kY, kF, 2>(a, max_chunks, stage, st);
  else grad_launch_rank<kX, kY, kF, 4>(a, max_chunks, stage, st);
}

template <int kF, int kOut, bool kBase, int kS>
static void grad_launch_input_rank(const GradArgs& a, hipStream_t st) {
  // A takes up to 64 registers: 4 kS words a column, twice for fp16's two terms; three
  // tiles of fp32 base up to 48, of 128 ranks 24
  constexpr int kC = std::min(kOut == GPTQ_F32 ? kS == 4 ? 2 : 4 : 8, 16 / (kS * (kF == GPTQ_F16 ? 2 : 1)));
  // in one round of two workgroups a CU
  const int64_t blocks = cdiv(a.side[0].K, 64 * kC);
  GradArgs b = a;
  b.input_tokens = (int)(cdiv(a.P, std::max<int64_t>(1, 512 / blocks) * 16) * 16);
  const int64_t wgs = blocks * cdiv(a.P, b.input_tokens);
  hipLaunchKernelGGL((lora_grad_input_kernel<kF, kOut, kBase, kS, kC>), dim3((unsigned)wgs), dim3(256), 0, st, b);
}

template <int kF, int kOut, bool kBase>
static void grad_launch_input(const GradArgs& a, hipStream_t st) {
  if (a.rk == 32) grad_launch_input_rank<kF, kOut, kBase, 1>(a, st);
  else if (a.rk == 64) grad_launch_input_rank<kF, kOut, kBase, 2>(a, st);
  else grad_launch_input_rank<kF, kOut, kBase, 4>(a, st);
}

template <int kF>
static void grad_launch(const GradArgs& a, bool codes, bool wide, int64_t max_chunks, GradStage stage, hipStream_t st) {
  if (stage == kGradInput) {
    if (a.wide_dx && a.base) grad_launch_input<kF, GPTQ_F32, true>(a, st);
    else if (a.wide_dx) grad_launch_input<kF, GPTQ_F32, false>(a, st);
    else if (a.base) grad_launch_input<kF, kF, true>(a, st);
    else grad_launch_input<kF, kF, false>(a, st);
  } else if (codes && wide) {
    grad_launch_types<GPTQ_E4M3, GPTQ_F32, kF>(a, max_chunks, stage, st);
  } else if (codes) {
    grad_launch_types<GPTQ_E4M3, kF, kF>(a, max_chunks, stage, st);
  } else if (wide) {
    grad_launch_types<kF, GPTQ_F32, kF>(a, max_chunks, stage, st);
  } else {
    grad_launch_types<kF, kF, kF>(a, max_chunks, stage, st);
  }
}

}  // namespace gq
