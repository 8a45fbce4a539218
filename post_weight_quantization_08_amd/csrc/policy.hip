// Clipped policy loss with a KL term: loss and gradient of rows.
//
// Of a row's softmax q only the answered token t matters, and the rest of the
// vocabulary as one sum.  With r a reference near the rest's maximum, c =
// log2(e) / T, s = sum over the rest of 2^((x - r) c), m the larger of r and x_t and
// S = s 2^((r - m) c) + 2^((x_t - m) c):
//   l = (x_t - m) / T - ln S, or -log1p(s 2^((r - x_t) c)) where x_t is the maximum,
//   dl/dx_t = s 2^((r - m) c) / (S T),   dl/dx_j = -2^((x_j - m) c) / (S T),
// so neither l near 0 nor 1 - q_t is a difference of nearly equal numbers.  The row's
// few other numbers (l, ratio, clipping, KL) are made by one wave in 64 bits, by functions
// of their own that leave the held blocks in their registers.
//
// The row kernel holds a row in registers (16-byte blocks as loaded), so a logit is
// read once and its gradient written once; the registers are refilled with the
// next row's as soon as a block's gradient is stored.  Few rows are split over
// workgroups, and rows too long for the registers of one, in two launches.
//
// 4096 x 131072 bf16 428 us (5.02 TB/s read and written, as a large copy); 777 x 50021
// fp16 51 us (512 workgroups have a row each, half of them a second); 8 x 32000 fp32 11 us,
// two launches of 3.5 and 4.6.
#include "rows.h"

namespace gq {

struct PlArgs {
  const void* x;
  int64_t ld;
  const int32_t* target;
  const float* old;
  const float* adv;
  const float* ref;
  const float* weight;
  float* loss;
  float* logprob;
  float* ratio;
  float* kl;
  void* grad;
  int64_t ld_g, n_rows;
  float c, inv_t, beta;
  double inv_td, low, high;   // 1 / T, and the interval that the ratio is held to
  int vocab;
  int parts, slots;           // part kernels: parts of a row, blocks a lane holds of one
  float* ws_sums;             // [rows][parts][2]: r, s
  float* ws_x;                // [rows]: the target's logit
};

// A row's answer, the same in every lane.
struct PlRow {
  int target;                 // -1: not scored
  float weight;
};
__device__ __forceinline__ PlRow pl_row(const PlArgs& a, int64_t row) {
  const int t = a.target[row];
  return PlRow{t >= 0 && t < a.vocab ? t : -1, a.weight ? a.weight[row] : 1.f};
}

// Where the target lies among a lane's blocks.
struct PlPlace {
  int slot, e;                // this lane's slot and element, slot -1 if it has it not
  bool edge;                  // the target is this lane's single logit
};
template <int kDt, int T>
__device__ __forceinline__ PlPlace pl_place(const Span<kDt>& sp, int target) {
  constexpr int E = Span<kDt>::E;
  PlPlace p{-1, 0, target >= 0 && sp.edge(threadIdx.x) == target};
  const int at = target - sp.head;
  if (target >= 0 && at >= 0 && at < sp.blocks * E && at / E % T == (int)threadIdx.x) {
    p.slot = at / E / T;
    p.e = at % E;
  }
  return p;
}

// What the gradient of a row is made of.
struct PlFinal {
  float r, rest, at;          // rest: rest * 2^((x - r) c); the target's gradient
  int zero, nan;
};

// A constant made where it is used: kept in registers from row to row, those of the functions
// below spill held blocks.
template <uint64_t kBits>
__device__ __forceinline__ double pl_const() {
  uint32_t lo, hi;
  asm volatile("v_mov_b32 %0, %2\n\tv_mov_b32 %1, %3" : "=&v"(lo), "=v"(hi) : "n"((int)(uint32_t)kBits), "n"((int)(uint32_t)(kBits >> 32)));
  return __hiloint2double((int)hi, (int)lo);
}
#define PL_CONST(x) pl_const<__builtin_bit_cast(uint64_t, (double)(x))>()

// e^d, e^d - 1 and e^d - 1 - d of a 64-bit d.  d = n ln 2 + f with |f| <= ln 2 / 2; at x =
// f / 8 the series of e^x - 1 - x, whose first term left out, x^9 / 9!, is 2^-49 of it; then
// three times from x to 2 x by e^(2 x) - 1 - 2 x = p^2 + 2 (p - x) with p = e^x - 1, in which
// nothing cancels.  A NaN stays one.
struct PlExp {
  double p, over, e;          // e^f - 1, e^f - 1 - f, e^d
  bool near;                  // n = 0: d = f
  __device__ __forceinline__ explicit PlExp(double d) {
    // beyond, e^d is 0 or infinite in 64 bits
    d = d > 720.0 ? 720.0 : d < -760.0 ? -760.0 : d;
    const double n = rint(d * PL_CONST(1.4426950408889634));
    // ln 2 in two parts, the first of 24 bits, so that n times it is exact
    double x = 0.125 * fma(n, PL_CONST(1.904654299957768e-09), fma(-n, PL_CONST(0.6931471824645996), d));
    double q = fma(PL_CONST(1.0 / 40320), x, PL_CONST(1.0 / 5040));
    q = fma(q, x, PL_CONST(1.0 / 720));
    q = fma(q, x, PL_CONST(1.0 / 120));
    q = fma(q, x, PL_CONST(1.0 / 24));
    q = fma(q, x, PL_CONST(1.0 / 6));
    q = fma(q, x, 0.5);
    over = x * x * q;
    p = x + over;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      over = fma(p, p, 2.0 * over);
      x *= 2.0;
      p = x + over;
    }
    e = ldexp(1.0 + p, (int)n);
    near = n == 0.0;
  }
  __device__ __forceinline__ double less_one() const { return near ? p : e - 1.0; }
  __device__ __forceinline__ double less_line(double d) const {   // e^d - 1 - d
    return near ? over : d == INFINITY ? d : less_one() - d;
  }
};

// ln x and ln(1 + x) of fp32 numbers, x > 0 and x >= 0: the 32-bit function and one step of
// Newton's, which leaves the square of its error.
__device__ __forceinline__ double pl_ln(float x) {
  int e;
  const float m = frexpf(x, &e), y = logf(m);
  return fma((double)e, PL_CONST(0.69314718055994530942), (double)y + fma((double)m, PlExp(-(double)y).e, -1.0));
}
__device__ __forceinline__ double pl_ln1p(float x) {
  const float y = log1pf(x);
  const float left = (float)((double)x - PlExp(y).less_one());
  return (double)y + (double)(left / (1.f + x));
}

// The row's outputs and what its gradient is made of, from the rest's sum and the
// target's logit.  `write`: this lane stores the outputs.
__device__ __forceinline__ PlFinal pl_final(const PlArgs& a, int64_t row, const PlRow& p, float r, float s, float xt,
                                            bool write) {
  PlFinal f{r, 0.f, 0.f, 1, 0};
  double loss = 0.0, lp = 0.0, ratio = 0.0, kl = 0.0;
  if (p.target >= 0) {
    const float m = fmaxf(xt, s > 0.f ? r : -INFINITY);
    const float up = s > 0.f ? exp2_hw((r - m) * a.c) : 0.f;
    const float mass = s != s ? s : s * up, et = exp2_hw((xt - m) * a.c), total = mass + et;
    const bool bad = !(total > 0.f && total < INFINITY);
    double coef = 0.0;
    if (bad) {
      loss = lp = ratio = kl = NAN;
    } else {
      lp = xt == m ? -pl_ln1p(mass) : ((double)xt - m) * a.inv_td - pl_ln(total);
      const double adv = a.adv[row], old = a.old[row];
      // a masked token has ratio 0 and no gradient, whatever the others' finite or infinite
      // numbers are; comparisons let a NaN through
      const bool gone = lp == -INFINITY;
      ratio = gone && old == old ? 0.0 : PlExp(lp - old).e;
      const double open = adv == 0.0 && ratio == INFINITY ? 0.0 : ratio * adv;
      const double held = (ratio < a.low ? a.low : ratio > a.high ? a.high : ratio) * adv;
      loss = open > held ? -held : -open;
      coef = open > held ? 0.0 : -open;
      if (a.ref) {
        const double ref = a.ref[row], d = gone && ref == ref ? INFINITY : ref - lp;
        const PlExp up(d);
        kl = up.less_line(d);
        float beta = a.beta;
        asm volatile("" : "+v"(beta));     // nor its 64 bits
        if (beta > 0.f) {                  // 0 times an infinite kl is nothing
          loss += beta * kl;
          coef -= beta * up.less_one();
        }
      }
      if (gone && coef == coef) coef = 0.0;
    }
    const float w = p.weight * a.inv_t;
    f.zero = w == 0.f;
    const float cf = f.zero ? 0.f : (float)(coef * w), inv_s = 1.f / total;
    f.nan = !f.zero && (bad || cf != cf);
    f.rest = s > 0.f ? -cf * (up * inv_s) : 0.f;
    f.at = cf * (mass * inv_s);
  }
  if (write) {
    a.loss[row] = (float)loss;
    if (a.logprob) a.logprob[row] = (float)lp;
    if (a.ratio) a.ratio[row] = (float)ratio;
    if (a.kl) a.kl[row] = (float)kl;
  }
  return f;
}

// Into scalar registers.
__device__ __forceinline__ PlFinal pl_fetch(const PlFinal& g) {
  return PlFinal{uniform(g.r), uniform(g.rest), uniform(g.at), __builtin_amdgcn_readfirstlane(g.zero),
                 __builtin_amdgcn_readfirstlane(g.nan)};
}

// A held block's logits as the rest's: the target's taken out into xt, blocks that
// the lane does not have masked.
template <int kDt>
__device__ __forceinline__ void pl_take(float (&v)[Span<kDt>::E], bool mine, int e, bool there, float& xt) {
  constexpr int E = Span<kDt>::E;
  if (mine) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      xt = i == e ? v[i] : xt;
      v[i] = i == e ? -INFINITY : v[i];
    }
  }
  if (!there) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = -INFINITY;
  }
}

// r, s of the rest, the slow way: around the true maximum, differences taken
// before they are scaled.  Reads the row again.
template <int kDt, int T>
__device__ __forceinline__ void pl_exact_sums(const PlArgs& a, const Span<kDt>& sp, const PlPlace& at, int slot0,
                                              int slots, float xe, float& r, float& s, float (&red)[T / 64][2]) {
  constexpr int E = Span<kDt>::E;
  const bool nan = s != s;
  auto get = [&](int i, float (&v)[E]) {
    const int first = (slot0 + i) * T, t = threadIdx.x;
    Blocks<kDt>::unpack(t < sp.blocks - first ? sp.load(first, t) : masked_block<kDt>(), v);
    hide<kDt>(v, slot0 + i == at.slot ? 1u << at.e : 0u);
  };
  float m = xe;
#pragma unroll 1
  for (int i = 0; i < slots; ++i) {
    float v[E];
    get(i, v);
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, v[e]);
  }
  m = wave_reduce(m, [](float p, float q) { return fmaxf(p, q); });
  lds_barrier();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][0] = m;
  lds_barrier();
#pragma unroll
  for (int i = 0; i < T / 64; ++i) m = fmaxf(m, red[i][0]);
  lds_barrier();
  r = -3.4028235e38f;
  s = 0.f;
  if (m == -INFINITY) {
    s = nan ? NAN : 0.f;
    return;
  }
  r = m;
  if (m == INFINITY) {
    s = NAN;
    return;
  }
#pragma unroll 1
  for (int i = 0; i < slots; ++i) {
    float v[E];
    get(i, v);
#pragma unroll
    for (int e = 0; e < E; ++e) s += exp2_hw((v[e] - m) * a.c);
  }
  s += exp2_hw((xe - m) * a.c);
  ds_join<T>(r, s, a.c, red);
}

// Gradients of a block.  kFast: rc is r c rounded and `rest` made for that.
template <int kDt, bool kFast>
__device__ __forceinline__ void pl_gradient(const PlFinal& f, float rest, float rc, float c,
                                            const float (&v)[Span<kDt>::E], float (&g)[Span<kDt>::E]) {
#pragma unroll
  for (int e = 0; e < Span<kDt>::E; ++e) g[e] = rest * exp2_hw(kFast ? fmaf(v[e], c, -rc) : (v[e] - f.r) * c);
}
template <int kDt>
__device__ __forceinline__ void pl_put(float (&g)[Span<kDt>::E], bool mine, int e, float at) {
  if (mine) {
#pragma unroll
    for (int i = 0; i < Span<kDt>::E; ++i) g[i] = i == e ? at : g[i];
  }
}
// A single logit's.
__device__ __forceinline__ float pl_edge(const PlFinal& f, float c, float xe, bool target) {
  if (f.zero || f.nan) return f.nan ? NAN : 0.f;
  return target ? f.at : f.rest * exp2_hw((xe - f.r) * c);
}

// Blocks a lane holds in registers; a row kernel's others lie in LDS, where direct
// loads put them.
constexpr int kPlHeld = 16;

// Row kernel: T threads hold a row of at most T NB blocks.
template <int kDt, int T, int NB, bool kGrad>
__global__ __launch_bounds__(T) __attribute__((amdgpu_waves_per_eu(4))) void policy_row_kernel(PlArgs a) {
  constexpr int E = Span<kDt>::E;
  constexpr int kHeld = NB < kPlHeld ? NB : kPlHeld;
  __shared__ float red[T / 64][2];
  __shared__ float target_x;
  __shared__ PlFinal fin;
  __shared__ __align__(16) u32x4 tail[NB > kHeld ? NB - kHeld : 1][NB > kHeld ? T : 1];
  const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  int64_t row = blockIdx.x;
  if (row >= a.n_rows) return;
  u32x4 w[kHeld];
  // the next row's block into the place of block i, which nothing reads any more
  auto refill = [&](const DsSource<kDt>& src, int i) {
    if (i < kHeld) w[i < kHeld ? i : 0] = src.load(i * T);
    else lds_load16(src.block(i * T), reinterpret_cast<char*>(&tail[i - kHeld][wave * 64]));
  };
  // together, and after all of them were read: a direct load in flight is waited
  // for at the next reading
  auto refill_tail = [&](const DsSource<kDt>& src) {
    if constexpr (NB > kHeld) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int i = kHeld; i < NB; ++i) refill(src, i);
    }
  };
  Span<kDt> sp(a.x, row, a.ld, a.vocab);
  PlRow p = pl_row(a, row);
  uint32_t edge_bits = load_bits<kDt>(sp.p, max(sp.edge(t), 0));
  {
    const DsSource<kDt> src(sp, true);
#pragma unroll
    for (int i = 0; i < NB; ++i) refill(src, i);
  }
  for (;;) {
    const int64_t next_row = row + gridDim.x;
    const bool more = next_row < a.n_rows;
    const Span<kDt> next(a.x, more ? next_row : row, a.ld, a.vocab);
    const DsSource<kDt> src(next, more);
    const PlPlace at = pl_place<kDt, T>(sp, p.target);
    const int held = max(sp.blocks - t + T - 1, 0) / T;   // slots of this lane with a block of its own
    float r = kDsFloor, rc = kDsFloor * a.c, s = 0.f, xt = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      float v[E];
      unpack_held<kDt>(w[i], v);
      pl_take<kDt>(v, i == at.slot, at.e, i < held, xt);
      ds_add_block<kDt>(r, rc, s, v, a.c);
      if constexpr (!kGrad) refill(src, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (NB > kHeld) {
      memory_done();   // this wave's part of the tail is there
#pragma unroll
      for (int i = kHeld; i < NB; ++i) {
        float v[E];
        Blocks<kDt>::unpack(tail[i - kHeld][t], v);
        pl_take<kDt>(v, i == at.slot, at.e, i < held, xt);
        ds_add_block<kDt>(r, rc, s, v, a.c);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!kGrad) refill_tail(src);
    }
    const float xe = sp.edge(t) >= 0 ? bits_value<kDt>(edge_bits) : -INFINITY;
    const float xr = at.edge ? -INFINITY : xe;
    if (t < 64) {
      float v[E];
      v[0] = xr;
#pragma unroll
      for (int e = 1; e < E; ++e) v[e] = -INFINITY;
      ds_add_block<kDt>(r, rc, s, v, a.c);
    }
    s *= exp2_hw(-fmaf(r, a.c, -rc));
    if (at.slot >= 0 || at.edge) target_x = at.edge ? xe : xt;
    const uint32_t edge_ahead = load_bits<kDt>(next.p, max(next.edge(t), 0));
    ds_join<T>(r, s, a.c, red);
    const float x_target = target_x;
    // a rest of -inf alone, or out of the fast way's range
    const bool exact = !(s > 0.f && s < INFINITY && fabsf(r) * a.c < kDsFast);
    if (exact) pl_exact_sums<kDt, T>(a, sp, at, 0, NB, xr, r, s, red);
    if (t < 64) {
      const PlFinal f = pl_final(a, row, p, r, s, x_target, t == 0);
      if (t == 0) fin = f;
    }
    lds_barrier();
    if constexpr (kGrad) {
      const PlFinal f = pl_fetch(fin);
      if (sp.edge(t) >= 0)
        store_el<kDt>(static_cast<char*>(a.grad) + row * a.ld_g * Span<kDt>::kSize, sp.edge(t), pl_edge(f, a.c, xe, at.edge));
      if (f.zero || f.nan) {
        float g[E];
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = f.nan ? NAN : 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          if (i < held) ds_store<kDt>(a.grad, a.ld_g, sp, row, i * T, t, g);
          if (i < kHeld) refill(src, i);
        }
        refill_tail(src);
      } else if (!exact) {
        const float frc = f.r * a.c;
        const float rest = f.rest * exp2_hw(-fmaf(f.r, a.c, -frc));
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          float v[E], g[E];
          if (i < kHeld) unpack_held<kDt>(w[i < kHeld ? i : 0], v);
          else Blocks<kDt>::unpack(tail[i < kHeld ? 0 : i - kHeld][t], v);
          pl_gradient<kDt, true>(f, rest, frc, a.c, v, g);
          pl_put<kDt>(g, i == at.slot, at.e, f.at);
          if (i < held) ds_store<kDt>(a.grad, a.ld_g, sp, row, i * T, t, g);
          if (i < kHeld) refill(src, i);
          __builtin_amdgcn_sched_barrier(0);   // one block's registers at a time
        }
        refill_tail(src);
      } else {
#pragma unroll 1
        for (int i = 0; i < held; ++i) {
          float v[E], g[E];
          Blocks<kDt>::unpack(sp.load(i * T, t), v);
          pl_gradient<kDt, false>(f, f.rest, 0.f, a.c, v, g);
          pl_put<kDt>(g, i == at.slot, at.e, f.at);
          ds_store<kDt>(a.grad, a.ld_g, sp, row, i * T, t, g);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) refill(src, i);
        refill_tail(src);
      }
    }
    if (!more) break;
    row = next_row;
    sp = next;
    edge_bits = edge_ahead;
    p = pl_row(a, row);
  }
  if constexpr (NB > kHeld) memory_done();   // no direct load ends after the workgroup
}

constexpr int kPlPartThreads = 256;
constexpr int kPlPartBlocks = 16;   // blocks a lane holds of a part, at most

// Part kernels.  kSums: r, s of a part's rest and the target's logit into the
// workspace.  Otherwise: the parts joined, the outputs (part 0), the part's gradients.
template <int kDt, int NB, bool kSums>
__global__ __launch_bounds__(kPlPartThreads) void policy_part_kernel(PlArgs a) {
  constexpr int T = kPlPartThreads;
  constexpr int E = Span<kDt>::E;
  __shared__ float red[T / 64][2];
  const int t = threadIdx.x;
  const int per_row = kSums || a.grad ? a.parts : 1;
  const int64_t row = blockIdx.x / per_row;
  const int part = blockIdx.x % per_row;
  const Span<kDt> sp(a.x, row, a.ld, a.vocab);
  const PlRow p = pl_row(a, row);
  const PlPlace at = pl_place<kDt, T>(sp, p.target);
  const bool edges = part == 0;
  const int slot0 = part * a.slots;
  const int held = min(max(sp.blocks - slot0 * T - t + T - 1, 0) / T, a.slots);
  u32x4 w[NB];
  float xe = -INFINITY;
  if (kSums || a.grad) {
    const DsSource<kDt> src(sp, true);
#pragma unroll
    for (int i = 0; i < NB; ++i) w[i] = src.load((slot0 + min(i, a.slots - 1)) * T);
    if (edges && sp.edge(t) >= 0) xe = load_el<kDt>(sp.p, sp.edge(t));
  }
  if constexpr (kSums) {
    float r = kDsFloor, rc = kDsFloor * a.c, s = 0.f, xt = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      float v[E];
      unpack_held<kDt>(w[i], v);
      pl_take<kDt>(v, slot0 + i == at.slot && i < held, at.e, i < held, xt);
      ds_add_block<kDt>(r, rc, s, v, a.c);
      __builtin_amdgcn_sched_barrier(0);
    }
    const float xr = at.edge ? -INFINITY : xe;
    if (edges && t < 64) {
      float v[E];
      v[0] = xr;
#pragma unroll
      for (int e = 1; e < E; ++e) v[e] = -INFINITY;
      ds_add_block<kDt>(r, rc, s, v, a.c);
    }
    if (at.slot >= slot0 && at.slot < slot0 + a.slots) a.ws_x[row] = xt;
    if (edges && at.edge) a.ws_x[row] = xe;
    s *= exp2_hw(-fmaf(r, a.c, -rc));
    ds_join<T>(r, s, a.c, red);
    if (!(s > 0.f && s < INFINITY && fabsf(r) * a.c < kDsFast))
      pl_exact_sums<kDt, T>(a, sp, at, slot0, a.slots, edges ? xr : -INFINITY, r, s, red);
    if (t == 0) {
      float* o = a.ws_sums + (row * a.parts + part) * 2;
      o[0] = r;
      o[1] = s;
    }
  } else {
    float r = -3.4028235e38f, s = 0.f;
    for (int i = t; i < a.parts; i += T) {
      const float* o = a.ws_sums + (row * a.parts + i) * 2;
      const float to = fmaxf(r, o[0]);
      s = (s == 0.f ? 0.f : s * exp2_hw((r - to) * a.c)) + (o[1] == 0.f ? 0.f : o[1] * exp2_hw((o[0] - to) * a.c));
      r = to;
    }
    ds_join<T>(r, s, a.c, red);
    const float xt = p.target >= 0 ? a.ws_x[row] : 0.f;
    const PlFinal f = pl_final(a, row, p, r, s, xt, part == 0 && t == 0);
    if (!a.grad) return;
    if (edges && sp.edge(t) >= 0)
      store_el<kDt>(static_cast<char*>(a.grad) + row * a.ld_g * Span<kDt>::kSize, sp.edge(t), pl_edge(f, a.c, xe, at.edge));
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if (i >= held) continue;
      float v[E], g[E];
      unpack_held<kDt>(w[i], v);
      pl_gradient<kDt, false>(f, f.rest, 0.f, a.c, v, g);
      pl_put<kDt>(g, slot0 + i == at.slot, at.e, f.at);
      if (f.zero || f.nan) {
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = f.nan ? NAN : 0.f;
      }
      ds_store<kDt>(a.grad, a.ld_g, sp, row, (slot0 + i) * T, t, g);
    }
  }
}

struct PlPlan {
  int threads, held;       // row kernel: threads and blocks a lane holds; threads 0: part kernels
  int parts, slots;
  size_t off_x, total;
};

// Whole rows, or parts of rows.  Few rows in whole leave CUs idle.  The smallest
// workgroups in which a row fits 16 blocks a lane; one of up to 4 blocks in
// registers for 4.
static PlPlan pl_plan(int64_t n_rows, int64_t vocab, int es) {
  PlPlan p{};
  const int64_t blocks = vocab * es / 16;
  const int64_t row_max = 1024 * 20;
  if (blocks <= 1024 || (n_rows > (blocks <= 256 * 16 ? 32 : 64) && blocks <= row_max)) {
    p.threads = blocks <= 256 * 16 ? 256 : blocks <= 512 * 16 ? 512 : 1024;
    p.held = blocks <= 256 * 4 ? 4 : blocks <= 1024 * 16 ? 16 : 20;
    return p;
  }
  // parts: enough for four workgroups per CU, of one block a lane or more
  int64_t slots = kPlPartBlocks;
  while (slots > 1 && n_rows * cdiv(blocks, slots * kPlPartThreads) < 1024) slots /= 2;
  p.slots = (int)slots;
  p.parts = (int)cdiv(blocks, slots * kPlPartThreads);
  p.off_x = align_up((size_t)n_rows * p.parts * 8, 256);
  p.total = p.off_x + (size_t)n_rows * 4;
  return p;
}

size_t policy_workspace_bytes(int64_t n_rows, int64_t vocab) {
  return std::max(pl_plan(n_rows, vocab, 2).total, pl_plan(n_rows, vocab, 4).total);
}

template <int kDt, int T, int NB>
static void pl_launch_rows(const PlArgs& a, int per_cu, hipStream_t st) {
  const dim3 grid((unsigned)std::min<int64_t>(a.n_rows, 256 * per_cu));
  if (a.grad) hipLaunchKernelGGL((policy_row_kernel<kDt, T, NB, true>), grid, dim3(T), 0, st, a);
  else hipLaunchKernelGGL((policy_row_kernel<kDt, T, NB, false>), grid, dim3(T), 0, st, a);
}

template <int kDt, int NB>
static void pl_launch_parts(const PlArgs& a, hipStream_t st) {
  const dim3 all((unsigned)(a.n_rows * a.parts)), rows((unsigned)a.n_rows);
  hipLaunchKernelGGL((policy_part_kernel<kDt, NB, true>), all, dim3(kPlPartThreads), 0, st, a);
  hipLaunchKernelGGL((policy_part_kernel<kDt, NB, false>), a.grad ? all : rows, dim3(kPlPartThreads), 0, st, a);
}

template <int kDt>
static void pl_dispatch(const PlArgs& a, const PlPlan& p, hipStream_t st) {
  if (p.threads == 256 && p.held == 4) pl_launch_rows<kDt, 256, 4>(a, 6, st);
  else if (p.threads == 256) pl_launch_rows<kDt, 256, 16>(a, 4, st);
  else if (p.threads == 512) pl_launch_rows<kDt, 512, 16>(a, 2, st);
  else if (p.threads == 1024 && p.held == 16) pl_launch_rows<kDt, 1024, 16>(a, 1, st);
  else if (p.threads == 1024) pl_launch_rows<kDt, 1024, 20>(a, 1, st);
  else if (p.slots <= 4) pl_launch_parts<kDt, 4>(a, st);
  else pl_launch_parts<kDt, kPlPartBlocks>(a, st);
}

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_policy_loss(const void* logits, int32_t x_dtype, int64_t n_rows, int64_t vocab, int64_t ld_x,
                                        const int32_t* targets, const float* old_logprob, const float* advantage,
                                        const float* ref_logprob, float clip_low, float clip_high, float kl_coef,
                                        float temperature, const float* weight, float* loss, float* logprob, float* ratio,
                                        float* kl, void* grad, int64_t ld_g, void* workspace, size_t ws_bytes,
                                        void* stream) {
  GQ_CHECK_ARG(x_dtype == GPTQ_F32 || x_dtype == GPTQ_F16 || x_dtype == GPTQ_BF16);
  GQ_CHECK_ARG(n_rows >= 0 && n_rows <= ((int64_t)1 << 22) && vocab >= 1 && vocab <= ((int64_t)1 << 30));
  GQ_CHECK_ARG(ld_x >= vocab && ld_x <= ((int64_t)1 << 36));
  GQ_CHECK_ARG(temperature >= 1e-4f && temperature <= 1e4f);
  GQ_CHECK_ARG(clip_low >= 0.f && clip_low <= 1.f && clip_high >= 0.f && clip_high <= 1e4f);
  GQ_CHECK_ARG(kl_coef >= 0.f && kl_coef <= 1e4f);
  GQ_CHECK_ARG(grad == nullptr || (ld_g >= vocab && ld_g <= ((int64_t)1 << 36)));
  if (vocab > ((int64_t)1 << 21)) return GPTQ_EUNSUPPORTED;
  if (n_rows == 0) return GPTQ_OK;
  GQ_CHECK_ARG(logits && targets && old_logprob && advantage && loss);
  GQ_CHECK_ARG(grad == nullptr || grad != logits || ld_g == ld_x);
  const int es = x_dtype == GPTQ_F32 ? 4 : 2;
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(logits) % es == 0 && reinterpret_cast<uintptr_t>(grad) % es == 0);
  const size_t need = policy_workspace_bytes(n_rows, vocab);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GPTQ_ENOMEM;
  const PlPlan pl = pl_plan(n_rows, vocab, es);
  GQ_CHECK_ARG(pl.threads != 0 || reinterpret_cast<uintptr_t>(workspace) % 256 == 0);
  PlArgs a{};
  a.x = logits;
  a.ld = ld_x;
  a.target = targets;
  a.old = old_logprob;
  a.adv = advantage;
  a.ref = ref_logprob;
  a.weight = weight;
  a.loss = loss;
  a.logprob = logprob;
  a.ratio = ratio;
  a.kl = kl;
  a.grad = grad;
  a.ld_g = ld_g;
  a.n_rows = n_rows;
  a.c = (float)(1.4426950408889634074 / temperature);
  a.inv_t = (float)(1.0 / temperature);
  a.beta = kl_coef;
  a.inv_td = 1.0 / temperature;
  a.low = 1.0 - (double)clip_low;
  a.high = 1.0 + (double)clip_high;
  a.vocab = (int)vocab;
  a.parts = pl.parts;
  a.slots = pl.slots;
  a.ws_sums = static_cast<float*>(workspace);
  a.ws_x = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.off_x);
  hipStream_t st = static_cast<hipStream_t>(stream);
  TimedScope ts(kTimePolicy, st);
  if (x_dtype == GPTQ_F32) pl_dispatch<GPTQ_F32>(a, pl, st);
  else if (x_dtype == GPTQ_F16) pl_dispatch<GPTQ_F16>(a, pl, st);
  else pl_dispatch<GPTQ_BF16>(a, pl, st);
  GQ_LAUNCHED();
  return GPTQ_OK;
}
