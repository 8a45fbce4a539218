// Log probabilities of given tokens, entropy and the best alternatives of
// rows of logits, each logit read from memory once.
//
// With c = log2(e) / T and a reference r, one pass keeps S = sum 2^a and U =
// sum 2^a a over a = (x - r) c.  Then
//   log p(t) = (x_t - r) / T - ln S,   lse = r / T + ln S,
//   entropy  = ln 2 (log2 S - U / S),
// and two (r, S, U) join by moving one to the other's reference: S' = S f,
// U' = f (U + d S), d = (r - r') c, f = 2^d.  The reference need not be the
// maximum: a lane takes a new one only when a logit's term would exceed 2^8,
// so the common step is one fused multiply-add, one exponential, an
// addition and a second fused multiply-add per logit.
//
// The k best alternatives come out of the same pass.  Every lane keeps the
// maximum of what it saw (disjoint parts of the row), and the maximum of
// every group of blocks goes to LDS.  The k-th largest of the lanes' maxima
// is a lower bound of the k-th largest logit that at least k logits reach,
// and only groups whose maximum reaches it can hold alternatives: about k
// of them, read again (a few percent of the row), their logits above the
// bound sorted by (value, index).
//
// Bound by memory: 2 or 4 bytes and about 6 operations, one exponential, per
// logit.  4096 rows of 131072 bf16, k = 64: 213 us, 5.0 TB/s of logits; 1000 of
// 50021 fp32, k = 1: 44 us, 4.5 TB/s.  One row of 131072: 12.3 us in two launches,
// of which the reading is a small part.
#include "answer.h"

namespace gq {

constexpr int kLpThreads = 256;
constexpr int kLpGroups = 2048;        // group maxima held in LDS
constexpr int kLpGroupBlocks = 16;     // blocks of a group when there are more blocks than kLpGroups
constexpr int kLpKeys = 1024;          // candidates held in LDS
constexpr int kLpMaxBlocks = kLpGroups * kLpGroupBlocks;   // blocks one workgroup can take

// The fast pass: no reference below kLpFloor (a power of two, so its product
// with c is exact; large negative masks never become one), none whose product
// with c is so large that its rounding could push terms out of range
// (kLpFast), and a new one when a logit is 2^kLpLag above the old (a lagging
// reference costs U / S and log2 S digits that their difference would lose).
constexpr float kLpFloor = -1048576.f, kLpFast = 268435456.f, kLpLag = 8.f;

struct LpArgs {
  const void* x;
  int64_t ld;
  const int32_t* targets;
  float c, inv_t;          // log2(e) / T, 1 / T
  int vocab, k, parts, blocks;   // parts of a row, blocks of a part
  float *logprob, *lse, *entropy, *top_lp;
  int32_t* top_id;
  float* ws_sums;          // [rows][parts][4]
  uint64_t* ws_keys;       // [rows][parts][k]
};

// Number of leading bits of order_of() that tell the values of a type apart:
// a bf16 has no more than 16, an fp16 widened to fp32 1 + 8 + 10.
template <int kDt>
constexpr int kOrderBits = kDt == GPTQ_F32 ? 32 : kDt == GPTQ_F16 ? 19 : 16;

struct LpShared {
  float gmax[kLpGroups];
  uint64_t keys[kLpKeys];
  uint16_t list[kLpGroups];
  uint32_t lane_order[kLpThreads];
  float red[4][4];
  int flagged, count;
};

// Sums and the maximum over a workgroup; every thread gets them.
__device__ __forceinline__ void lp_join(Sums& a, float& m, float c, LpShared& sh) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  auto fmax2 = [](float p, float q) { return fmaxf(p, q); };
  auto add2 = [](float p, float q) { return p + q; };
  const float rw = wave_reduce(a.r, fmax2);
  a = moved(a, rw, c);
  a.s = wave_reduce(a.s, add2);
  a.u = wave_reduce(a.u, add2);
  m = wave_reduce(m, fmax2);
  if (lane == 0) {
    sh.red[wave][0] = a.r;
    sh.red[wave][1] = a.s;
    sh.red[wave][2] = a.u;
    sh.red[wave][3] = m;
  }
  __syncthreads();
  float r = sh.red[0][0];
  m = sh.red[0][3];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    r = fmaxf(r, sh.red[w][0]);
    m = fmaxf(m, sh.red[w][3]);
  }
  a = Sums{r, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const Sums b = moved(Sums{sh.red[w][0], sh.red[w][1], sh.red[w][2]}, r, c);
    a.s += b.s;
    a.u += b.u;
  }
  __syncthreads();
}

struct LpOut {
  Sums s;
  float log_s, inv_t;
  bool dead;               // nothing above -inf
  __device__ __forceinline__ LpOut(Sums a, float it) : s(a), log_s(kLn2 * log2f(a.s)), inv_t(it), dead(a.s == 0.f) {}
  __device__ __forceinline__ float logprob(float x) const { return dead ? -INFINITY : (x - s.r) * inv_t - log_s; }
  __device__ __forceinline__ float lse() const { return dead ? -INFINITY : fmaf(s.r, inv_t, log_s); }
  __device__ __forceinline__ float entropy() const {
    const float h = log_s - kLn2 * (s.u / s.s);
    return dead || h < 0.f ? 0.f : h;
  }
};

__device__ __forceinline__ void lp_write_row(const LpArgs& a, int64_t row, const LpOut& o, float x_target, bool scored) {
  if (a.logprob) a.logprob[row] = scored ? o.logprob(x_target) : 0.f;
  if (a.lse) a.lse[row] = o.lse();
  if (a.entropy) a.entropy[row] = o.entropy();
}

// The k-th largest of 256 values of kBits bits (0 if fewer than k are not 0),
// from LDS, by every wave for itself: the answer's bits from the top, each
// kept if k values still reach it.
template <int kBits>
__device__ __forceinline__ uint32_t kth_largest(const uint32_t* v, int k) {
  const int lane = threadIdx.x & 63;
  const uint32_t a0 = v[lane], a1 = v[lane + 64], a2 = v[lane + 128], a3 = v[lane + 192];
  uint32_t t = 0;
  for (int b = kBits - 1; b >= 0; --b) {
    const uint32_t cand = t | 1u << b;
    const int n = __popcll(__ballot(a0 >= cand)) + __popcll(__ballot(a1 >= cand)) + __popcll(__ballot(a2 >= cand)) +
                  __popcll(__ballot(a3 >= cand));
    if (n >= k) t = cand;
  }
  return t;
}

// Position of `key` in descending order among n keys in LDS.
__device__ __forceinline__ int rank_of(uint64_t key, const uint64_t* keys, int n) {
  int r = 0;
  int i = 0;
  for (; i + 8 <= n; i += 8) {
    uint64_t q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = keys[i + e];
#pragma unroll
    for (int e = 0; e < 8; ++e) r += q[e] > key;
  }
  for (; i < n; ++i) r += keys[i] > key;
  return r;
}

// keys[0..n) -> its k largest, sorted, in keys[0..k).  n <= kLpKeys.
__device__ __forceinline__ void sort_top(LpShared& sh, int n, int k) {
  uint64_t key[kLpKeys / kLpThreads];
  int rank[kLpKeys / kLpThreads];
#pragma unroll
  for (int i = 0; i < kLpKeys / kLpThreads; ++i) {
    const int at = threadIdx.x + i * kLpThreads;
    rank[i] = kLpKeys;
    if (at < n) {
      key[i] = sh.keys[at];
      rank[i] = rank_of(key[i], sh.keys, n);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kLpKeys / kLpThreads; ++i)
    if (rank[i] < k) sh.keys[rank[i]] = key[i];
  __syncthreads();
}

// The keys of a part's logits whose order (kShift bits down) is at least
// `bound`, or above it for kAbove, appended to sh.keys in any order; gives up
// once they are more than kLpKeys (sh.count then is, too).
template <int kDt, int kGs, bool kAbove>
__device__ void lp_collect(const LpArgs& a, const Blocks<kDt>& bl, int b0, int b1, uint32_t bound, LpShared& sh) {
  constexpr int E = Blocks<kDt>::E;
  constexpr int kShift = 32 - kOrderBits<kDt>;
  const int tid = threadIdx.x;
  auto reaches = [&](float x) { return kAbove ? order_of(x) >> kShift > bound : order_of(x) >> kShift >= bound; };
  const int groups = (b1 - b0 + kGs - 1) / kGs;
  __syncthreads();
  if (tid == 0) sh.flagged = sh.count = 0;
  __syncthreads();
  for (int g = tid; g < groups; g += kLpThreads)
    if (reaches(sh.gmax[g])) sh.list[atomicAdd(&sh.flagged, 1)] = (uint16_t)g;
  __syncthreads();
  const int items = sh.flagged * kGs;
  for (int i0 = tid; i0 < items; i0 += 2 * kLpThreads) {
    if (*(volatile int*)&sh.count > kLpKeys) break;
    float v[2][E];
    int blk[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = i0 + q * kLpThreads;
      blk[q] = i < items ? b0 + sh.list[i / kGs] * kGs + i % kGs : b1;
      if (blk[q] < b1) bl.fetch(blk[q], v[q]);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (blk[q] < b1)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int j = bl.element(blk[q], e);
          if (reaches(v[q][e]) && j >= 0 && j < a.vocab) {
            const int at = atomicAdd(&sh.count, 1);
            if (at < kLpKeys) sh.keys[at] = key_of(v[q][e], j);
          }
        }
  }
  __syncthreads();
}

// Walks a part in order, one logit a thread and round, and appends keys:
// kTies: the logits at the bound, until there are k keys in all (the rest of
// the ties have higher indices).  Otherwise every logit above the k-th best so
// far, in a buffer that is cut to its k best when it is nearly full; without
// kWhole only groups are read whose maximum says that they hold one (NaN is
// in no maximum).
template <int kDt, int kGs, bool kTies, bool kWhole>
__device__ void lp_walk(const LpArgs& a, const Blocks<kDt>& bl, int b0, int b1, uint32_t bound, LpShared& sh) {
  constexpr int E = Blocks<kDt>::E;
  constexpr int kStep = kLpThreads / E;   // blocks a round
  constexpr int kShift = 32 - kOrderBits<kDt>;
  uint64_t low = 0;                       // the k-th best so far
  int n = kTies ? sh.count : 0;
  __syncthreads();
  if (threadIdx.x == 0) sh.count = n;
  __syncthreads();
  for (int b = b0; b < b1; b += kStep) {
    if constexpr (!kWhole) {
      bool any = false;
      for (int g = (b - b0) / kGs; !any && g * kGs < b + kStep - b0 && g * kGs < b1 - b0; ++g) {
        const int first = max(bl.element(b0 + g * kGs, 0), 0);
        any = order_of(sh.gmax[g]) >> kShift >= bound && key_of(sh.gmax[g], first) > low;
      }
      if (!any) continue;
    }
    const int blk = b + threadIdx.x / E, e = threadIdx.x % E;
    const int j = bl.element(blk, e);
    uint64_t key = 0;
    if (blk < b1 && j >= 0 && j < a.vocab) key = key_of(load_el<kDt>(bl.p0, (int64_t)blk * E + e), j);
    const bool take = kTies ? key != 0 && (uint32_t)(key >> 32) >> kShift == bound : key > low;
    if (take) sh.keys[atomicAdd(&sh.count, 1)] = key;
    __syncthreads();
    n = sh.count;
    __syncthreads();
    if constexpr (kTies) {
      if (n >= a.k) break;
    } else if (n > kLpKeys - kLpThreads) {
      sort_top(sh, n, a.k);
      if (threadIdx.x == 0) sh.count = a.k;
      low = sh.keys[a.k - 1];
      __syncthreads();
    }
  }
}

// One workgroup per part of a row: sums, then the part's best.  Seven
// workgroups fit a CU's LDS; rows of fp32 are held to the registers for that
// (1500 rows of 50021, k = 1: 72 -> 67 us).
template <int kDt, bool kTop, int kGs, bool kSplit>
__global__ __launch_bounds__(kLpThreads, kDt == GPTQ_F32 && !kSplit ? 7 : 1) void logprobs_kernel(LpArgs a) {
  __shared__ LpShared sh;
  constexpr int E = Blocks<kDt>::E;
  constexpr int kU = 4;                   // blocks in flight per lane
  constexpr int kShift = 32 - kOrderBits<kDt>;
  const int tid = threadIdx.x;
  const int64_t row = kSplit ? blockIdx.x / a.parts : blockIdx.x;
  const int part = kSplit ? blockIdx.x % a.parts : 0;
  const Blocks<kDt> bl(a.x, row, a.ld, a.vocab);
  const int b0 = part * a.blocks;
  const int b1 = min(b0 + a.blocks, bl.n);
  bool scored = false;
  float x_target = 0.f;
  if (!kSplit && tid == 0 && a.logprob) {
    const int t = a.targets[row];
    scored = t >= 0 && t < a.vocab;
    if (scored) x_target = load_el<kDt>(bl.p0, (int64_t)bl.h + t);
  }

  Sums sum{kLpFloor, 0.f, 0.f};
  float rc = kLpFloor * a.c;              // the reference as the fast pass subtracts it
  float m = -INFINITY;
  auto add_block = [&](const float (&v)[E], int b) {
    float vm = fmaxf(v[0], v[1]);
#pragma unroll
    for (int e = 2; e < E; ++e) vm = fmaxf(vm, v[e]);
    m = fmaxf(m, vm);
    if constexpr (kTop) {
      if constexpr (kGs == 1) {
        sh.gmax[b - b0] = vm;
      } else {
        // 16 lanes hold 16 blocks in a row
        const float g = row_reduce(vm, [](float p, float q) { return fmaxf(p, q); });
        if ((tid & (kGs - 1)) == 0) sh.gmax[(b - b0) / kGs] = g;
      }
    }
    if (fmaf(vm, a.c, -rc) > kLpLag) {
      // S and U stand at rc, not at r c: both roundings go into the move
      const float skew = fmaf(vm, a.c, -(vm * a.c)) - fmaf(sum.r, a.c, -rc);
      sum = moved(sum, vm, a.c);
      rc = vm * a.c;
      const float f = exp2_hw(skew);
      sum.u = f * fmaf(skew, sum.s, sum.u);
      sum.s *= f;
    }
    // a block's terms are added among themselves first: a lane then rounds once
    // per block, not once per logit, at the size of the running sums
    float s0 = 0.f, s1 = 0.f, u0 = 0.f, u1 = 0.f;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float d0 = fmaf(v[e], a.c, -rc), d1 = fmaf(v[e + 1], a.c, -rc);
      const float p0 = exp2_hw(d0), p1 = exp2_hw(d1);
      s0 += p0;
      s1 += p1;
      u0 = fmaf(p0, fmaxf(d0, -200.f), u0);   // 0 times the distance of a masked logit is 0
      u1 = fmaf(p1, fmaxf(d1, -200.f), u1);
    }
    sum.s += s0 + s1;
    sum.u += u0 + u1;
  };
  {
    int b = b0;
    const int w0 = max(b0, bl.first_whole()), w1 = min(b1, bl.end_whole());
    while (b < b1) {
      if (b >= w0 && b + kU * kLpThreads <= w1) {
        u32x4 w[kU];
#pragma unroll
        for (int i = 0; i < kU; ++i) w[i] = bl.load(b + i * kLpThreads + tid);
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          float v[E];
          Blocks<kDt>::unpack(w[i], v);
          add_block(v, b + i * kLpThreads + tid);
        }
        b += kU * kLpThreads;
      } else {
        // the row's ends; lanes past the part's end hold -inf and their group
        // maxima fall into the last group or beyond the ones looked at
        float v[E];
        const int at = b + tid;
        if (at < b1) bl.fetch(at, v);
        else
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = -INFINITY;
        if (kGs > 1 || at < b1) add_block(v, at);
        b += kLpThreads;
      }
    }
  }
  {
    const float skew = -fmaf(sum.r, a.c, -rc);
    const float f = exp2_hw(skew);
    sum.u = f * fmaf(skew, sum.s, sum.u);
    sum.s *= f;
  }
  const bool has = b0 + tid < b1;
  const float m_lane = m;
  lp_join(sum, m, a.c, sh);
  const bool fast_nan = !(sum.s == sum.s);
  if (!(sum.s > 0.f && sum.s < INFINITY && sum.u == sum.u && fabsf(sum.r) * a.c < kLpFast)) {
    // nothing reached the lowest reference, or something is out of range or no
    // number: once more around the true maximum, with the difference taken
    // before it is scaled
    if (m == -INFINITY) {
      sum = Sums{-3.4028235e38f, fast_nan ? NAN : 0.f, 0.f};
    } else if (m == INFINITY) {
      sum = Sums{0.f, NAN, 0.f};
    } else {
      sum = Sums{m, 0.f, 0.f};
      for (int b = b0 + tid; b < b1; b += kLpThreads) {
        float v[E];
        bl.fetch(b, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float d = (v[e] - m) * a.c;
          const float p = exp2_hw(d);
          sum.s += p;
          sum.u = fmaf(p, fmaxf(d, -200.f), sum.u);
        }
      }
      float unused = 0.f;
      lp_join(sum, unused, a.c, sh);
    }
  }
  const LpOut out(sum, a.inv_t);
  if constexpr (kSplit) {
    if (tid == 0) {
      float* w = a.ws_sums + (row * a.parts + part) * 4;
      w[0] = sum.r;
      w[1] = sum.s;
      w[2] = sum.u;
    }
  } else if (tid == 0) {
    lp_write_row(a, row, out, x_target, scored);
  }
  if constexpr (kTop) {
    const bool broken = !(sum.s == sum.s);
    sh.lane_order[tid] = has ? order_of(m_lane) >> kShift : 0u;
    __syncthreads();
    const uint32_t bound = kth_largest<kOrderBits<kDt>>(sh.lane_order, a.k);
    if (broken) {
      lp_walk<kDt, kGs, false, true>(a, bl, b0, b1, bound, sh);
    } else {
      // a bound that is the type's lowest value or -inf means a masked part
      // where next to everything ties: not worth a collection
      const float lowest = kDt == GPTQ_F16 ? -65504.f : kDt == GPTQ_BF16 ? -3.3895314e38f : -3.4028235e38f;
      const bool masked = bound != 0 && bound <= order_of(lowest) >> kShift;
      if (!masked) lp_collect<kDt, kGs, false>(a, bl, b0, b1, bound, sh);
      if (masked || sh.count > kLpKeys) {
        // ties at the bound: what is above it, then the first of the ties
        lp_collect<kDt, kGs, true>(a, bl, b0, b1, bound, sh);
        if (sh.count < a.k) lp_walk<kDt, kGs, true, false>(a, bl, b0, b1, bound, sh);
        else if (sh.count > kLpKeys) lp_walk<kDt, kGs, false, false>(a, bl, b0, b1, bound, sh);
      }
    }
    __syncthreads();
    const int n = sh.count;
    for (int at = tid; at < n; at += kLpThreads) {
      const uint64_t key = sh.keys[at];
      const int r = rank_of(key, sh.keys, n);
      if (r >= a.k) continue;
      if constexpr (kSplit) {
        a.ws_keys[(row * a.parts + part) * a.k + r] = key;
      } else {
        a.top_lp[row * a.k + r] = out.logprob(value_of((uint32_t)(key >> 32)));
        a.top_id[row * a.k + r] = (int32_t)index_of(key);
      }
    }
    if constexpr (kSplit)
      for (int r = n + tid; r < a.k; r += kLpThreads) a.ws_keys[(row * a.parts + part) * a.k + r] = 0;
  }
}

// Joins the parts of a row: their sums, and the best of their best.
template <int kDt>
__global__ __launch_bounds__(kLpThreads) void logprobs_join_kernel(LpArgs a) {
  __shared__ LpShared sh;
  constexpr int kShift = 32 - kOrderBits<kDt>;
  constexpr int kMine = 16;               // keys a thread holds: parts * k <= 4096
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const uint64_t* src = a.ws_keys + row * a.parts * a.k;
  const int total = a.parts * a.k;
  uint64_t key[kMine];
  uint64_t best = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int at = tid + i * kLpThreads;
    key[i] = at < total ? src[at] : 0;
    best = key[i] > best ? key[i] : best;
  }
  bool scored = false;
  float x_target = 0.f;
  if (tid == 0 && a.logprob) {
    const int t = a.targets[row];
    scored = t >= 0 && t < a.vocab;
    if (scored) x_target = load_el<kDt>(a.x, row * a.ld + t);
  }
  Sums sum{-3.4028235e38f, 0.f, 0.f};
  if (tid < a.parts) {
    const float* w = a.ws_sums + (row * a.parts + tid) * 4;
    sum = Sums{w[0], w[1], w[2]};
  }
  float unused = 0.f;
  lp_join(sum, unused, a.c, sh);
  const LpOut out(sum, a.inv_t);
  if (tid == 0) lp_write_row(a, row, out, x_target, scored);
  if (a.k == 0) return;
  sh.lane_order[tid] = (uint32_t)(best >> 32) >> kShift;
  if (tid == 0) sh.count = sh.flagged = 0;
  __syncthreads();
  const uint32_t bound = kth_largest<kOrderBits<kDt>>(sh.lane_order, a.k);
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (key[i] != 0 && (uint32_t)(key[i] >> 32) >> kShift >= bound) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kLpThreads) sh.keys[at] = key[i];
    }
  __syncthreads();
  const int n = sh.count;
  if (n <= kLpThreads) {
    if (tid < n) {
      const uint64_t q = sh.keys[tid];
      const int r = rank_of(q, sh.keys, n);
      if (r < a.k) {
        a.top_lp[row * a.k + r] = out.logprob(value_of((uint32_t)(q >> 32)));
        a.top_id[row * a.k + r] = (int32_t)index_of(q);
      }
    }
  } else {
    // many ties at the bound (masked parts hold only such): the k-th largest
    // key (they differ) itself, its bits from the top: the value's, then those
    // of 0xFFFFFFFF - index that an index below 2^21 can clear; only the k keys
    // that reach it are ranked
    uint64_t kth = 0;
    int turn = 0;
    auto settle = [&](int bit, uint64_t fixed) {
      const uint64_t cand = kth | fixed | 1ull << bit;
      int c = 0;
#pragma unroll
      for (int i = 0; i < kMine; ++i) c += __popcll(__ballot(key[i] >= cand));
      if ((tid & 63) == 0) sh.list[(turn & 1) * 4 + (tid >> 6)] = (uint16_t)c;
      __syncthreads();
      const uint16_t* got = sh.list + (turn & 1) * 4;
      if (got[0] + got[1] + got[2] + got[3] >= a.k) kth = cand;
      ++turn;
    };
    for (int b = 63; b >= 32 + kShift; --b) settle(b, 0);
    // a 16-bit value's order ends in zeros, a negative one's or a NaN's in ones
    const uint32_t top = (uint32_t)(kth >> 32) >> kShift;
    const bool ones = top >> (31 - kShift) == 0 || top == 0xFFFFFFFFu >> kShift;
    const uint64_t fixed = 0xFFE00000ull | (ones ? ((1ull << kShift) - 1) << 32 : 0ull);
    for (int b = 20; b >= 0; --b) settle(b, fixed);
    kth |= fixed;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (key[i] == 0 || key[i] < kth) continue;
      sh.keys[atomicAdd(&sh.flagged, 1)] = key[i];
    }
    __syncthreads();
    if (tid < a.k) {
      const uint64_t q = sh.keys[tid];
      const int r = rank_of(q, sh.keys, a.k);
      a.top_lp[row * a.k + r] = out.logprob(value_of((uint32_t)(q >> 32)));
      a.top_id[row * a.k + r] = (int32_t)index_of(q);
    }
  }
}

struct LpPlan {
  int parts, blocks;
  size_t off_keys, total;
};

// Parts of a row: one workgroup per row when that gives every CU one, else
// enough parts for four, of at least two blocks a lane.  The join is a second
// launch and a part ends in a search of its own, which only long rows pay for.
// Whole / in parts, us, k = 5, blocks of 16 bytes in a row (calls on a few inputs
// in turn, recorded in a graph; 1000 rows of 50021 fp32 take 46 us there):
//   up to 48 rows: 1 row of 2000 blocks 8.4 / 11.3, 4000 10.1 / 11.3, 6250 12.4 /
//     11.4, 16384 22 / 11.5; 48 rows of 4000 11.6 / 12.7, 6250 15.6 / 14.2
//   100 rows of 12500, k = 1, 21.0 / 17.6; 128 rows of 8192 16.8 / 16.2 (masked 18.8 /
//     22.8), 16384 fp32 22.8 / 19.9; 200 of 8192 17.1 / 18.9, 12500 21.2 / 22.9, 16384
//     fp32 26.7 / 25.0; 240 of 16384 31.0 / 27.1 (k = 10)
//   512 rows of 16384, k = 20, 40.3 / 43.3; 1000 of 12500, k = 1, 46.3 / 56.7
static LpPlan lp_plan(int64_t n_rows, int64_t vocab, int64_t k, int es) {
  const int64_t blocks = cdiv(vocab * es, 16) + 1;   // a row that starts inside a block has one more
  int64_t parts = 1;
  if (n_rows < 256 && blocks > std::min<int64_t>(std::max<int64_t>(4096, 80 * n_rows), 12800))
    parts = std::min<int64_t>(cdiv(1024, std::max<int64_t>(n_rows, 1)), blocks / 512);
  parts = std::min<int64_t>(parts, std::min<int64_t>(64, 4096 / std::max<int64_t>(k, 1)));
  parts = std::max<int64_t>(parts, std::max<int64_t>(cdiv(blocks, kLpMaxBlocks), 1));
  LpPlan p;
  p.blocks = (int)(cdiv(cdiv(blocks, parts), 64) * 64);
  p.parts = (int)cdiv(blocks, p.blocks);
  p.off_keys = align_up((size_t)n_rows * p.parts * 16, 256);
  p.total = p.parts > 1 ? p.off_keys + (size_t)n_rows * p.parts * std::max<int64_t>(k, 1) * 8 : 0;
  return p;
}

size_t logprobs_workspace_bytes(int64_t n_rows, int64_t vocab, int64_t k) {
  return std::max(lp_plan(n_rows, vocab, k, 2).total, lp_plan(n_rows, vocab, k, 4).total);
}

template <int kDt, bool kTop, int kGs>
static void lp_launch(const LpArgs& a, int64_t n_rows, hipStream_t st) {
  if (a.parts == 1) {
    hipLaunchKernelGGL((logprobs_kernel<kDt, kTop, kGs, false>), dim3((unsigned)n_rows), dim3(kLpThreads), 0, st, a);
  } else {
    hipLaunchKernelGGL((logprobs_kernel<kDt, kTop, kGs, true>), dim3((unsigned)(n_rows * a.parts)), dim3(kLpThreads), 0,
                       st, a);
    hipLaunchKernelGGL(logprobs_join_kernel<kDt>, dim3((unsigned)n_rows), dim3(kLpThreads), 0, st, a);
  }
}

template <int kDt>
static void lp_dispatch(const LpArgs& a, int64_t n_rows, hipStream_t st) {
  if (a.k == 0) lp_launch<kDt, false, 1>(a, n_rows, st);
  else if (a.blocks <= kLpGroups) lp_launch<kDt, true, 1>(a, n_rows, st);
  else lp_launch<kDt, true, kLpGroupBlocks>(a, n_rows, st);
}

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_token_logprobs(const void* logits, int32_t x_dtype, int64_t n_rows, int64_t vocab,
                                           int64_t ld_x, const int32_t* targets, float temperature, int32_t k,
                                           float* logprob, float* lse, float* entropy, float* top_logprob,
                                           int32_t* top_id, void* workspace, size_t ws_bytes, void* stream) {
  GQ_CHECK_ARG(x_dtype == GPTQ_F32 || x_dtype == GPTQ_F16 || x_dtype == GPTQ_BF16);
  // a launch holds fewer than 2^32 threads
  GQ_CHECK_ARG(n_rows >= 0 && n_rows < ((int64_t)1 << 32) / kLpThreads && vocab >= 1 && vocab <= ((int64_t)1 << 30));
  GQ_CHECK_ARG(ld_x >= vocab && ld_x <= ((int64_t)1 << 36));
  GQ_CHECK_ARG(temperature >= 1e-4f && temperature <= 1e4f);
  GQ_CHECK_ARG(k >= 0 && k <= vocab);
  if (k > 128 || vocab > ((int64_t)1 << 21)) return GPTQ_EUNSUPPORTED;
  if (n_rows == 0) return GPTQ_OK;
  GQ_CHECK_ARG(logprob == nullptr || targets != nullptr);
  GQ_CHECK_ARG(k == 0 || (top_logprob && top_id));
  GQ_CHECK_ARG(logprob || lse || entropy || k > 0);
  const int es = x_dtype == GPTQ_F32 ? 4 : 2;
  GQ_CHECK_ARG(logits != nullptr && reinterpret_cast<uintptr_t>(logits) % es == 0);
  const size_t need = logprobs_workspace_bytes(n_rows, vocab, k);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GPTQ_ENOMEM;
  const LpPlan pl = lp_plan(n_rows, vocab, k, es);
  GQ_CHECK_ARG(pl.parts == 1 || reinterpret_cast<uintptr_t>(workspace) % 256 == 0);
  LpArgs a{};
  a.x = logits;
  a.ld = ld_x;
  a.targets = targets;
  a.c = (float)(1.4426950408889634074 / temperature);
  a.inv_t = (float)(1.0 / temperature);
  a.vocab = (int)vocab;
  a.k = k;
  a.parts = pl.parts;
  a.blocks = pl.blocks;
  a.logprob = logprob;
  a.lse = lse;
  a.entropy = entropy;
  a.top_lp = top_logprob;
  a.top_id = top_id;
  a.ws_sums = static_cast<float*>(workspace);
  a.ws_keys = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + pl.off_keys);
  hipStream_t st = static_cast<hipStream_t>(stream);
  TimedScope ts(kTimeLogprobs, st);
  if (x_dtype == GPTQ_F32) lp_dispatch<GPTQ_F32>(a, n_rows, st);
  else if (x_dtype == GPTQ_F16) lp_dispatch<GPTQ_F16>(a, n_rows, st);
  else lp_dispatch<GPTQ_BF16>(a, n_rows, st);
  GQ_LAUNCHED();
  return GPTQ_OK;
}
