// Distillation from a teacher's top logits: loss and gradient of rows.
//
// The listed tokens K and the rest of the vocabulary are kept apart.  For the
// rest one pass keeps a reference r and s = sum 2^((x - r) c), c = log2(e) / T;
// the listed ones (at most 128) give their own maximum and sum.  Joined, with
// m the larger reference and S = s 2^((r - m) c) + s_K 2^((m_K - m) c):
//   log q_k = (x_k - m) / T - ln S,   log q_r = (r - m) / T + ln s - ln S,
// so the student's mass in the tail is never the difference of nearly equal
// sums (the teacher's is 1 less its list's: below the rounding of the listed
// log probabilities it counts as far as the student's reaches), and
//   gradient in the rest = w / T 2^((x - r) c) (2^((r - m) c) / S - p_r / s)
//   gradient in K        = w / T (2^((x - m) c) / S - p_k).
//
// Row kernel: one workgroup holds a whole row in registers (16-byte blocks as
// loaded), so a logit is read once and its gradient written once: the same
// traffic as a copy.  Workgroups stay and take row after row; a block's
// registers are refilled with the next row's as soon as its gradient is
// stored, so the loads of one row run under the stores of the one before.
// Part kernels: few rows are split over workgroups (and rows too long for the
// registers of one): sums per part, then each part joins them and writes its
// own gradients.
//
// Listed tokens are kept out of the rest by one bit per held logit, which the
// list's entries set in LDS for the lanes that own them.  Their gradients are
// made by the entries and stored over the rest's once those are known to be
// written: a row later, after a wait that the row kernel makes anyway.
//
// Bound by memory: 4096 rows of 131072 bf16, k = 64, take 465 us with gradient,
// 4.6 TB/s read and written; 2048 rows of 32000 bf16, loss alone, 34.5 us, 3.8
// TB/s, where the workgroups' sums between two rows show; 777 odd rows of
// 50021 fp16 48 us, 3.2 TB/s: 512 workgroups, of which half take a second row.
#include "rows.h"

namespace gq {

constexpr int kDsMaxK = 128;

struct DsArgs {
  const void* x;
  int64_t ld;
  const int32_t* id;
  const float* lp;
  const float* weight;
  float* loss;
  void* grad;
  int64_t ld_g, n_rows;
  float c, inv_t;
  double inv_td;           // 1 / T
  int vocab, k, tail;
  int parts, slots;        // part kernels: parts of a row, blocks a lane holds of one
  float* ws_sums;          // [rows][parts][2]: r, s
  float* ws_list;          // [rows][8]: the listed tokens' sums
};

// What the listed tokens of a row give.
struct DsList {
  float m, s;              // maximum of x, sum of 2^((x - m) c)
  float mass, norm;        // sum of p before (tail) / 1 after normalization; p = e^(l - norm)
  float left;              // 1 - sum p (0 without a tail); negative: it may be nothing but the rounding of the l
  double gap;              // sum p (log p - (x - m) / T)
  float count;
};

// What the gradient of a row is made of.
struct DsFinal {
  float m, inv_s;          // listed: w (2^((x - m) c) inv_s - p)
  float r, rest;           // rest: rest * 2^((x - r) c)
  float w, norm;
  float total, tail_q, pr; // S, q_r (0 also where it is below 2^-126) and p_r, for the loss
  int zero, nan, bad;
};

// LDS of a workgroup of T threads with W words of bits per lane.
template <int T, int W>
struct DsShared {
  __align__(16) int id[kDsMaxK];   // -1: absent
  float lp[kDsMaxK];       // -inf: absent, or not the id's first place
  float x[kDsMaxK];
  uint32_t listed[W][T];   // a bit per held logit
  uint32_t edge[16];       // the single logits' bits
  float red[T / 64][2];
  DsFinal fin;
};

// A thread's list entry of a row as read from memory.  Its logit stays as
// loaded: looking at it would wait for it, and for everything loaded before.
struct DsEntry {
  int id;
  float lp;
  uint32_t x;
};

template <int kDt, int T, int NB>
struct DsRow {
  static constexpr int E = Span<kDt>::E;
  static constexpr int kMaskWords = (NB * E + 31) / 32;
  using Shared = DsShared<T, kMaskWords>;
  Shared& sh;
  const DsArgs& a;
  uint32_t mask[kMaskWords];   // held logits that are not the rest's: listed, or behind the row's end
  bool edge_listed;

  __device__ __forceinline__ DsRow(Shared& s, const DsArgs& args) : sh(s), a(args) {}

  __device__ __forceinline__ void clear_bits() const {
#pragma unroll
    for (int i = 0; i < kMaskWords; ++i) sh.listed[i][threadIdx.x] = 0;
    if (threadIdx.x < 16) sh.edge[threadIdx.x] = 0;
  }

  // Thread and slot that hold token j of a row; slot -1: the lane's single logit.
  static __device__ __forceinline__ void owner(const Span<kDt>& sp, int j, int& thread, int& slot, int& e) {
    if (j < sp.head) {
      thread = j;
      slot = -1;
      e = 0;
    } else if (j >= sp.head + sp.blocks * E) {
      thread = 8 + j - sp.head - sp.blocks * E;
      slot = -1;
      e = 0;
    } else {
      const int b = (j - sp.head) / E;
      thread = b % T;
      slot = b / T;
      e = (j - sp.head) % E;
    }
  }

  // Every lane reads (lanes without an entry the last one's), so that the
  // compiler can count these loads, too.
  __device__ __forceinline__ DsEntry read_entry(int64_t row) const {
    const int64_t at = row * a.k + min((int)threadIdx.x, a.k - 1);
    return DsEntry{a.id[at], a.lp[at], 0};
  }
  __device__ __forceinline__ bool present(const DsEntry& n) const {
    return (int)threadIdx.x < a.k && n.id >= 0 && n.id < a.vocab && n.lp != -INFINITY;
  }
  __device__ __forceinline__ void read_logit(DsEntry& n, const Span<kDt>& sp) const {
    n.x = load_bits<kDt>(sp.p, min(max(n.id, 0), a.vocab - 1));
  }
  __device__ __forceinline__ uint32_t read_edge(const Span<kDt>& sp) const {
    return load_bits<kDt>(sp.p, max(sp.edge(threadIdx.x), 0));
  }

  // The entries' logits into LDS.
  __device__ __forceinline__ void put_logits(const DsEntry& n) const {
    if (present(n)) sh.x[threadIdx.x] = bits_value<kDt>(n.x);
  }

  // The row's list (without its logits) into LDS and this lane's bits out of it.
  // Slots [slot0, slot0 + slots) are the held ones; `edges`: the single logits,
  // too.  The bits in LDS are clear before, and stay until clear_bits().  One
  // barrier; absent and repeated entries are marked only after another one.
  __device__ __forceinline__ void take_list(const Span<kDt>& sp, const DsEntry& n, int slot0, int slots, bool edges) {
    const int t = threadIdx.x;
    if (t < a.k) {
      const bool there = present(n);
      sh.id[t] = there ? n.id : -1;
      sh.lp[t] = n.lp;
      int thread, slot, e;
      owner(sp, n.id, thread, slot, e);
      if (there && slot < 0) {
        if (edges) sh.edge[thread] = 1;
      } else if (there && slot >= slot0 && slot < slot0 + slots) {
        const int bit = (slot - slot0) * E + e;
        atomicOr(&sh.listed[bit / 32][thread], 1u << (bit % 32));
      }
    }
    lds_barrier();
    read_bits(sp, slot0, slots);
    edge_listed = t < 16 && sh.edge[t & 15] != 0;
    // an id counts at its first place: every entry against a share of the
    // entries before it
    const int i = t % kDsMaxK, share = t / kDsMaxK;
    if (i < a.k) {
      const int id = sh.id[i];
      constexpr int kPer = kDsMaxK / (T / kDsMaxK);
      bool again = false;
      const int end = min((share + 1) * kPer, i);
      for (int o = share * kPer; o < end; o += 4) {
        const int4 v = *reinterpret_cast<const int4*>(sh.id + o);
        again = again || (v.x == id) || (v.y == id && o + 1 < i) || (v.z == id && o + 2 < i) || (v.w == id && o + 3 < i);
      }
      if (again) sh.lp[i] = -INFINITY;
    }
  }

  // The bits of listed logits, of blocks behind the span's end and of slots not held.
  __device__ __forceinline__ void read_bits(const Span<kDt>& sp, int slot0, int slots) {
    // this lane's first slot without a block, as a bit number
    const int end = sp.blocks - slot0 * T - (int)threadIdx.x;
    const int bits = min(max(end + T - 1, 0) / T, slots) * E;
#pragma unroll
    for (int i = 0; i < kMaskWords; ++i)
      mask[i] = sh.listed[i][threadIdx.x] |
                (bits <= 32 * i ? ~0u : bits >= 32 * i + 32 ? 0u : ~0u << (bits - 32 * i));
  }

  // Listed bits of held block i (i known to the compiler, or any).
  __device__ __forceinline__ uint32_t bits(int i) const {
    return mask[i * E / 32] >> (i * E % 32) & ((1u << E) - 1u);
  }
  __device__ __forceinline__ uint32_t bits_any(int i) const {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) m = w == i * E / 32 ? mask[w] : m;
    return m >> (i * E % 32) & ((1u << E) - 1u);
  }

  // The listed tokens' sums, by one wave.
  __device__ __forceinline__ DsList list_sums() const {
    auto fmax2 = [](float p, float q) { return fmaxf(p, q); };
    auto add2 = [](float p, float q) { return p + q; };
    const int lane = threadIdx.x & 63;
    float l[2], x[2], p[2];
    bool has[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = lane + 64 * i;
      has[i] = at < a.k && sh.id[at < a.k ? at : 0] >= 0;
      l[i] = has[i] ? sh.lp[at] : -INFINITY;
      has[i] = has[i] && l[i] != -INFINITY;
      x[i] = has[i] ? sh.x[at] : -INFINITY;
    }
    DsList d;
    d.count = (float)(__popcll(__ballot(has[0])) + __popcll(__ballot(has[1])));
    d.m = wave_reduce(fmaxf(x[0], x[1]), fmax2);
    const float lm = a.tail ? 0.f : wave_reduce(fmaxf(l[0], l[1]), fmax2);
#pragma unroll
    for (int i = 0; i < 2; ++i) p[i] = has[i] ? exp2_hw((l[i] - lm) * kLog2e) : 0.f;
    // in 64 bits: what is left of 1 may be as small as the rounding of the l
    const double sum = wave_reduce((double)p[0] + (double)p[1], [](double q, double w) { return q + w; });
    d.mass = (float)sum;
    d.norm = 0.f;
    d.left = 0.f;
    if (a.tail) {
      // The l of a complete list share the rounding of a log-sum below 16 (a few
      // steps of 2^-21, up to 2^-19) and carry a few of their own, 2^-24 |l| each.
      const float size = wave_reduce((p[0] > 0.f ? p[0] * fabsf(l[0]) : 0.f) + (p[1] > 0.f ? p[1] * fabsf(l[1]) : 0.f), add2);
      const float left = (float)fmax(1.0 - sum, 0.0);
      d.left = left > 0x1p-19f + 0x1p-22f * size ? left : -left;
    } else {
      d.norm = lm + logf(d.mass);
      p[0] /= d.mass;
      p[1] /= d.mass;
      d.mass = 1.f;
    }
    float s = 0.f;
    double gap = 0.0;   // the loss is what is left of sums larger than it: 64 bits for these few
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float far = x[i] == -INFINITY ? -INFINITY : x[i] - d.m;
      if (has[i]) s += exp2_hw(far * a.c);
      if (p[i] > 0.f) gap += (double)p[i] * ((double)l[i] - d.norm - (double)far * a.inv_td);
    }
    d.s = wave_reduce(s, add2);
    d.gap = wave_reduce(gap, [](double q, double w) { return q + w; });
    return d;
  }
};

// loss of a row: sum p (log p - log q) over the list, p_r (log p_r - log q_r).
__device__ __forceinline__ float ds_loss(const DsArgs& a, const DsList& l, const DsFinal& f, float r, float s) {
  if (l.count == 0.f) return 0.f;
  if (f.bad) return NAN;
  const double log_s = ln_wide(f.total);
  double loss = l.gap;
  if (l.mass > 0.f) loss -= (double)l.mass * ((double)(l.m - f.m) * a.inv_td - log_s);
  if (f.pr > 0.f) {
    if (!(s > 0.f)) return INFINITY;
    const double lq = f.tail_q > 0.f ? ln_wide(f.tail_q) : (double)(r - f.m) * a.inv_td + ln_wide(s) - log_s;
    loss += (double)f.pr * (ln_wide(f.pr) - lq);
  }
  return (float)loss;
}

__device__ __forceinline__ DsFinal ds_final(const DsArgs& a, float weight, const DsList& l, float r, float s) {
  DsFinal f;
  f.m = fmaxf(l.m, s > 0.f ? r : -INFINITY);
  const float up = s > 0.f ? exp2_hw((r - f.m) * a.c) : 0.f;
  const float total = (l.s > 0.f || l.s != l.s ? l.s * exp2_hw((l.m - f.m) * a.c) : 0.f) + (s != s ? s : s * up);
  const bool bad = !(total > 0.f && total < INFINITY);
  f.total = total;
  f.tail_q = s * up / total;
  // Rounding is no mass that the student lacks: it counts only where the
  // student's tail is as large.  p_r log(p_r / q_r) is 0 where that ends.
  const float pr = l.left >= 0.f || f.tail_q >= -l.left ? fabsf(l.left) : 0.f;
  f.pr = pr;
  f.bad = bad;
  f.w = weight * a.inv_t;
  f.zero = f.w == 0.f || l.count == 0.f;
  f.nan = bad && !f.zero;
  f.inv_s = 1.f / total;
  f.r = r;
  f.norm = l.norm;
  f.rest = s > 0.f && !f.zero ? f.w * (up * f.inv_s - pr / s) : 0.f;
  return f;
}

// What every wave needs of it, from LDS into scalar registers.
__device__ __forceinline__ DsFinal ds_fetch(const DsFinal& g, float r) {
  DsFinal f;
  f.m = uniform(g.m);
  f.inv_s = uniform(g.inv_s);
  f.rest = uniform(g.rest);
  f.w = uniform(g.w);
  f.norm = uniform(g.norm);
  f.zero = __builtin_amdgcn_readfirstlane(g.zero);
  f.nan = __builtin_amdgcn_readfirstlane(g.nan);
  f.r = r;
  return f;
}

// r, s of the rest among the workgroup's blocks, the slow way: around the true
// maximum, differences taken before they are scaled.  Reads the row again, so
// that the common way needs no registers for this.
template <int kDt, int T, int NB>
__device__ __forceinline__ void ds_exact_sums(DsRow<kDt, T, NB>& d, const Span<kDt>& sp, int slot0, int slots, float xe,
                                              float& r, float& s, typename DsRow<kDt, T, NB>::Shared& sh) {
  constexpr int E = Span<kDt>::E;
  const bool nan = s != s;
  d.read_bits(sp, slot0, slots);
  auto get = [&](int i, float (&v)[E]) {
    const int first = (slot0 + i) * T, t = threadIdx.x;
    Blocks<kDt>::unpack(t < sp.blocks - first ? sp.load(first, t) : masked_block<kDt>(), v);
    hide<kDt>(v, d.bits_any(i));
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
  if ((threadIdx.x & 63) == 0) sh.red[threadIdx.x >> 6][0] = m;
  lds_barrier();
#pragma unroll
  for (int i = 0; i < T / 64; ++i) m = fmaxf(m, sh.red[i][0]);
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
    for (int e = 0; e < E; ++e) s += exp2_hw((v[e] - m) * d.a.c);
  }
  s += exp2_hw((xe - m) * d.a.c);
  ds_join<T>(r, s, d.a.c, sh.red);
}

// Gradients of n logits of the rest.  kFast: rc is r c rounded, `rest` made
// for that, and the row none of zeros or NaN.
template <bool kFast>
__device__ __forceinline__ void ds_gradient(const DsFinal& f, float rest, float rc, float c, const float* v, float* g,
                                            int n) {
#pragma unroll
  for (int e = 0; e < n; ++e) {
    g[e] = rest * exp2_hw(kFast ? fmaf(v[e], c, -rc) : (v[e] - f.r) * c);
    if (!kFast && (f.zero || f.nan)) g[e] = f.nan ? NAN : 0.f;
  }
}

// The gradient of a list's entry: id -1 where there is nothing to store.
struct DsFix {
  int id;
  float g;
};
template <int kDt, int T, int NB>
__device__ __forceinline__ DsFix ds_fix(const DsRow<kDt, T, NB>& d, const DsFinal& f) {
  DsFix x{-1, 0.f};
  const int t = threadIdx.x;
  if (t < d.a.k && !(f.zero || f.nan)) {
    const float l = d.sh.lp[t];
    if (l != -INFINITY) x.id = d.sh.id[t];
    x.g = f.w * (exp2_hw((d.sh.x[t] - f.m) * d.a.c) * f.inv_s - exp2_hw((l - f.norm) * kLog2e));
  }
  return x;
}
template <int kDt>
__device__ __forceinline__ void ds_store_fix(const DsArgs& a, int64_t row, const DsFix& x) {
  if (x.id >= 0) store_el<kDt>(a.grad, row * a.ld_g + x.id, x.g);
}

// Blocks a lane holds in registers; a row kernel's others lie in LDS, where
// direct loads put them.  2048 rows of 151936 bf16, k = 64, take 295 us with
// gradient, 4.2 TB/s, and 123 us without; with all 20 blocks in registers up to
// 47 of 128 registers were spilled, and it took 339 and 144.
constexpr int kDsHeld = 16;

// Row kernel: T threads hold a row of at most T NB blocks.
//
// What is read ahead is waited for only where nothing younger is in flight:
// the memory operations of a wave complete in order, so a wait for one is a
// wait for all before it, and the compiler counts none of the conditional ones
// after it.  So the next row's ids are looked at after this row's blocks are
// used up, its blocks and listed logits are asked for after that, and the
// listed logits are looked at after its blocks.
template <int kDt, int T, int NB, bool kGrad>
__global__ __launch_bounds__(T) __attribute__((amdgpu_waves_per_eu(4))) void distill_row_kernel(DsArgs a) {
  __shared__ typename DsRow<kDt, T, NB>::Shared sh;
  constexpr int E = Span<kDt>::E;
  const int t = threadIdx.x;
  int64_t row = blockIdx.x;
  if (row >= a.n_rows) return;
  DsRow<kDt, T, NB> d(sh, a);
  d.clear_bits();
  constexpr int kHeld = NB < kDsHeld ? NB : kDsHeld;
  __shared__ __align__(16) u32x4 tail[NB > kHeld ? NB - kHeld : 1][NB > kHeld ? T : 1];
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  u32x4 w[kHeld];
  // the next row's block into the place of block i, which nothing reads any more
  auto refill = [&](const DsSource<kDt>& src, int i) {
    if (i < kHeld) w[i < kHeld ? i : 0] = src.load(i * T);
    else lds_load16(src.block(i * T), reinterpret_cast<char*>(&tail[i - kHeld][wave * 64]));
  };
  // together, and after all of them were read: a direct load in flight is
  // waited for at the next reading
  auto refill_tail = [&](const DsSource<kDt>& src) {
    if constexpr (NB > kHeld) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int i = kHeld; i < NB; ++i) refill(src, i);
    }
  };
  Span<kDt> sp(a.x, row, a.ld, a.vocab);
  DsEntry n = d.read_entry(row);
  d.read_logit(n, sp);
  uint32_t edge_bits = d.read_edge(sp);
  {
    const DsSource<kDt> src(sp, true);
#pragma unroll
    for (int i = 0; i < NB; ++i) refill(src, i);
  }
  lds_barrier();
  DsFix fix{-1, 0.f};
  int64_t fix_row = row;
  for (;;) {
    const int64_t next_row = row + gridDim.x;
    const bool more = next_row < a.n_rows;
    const Span<kDt> next(a.x, more ? next_row : row, a.ld, a.vocab);
    const DsSource<kDt> src(next, more);
    d.take_list(sp, n, 0, NB, true);
    DsEntry ahead = d.read_entry(more ? next_row : row);
    const float* weights = a.weight ? a.weight + row : a.lp;
    float weight = *weights;
    float r = kDsFloor, rc = kDsFloor * a.c, s = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      float v[E];
      unpack_held<kDt>(w[i], v);
      hide<kDt>(v, d.bits(i));
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
        hide<kDt>(v, d.bits(i));
        ds_add_block<kDt>(r, rc, s, v, a.c);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!kGrad) refill_tail(src);
    }
    const float xe = sp.edge(t) >= 0 ? bits_value<kDt>(edge_bits) : -INFINITY;
    const float xr = d.edge_listed ? -INFINITY : xe;
    if (t < 64) {
      float v[E];
      v[0] = xr;
#pragma unroll
      for (int e = 1; e < E; ++e) v[e] = -INFINITY;
      ds_add_block<kDt>(r, rc, s, v, a.c);
    }
    s *= exp2_hw(-fmaf(r, a.c, -rc));
    d.put_logits(n);
    // the ids read ahead, and the last row's gradients in memory
    if constexpr (kGrad) memory_done();
    asm volatile("" : "+v"(ahead.id), "+v"(ahead.lp), "+v"(weight));
    d.read_logit(ahead, next);
    const uint32_t edge_ahead = d.read_edge(next);
    ds_join<T>(r, s, a.c, sh.red);
    if constexpr (kGrad) ds_store_fix<kDt>(a, fix_row, fix);
    // a rest of -inf alone, or out of the fast way's range
    const bool exact = !(s > 0.f && s < INFINITY && fabsf(r) * a.c < kDsFast);
    if (exact) ds_exact_sums<kDt, T, NB>(d, sp, 0, NB, xr, r, s, sh);
    if (t < 64) {
      const DsList l = d.list_sums();
      if (t == 0) {
        sh.fin = ds_final(a, a.weight ? weight : 1.f, l, r, s);
        if (a.loss) a.loss[row] = ds_loss(a, l, sh.fin, r, s);
      }
    }
    d.clear_bits();
    lds_barrier();
    if constexpr (kGrad) {
      const DsFinal f = ds_fetch(sh.fin, r);
      fix = ds_fix<kDt, T, NB>(d, f);
      fix_row = row;
      if (sp.edge(t) >= 0) {
        float g[1];
        ds_gradient<false>(f, f.rest, 0.f, a.c, &xe, g, 1);
        store_el<kDt>(static_cast<char*>(a.grad) + row * a.ld_g * Span<kDt>::kSize, sp.edge(t), g[0]);
      }
      if (f.zero || f.nan) {
        float g[E];
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] = f.nan ? NAN : 0.f;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          if (t < sp.blocks - i * T) ds_store<kDt>(a.grad, a.ld_g, sp, row, i * T, t, g);
          if (i < kHeld) refill(src, i);
        }
        refill_tail(src);
      } else if (!exact) {
        const float frc = r * a.c;
        const float rest = f.rest * exp2_hw(-fmaf(r, a.c, -frc));
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          float v[E], g[E];
          if (i < kHeld) unpack_held<kDt>(w[i < kHeld ? i : 0], v);
          else Blocks<kDt>::unpack(tail[i < kHeld ? 0 : i - kHeld][t], v);
          ds_gradient<true>(f, rest, frc, a.c, v, g, E);
          if (t < sp.blocks - i * T) ds_store<kDt>(a.grad, a.ld_g, sp, row, i * T, t, g);
          if (i < kHeld) refill(src, i);
          __builtin_amdgcn_sched_barrier(0);   // one block's registers at a time
        }
        refill_tail(src);
      } else {
#pragma unroll 1
        for (int i = 0; i < NB; ++i) {
          if (t >= sp.blocks - i * T) break;
          float v[E], g[E];
          Blocks<kDt>::unpack(sp.load(i * T, t), v);
          ds_gradient<false>(f, f.rest, 0.f, a.c, v, g, E);
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
    n = ahead;
    edge_bits = edge_ahead;
  }
  if constexpr (kGrad || NB > kHeld) memory_done();   // no direct load ends after the workgroup
  if constexpr (kGrad) {
    lds_barrier();
    ds_store_fix<kDt>(a, fix_row, fix);
  }
}

constexpr int kDsPartThreads = 256;
constexpr int kDsPartBlocks = 16;   // blocks a lane holds of a part, at most

// Part kernels.  kSums: r, s of a part's rest (and from part 0 the listed
// tokens' sums) into the workspace.  Otherwise: the parts joined, the loss
// (part 0), the part's gradients.
template <int kDt, int NB, bool kSums>
__global__ __launch_bounds__(kDsPartThreads) void distill_part_kernel(DsArgs a) {
  constexpr int T = kDsPartThreads;
  constexpr int E = Span<kDt>::E;
  __shared__ typename DsRow<kDt, T, NB>::Shared sh;
  const int t = threadIdx.x;
  const int per_row = kSums || a.grad ? a.parts : 1;
  const int64_t row = blockIdx.x / per_row;
  const int part = blockIdx.x % per_row;
  const Span<kDt> sp(a.x, row, a.ld, a.vocab);
  DsRow<kDt, T, NB> d(sh, a);
  d.clear_bits();
  u32x4 w[NB];
  const bool edges = part == 0;
  const int slot0 = part * a.slots;
  float xe = -INFINITY;
  if (kSums || a.grad) {
    const DsSource<kDt> src(sp, true);
#pragma unroll
    for (int i = 0; i < NB; ++i) w[i] = src.load((slot0 + min(i, a.slots - 1)) * T);
    if (edges && sp.edge(t) >= 0) xe = load_el<kDt>(sp.p, sp.edge(t));
  }
  DsEntry n = d.read_entry(row);
  bool own = part == 0;
  if (!kSums && d.present(n)) {
    // only what this part holds: in place, other parts are being overwritten
    int thread, slot, e;
    DsRow<kDt, T, NB>::owner(sp, n.id, thread, slot, e);
    own = slot < 0 ? edges : slot >= slot0 && slot < slot0 + a.slots;
  }
  if (own) d.read_logit(n, sp);
  lds_barrier();
  d.take_list(sp, n, slot0, a.slots, edges);
  d.put_logits(n);
  lds_barrier();
  if constexpr (kSums) {
    if (part == 0 && t < 64) {
      const DsList l = d.list_sums();
      if (t == 0) {
        float* o = a.ws_list + row * 8;
        o[0] = l.m;
        o[1] = l.s;
        o[2] = l.mass;
        o[3] = l.norm;
        o[4] = l.count;
        o[5] = l.left;
        *reinterpret_cast<double*>(o + 6) = l.gap;
      }
    }
    float r = kDsFloor, rc = kDsFloor * a.c, s = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      float v[E];
      unpack_held<kDt>(w[i], v);
      hide<kDt>(v, d.bits(i));
      ds_add_block<kDt>(r, rc, s, v, a.c);
      __builtin_amdgcn_sched_barrier(0);
    }
    const float xr = d.edge_listed ? -INFINITY : xe;
    if (edges && t < 64) {
      float v[E];
      v[0] = xr;
#pragma unroll
      for (int e = 1; e < E; ++e) v[e] = -INFINITY;
      ds_add_block<kDt>(r, rc, s, v, a.c);
    }
    s *= exp2_hw(-fmaf(r, a.c, -rc));
    ds_join<T>(r, s, a.c, sh.red);
    if (!(s > 0.f && s < INFINITY && fabsf(r) * a.c < kDsFast)) ds_exact_sums<kDt, T, NB>(d, sp, slot0, a.slots, xr, r, s, sh);
    if (t == 0) {
      float* o = a.ws_sums + (row * a.parts + part) * 2;
      o[0] = r;
      o[1] = s;
    }
  } else {
    float r = -3.4028235e38f, s = 0.f;
    for (int p = t; p < a.parts; p += T) {
      const float* o = a.ws_sums + (row * a.parts + p) * 2;
      const float to = fmaxf(r, o[0]);
      s = (s == 0.f ? 0.f : s * exp2_hw((r - to) * a.c)) + (o[1] == 0.f ? 0.f : o[1] * exp2_hw((o[0] - to) * a.c));
      r = to;
    }
    ds_join<T>(r, s, a.c, sh.red);
    const float* o = a.ws_list + row * 8;
    const DsList list{o[0], o[1], o[2], o[3], o[5], *reinterpret_cast<const double*>(o + 6), o[4]};
    const DsFinal f = ds_final(a, a.weight ? a.weight[row] : 1.f, list, r, s);
    if (part == 0 && t == 0 && a.loss) a.loss[row] = ds_loss(a, list, f, r, s);
    if (!a.grad) return;
    if (edges && sp.edge(t) >= 0) {
      float g[1];
      ds_gradient<false>(f, f.rest, 0.f, a.c, &xe, g, 1);
      store_el<kDt>(static_cast<char*>(a.grad) + row * a.ld_g * Span<kDt>::kSize, sp.edge(t), g[0]);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int first = (slot0 + i) * T;
      if (i >= a.slots || t >= sp.blocks - first) continue;
      float v[E], g[E];
      unpack_held<kDt>(w[i], v);
      ds_gradient<false>(f, f.rest, 0.f, a.c, v, g, E);
      ds_store<kDt>(a.grad, a.ld_g, sp, row, first, t, g);
    }
    const DsFix fix = ds_fix<kDt, T, NB>(d, f);
    memory_done();
    lds_barrier();
    if (own) ds_store_fix<kDt>(a, row, fix);
  }
}

struct DsPlan {
  int threads, held;       // row kernel: threads and blocks a lane holds; threads 0: part kernels
  int parts, slots;
  size_t off_list, total;
};

// Whole rows, or parts of rows.  Few rows in whole leave CUs idle: 32 rows of
// 131072 bf16 take 19.4 us whole and 14.5 in parts, 128 take 25 and 29; of 32000,
// 32 rows 11.6 and 11.9, 128 rows 12.4 and 15.1.  The smallest workgroups in
// which a row fits 16 blocks a lane; one of up to 4 blocks in registers for 4.
static DsPlan ds_plan(int64_t n_rows, int64_t vocab, int es) {
  DsPlan p{};
  const int64_t blocks = vocab * es / 16;
  const int64_t row_max = 1024 * 20;
  if (blocks <= 1024 || (n_rows > (blocks <= 256 * 16 ? 32 : 64) && blocks <= row_max)) {
    p.threads = blocks <= 256 * 16 ? 256 : blocks <= 512 * 16 ? 512 : 1024;
    p.held = blocks <= 256 * 4 ? 4 : blocks <= 1024 * 16 ? 16 : 20;
    return p;
  }
  // parts: enough for four workgroups per CU, of one block a lane or more
  int64_t slots = kDsPartBlocks;
  while (slots > 1 && n_rows * cdiv(blocks, slots * kDsPartThreads) < 1024) slots /= 2;
  p.slots = (int)slots;
  p.parts = (int)cdiv(blocks, slots * kDsPartThreads);
  p.off_list = align_up((size_t)n_rows * p.parts * 8, 256);
  p.total = p.off_list + (size_t)n_rows * 32;
  return p;
}

size_t distill_workspace_bytes(int64_t n_rows, int64_t vocab, int64_t) {
  return std::max(ds_plan(n_rows, vocab, 2).total, ds_plan(n_rows, vocab, 4).total);
}

template <int kDt, int T, int NB>
static void ds_launch_rows(const DsArgs& a, int per_cu, hipStream_t st) {
  const dim3 grid((unsigned)std::min<int64_t>(a.n_rows, 256 * per_cu));
  if (a.grad) hipLaunchKernelGGL((distill_row_kernel<kDt, T, NB, true>), grid, dim3(T), 0, st, a);
  else hipLaunchKernelGGL((distill_row_kernel<kDt, T, NB, false>), grid, dim3(T), 0, st, a);
}

template <int kDt, int NB>
static void ds_launch_parts(const DsArgs& a, hipStream_t st) {
  const dim3 all((unsigned)(a.n_rows * a.parts)), rows((unsigned)a.n_rows);
  hipLaunchKernelGGL((distill_part_kernel<kDt, NB, true>), all, dim3(kDsPartThreads), 0, st, a);
  hipLaunchKernelGGL((distill_part_kernel<kDt, NB, false>), a.grad ? all : rows, dim3(kDsPartThreads), 0, st, a);
}

template <int kDt>
static void ds_dispatch(const DsArgs& a, const DsPlan& p, hipStream_t st) {
  if (p.threads == 256 && p.held == 4) ds_launch_rows<kDt, 256, 4>(a, 6, st);
  else if (p.threads == 256) ds_launch_rows<kDt, 256, 16>(a, 4, st);
  else if (p.threads == 512) ds_launch_rows<kDt, 512, 16>(a, 2, st);
  else if (p.threads == 1024 && p.held == 16) ds_launch_rows<kDt, 1024, 16>(a, 1, st);
  else if (p.threads == 1024) ds_launch_rows<kDt, 1024, 20>(a, 1, st);
  else if (p.slots <= 4) ds_launch_parts<kDt, 4>(a, st);
  else ds_launch_parts<kDt, kDsPartBlocks>(a, st);
}

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_distill_topk(const void* logits, int32_t x_dtype, int64_t n_rows, int64_t vocab,
                                         int64_t ld_x, const int32_t* top_id, const float* top_logprob, int32_t k,
                                         float temperature, int32_t tail, const float* weight, float* loss, void* grad,
                                         int64_t ld_g, void* workspace, size_t ws_bytes, void* stream) {
  GQ_CHECK_ARG(x_dtype == GPTQ_F32 || x_dtype == GPTQ_F16 || x_dtype == GPTQ_BF16);
  GQ_CHECK_ARG(n_rows >= 0 && n_rows <= ((int64_t)1 << 22) && vocab >= 1 && vocab <= ((int64_t)1 << 30));
  GQ_CHECK_ARG(ld_x >= vocab && ld_x <= ((int64_t)1 << 36));
  GQ_CHECK_ARG(temperature >= 1e-4f && temperature <= 1e4f);
  GQ_CHECK_ARG(k >= 1 && (tail == 0 || tail == 1));
  GQ_CHECK_ARG(grad == nullptr || (ld_g >= vocab && ld_g <= ((int64_t)1 << 36)));
  if (k > kDsMaxK || vocab > ((int64_t)1 << 21)) return GPTQ_EUNSUPPORTED;
  if (n_rows == 0) return GPTQ_OK;
  GQ_CHECK_ARG(loss || grad);
  GQ_CHECK_ARG(grad == nullptr || grad != logits || ld_g == ld_x);
  const int es = x_dtype == GPTQ_F32 ? 4 : 2;
  GQ_CHECK_ARG(logits && top_id && top_logprob && reinterpret_cast<uintptr_t>(logits) % es == 0 &&
               reinterpret_cast<uintptr_t>(grad) % es == 0);
  const size_t need = distill_workspace_bytes(n_rows, vocab, k);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GPTQ_ENOMEM;
  const DsPlan pl = ds_plan(n_rows, vocab, es);
  GQ_CHECK_ARG(pl.threads != 0 || reinterpret_cast<uintptr_t>(workspace) % 256 == 0);
  DsArgs a{};
  a.x = logits;
  a.ld = ld_x;
  a.id = top_id;
  a.lp = top_logprob;
  a.weight = weight;
  a.loss = loss;
  a.grad = grad;
  a.ld_g = ld_g;
  a.n_rows = n_rows;
  a.c = (float)(1.4426950408889634074 / temperature);
  a.inv_t = (float)(1.0 / temperature);
  a.inv_td = 1.0 / temperature;
  a.vocab = (int)vocab;
  a.k = k;
  a.tail = tail;
  a.parts = pl.parts;
  a.slots = pl.slots;
  a.ws_sums = static_cast<float*>(workspace);
  a.ws_list = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.off_list);
  hipStream_t st = static_cast<hipStream_t>(stream);
  TimedScope ts(kTimeDistill, st);
  if (x_dtype == GPTQ_F32) ds_dispatch<GPTQ_F32>(a, pl, st);
  else if (x_dtype == GPTQ_F16) ds_dispatch<GPTQ_F16>(a, pl, st);
  else ds_dispatch<GPTQ_BF16>(a, pl, st);
  GQ_LAUNCHED();
  return GPTQ_OK;
}
