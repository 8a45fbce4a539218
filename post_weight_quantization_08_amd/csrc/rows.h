// Rows of logits held in registers between their sums and their gradients:
// 16-byte blocks as loaded, dealt to the threads of a workgroup.
#pragma once

#include "answer.h"

namespace gq {

// References as in the log probabilities: none below the floor (a power of
// two), a new one when a term would exceed 2^8, another way when r c is so
// large that its rounding matters.
constexpr float kDsFloor = -1048576.f, kDsFast = 268435456.f, kDsLag = 8.f;

// A row as `head` single logits, `blocks` 16-byte blocks on 16-byte addresses
// and `rest` single logits.
template <int kDt>
struct Span {
  static constexpr int E = kDt == GPTQ_F32 ? 4 : 8;
  static constexpr int kSize = 16 / E;
  const char* p;           // first element
  int head, blocks, rest;
  __device__ __forceinline__ Span(const void* x, int64_t row, int64_t ld, int vocab) {
    p = static_cast<const char*>(x) + row * ld * kSize;
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15) / kSize;
    head = min(vocab, off ? E - off : 0);
    blocks = (vocab - head) / E;
    rest = vocab - head - blocks * E;
  }
  // block first + lane, `first` the same in every lane
  __device__ __forceinline__ u32x4 load(int first, int lane) const {
    return *reinterpret_cast<const u32x4*>(p + head * kSize + (int64_t)first * 16 + (uint32_t)lane * 16u);
  }
  // the single logit of thread t (threads 0..7 the head's, 8..15 the rest's), or -1
  __device__ __forceinline__ int edge(int t) const {
    if (t < 8) return t < head ? t : -1;
    return t < 16 && t - 8 < rest ? head + blocks * E + t - 8 : -1;
  }
};

template <int kDt>
__device__ __forceinline__ u32x4 masked_block() {
  const uint32_t w = kDt == GPTQ_F32 ? 0xFF800000u : kDt == GPTQ_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
  return u32x4{w, w, w, w};
}

template <int kDt>
__device__ __forceinline__ u32x4 pack_block(const float (&g)[Span<kDt>::E]) {
  u32x4 w;
  if constexpr (kDt == GPTQ_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(g[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kDt == GPTQ_BF16) {
        uint32_t h;   // two roundings to nearest even in one instruction
        asm("v_cvt_pk_bf16_f32 %0, %1, %2" : "=v"(h) : "v"(g[2 * i]), "v"(g[2 * i + 1]));
        w[i] = h;
      } else {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const f16x2 h = {(_Float16)g[2 * i], (_Float16)g[2 * i + 1]};
        w[i] = __builtin_bit_cast(uint32_t, h);
      }
    }
  }
  return w;
}

// Where a lane reads that has no block to read: every load is made, so that
// the compiler can count the ones behind it and wait for one block at a time.
static __device__ u32x4 ds_pad[1];

// Blocks of a span as a lane reads them: block first + lane, or the last one
// in its place (or the pad, if there is none).
template <int kDt>
struct DsSource {
  const char* base;
  uint32_t last, lane;     // byte offsets: of the last block, of the lane's first
  __device__ __forceinline__ DsSource(const Span<kDt>& sp, bool real) {
    const bool any = real && sp.blocks > 0;
    base = any ? sp.p + sp.head * Span<kDt>::kSize : reinterpret_cast<const char*>(ds_pad);
    last = any ? (uint32_t)(sp.blocks - 1) * 16u : 0u;
    lane = threadIdx.x * 16u;
    asm volatile("" : "+v"(lane));   // a row's own value: offsets of all slots are not kept from row to row
  }
  __device__ __forceinline__ const u32x4* block(int first) const {
    const uint32_t at = (uint32_t)first * 16u + lane;
    return reinterpret_cast<const u32x4*>(base + (at < last ? at : last));
  }
  __device__ __forceinline__ u32x4 load(int first) const { return *block(first); }
};

// The block's logits.  The empty asm makes every use of a held block a value
// of its own: without it the compiler keeps the unpacked logits of the sums
// for the gradients, eight registers for every four held.
template <int kDt>
__device__ __forceinline__ void unpack_held(u32x4 w, float (&v)[Span<kDt>::E]) {
  asm volatile("" : "+v"(w));
  Blocks<kDt>::unpack(w, v);
}

template <int kDt>
__device__ __forceinline__ void hide(float (&v)[Span<kDt>::E], uint32_t listed) {
  if (listed) {
#pragma unroll
    for (int e = 0; e < Span<kDt>::E; ++e) v[e] = listed >> e & 1u ? -INFINITY : v[e];
  }
}

// The rest's sum over what a lane holds.
template <int kDt>
__device__ __forceinline__ void ds_add_block(float& r, float& rc, float& s, const float (&v)[Span<kDt>::E], float c) {
  constexpr int E = Span<kDt>::E;
  float vm = fmaxf(v[0], v[1]);
#pragma unroll
  for (int e = 2; e < E; ++e) vm = fmaxf(vm, v[e]);
  if (fmaf(vm, c, -rc) > kDsLag) {
    // s stands at rc, not at r c: both roundings go into the move
    const float skew = fmaf(vm, c, -(vm * c)) - fmaf(r, c, -rc);
    s *= exp2_hw(fmaxf((r - vm) * c, -1e30f) + skew);
    r = vm;
    rc = vm * c;
  }
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    s0 += exp2_hw(fmaf(v[e], c, -rc));
    s1 += exp2_hw(fmaf(v[e + 1], c, -rc));
  }
  s += s0 + s1;
}

// Reference and sum joined over the workgroup; every thread gets them.
template <int T>
__device__ __forceinline__ void ds_join(float& r, float& s, float c, float (&red)[T / 64][2]) {
  auto fmax2 = [](float p, float q) { return fmaxf(p, q); };
  auto add2 = [](float p, float q) { return p + q; };
  const float rw = wave_reduce(r, fmax2);
  s = wave_reduce(s * exp2_hw((r - rw) * c), add2);
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6][0] = rw;
    red[threadIdx.x >> 6][1] = s;
  }
  lds_barrier();
  static_assert(T / 64 <= 16, "a wave's partial per lane of sixteen");
  const int w = threadIdx.x & (T / 64 - 1) & 15;
  const float rl = red[w][0], sl = red[w][1];
  r = uniform(row_reduce(rl, fmax2));
  // every wave's partial stands 16 / (T / 64) times in a row of sixteen lanes
  const float mine = (threadIdx.x & 15) < T / 64 ? sl * exp2_hw((rl - r) * c) : 0.f;
  s = uniform(row_reduce(mine, add2));
}

// Every memory operation of this wave is done.
__device__ __forceinline__ void memory_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A block's gradients, 16 bytes in one store wherever they start (the gradient's
// rows need not start on their 16 bytes where the logits' do).
template <int kDt>
__device__ __forceinline__ void ds_store(void* grad, int64_t ld_g, const Span<kDt>& sp, int64_t row, int first, int lane,
                                         const float (&g)[Span<kDt>::E]) {
  char* p = static_cast<char*>(grad) + (row * ld_g + sp.head) * Span<kDt>::kSize + (int64_t)first * 16 +
            (uint32_t)lane * 16u;
  const u32x4 w = pack_block<kDt>(g);
  if constexpr (kDt == GPTQ_F32) __builtin_memcpy(__builtin_assume_aligned(p, 4), &w, 16);
  else __builtin_memcpy(__builtin_assume_aligned(p, 2), &w, 16);
}

// ln x in 64 bits of a 32-bit x: the exponent apart, so that the logarithm of
// a large sum keeps the digits that the loss is made of.
__device__ __forceinline__ double ln_wide(float x) {
  int e;
  const float m = frexpf(x, &e);
  return (double)e * 0.69314718055994530942 + (double)logf(m);
}

}  // namespace gq
