// Log probabilities of given tokens, entropy and the best alternatives of
// rows of logits.
#include "answer.h"

namespace gq {

struct LpArgs {
  const void* x;
  int64_t ld;
  const int32_t* targets;
  float c, inv_t;          // log2(e) / T, 1 / T
  int vocab, k;
  float *logprob, *lse, *entropy, *top_lp;
  int32_t* top_id;
};

template <class T, class F>
__device__ T block_reduce(T v, T* lds, F f) {
  __syncthreads();
  lds[threadIdx.x] = v;
  for (int s = 128; s > 0; s >>= 1) {
    __syncthreads();
    if (threadIdx.x < s) lds[threadIdx.x] = f(lds[threadIdx.x], lds[threadIdx.x + s]);
  }
  __syncthreads();
  return lds[0];
}

// One workgroup of 256 per row: the maximum, the sums, then one pass over the
// row for every alternative (the largest key below the last one).
template <int kDt>
__global__ __launch_bounds__(256) void logprobs_kernel(LpArgs a) {
  __shared__ float f_lds[256];
  __shared__ uint64_t k_lds[256];
  const int64_t row = blockIdx.x;
  const char* x = static_cast<const char*>(a.x) + row * a.ld * (kDt == GPTQ_F32 ? 4 : 2);
  float m = -INFINITY;
  for (int j = threadIdx.x; j < a.vocab; j += 256) m = fmaxf(m, load_el<kDt>(x, j));
  m = block_reduce(m, f_lds, [](float p, float q) { return fmaxf(p, q); });
  float s = 0.f, u = 0.f;
  if (m > -INFINITY || m != m)
    for (int j = threadIdx.x; j < a.vocab; j += 256) {
      const float d = (load_el<kDt>(x, j) - m) * a.c;
      const float e = exp2f(d);
      s += e;
      u += e * fmaxf(d, -200.f);
    }
  s = block_reduce(s, f_lds, [](float p, float q) { return p + q; });
  u = block_reduce(u, f_lds, [](float p, float q) { return p + q; });
  const bool dead = s == 0.f;
  const float log2s = log2f(s);
  auto lp_of = [&](float v) { return dead ? v == v ? -INFINITY : v : (v - m) * a.inv_t - kLn2 * log2s; };
  if (threadIdx.x == 0) {
    if (a.logprob) {
      const int t = a.targets[row];
      a.logprob[row] = t >= 0 && t < a.vocab ? lp_of(load_el<kDt>(x, t)) : 0.f;
    }
    if (a.lse) a.lse[row] = dead ? -INFINITY : m * a.inv_t + kLn2 * log2s;
    if (a.entropy) {
      const float h = kLn2 * (log2s - u / s);
      a.entropy[row] = dead || h < 0.f ? 0.f : h;
    }
  }
  uint64_t last = ~0ull;
  for (int r = 0; r < a.k; ++r) {
    uint64_t best = 0;
    for (int j = threadIdx.x; j < a.vocab; j += 256) {
      const uint64_t key = key_of(load_el<kDt>(x, j), j);
      if (key < last || r == 0) best = key > best ? key : best;
    }
    last = block_reduce(best, k_lds, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
    if (threadIdx.x == 0) {
      a.top_lp[row * a.k + r] = lp_of(value_of((uint32_t)(last >> 32)));
      a.top_id[row * a.k + r] = (int32_t)index_of(last);
    }
  }
}

size_t logprobs_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_token_logprobs(const void* logits, int32_t x_dtype, int64_t n_rows, int64_t vocab,
                                           int64_t ld_x, const int32_t* targets, float temperature, int32_t k,
                                           float* logprob, float* lse, float* entropy, float* top_logprob,
                                           int32_t* top_id, void* workspace, size_t ws_bytes, void* stream) {
  GQ_CHECK_ARG(x_dtype == GPTQ_F32 || x_dtype == GPTQ_F16 || x_dtype == GPTQ_BF16);
  GQ_CHECK_ARG(n_rows >= 0 && n_rows <= ((int64_t)1 << 24) && vocab >= 1 && vocab <= ((int64_t)1 << 30));
  GQ_CHECK_ARG(ld_x >= vocab && ld_x <= ((int64_t)1 << 40));
  GQ_CHECK_ARG(temperature >= 1e-4f && temperature <= 1e4f);
  GQ_CHECK_ARG(k >= 0 && k <= vocab);
  GQ_CHECK_ARG(logprob == nullptr || targets != nullptr);
  GQ_CHECK_ARG(k == 0 || (top_logprob && top_id));
  GQ_CHECK_ARG(logprob || lse || entropy || k > 0);
  if (k > 128) return GPTQ_EUNSUPPORTED;
  if (n_rows == 0) return GPTQ_OK;
  GQ_CHECK_ARG(logits != nullptr && reinterpret_cast<uintptr_t>(logits) % (x_dtype == GPTQ_F32 ? 4 : 2) == 0);
  const size_t need = logprobs_workspace_bytes(n_rows, vocab, k);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GPTQ_ENOMEM;
  LpArgs a{logits, ld_x, targets, (float)(1.4426950408889634074 / temperature), (float)(1.0 / temperature), (int)vocab,
           k, logprob, lse, entropy, top_logprob, top_id};
  hipStream_t st = static_cast<hipStream_t>(stream);
  TimedScope ts(kTimeLogprobs, st);
  const dim3 grid((unsigned)n_rows);
  if (x_dtype == GPTQ_F32) hipLaunchKernelGGL(logprobs_kernel<GPTQ_F32>, grid, dim3(256), 0, st, a);
  else if (x_dtype == GPTQ_F16) hipLaunchKernelGGL(logprobs_kernel<GPTQ_F16>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(logprobs_kernel<GPTQ_BF16>, grid, dim3(256), 0, st, a);
  GQ_LAUNCHED();
  return GPTQ_OK;
}
