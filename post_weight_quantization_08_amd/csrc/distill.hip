// Distillation from a teacher's top logits: loss and gradient of rows.
#include "answer.h"

namespace gq {

struct DsArgs {
  const void* x;
  int64_t ld;
  const int32_t* id;
  const float* lp;
  const float* weight;
  float* loss;
  void* grad;
  int64_t ld_g;
  float c, inv_t;
  int vocab, k, tail;
};

template <class F>
__device__ float block_reduce_f(float v, float* lds, F f) {
  __syncthreads();
  lds[threadIdx.x] = v;
  for (int s = 128; s > 0; s >>= 1) {
    __syncthreads();
    if (threadIdx.x < s) lds[threadIdx.x] = f(lds[threadIdx.x], lds[threadIdx.x + s]);
  }
  __syncthreads();
  return lds[0];
}

// One workgroup of 256 per row.  The tail's maximum and sum are taken over
// the tokens outside the teacher's list, the listed ones join afterwards.
template <int kDt>
__global__ __launch_bounds__(256) void distill_kernel(DsArgs a) {
  __shared__ float lds[256];
  __shared__ int ids[128];
  __shared__ float lps[128], xs[128];
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x;
  const char* x = static_cast<const char*>(a.x) + row * a.ld * (kDt == GPTQ_F32 ? 4 : 2);
  if (t < a.k) {
    const int id = a.id[row * a.k + t];
    const float lp = a.lp[row * a.k + t];
    bool ok = id >= 0 && id < a.vocab && !(lp == -INFINITY);
    if (ok)
      for (int i = 0; i < t; ++i) ok = ok && !(a.id[row * a.k + i] == id && !(a.lp[row * a.k + i] == -INFINITY));
    ids[t] = ok ? id : -1;
    lps[t] = lp;
    xs[t] = ok ? load_el<kDt>(x, id) : -INFINITY;
  }
  __syncthreads();
  auto listed = [&](int j) {
    int at = -1;
    for (int i = 0; i < a.k; ++i) at = ids[i] == j ? i : at;
    return at;
  };
  auto fmax2 = [](float p, float q) { return fmaxf(p, q); };
  auto add2 = [](float p, float q) { return p + q; };
  float mr = -INFINITY;
  for (int j = t; j < a.vocab; j += 256)
    if (listed(j) < 0) mr = fmaxf(mr, load_el<kDt>(x, j));
  mr = block_reduce_f(mr, lds, fmax2);
  float sr = 0.f;
  if (mr > -INFINITY)
    for (int j = t; j < a.vocab; j += 256) {
      const float v = load_el<kDt>(x, j);
      if (listed(j) < 0) sr += exp2f((v - mr) * a.c);
      else if (v != v) sr += v;
    }
  else
    for (int j = t; j < a.vocab; j += 256) {
      const float v = load_el<kDt>(x, j);
      if (v != v) sr += v;
    }
  sr = block_reduce_f(sr, lds, add2);
  // the listed tokens
  const bool has = t < a.k && ids[t < a.k ? t : 0] >= 0;
  const float lp = has ? lps[t] : -INFINITY, xk = has ? xs[t] : -INFINITY;
  const float m = block_reduce_f(fmaxf(xk, mr), lds, fmax2);
  const float lm = block_reduce_f(lp, lds, fmax2);
  const int count = (int)block_reduce_f(has ? 1.f : 0.f, lds, add2);
  float p = has ? expf(a.tail ? lp : lp - lm) : 0.f;
  const float mass = block_reduce_f(p, lds, add2);
  float l = lp;
  if (!a.tail) {
    p /= mass;
    l = lp - lm - logf(mass);
  }
  const float s = block_reduce_f(has ? exp2f((xk - m) * a.c) : 0.f, lds, add2) +
                  (sr != 0.f ? sr * exp2f((mr - m) * a.c) : 0.f);
  const float log2s = log2f(s);
  float term = 0.f;
  if (has && p > 0.f) term = p * (l - ((xk - m) * a.inv_t - kLn2 * log2s));
  float loss = block_reduce_f(term, lds, add2);
  const float pr = a.tail ? fmaxf(1.f - mass, 0.f) : 0.f;
  const float lqr = sr != 0.f ? (mr - m) * a.inv_t + kLn2 * (log2f(sr) - log2s) : -INFINITY;
  if (pr > 0.f) loss += pr * (logf(pr) - lqr);
  const bool bad = !(m > -INFINITY) || s != s || m == INFINITY;
  if (count == 0) loss = 0.f;
  else if (bad) loss = NAN;
  if (t == 0 && a.loss) a.loss[row] = loss;
  if (!a.grad) return;
  char* g = static_cast<char*>(a.grad) + row * a.ld_g * (kDt == GPTQ_F32 ? 4 : 2);
  const float w = (a.weight ? a.weight[row] : 1.f) * a.inv_t;
  const float inv_s = 1.f / s;
  for (int j = t; j < a.vocab; j += 256) {
    float d = 0.f;
    if (w != 0.f && count > 0) {
      const float v = load_el<kDt>(x, j);
      const int at = listed(j);
      const float q = exp2f((v - m) * a.c) * inv_s;
      if (at >= 0) d = q - (a.tail ? expf(lps[at]) : expf(lps[at] - lm) / mass);
      else if (a.tail) d = sr > 0.f ? q - pr * exp2f((v - mr) * a.c) / sr : 0.f;
      else d = q;
      d = bad ? NAN : d * w;
    }
    store_el<kDt>(g, j, d);
  }
}

size_t distill_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_distill_topk(const void* logits, int32_t x_dtype, int64_t n_rows, int64_t vocab,
                                         int64_t ld_x, const int32_t* top_id, const float* top_logprob, int32_t k,
                                         float temperature, int32_t tail, const float* weight, float* loss, void* grad,
                                         int64_t ld_g, void* workspace, size_t ws_bytes, void* stream) {
  GQ_CHECK_ARG(x_dtype == GPTQ_F32 || x_dtype == GPTQ_F16 || x_dtype == GPTQ_BF16);
  GQ_CHECK_ARG(n_rows >= 0 && n_rows <= ((int64_t)1 << 24) && vocab >= 1 && vocab <= ((int64_t)1 << 30));
  GQ_CHECK_ARG(ld_x >= vocab && ld_x <= ((int64_t)1 << 40));
  GQ_CHECK_ARG(temperature >= 1e-4f && temperature <= 1e4f);
  GQ_CHECK_ARG(k >= 1 && (tail == 0 || tail == 1));
  GQ_CHECK_ARG(loss || grad);
  GQ_CHECK_ARG(grad == nullptr || (ld_g >= vocab && ld_g <= ((int64_t)1 << 40)));
  GQ_CHECK_ARG(grad == nullptr || grad != logits || ld_g == ld_x);
  if (k > 128) return GPTQ_EUNSUPPORTED;
  if (n_rows == 0) return GPTQ_OK;
  const size_t es = x_dtype == GPTQ_F32 ? 4 : 2;
  GQ_CHECK_ARG(logits && top_id && top_logprob && reinterpret_cast<uintptr_t>(logits) % es == 0 &&
               reinterpret_cast<uintptr_t>(grad) % es == 0);
  const size_t need = distill_workspace_bytes(n_rows, vocab, k);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return GPTQ_ENOMEM;
  DsArgs a{logits, ld_x, top_id, top_logprob, weight, loss, grad, ld_g, (float)(1.4426950408889634074 / temperature),
           (float)(1.0 / temperature), (int)vocab, k, tail};
  hipStream_t st = static_cast<hipStream_t>(stream);
  TimedScope ts(kTimeDistill, st);
  const dim3 grid((unsigned)n_rows);
  if (x_dtype == GPTQ_F32) hipLaunchKernelGGL(distill_kernel<GPTQ_F32>, grid, dim3(256), 0, st, a);
  else if (x_dtype == GPTQ_F16) hipLaunchKernelGGL(distill_kernel<GPTQ_F16>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(distill_kernel<GPTQ_BF16>, grid, dim3(256), 0, st, a);
  GQ_LAUNCHED();
  return GPTQ_OK;
}
