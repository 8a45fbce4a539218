// Low-rank adapters of many requests beside a shared projection.
#include "answer.h"

namespace gq {

size_t w4a16_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out);

struct LoraArgs {
  const uint16_t* X;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const int32_t* adapter;
  const void* base;
  void* Y;
  float* T;                // [M][rank], scaled
  int64_t ld_x, ld_b, ld_y, M, d_out;
  int d_in, rank, n;
};

// T[m][r] = scale X[m] . A_a[r]: one wave per (token, rank).
template <int kDt>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs a) {
  const int64_t m = blockIdx.x;
  const int ad = a.adapter[m];
  if (ad < 0 || ad >= a.n) return;
  const int lane = threadIdx.x & 63;
  for (int r = threadIdx.x >> 6; r < a.rank; r += 4) {
    const uint16_t* Ar = a.A + ((int64_t)ad * a.rank + r) * a.d_in;
    float s = 0.f;
    for (int i = lane; i < a.d_in; i += 64) s = fmaf(load_el<kDt>(a.X, m * a.ld_x + i), load_el<kDt>(Ar, i), s);
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    if (lane == 0) a.T[m * a.rank + r] = (a.scale ? a.scale[ad] : 1.f) * s;
  }
}

// Y[m][n] = base[m][n] + T[m] . B_a[n].
template <int kDt, int kY>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
  const int64_t m = blockIdx.x;
  const int ad = a.adapter[m];
  const bool on = ad >= 0 && ad < a.n;
  for (int64_t n = threadIdx.x; n < a.d_out; n += 256) {
    float s = a.base ? load_el<kY>(a.base, m * a.ld_b + n) : 0.f;
    if (on) {
      float d = 0.f;
      const uint16_t* b = a.B + ((int64_t)ad * a.d_out + n) * a.rank;
      for (int r = 0; r < a.rank; ++r) d = fmaf(a.T[m * a.rank + r], load_el<kDt>(b, r), d);
      s += d;
    }
    store_el<kY>(a.Y, m * a.ld_y + n, s);
  }
}

size_t lora_workspace_bytes(int64_t M, int64_t, int64_t, int64_t rank) { return align_up((size_t)M * rank * 4, 256); }

size_t w4a16_lora_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out, int64_t rank) {
  return align_up(w4a16_workspace_bytes(M, d_in, d_out), 256) + lora_workspace_bytes(M, d_in, d_out, rank);
}

template <int kDt>
static void lora_launch(const LoraArgs& a, int32_t y_dtype, hipStream_t st) {
  const dim3 grid((unsigned)a.M);
  hipLaunchKernelGGL(lora_down_kernel<kDt>, grid, dim3(256), 0, st, a);
  if (y_dtype == GPTQ_F32) hipLaunchKernelGGL((lora_up_kernel<kDt, GPTQ_F32>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((lora_up_kernel<kDt, kDt>), grid, dim3(256), 0, st, a);
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
  if (rank > 128) return GPTQ_EUNSUPPORTED;
  if (M == 0) return GPTQ_OK;
  const size_t ys = y_dtype == GPTQ_F32 ? 4 : 2;
  GQ_CHECK_ARG(X && A && B && adapter && Y);
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(X) % 2 == 0 && reinterpret_cast<uintptr_t>(A) % 2 == 0 &&
               reinterpret_cast<uintptr_t>(B) % 2 == 0 && reinterpret_cast<uintptr_t>(Y) % ys == 0 &&
               reinterpret_cast<uintptr_t>(base) % ys == 0);
  if (workspace == nullptr || ws_bytes < lora_workspace_bytes(M, d_in, d_out, rank)) return GPTQ_ENOMEM;
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(workspace) % 256 == 0);
  LoraArgs a{static_cast<const uint16_t*>(X), static_cast<const uint16_t*>(A), static_cast<const uint16_t*>(B), scale,
             adapter, base, Y, static_cast<float*>(workspace), ld_x, ld_b, ld_y, M, d_out, (int)d_in, rank,
             (int)n_adapters};
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
  if (rank > 128 || M > 64) return GPTQ_EUNSUPPORTED;
  if (workspace != nullptr && ws_bytes < w4a16_lora_workspace_bytes(M, d_in, d_out, rank)) return GPTQ_ENOMEM;
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(workspace) % 256 == 0);
  const size_t w4 = align_up(w4a16_workspace_bytes(M, d_in, d_out), 256);
  const gptq_status s = gptq_w4a16_matmul(X, x_dtype, M, d_in, ld_x, qweight, scales, zeros, perm, d_out, group_size,
                                          Y, ld_y, workspace, ws_bytes, stream);
  if (s != GPTQ_OK) return s;
  return gptq_lora_add(X, x_dtype, M, d_in, ld_x, A, B, n_adapters, rank, scale, adapter, Y, ld_y, Y, GPTQ_F32, d_out,
                       ld_y, static_cast<char*>(workspace) + w4, ws_bytes - w4, stream);
}
