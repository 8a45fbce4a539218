// Gradients of low-rank adapters: the launches that no type changes, and the host's part.
#include "lora_grad.h"

namespace gq {

// U and T: the parts of their sums added up, scaled and laid out by position as three
// bf16 terms, zero where a run is only filled up: [rank][position] for the sums over
// tokens, [position][rank] for dX.
__global__ __launch_bounds__(256) void lora_grad_terms_kernel(GradArgs a) {
  const GradSide& s = a.side[blockIdx.y];
  const int pos = blockIdx.x * 64 + (threadIdx.x & 63);
  if (pos >= a.at.count[1]) return;
  const int v = a.at.order[pos];
  const int64_t m = v ^ (v >> 31);
  const float by = v < 0 ? 0.f : a.scale ? a.scale[a.adapter[m]] : 1.f;
  for (int r = (threadIdx.x >> 6) * 4; r < a.r16; r += 16) {
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (v >= 0 && r < a.rp) {
      const float* src = s.sums + m * a.rp + r;
      const int64_t step = a.M * a.rp;
      int p = 0;
      for (; p + 8 <= s.splits; p += 8) {
        f32x4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const f32x4*>(src + (p + i) * step);
#pragma unroll
        for (int i = 0; i < 8; ++i) x += w[i];
      }
      for (; p < s.splits; ++p) x += *reinterpret_cast<const f32x4*>(src + p * step);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] *= by;
    }
    uint32_t h[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float left = x[i];
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        h[t][i] = value_bits<GPTQ_BF16>(left);
        s.turned[(int64_t)(t * a.r16 + r + i) * a.P + pos] = (uint16_t)h[t][i];
        left = isinf(bf16_bits_to_f32(h[t][i])) ? 0.f : left - bf16_bits_to_f32(h[t][i]);   // an infinity is one term
      }
    }
    if (s.flat) {
#pragma unroll
      for (int t = 0; t < 3; ++t)
        *reinterpret_cast<uint2*>(s.flat + ((int64_t)t * a.P + pos) * a.rk + r) =
            uint2{h[t][0] | h[t][1] << 16, h[t][2] | h[t][3] << 16};
    }
  }
  // a step of 32 ranks may end behind the tiles of 16
  if (s.flat && a.r16 < a.rk && threadIdx.x < 64) {
#pragma unroll
    for (int t = 0; t < 3; ++t)
      for (int r = a.r16; r < a.rk; r += 4)
        *reinterpret_cast<uint2*>(s.flat + ((int64_t)t * a.P + pos) * a.rk + r) = uint2{0u, 0u};
  }
}

// The parts of adapters that have several, added up in order.
__global__ __launch_bounds__(256) void lora_grad_join_kernel(GradArgs a) {
  const GradSide& s = a.side[blockIdx.z];
  const int ad = blockIdx.y, slot = a.at.parts[2 * ad], parts = a.at.parts[2 * ad + 1];
  if (parts < 2) return;
  const int64_t each = (int64_t)a.rank * s.K;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < each; i += (int64_t)gridDim.x * 256) {
    float v = 0.f;
    for (int p = 0; p < parts; ++p) v += s.part[(slot + p) * each + i];
    s.grad[ad * each + i] = v;
  }
}

struct GradPlan {
  int rp, r16, rk, chunk, splits[2], per[2];
  int64_t P, max_chunks, slots;
  size_t order, chunks, parts, count, flat, sums[2], turned[2], part[2], total;
};

// The last: a launch has fewer than 2^32 threads, and the sums over tokens 512 for every 256
// columns, 64 ranks and chunk, of which an adapter has one whether it has tokens or not.
static bool grad_supported(int64_t M, int64_t d_in, int64_t d_out, int64_t rank, int64_t n) {
  const int64_t most = (int64_t)1 << 22;
  return rank <= kGradMaxRank && n <= kGradMaxAdapters && M <= most && d_in <= most && d_out <= most &&
         n * (d_in + d_out) <= ((int64_t)1 << 29);
}

static GradPlan grad_plan(int64_t M, int64_t d_in, int64_t d_out, int64_t rank, int64_t n) {
  GradPlan p{};
  p.rp = (int)(cdiv(rank, 8) * 8);
  p.r16 = rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128;
  p.rk = std::max(p.r16, 32);
  const int64_t blocks = cdiv(d_in, 256) + cdiv(d_out, 256);
  // chunks: a workgroup for every CU in one round, or two where registers and LDS have
  // room for them, of a step for every wave or more
  const int64_t want = std::max<int64_t>(1, std::min((p.r16 >= 64 ? 256 : 512) / blocks, M / 128));
  p.chunk = (int)(cdiv(cdiv(M, want), 32) * 32);
  p.P = align_up(M + 32 * n + 32, 64);
  p.max_chunks = cdiv(M, p.chunk) + n;
  // an adapter of k > 1 chunks has more than (k - 1) chunk tokens, k / 2 chunk of them
  p.slots = M > p.chunk ? 2 * cdiv(M, p.chunk) : 0;
  const int64_t widths[2] = {d_in, d_out};
  Carver c(nullptr);
  auto take = [&](size_t bytes) {
    c.take<char>(bytes);
    return c.used - bytes;
  };
  p.order = take((size_t)p.P * 4);
  p.chunks = take((size_t)p.max_chunks * sizeof(GradChunk));
  p.parts = take((size_t)n * 8);
  p.count = take(12);
  p.flat = take((size_t)3 * p.P * p.rk * 2);
  // parts of the sums: as many as one round of two workgroups a CU takes, of both sides
  const int64_t nb[2] = {cdiv(d_in, kF8Block), cdiv(d_out, kF8Block)};
  const int64_t parts = std::max<int64_t>(2, 512 / (cdiv(M, 4 * kGradTile) * (p.r16 > 64 ? 2 : 1)));
  int64_t per = cdiv(nb[0] + nb[1], parts);
  while (cdiv(nb[0], per) + cdiv(nb[1], per) > parts) ++per;
  for (int i = 0; i < 2; ++i) {
    p.splits[i] = (int)cdiv(nb[i], per);
    p.per[i] = (int)cdiv(nb[i], p.splits[i]);
    p.sums[i] = take((size_t)p.splits[i] * M * p.rp * 4);
    p.turned[i] = take((size_t)3 * p.r16 * p.P * 2);
    p.part[i] = take((size_t)p.slots * rank * widths[i] * 4);
  }
  p.total = align_up(c.used, 256);
  return p;
}

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_lora_grad_workspace_size(int64_t M, int64_t d_in, int64_t d_out, int32_t rank,
                                                     int64_t n_adapters, size_t* bytes_out) {
  GQ_CHECK_ARG(bytes_out && M >= 0 && d_in >= 1 && d_out >= 1 && rank >= 1 && n_adapters >= 1);
  if (!grad_supported(M, d_in, d_out, rank, n_adapters)) return GPTQ_EUNSUPPORTED;
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
  if (!grad_supported(M, d_in, d_out, rank, n_adapters)) return GPTQ_EUNSUPPORTED;
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

  GradArgs a{};
  a.at = GradPlace{reinterpret_cast<int32_t*>(ws + p.order), reinterpret_cast<GradChunk*>(ws + p.chunks),
                   reinterpret_cast<int32_t*>(ws + p.parts), reinterpret_cast<int32_t*>(ws + p.count)};
  a.adapter = adapter;
  a.scale = scale;
  a.base = base;
  a.dX = dX;
  a.ld_b = ld_b;
  a.ld_dx = ld_dx;
  a.wide_dx = dx_dtype == GPTQ_F32;
  a.M = M;
  a.P = p.P;
  a.n = (int)n_adapters;
  a.rank = rank;
  a.rp = p.rp;
  a.r16 = p.r16;
  a.rk = p.rk;
  a.chunk = p.chunk;
  a.halves = p.r16 > 64 ? 2 : 1;
  a.groups = (int)cdiv(M, 4 * kGradTile);
  for (int i = 0; i < 2; ++i) {     // X with A, dY with B
    GradSide& s = a.side[i];
    s.D = i ? dY : X;
    s.scales = i ? nullptr : x_scales;
    s.ld = i ? ld_dy : ld_x;
    s.K = (int)(i ? d_out : d_in);
    s.nb = (int)cdiv(s.K, kF8Block);
    s.F = static_cast<const uint16_t*>(i ? B : A);
    s.splits = p.splits[i];
    s.per = p.per[i];
    s.sums = reinterpret_cast<float*>(ws + p.sums[i]);
    s.flat = i && dX ? reinterpret_cast<uint16_t*>(ws + p.flat) : nullptr;
    s.turned = reinterpret_cast<uint16_t*>(ws + p.turned[i]);
    s.by = reinterpret_cast<uint16_t*>(ws + p.turned[1 - i]);
    s.grad = i ? dB : dA;
    s.part = reinterpret_cast<float*>(ws + p.part[i]);
    s.blocks = (int)cdiv(s.K, 256);
  }
  const bool codes = x_dtype == GPTQ_E4M3, wide = dy_dtype == GPTQ_F32;
  const auto launch = dtype == GPTQ_F16 ? grad_launch_f16 : grad_launch_bf16;
  launch(a, codes, wide, p.max_chunks, kGradProject, st);
  GQ_LAUNCHED();
  hipLaunchKernelGGL(lora_grad_terms_kernel, dim3((unsigned)cdiv(p.P, 64), 2), dim3(256), 0, st, a);
  GQ_LAUNCHED();
  launch(a, codes, wide, p.max_chunks, kGradOuter, st);
  GQ_LAUNCHED();
  if (p.slots > 0) {
    const int64_t each = (int64_t)rank * std::max(d_in, d_out);
    hipLaunchKernelGGL(lora_grad_join_kernel, dim3((unsigned)std::min<int64_t>(cdiv(each, 256), 4096), (unsigned)n_adapters, 2),
                       dim3(256), 0, st, a);
    GQ_LAUNCHED();
  }
  if (dX && M > 0) {
    launch(a, codes, wide, p.max_chunks, kGradInput, st);
    GQ_LAUNCHED();
  }
  return GPTQ_OK;
}
