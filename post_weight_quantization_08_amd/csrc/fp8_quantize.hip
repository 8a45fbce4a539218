// Rows, or 128 x 128 tiles, to e4m3 codes with a power-of-two scale for each
// block of 128:  b = 127 + ceil(log2(max |x| / 448)), code = e4m3(x 2^(127 - b)).
//
// Bound by memory: every element is read once, kept in registers between the
// maximum and the rounding, and leaves as one byte (two with the transpose).
// 8192 x 11008 bf16 in rows 52 us (5.2 TB/s; a large copy runs at 5.0); 28672 x 8192
// in tiles with the transpose 188 us (5.0 TB/s).
#include "fp8.h"

namespace gq {

struct F8Args {
  const void* X;
  uint8_t* codes;
  uint8_t* scales;
  uint8_t* codes_t;        // tiles: the transpose's, or null
  uint8_t* scales_t;
  int64_t ld_x, ld_c, ld_ct, rows;
  int cols, blocks;        // blocks of a row
  int row_tiles;
  uint32_t total;          // rows mode: blocks of all rows
};

// Sixteen lanes take a block, eight elements each, so a wave's loads and stores
// lie next to each other; kU blocks of a lane are asked for before the first is
// looked at.
constexpr int kF8U = 4;

template <int kDt>
__global__ __launch_bounds__(256) void fp8_rows_kernel(F8Args a) {
  const int group = threadIdx.x >> 4, k = (threadIdx.x & 15) * 8;
  float v[kF8U][8];
  uint32_t row[kF8U], block[kF8U];
#pragma unroll
  for (int u = 0; u < kF8U; ++u) {
    const uint32_t at = (blockIdx.x * kF8U + u) * 16 + group;
    row[u] = at < a.total ? at / (uint32_t)a.blocks : 0xFFFFFFFFu;
    block[u] = at - row[u] * (uint32_t)a.blocks;
    if (at < a.total) {
      const char* p = static_cast<const char*>(a.X) + (int64_t)row[u] * a.ld_x * (kDt == GPTQ_F32 ? 4 : 2);
      f8_load8<kDt>(p, (int)block[u] * kF8Block + k, a.cols, v[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kF8U; ++u) {
    if (row[u] == 0xFFFFFFFFu) continue;
    // the sixteen lanes of a block are active together
    const uint32_t top = row_reduce(f8_top8(v[u]), [](uint32_t p, uint32_t q) { return max(p, q); });
    const uint32_t b = f8_scale(top);
    const uint2 w = {f8_codes4(v[u][0], v[u][1], v[u][2], v[u][3], b), f8_codes4(v[u][4], v[u][5], v[u][6], v[u][7], b)};
    *reinterpret_cast<uint2*>(a.codes + (int64_t)row[u] * a.ld_c + (int64_t)block[u] * kF8Block + k) = w;
    if ((threadIdx.x & 15) == 0) a.scales[(int64_t)row[u] * a.blocks + block[u]] = (uint8_t)b;
  }
}

// One workgroup per 128 x 128 tile: a thread holds eight rows of eight columns.
// The transpose goes through LDS, 16 bytes behind every 128 so that the columns
// of a store fall into different banks.
// Tiles are taken in bands of eight row tiles, so that what runs at one time reads and
// writes several lines next to each other of every row, of the transpose's too: 28672 x
// 8192 bf16 in one column of tiles after another 241 us, in bands of 8, 16, 32, 64 rows of
// tiles 189, 195, 197, 213; 131072 x 4096 528, and 422, 428, 451, 478.
constexpr int kF8Band = 8;

template <int kDt>
__global__ __launch_bounds__(256) void fp8_tiles_kernel(F8Args a) {
  constexpr int kPitch = kF8Block + 8;
  __shared__ uint32_t tops[4];
  __shared__ __align__(16) uint8_t turned[kF8Block * kPitch];
  const int t = threadIdx.x, group = t >> 4, k = (t & 15) * 8;
  const int band = blockIdx.x / (kF8Band * a.blocks), first = band * kF8Band, in = blockIdx.x - first * a.blocks;
  const int height = min(kF8Band, a.row_tiles - first);
  const int row_tile = first + in % height, col_tile = in / height;
  const int64_t r0 = (int64_t)row_tile * kF8Block + group * 8;
  const int c0 = col_tile * kF8Block;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + i < a.rows) {
      const char* p = static_cast<const char*>(a.X) + (r0 + i) * a.ld_x * (kDt == GPTQ_F32 ? 4 : 2);
      f8_load8<kDt>(p, c0 + k, a.cols, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
  auto larger = [](uint32_t p, uint32_t q) { return max(p, q); };
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, f8_top8(v[i]));
  top = row_reduce(top, larger);
  top = max(top, (uint32_t)__shfl_xor((int)top, 16));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32));
  if ((t & 63) == 0) tops[t >> 6] = top;
  __syncthreads();
  top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
  const uint32_t b = f8_scale(top);
  uint32_t w[8][2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i][0] = f8_codes4(v[i][0], v[i][1], v[i][2], v[i][3], b);
    w[i][1] = f8_codes4(v[i][4], v[i][5], v[i][6], v[i][7], b);
    if (r0 + i < a.rows)
      *reinterpret_cast<uint2*>(a.codes + (r0 + i) * a.ld_c + c0 + k) = uint2{w[i][0], w[i][1]};
  }
  if (t == 0) {
    a.scales[(int64_t)row_tile * a.blocks + col_tile] = (uint8_t)b;
    if (a.codes_t) a.scales_t[(int64_t)col_tile * a.row_tiles + row_tile] = (uint8_t)b;
  }
  if (!a.codes_t) return;
  // byte e of rows 0..3 and 4..7 side by side: two exchanges of halves and bytes
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t col[4][2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t x0 = w[4 * g][h], x1 = w[4 * g + 1][h], x2 = w[4 * g + 2][h], x3 = w[4 * g + 3][h];
      const uint32_t lo01 = __builtin_amdgcn_perm(x1, x0, 0x05010400u), hi01 = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
      const uint32_t lo23 = __builtin_amdgcn_perm(x3, x2, 0x05010400u), hi23 = __builtin_amdgcn_perm(x3, x2, 0x07030602u);
      col[0][g] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
      col[1][g] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
      col[2][g] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
      col[3][g] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<uint2*>(turned + (k + 4 * h + e) * kPitch + group * 8) = uint2{col[e][0], col[e][1]};
  }
  __syncthreads();
  // rows of the transpose, 128 bytes by sixteen lanes
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = i * 16 + group;
    if (c0 + c < a.cols)
      *reinterpret_cast<uint2*>(a.codes_t + (int64_t)(c0 + c) * a.ld_ct + (int64_t)row_tile * kF8Block + k) =
          *reinterpret_cast<const uint2*>(turned + c * kPitch + k);
  }
}

void f8_quantize_rows(const void* X, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* codes,
                      int64_t ld_c, uint8_t* scales, hipStream_t st) {
  F8Args a{};
  a.X = X;
  a.codes = codes;
  a.scales = scales;
  a.ld_x = ld_x;
  a.ld_c = ld_c;
  a.rows = rows;
  a.cols = (int)cols;
  a.blocks = (int)cdiv(cols, kF8Block);
  a.total = (uint32_t)(rows * a.blocks);
  const dim3 grid((unsigned)cdiv(a.total, 16 * kF8U));
  if (x_dtype == GPTQ_F32) hipLaunchKernelGGL((fp8_rows_kernel<GPTQ_F32>), grid, dim3(256), 0, st, a);
  else if (x_dtype == GPTQ_F16) hipLaunchKernelGGL((fp8_rows_kernel<GPTQ_F16>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((fp8_rows_kernel<GPTQ_BF16>), grid, dim3(256), 0, st, a);
}

}  // namespace gq

using namespace gq;

extern "C" gptq_status gptq_fp8_quantize(const void* X, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                                         int32_t block_rows, uint8_t* codes, int64_t ld_c, uint8_t* scales,
                                         uint8_t* codes_t, int64_t ld_ct, uint8_t* scales_t, void* stream) {
  GQ_CHECK_ARG(x_dtype == GPTQ_F32 || x_dtype == GPTQ_F16 || x_dtype == GPTQ_BF16);
  GQ_CHECK_ARG(rows >= 0 && rows < ((int64_t)1 << 31) && cols >= 1 && cols <= ((int64_t)1 << 30));
  GQ_CHECK_ARG(ld_x >= cols && ld_x <= ((int64_t)1 << 36));
  GQ_CHECK_ARG(block_rows == 1 || block_rows == kF8Block);
  const int64_t blocks = cdiv(cols, kF8Block), row_tiles = cdiv(rows, kF8Block);
  GQ_CHECK_ARG(ld_c >= blocks * kF8Block && ld_c % 16 == 0 && ld_c <= ((int64_t)1 << 36));
  const bool turn = codes_t != nullptr || scales_t != nullptr;
  GQ_CHECK_ARG(!turn || (block_rows == kF8Block && codes_t && scales_t && ld_ct >= row_tiles * kF8Block &&
                         ld_ct % 16 == 0 && ld_ct <= ((int64_t)1 << 36)));
  if (rows * blocks > kF8MostBlocks) return GPTQ_EUNSUPPORTED;
  if (rows == 0) return GPTQ_OK;
  GQ_CHECK_ARG(X && codes && scales && reinterpret_cast<uintptr_t>(X) % f8_elem(x_dtype) == 0);
  GQ_CHECK_ARG(reinterpret_cast<uintptr_t>(codes) % 16 == 0 && reinterpret_cast<uintptr_t>(codes_t) % 16 == 0);
  hipStream_t st = static_cast<hipStream_t>(stream);
  TimedScope ts(kTimeFp8, st);
  if (block_rows == 1) {
    f8_quantize_rows(X, x_dtype, rows, cols, ld_x, codes, ld_c, scales, st);
  } else {
    F8Args a{};
    a.X = X;
    a.codes = codes;
    a.scales = scales;
    a.codes_t = codes_t;
    a.scales_t = scales_t;
    a.ld_x = ld_x;
    a.ld_c = ld_c;
    a.ld_ct = ld_ct;
    a.rows = rows;
    a.cols = (int)cols;
    a.blocks = (int)blocks;
    a.row_tiles = (int)row_tiles;
    const dim3 grid((unsigned)(row_tiles * blocks));
    if (x_dtype == GPTQ_F32) hipLaunchKernelGGL((fp8_tiles_kernel<GPTQ_F32>), grid, dim3(256), 0, st, a);
    else if (x_dtype == GPTQ_F16) hipLaunchKernelGGL((fp8_tiles_kernel<GPTQ_F16>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((fp8_tiles_kernel<GPTQ_BF16>), grid, dim3(256), 0, st, a);
  }
  GQ_LAUNCHED();
  return GPTQ_OK;
}
