// FP8 rows and FP8 blocks from bf16 or fp32.
#include "fp4mi_moe.h"
#include "host_common.hpp"
#include "rows_common.hpp"

namespace fp4mi {
namespace {

// Parts of the whole tensor in turn: blocks of 128 never straddle rows, as cols is a
// multiple of 128, so a block's lanes are neighbours wherever they stand.  Bound by
// memory: 16384 x 7168 bf16 55 us (6.4 TB/s), fp32 90 us (6.6 TB/s).
constexpr int kRowParts = 2;   // parts a thread
template <bool BF16>
__global__ __launch_bounds__(kThreads) void fp8_rows_kernel(const void* x, uint8_t* q, float* scales,
                                                            int64_t parts, int64_t blk0) {
  constexpr int V = Part<BF16>::kValues;
  const int64_t i0 = ((int64_t)blockIdx.x + blk0) * (kThreads * kRowParts) + threadIdx.x;
  u32x4 raw[kRowParts];
#pragma unroll
  for (int c = 0; c < kRowParts; ++c)
    if (i0 + c * kThreads < parts) raw[c] = ld_u32x4(static_cast<const u32x4*>(x) + i0 + c * kThreads);
#pragma unroll
  for (int c = 0; c < kRowParts; ++c) {
    const int64_t i = i0 + c * kThreads;
    if (i >= parts) continue;   // a block's lanes leave together
    float z[V];
    part_values<BF16>(raw[c], z);
    quantize_part<true, false, V>(z, i, q, scales);
  }
}

// One workgroup a tile: a thread holds one part of every row that is its own.
// The transposed copy goes through LDS: a thread reads 4 columns of 16 rows, a
// word each, and turns them in registers.  Bound by memory: four 4096 x 7168 fp32
// weights with the copy 119 us (5.9 TB/s), bf16 73 us (6.4 TB/s).
struct BlockArgs {
  const void* x;
  uint8_t* q;
  float* scales;
  uint8_t* qt;
  float* scales_t;
  int64_t rows;
  int cols;
  int64_t row_tiles;
  int col_tiles;
};
constexpr int kTilePitch = 33;   // words of a row of codes in LDS
template <bool BF16>
__global__ __launch_bounds__(kThreads) void fp8_blocks_kernel(BlockArgs p, int64_t blk0) {
  __shared__ uint32_t codes[128 * kTilePitch];
  __shared__ float top[4];
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int ct = (int)(blk % p.col_tiles);
  const int64_t bt = blk / p.col_tiles, rt = bt % p.row_tiles, b = bt / p.row_tiles;
  constexpr int V = Part<BF16>::kValues, L = Part<BF16>::kLanes, R = kThreads / L, N = 128 / R;   // N rows a thread
  const int tid = threadIdx.x, part = tid % L, r0 = tid / L;
  const int rows = (int)min(p.rows - rt * 128, (int64_t)128), width = p.cols / V;
  const int64_t first = (b * p.rows + rt * 128) * width + ct * L + part;
  u32x4 raw[N];
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    raw[i] = {};
    if (r0 + R * i < rows) raw[i] = ld_u32x4(static_cast<const u32x4*>(p.x) + first + (int64_t)(r0 + R * i) * width);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float z[V];
    part_values<BF16>(raw[i], z);
    am = part_max(z, am);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) am = fmaxf(am, __shfl_xor(am, d));
  if ((tid & 63) == 0) top[tid >> 6] = am;
  __syncthreads();
  am = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  const int k = fp8_block_exponent(am);
  if (tid == 0) {
    const float s = fp8_scale(am, k);
    p.scales[(b * p.row_tiles + rt) * p.col_tiles + ct] = s;
    if (p.qt) p.scales_t[(b * p.col_tiles + ct) * p.row_tiles + rt] = s;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + R * i;
    float z[V];
    part_values<BF16>(raw[i], z);
    uint8_t* to = p.q + V * (first + (int64_t)r * width);
    if constexpr (BF16) {
      const u32x2 c = fp8_codes8(z, k);
      if (r < rows) *reinterpret_cast<u32x2*>(to) = c;
      if (p.qt) {
        codes[r * kTilePitch + 2 * part] = c.x;
        codes[r * kTilePitch + 2 * part + 1] = c.y;
      }
    } else {
      const uint32_t c = fp8_codes4(z, k);
      if (r < rows) *reinterpret_cast<uint32_t*>(to) = c;
      if (p.qt) codes[r * kTilePitch + part] = c;
    }
  }
  if (!p.qt) return;
  __syncthreads();
  // rows 16 (tid % 8) .. + 15 of columns 4 (tid / 8) .. + 3: eight lanes write a
  // column's 128 bytes
  const int rg = tid & 7, cg = tid >> 3;
  uint32_t col[4][4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t w[4], t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = codes[(rg * 16 + h * 4 + j) * kTilePitch + cg];
    transpose_bytes(w, t);
#pragma unroll
    for (int j = 0; j < 4; ++j) col[j][h] = t[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    st_u32x4(p.qt + ((b * p.cols + ct * 128 + cg * 4 + j) * p.rows + rt * 128 + rg * 16),
             u32x4{col[j][0], col[j][1], col[j][2], col[j][3]});
}

}  // namespace
}  // namespace fp4mi

using namespace fp4mi;

extern "C" int fp8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, uint8_t* q,
                            float* scales, void* stream) {
  const int isz = dtype_size(dtype);
  if (!isz) return FP4_EDTYPE;
  int64_t n;
  if (cols % 128 || !checked_count(rows, cols, &n)) return FP4_ESHAPE;
  if (n == 0) return FP4_OK;
  if (!x || !q || !scales) return FP4_EINVAL;
  if (!is_aligned(x, 16) || !is_aligned(q, 16) || !is_aligned(scales, 4)) return FP4_EALIGN;
  if (overlaps(q, n, x, n * isz) || overlaps(scales, n / 32, x, n * isz) || overlaps(q, n, scales, n / 32))
    return FP4_EOVERLAP;
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const int64_t parts = n * isz / 16, blocks = blocks_for(parts, kRowParts);
  if (dtype == FP4_DTYPE_BF16)
    launch_1d(fp8_rows_kernel<true>, blocks, kThreads, st, x, q, scales, parts);
  else
    launch_1d(fp8_rows_kernel<false>, blocks, kThreads, st, x, q, scales, parts);
  return launch_status();
}

extern "C" int fp8_quantize_blocks(const void* x, int dtype, int64_t batch, int64_t rows,
                                   int64_t cols, uint8_t* q, float* scales, uint8_t* q_t,
                                   float* scales_t, void* stream) {
  const int isz = dtype_size(dtype);
  if (!isz) return FP4_EDTYPE;
  int64_t m, n;
  if (batch < 0 || cols % 128 || cols >= (int64_t(1) << 31) || !checked_count(rows, cols, &m) ||
      !checked_count(batch, m, &n))
    return FP4_ESHAPE;
  if (q_t && rows % 128) return FP4_ESHAPE;
  if (!q_t != !scales_t) return FP4_EINVAL;
  if (n == 0) return FP4_OK;
  if (!x || !q || !scales) return FP4_EINVAL;
  if (!is_aligned(x, 16) || !is_aligned(q, 16) || !is_aligned(scales, 4) || !is_aligned(q_t, 16) ||
      !is_aligned(scales_t, 4))
    return FP4_EALIGN;
  const int64_t row_tiles = (rows + 127) / 128, tiles = batch * row_tiles * (cols / 128);
  const void* outs[4] = {q, scales, q_t, scales_t};
  const int64_t outn[4] = {n, tiles * 4, q_t ? n : 0, q_t ? tiles * 4 : 0};
  for (int i = 0; i < 4; ++i) {
    if (overlaps(outs[i], outn[i], x, n * isz)) return FP4_EOVERLAP;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outn[i], outs[j], outn[j])) return FP4_EOVERLAP;
  }
  BlockArgs p = {x, q, scales, q_t, scales_t, rows, (int)cols, row_tiles, (int)(cols / 128)};
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  if (dtype == FP4_DTYPE_BF16)
    launch_1d(fp8_blocks_kernel<true>, tiles, kThreads, st, p);
  else
    launch_1d(fp8_blocks_kernel<false>, tiles, kThreads, st, p);
  return launch_status();
}
