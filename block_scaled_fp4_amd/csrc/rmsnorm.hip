// RMS norm with residual addition and quantized rows, and its gradient.
#include <math.h>

#include "fp4mi_ops.h"
#include "host_common.hpp"
#include "device_common.hpp"

namespace fp4mi {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Largest |v| over the L lanes (4 or 16) that share a quantization block.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  v = fmaxf(v, lane_xor1(v));
  v = fmaxf(v, lane_xor2(v));
  if constexpr (L == 16) {
    v = fmaxf(v, __shfl_xor(v, 4));
    v = fmaxf(v, __shfl_xor(v, 8));
  }
  return v;
}

// Least k in [-126, 127] with amax <= 448 * 2^k = 1.75 * 2^(k+8).
__device__ __forceinline__ int fp8_block_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(k, -126);
}

// One octet z of a row -> its codes; the block's first lane stores the scale.
// i: octet index in the tensor.
template <bool FP8>
__device__ __forceinline__ void quantize_octet(const float (&z)[8], int64_t i, uint8_t* q,
                                               void* scales) {
  float am = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(z[j]));
  am = lanes_max<FP8 ? 16 : 4>(am);
  float v[8];
  if constexpr (FP8) {
    const int k = fp8_block_exponent(am);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_ldexpf(z[j], -k);
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    *reinterpret_cast<u32x2*>(q + 8 * i) = u32x2{(uint32_t)lo, (uint32_t)hi};
    if ((i & 15) == 0)
      static_cast<float*>(scales)[i >> 4] =
          am > 0.0f ? __uint_as_float((uint32_t)(k + 127) << 23) : 0x1p-127f;
  } else {
    const int b = max((int)(__float_as_uint(am) >> 23) - 2, 0);   // floor(log2 amax) - 2 + 127
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_ldexpf(z[j], 127 - b);
    *reinterpret_cast<uint32_t*>(q + 4 * i) = rtn8_unit(v);
    if ((i & 3) == 0) static_cast<uint8_t*>(scales)[i >> 2] = (uint8_t)b;
  }
}

struct NormArgs {
  const void* x;
  const void* res;
  const void* w;
  void* q;
  void* scales;
  float* row_scale;
  void* h;
  int64_t rows;
  int cols;
  float eps;
};

// One wave per row.
template <bool BF16, bool WBF16, bool FP8>
__global__ __launch_bounds__(kThreads) void rmsnorm_quantize_kernel(NormArgs p, int64_t blk0) {
  const int lane = threadIdx.x & 63;
  const int64_t row = ((int64_t)blockIdx.x + blk0) * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= p.rows) return;
  const int octets = p.cols >> 3;
  float sum = 0.0f;
  for (int o0 = 0; o0 < octets; o0 += 64) {
    const int o = o0 + lane;
    const bool in = o < octets;                 // whole blocks are in or out together
    const int64_t i = row * octets + (in ? o : 0);
    float h[8], w[8];
    load8<BF16>(p.x, i, h);
    if (p.res) {
      float r[8];
      load8<BF16>(p.res, i, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] += r[j];
      if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint32_t b = pack_bf16x2(h[j], h[j + 1]);
          h[j] = bf16_lo(b);
          h[j + 1] = bf16_hi(b);
        }
      }
    }
    load8<WBF16>(p.w, in ? o : 0, w);
    if (in && p.h) store8<BF16>(p.h, i, h);
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (in) sum = fmaf(h[j], h[j], sum);
      z[j] = h[j] * w[j];
    }
    if (in) quantize_octet<FP8>(z, i, static_cast<uint8_t*>(p.q), p.scales);
  }
  sum = wave_sum(sum);
  if (lane == 0) p.row_scale[row] = 1.0f / sqrtf(sum / (float)p.cols + p.eps);
}

struct NormGradArgs {
  const void* dy;
  const void* h;
  const void* dh;
  const void* w;
  const float* row_scale;
  void* dx;
  float* dot;        // [rows]: r^2 mean(g h)
  float* partial;    // [chunks, cols]
  float* dweight;
  int64_t rows;
  int cols;
  int64_t chunk_rows;
  int chunks;
};

template <bool BF16, bool WBF16>
__global__ __launch_bounds__(kThreads) void rmsnorm_dot_kernel(NormGradArgs p, int64_t blk0) {
  const int lane = threadIdx.x & 63;
  const int64_t row = ((int64_t)blockIdx.x + blk0) * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= p.rows) return;
  const int octets = p.cols >> 3;
  float sum = 0.0f;
  for (int o = lane; o < octets; o += 64) {
    float d[8], h[8], w[8];
    load8<BF16>(p.dy, row * octets + o, d);
    load8<BF16>(p.h, row * octets + o, h);
    load8<WBF16>(p.w, o, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(d[j] * w[j], h[j], sum);
  }
  sum = wave_sum(sum);
  const float r = p.row_scale[row];
  if (lane == 0) p.dot[row] = r * r * (sum / (float)p.cols);
}

// One workgroup per 2048 columns and chunk of rows; a thread owns 8 columns.
template <bool BF16, bool WBF16>
__global__ __launch_bounds__(kThreads) void rmsnorm_grad_kernel(NormGradArgs p) {
  const int octets = p.cols >> 3, o = blockIdx.x * kThreads + threadIdx.x;
  if (o >= octets) return;
  float w[8], acc[8] = {};
  load8<WBF16>(p.w, o, w);
  const int64_t r0 = blockIdx.y * p.chunk_rows, r1 = min(r0 + p.chunk_rows, p.rows);
  for (int64_t row = r0; row < r1; ++row) {
    const float r = p.row_scale[row], c = p.dot[row];
    float d[8], h[8], out[8];
    load8<BF16>(p.dy, row * octets + o, d);
    load8<BF16>(p.h, row * octets + o, h);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      out[j] = r * fmaf(-h[j], c, d[j] * w[j]);
      acc[j] = fmaf(d[j], h[j] * r, acc[j]);
    }
    if (p.dh) {
      float e[8];
      load8<BF16>(p.dh, row * octets + o, e);
#pragma unroll
      for (int j = 0; j < 8; ++j) out[j] += e[j];
    }
    store8<BF16>(p.dx, row * octets + o, out);
  }
  store8<false>(p.partial, (int64_t)blockIdx.y * octets + o, acc);
}

__global__ __launch_bounds__(kThreads) void rmsnorm_dweight_kernel(NormGradArgs p) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.cols) return;
  float s = 0.0f;
  for (int k = 0; k < p.chunks; ++k) s += p.partial[(int64_t)k * p.cols + c];
  p.dweight[c] = s;
}

int64_t grad_chunks(int64_t rows) { return rows < 512 ? (rows + 1) / 2 : 256; }

bool norm_shape_ok(int64_t rows, int64_t cols, int block, int64_t* n) {
  return rows >= 0 && cols > 0 && cols < (int64_t(1) << 21) && cols % block == 0 &&
         checked_count(rows, cols, n);
}

}  // namespace
}  // namespace fp4mi

using namespace fp4mi;

extern "C" int rmsnorm_quantize(const void* x, const void* residual, int dtype, const void* weight,
                                int weight_dtype, int64_t rows, int64_t cols, float eps, int fmt,
                                void* q, void* scales, float* row_scale, void* h, void* stream) {
  if (fmt != FP4_ROWS_MXFP4 && fmt != FP4_ROWS_FP8) return FP4_EINVAL;
  const int sz = dtype_size(dtype), wsz = dtype_size(weight_dtype);
  if (!sz || !wsz) return FP4_EDTYPE;
  if (!(eps >= 0.0f) || isinf(eps)) return FP4_EINVAL;
  const bool fp8 = fmt == FP4_ROWS_FP8;
  int64_t n;
  if (!norm_shape_ok(rows, cols, fp8 ? 128 : 32, &n)) return FP4_ESHAPE;
  if (n == 0) return FP4_OK;
  if (!x || !weight || !q || !scales || !row_scale) return FP4_EINVAL;
  if (!is_aligned(x, 16) || !is_aligned(residual, 16) || !is_aligned(weight, 16) ||
      !is_aligned(q, 16) || !is_aligned(scales, 4) || !is_aligned(row_scale, 4) ||
      !is_aligned(h, 16))
    return FP4_EALIGN;
  const void* ins[3] = {x, residual, weight};
  const int64_t inn[3] = {n * sz, n * sz, cols * wsz};
  const void* outs[4] = {q, scales, row_scale, h};
  const int64_t outn[4] = {fp8 ? n : n / 2, fp8 ? n / 128 * 4 : n / 32, rows * 4, n * sz};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 3; ++i) {
      if (o == 3 && i < 2 && h == ins[i]) continue;   // the sum in place of an addend
      if (overlaps(outs[o], outn[o], ins[i], inn[i])) return FP4_EOVERLAP;
    }
    for (int i = 0; i < o; ++i)
      if (overlaps(outs[o], outn[o], outs[i], outn[i])) return FP4_EOVERLAP;
  }
  const NormArgs p = {x, residual, weight, q, scales, row_scale, h, rows, (int)cols, eps};
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const int64_t blocks = (rows + kThreads / 64 - 1) / (kThreads / 64);
  auto go = [&](auto kernel) { launch_1d(kernel, blocks, kThreads, st, p); };
  const bool b = dtype == FP4_DTYPE_BF16, wb = weight_dtype == FP4_DTYPE_BF16;
  if (b && wb) fp8 ? go(rmsnorm_quantize_kernel<true, true, true>) : go(rmsnorm_quantize_kernel<true, true, false>);
  else if (b) fp8 ? go(rmsnorm_quantize_kernel<true, false, true>) : go(rmsnorm_quantize_kernel<true, false, false>);
  else if (wb) fp8 ? go(rmsnorm_quantize_kernel<false, true, true>) : go(rmsnorm_quantize_kernel<false, true, false>);
  else fp8 ? go(rmsnorm_quantize_kernel<false, false, true>) : go(rmsnorm_quantize_kernel<false, false, false>);
  return launch_status();
}

extern "C" int64_t rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  int64_t n;
  if (!norm_shape_ok(rows, cols, 32, &n) || n == 0) return 0;
  return ((rows + 3) / 4 * 4 + grad_chunks(rows) * cols) * 4;
}

extern "C" int rmsnorm_backward(const void* dy, const void* h, const void* dh, int dtype,
                                const void* weight, int weight_dtype, const float* row_scale,
                                int64_t rows, int64_t cols, void* dx, float* dweight,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  const int sz = dtype_size(dtype), wsz = dtype_size(weight_dtype);
  if (!sz || !wsz) return FP4_EDTYPE;
  int64_t n;
  if (!norm_shape_ok(rows, cols, 32, &n)) return FP4_ESHAPE;
  const int64_t need = rmsnorm_backward_workspace(rows, cols);
  if (!dweight) return FP4_EINVAL;
  if (n && (!dy || !h || !weight || !row_scale || !dx || !workspace)) return FP4_EINVAL;
  if (workspace_bytes < need) return FP4_ESHAPE;
  if (!is_aligned(dy, 16) || !is_aligned(h, 16) || !is_aligned(dh, 16) || !is_aligned(weight, 16) ||
      !is_aligned(row_scale, 4) || !is_aligned(dx, 16) || !is_aligned(dweight, 16) ||
      !is_aligned(workspace, 16))
    return FP4_EALIGN;
  const void* ins[5] = {dy, dh, h, weight, row_scale};
  const int64_t inn[5] = {n * sz, n * sz, n * sz, cols * wsz, rows * 4};
  const void* outs[3] = {dx, dweight, workspace};
  const int64_t outn[3] = {n * sz, cols * 4, need};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 5; ++i) {
      if (o == 0 && i < 2 && dx == ins[i]) continue;   // in place of a gradient
      if (overlaps(outs[o], outn[o], ins[i], inn[i])) return FP4_EOVERLAP;
    }
    for (int i = 0; i < o; ++i)
      if (overlaps(outs[o], outn[o], outs[i], outn[i])) return FP4_EOVERLAP;
  }
  NormGradArgs p = {dy, h, dh, weight, row_scale, dx, static_cast<float*>(workspace), nullptr,
                    dweight, rows, (int)cols, 1, n ? (int)grad_chunks(rows) : 0};
  p.partial = p.dot + (rows + 3) / 4 * 4;
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  if (n) {
    p.chunk_rows = (rows + p.chunks - 1) / p.chunks;
    const int64_t blocks = (rows + kThreads / 64 - 1) / (kThreads / 64);
    const dim3 grid((unsigned)((cols / 8 + kThreads - 1) / kThreads), (unsigned)p.chunks);
    auto go = [&](auto dot, auto grad) {
      launch_1d(dot, blocks, kThreads, st, p);
      hipLaunchKernelGGL(grad, grid, dim3(kThreads), 0, st, p);
    };
    const bool b = dtype == FP4_DTYPE_BF16, wb = weight_dtype == FP4_DTYPE_BF16;
    if (b && wb) go(rmsnorm_dot_kernel<true, true>, rmsnorm_grad_kernel<true, true>);
    else if (b) go(rmsnorm_dot_kernel<true, false>, rmsnorm_grad_kernel<true, false>);
    else if (wb) go(rmsnorm_dot_kernel<false, true>, rmsnorm_grad_kernel<false, true>);
    else go(rmsnorm_dot_kernel<false, false>, rmsnorm_grad_kernel<false, false>);
  }
  hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((unsigned)((cols + kThreads - 1) / kThreads)),
                     dim3(kThreads), 0, st, p);
  return launch_status();
}
