// RMS norm with residual addition and quantized rows, and its gradient.
#include <math.h>

#include <algorithm>
#include <type_traits>

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

// Loads and stores of octet i, kept raw until they are needed.
template <bool BF16>
struct Octet {
  u32x4 a, b;   // bf16: a alone
};
template <bool BF16>
__device__ __forceinline__ Octet<BF16> octet_load(const void* base, int64_t i) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i * (BF16 ? 16 : 32);
  Octet<BF16> o;
  o.a = ld_u32x4(p);
  if constexpr (!BF16) o.b = ld_u32x4(p + 16);
  return o;
}
template <bool BF16>
__device__ __forceinline__ void octet_values(const Octet<BF16>& o, float (&v)[8]) {
  if constexpr (BF16) {
    v[0] = bf16_lo(o.a.x); v[1] = bf16_hi(o.a.x); v[2] = bf16_lo(o.a.y); v[3] = bf16_hi(o.a.y);
    v[4] = bf16_lo(o.a.z); v[5] = bf16_hi(o.a.z); v[6] = bf16_lo(o.a.w); v[7] = bf16_hi(o.a.w);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(o.a[j]);
      v[4 + j] = __uint_as_float(o.b[j]);
    }
  }
}
// Weights are read by every workgroup: a plain load keeps them cached.
template <bool BF16>
__device__ __forceinline__ void load_weights(const void* base, int i, float (&v)[8]) {
  Octet<BF16> o;
  const uint8_t* p = static_cast<const uint8_t*>(base) + (int64_t)i * (BF16 ? 16 : 32);
  o.a = ld_u32x4_keep(p);
  if constexpr (!BF16) o.b = ld_u32x4_keep(p + 16);
  octet_values<BF16>(o, v);
}

// h of one octet: the sum rounded to the row's type.
template <bool BF16>
__device__ __forceinline__ void residual_sum(const Octet<BF16>& x, const Octet<BF16>& res, bool has,
                                             float (&h)[8]) {
  octet_values<BF16>(x, h);
  if (!has) return;
  float r[8];
  octet_values<BF16>(res, r);
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

// A workgroup owns whole rows, a thread the octets tid, tid + T, .. of each:
// its weights stay in registers, and as neither codes nor block scales wait for
// the row's mean, rows follow each other without a barrier.  The waves' sums of
// squares meet in LDS at the end, in a fixed order.  Bound by memory: bf16 rows
// with a residual move 7 bytes an element, 16384 x 7168 in 130 us (6.3 TB/s; with
// a wave per row and the weights read for each it was 181).
constexpr int kNormRows = 32;   // rows of a workgroup at most
template <bool BF16, bool WBF16, bool FP8, int CH>
__global__ __launch_bounds__(1024) void rmsnorm_quantize_kernel(NormArgs p, int rows_per, int64_t blk0) {
  __shared__ float sums[kNormRows][16];
  const int tid = threadIdx.x, T = blockDim.x, octets = p.cols >> 3;
  const int64_t r0 = ((int64_t)blockIdx.x + blk0) * rows_per;
  const int rows = (int)min((int64_t)rows_per, p.rows - r0);
  float w[CH][8];
  Octet<BF16> x[CH], e[CH];
  auto fetch = [&](int row) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int o = tid + c * T;
      if (o >= octets) continue;
      x[c] = octet_load<BF16>(p.x, (r0 + row) * octets + o);
      if (p.res) e[c] = octet_load<BF16>(p.res, (r0 + row) * octets + o);
    }
  };
  fetch(0);
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (tid + c * T < octets) load_weights<WBF16>(p.w, tid + c * T, w[c]);
  for (int row = 0; row < rows; ++row) {
    float h[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) residual_sum<BF16>(x[c], e[c], p.res != nullptr, h[c]);
    if (row + 1 < rows) fetch(row + 1);
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int o = tid + c * T;
      if (o >= octets) continue;   // whole blocks are in or out together
      const int64_t i = (r0 + row) * octets + o;
      float z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = fmaf(h[c][j], h[c][j], sum);
        z[j] = h[c][j] * w[c][j];
      }
      if (p.h) store8<BF16>(p.h, i, h[c]);
      quantize_octet<FP8>(z, i, static_cast<uint8_t*>(p.q), p.scales);
    }
    sum = wave_sum(sum);
    if ((tid & 63) == 0) sums[row][tid >> 6] = sum;
  }
  __syncthreads();
  if (tid < rows) {
    float s = 0.0f;
    for (int k = 0; k < T / 64; ++k) s += sums[tid][k];
    p.row_scale[r0 + tid] = 1.0f / sqrtf(s / (float)p.cols + p.eps);
  }
}

// Rows too long for a workgroup's registers: one workgroup per row, octet by
// octet.
template <bool BF16, bool WBF16, bool FP8>
__global__ __launch_bounds__(1024) void rmsnorm_quantize_long_kernel(NormArgs p, int64_t blk0) {
  __shared__ float sums[16];
  const int tid = threadIdx.x, octets = p.cols >> 3;
  const int64_t row = (int64_t)blockIdx.x + blk0;
  float sum = 0.0f;
  for (int o = tid; o < octets; o += 1024) {   // a block's lanes leave together
    const int64_t i = row * octets + o;
    Octet<BF16> x = octet_load<BF16>(p.x, i), e = x;
    if (p.res) e = octet_load<BF16>(p.res, i);
    float h[8], w[8], z[8];
    residual_sum<BF16>(x, e, p.res != nullptr, h);
    load_weights<WBF16>(p.w, o, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(h[j], h[j], sum);
      z[j] = h[j] * w[j];
    }
    if (p.h) store8<BF16>(p.h, i, h);
    quantize_octet<FP8>(z, i, static_cast<uint8_t*>(p.q), p.scales);
  }
  sum = wave_sum(sum);
  if ((tid & 63) == 0) sums[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) {
    float s = 0.0f;
    for (int k = 0; k < 16; ++k) s += sums[k];
    p.row_scale[row] = 1.0f / sqrtf(s / (float)p.cols + p.eps);
  }
}

struct NormGradArgs {
  const void* dy;
  const void* h;
  const void* dh;
  const void* w;
  const float* row_scale;
  void* dx;
  float* dot;        // [rows]: r^2 mean(g h), long rows only
  float* partial;    // [chunks, cols]
  float* dweight;
  int64_t rows;
  int cols;
  int64_t chunk_rows;
  int chunks;
};

// Gradient, rows owned as above: a row's dy and h stay in registers between
// the sum of g h and dx, so every input is read once; the next row's loads are
// in flight over the one barrier a row needs.  A thread adds its columns' dy h r
// over its rows, and each workgroup leaves one row of partial sums.  16384 x 7168
// bf16 with dh in 187 us (5.0 TB/s; 382 in two passes over dy and h).
template <bool BF16, bool WBF16, int CH>
__global__ __launch_bounds__(1024) void rmsnorm_grad_kernel(NormGradArgs p) {
  __shared__ float sums[2][16];
  const int tid = threadIdx.x, T = blockDim.x, octets = p.cols >> 3;
  const int64_t r0 = blockIdx.x * p.chunk_rows, r1 = min(r0 + p.chunk_rows, p.rows);
  float w[CH][8], acc[CH][8] = {};
  Octet<BF16> d[CH], h[CH], e[CH];
  float r = 0.0f;
  auto fetch = [&](int64_t row) {
    r = p.row_scale[row];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int o = tid + c * T;
      if (o >= octets) continue;
      d[c] = octet_load<BF16>(p.dy, row * octets + o);
      h[c] = octet_load<BF16>(p.h, row * octets + o);
      if (p.dh) e[c] = octet_load<BF16>(p.dh, row * octets + o);
    }
  };
  if (r0 < r1) fetch(r0);
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (tid + c * T < octets) load_weights<WBF16>(p.w, tid + c * T, w[c]);
  for (int64_t row = r0; row < r1; ++row) {
    const Octet<BF16> (&dc)[CH] = d;
    float sum = 0.0f;
    Octet<BF16> dk[CH], hk[CH], ek[CH];
    const float rk = r;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      dk[c] = dc[c];
      hk[c] = h[c];
      ek[c] = e[c];
      if (tid + c * T >= octets) continue;
      float dv[8], hv[8];
      octet_values<BF16>(dk[c], dv);
      octet_values<BF16>(hk[c], hv);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(dv[j] * w[c][j], hv[j], sum);
    }
    if (row + 1 < r1) fetch(row + 1);
    sum = wave_sum(sum);
    const int b = (int)(row - r0) & 1;   // the other row's sums may still be read
    if ((tid & 63) == 0) sums[b][tid >> 6] = sum;
    __syncthreads();
    float s = 0.0f;
    for (int k = 0; k < T / 64; ++k) s += sums[b][k];
    const float dot = rk * rk * (s / (float)p.cols);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int o = tid + c * T;
      if (o >= octets) continue;
      float dv[8], hv[8], out[8];
      octet_values<BF16>(dk[c], dv);
      octet_values<BF16>(hk[c], hv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        out[j] = rk * fmaf(-hv[j], dot, dv[j] * w[c][j]);
        acc[c][j] = fmaf(dv[j], hv[j] * rk, acc[c][j]);
      }
      if (p.dh) {
        float ev[8];
        octet_values<BF16>(ek[c], ev);
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] += ev[j];
      }
      store8<BF16>(p.dx, row * octets + o, out);
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (tid + c * T < octets)
      store8<false>(p.partial, (int64_t)blockIdx.x * octets + tid + c * T, acc[c]);
}

// Long rows: the dot products first (one workgroup per row), then columns.
template <bool BF16, bool WBF16>
__global__ __launch_bounds__(1024) void rmsnorm_dot_kernel(NormGradArgs p, int64_t blk0) {
  __shared__ float sums[16];
  const int tid = threadIdx.x, octets = p.cols >> 3;
  const int64_t row = (int64_t)blockIdx.x + blk0;
  float sum = 0.0f;
  for (int o = tid; o < octets; o += 1024) {
    float d[8], h[8], w[8];
    load8<BF16>(p.dy, row * octets + o, d);
    load8<BF16>(p.h, row * octets + o, h);
    load_weights<WBF16>(p.w, o, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(d[j] * w[j], h[j], sum);
  }
  sum = wave_sum(sum);
  if ((tid & 63) == 0) sums[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) {
    float s = 0.0f;
    for (int k = 0; k < 16; ++k) s += sums[k];
    const float r = p.row_scale[row];
    p.dot[row] = r * r * (s / (float)p.cols);
  }
}

// One workgroup per 2048 columns and chunk of rows; a thread owns 8 columns.
template <bool BF16, bool WBF16>
__global__ __launch_bounds__(kThreads) void rmsnorm_grad_long_kernel(NormGradArgs p) {
  const int octets = p.cols >> 3, o = blockIdx.x * kThreads + threadIdx.x;
  if (o >= octets) return;
  float w[8], acc[8] = {};
  load_weights<WBF16>(p.w, o, w);
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

// Sum of the chunks' partial sums: 64 columns a workgroup, 16 waves each taking
// every 16th chunk.
__global__ __launch_bounds__(1024) void rmsnorm_dweight_kernel(NormGradArgs p) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < p.cols) {
#pragma unroll 8
    for (int k = wave; k < p.chunks; k += 16) s += p.partial[(int64_t)k * p.cols + c];
  }
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < p.cols) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += part[k][lane];
    p.dweight[c] = s;
  }
}

// Threads and octets a thread for rows of `octets` (up to 16384 columns; with
// more octets the registers of 1024 threads run out); 0 octets: too long.  The
// gradient of fp32 rows keeps registers in scratch with two octets already, as
// it is built for 1024 threads (16384 x 7168 in 706 us, 2.7 TB/s).
struct RowShape {
  int threads, ch;
};
RowShape row_shape(int octets) {
  for (int ch = 1; ch <= 2; ++ch) {
    const int t = ((octets + ch - 1) / ch + 63) / 64 * 64;
    if (t <= 512 * ch) return {t, ch};
  }
  return {1024, 0};
}

// Chunks of rows of the gradient: one partial sum of dweight each, written and
// read again, so no more than keep the card busy.
int64_t grad_chunks(int64_t rows) { return rows < 1024 ? (rows + 1) / 2 : 512; }

// f(is x bf16, are the weights) as types
template <typename F>
void by_types(int dtype, int weight_dtype, F f) {
  constexpr std::true_type y{};
  constexpr std::false_type n{};
  const bool b = dtype == FP4_DTYPE_BF16, w = weight_dtype == FP4_DTYPE_BF16;
  if (b) w ? f(y, y) : f(y, n);
  else w ? f(n, y) : f(n, n);
}

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
  const RowShape sh = row_shape((int)cols / 8);
  // enough workgroups to fill the card first, then rows that share the weights
  const int per = (int)std::min<int64_t>(kNormRows, std::max<int64_t>(1, rows / 2048));
  auto go = [&](auto bf16, auto wbf16, auto f8) {
    constexpr bool B = decltype(bf16)::value, W = decltype(wbf16)::value, F = decltype(f8)::value;
    const int64_t blocks = (rows + per - 1) / per;
    if (sh.ch == 1) launch_1d(rmsnorm_quantize_kernel<B, W, F, 1>, blocks, sh.threads, st, p, per);
    else if (sh.ch == 2) launch_1d(rmsnorm_quantize_kernel<B, W, F, 2>, blocks, sh.threads, st, p, per);
    else launch_1d(rmsnorm_quantize_long_kernel<B, W, F>, rows, 1024, st, p);
  };
  by_types(dtype, weight_dtype, [&](auto b, auto w) { fp8 ? go(b, w, std::true_type()) : go(b, w, std::false_type()); });
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
    const RowShape sh = row_shape((int)cols / 8);
    by_types(dtype, weight_dtype, [&](auto bf16, auto wbf16) {
      constexpr bool B = decltype(bf16)::value, W = decltype(wbf16)::value;
      const dim3 grid((unsigned)p.chunks), thr((unsigned)sh.threads);
      if (sh.ch == 1) hipLaunchKernelGGL((rmsnorm_grad_kernel<B, W, 1>), grid, thr, 0, st, p);
      else if (sh.ch == 2) hipLaunchKernelGGL((rmsnorm_grad_kernel<B, W, 2>), grid, thr, 0, st, p);
      else {
        launch_1d(rmsnorm_dot_kernel<B, W>, rows, 1024, st, p);
        hipLaunchKernelGGL((rmsnorm_grad_long_kernel<B, W>),
                           dim3((unsigned)((cols / 8 + kThreads - 1) / kThreads), (unsigned)p.chunks),
                           dim3(kThreads), 0, st, p);
      }
    });
  }
  hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, st,
                     p);
  return launch_status();
}
