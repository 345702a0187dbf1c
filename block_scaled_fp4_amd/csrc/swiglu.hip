// SwiGLU into quantized rows with an 8-bit checkpoint, and its gradient.
#include <string.h>

#include "fp4mi_moe.h"
#include "host_common.hpp"
#include "rows_common.hpp"

namespace fp4mi {
namespace {

// s = 1 / (1 + exp(-g)), 0 where exp(-g) is past fp32, and `rest` = 1 - s as exp(-g) s:
// the difference would lose what is left for large g, and where s is 0 nothing takes
// it.  BF16: g has 9 significant bits at most, so its product with the first 15 of
// log2(e) is exact, and exp2 of it lacks of exp(-g) the factor 1 - g L, L = ln 2 times
// the rest of log2(e) (|g L| < 2^-11, half its square is below 2^-23).  Without
// it e is off by |g| 2^-24 of itself; with it the gradient of 65536 x 2048 into FP8 rows, which
// instructions bound, takes 135 us for 130, into bf16 159 both.  FINITE: g is a
// checkpoint's, a number or NaN.
template <bool BF16, bool FINITE>
__device__ __forceinline__ float sigmoid(float g, float& rest) {
  float e;
  if constexpr (BF16) {
    e = __builtin_amdgcn_exp2f(g * -0x1.7154p+0f);
    const float more = g * -0x1.480fb6p-18f;
    e = fmaf(e, FINITE ? more : fmaxf(more, -1.0f), e);   // e is 0 where g is infinite
  } else {
    e = exp_f32(-g);
  }
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  rest = __uint_as_float(min(__float_as_uint(e), 0x7F7FFFFFu)) * s;   // not 0 times infinity
  return s;
}

// Row and part of flat part `i0 + local` of a tensor of d parts a row, from those of
// i0 (the workgroup's, so its 64-bit division is scalar); local < kSpan.  magic = 2^32
// / d rounded up gives the quotient or, of operands below 2^20, one more.
constexpr int kSpan = 512;   // parts a workgroup
struct Place {
  int64_t row;
  int part;
};
__device__ __forceinline__ Place place_of(int64_t row0, uint32_t part0, uint32_t local, uint32_t d, uint32_t magic) {
  const uint32_t o = part0 + local, q = __umulhi(o, magic);
  const int part = (int)(o - q * d);
  return {row0 + q - (part < 0 ? 1 : 0), part < 0 ? part + (int)d : part};
}

struct SwigluArgs {
  const void* x;        // forward: [rows, 2 ffn]; backward: dy [rows, ffn]
  uint8_t* ckpt;
  float* ckpt_scales;
  void* q;
  void* scales;
  void* dx;
  int64_t parts;        // of 16 bytes of dtype in rows * ffn
  uint32_t d, magic;    // parts of ffn
};

// A thread takes a part of y: those of g and u, of the same row.  Lanes that share
// a block of y share blocks of g and u too.  Bound by memory: 65536 x 2048 bf16 with
// the checkpoint 7.1 bytes a pair, 140 us (6.8 TB/s); the checkpoint is stored past the
// caches, where it would push out y (170 us before), and the maxima of a block meet
// as integers (each step one instruction).
template <bool BF16, bool FP8>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(SwigluArgs p, int64_t blk0) {
  constexpr int U = kSpan / kThreads, V = Part<BF16>::kValues;
  const int64_t i0 = ((int64_t)blockIdx.x + blk0) * kSpan;
  const int64_t row0 = i0 / p.d;
  const uint32_t part0 = (uint32_t)(i0 - row0 * p.d);
  u32x4 g[U], u[U];
  int64_t at[U];
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const uint32_t local = c * kThreads + threadIdx.x;
    const Place o = place_of(row0, part0, local, p.d, p.magic);
    at[c] = o.row * (2 * (int64_t)p.d) + o.part;
    if (i0 + local < p.parts) {
      g[c] = ld_u32x4(static_cast<const u32x4*>(p.x) + at[c]);
      u[c] = ld_u32x4(static_cast<const u32x4*>(p.x) + at[c] + p.d);
    }
  }
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const int64_t i = i0 + c * kThreads + threadIdx.x;
    if (i >= p.parts) continue;   // a block's lanes leave together
    float gv[V], uv[V], y[V];
    part_values<BF16>(g[c], gv);
    part_values<BF16>(u[c], uv);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float rest;
      y[j] = gv[j] * sigmoid<BF16, false>(gv[j], rest) * uv[j];
    }
    quantize_part<FP8, false, V>(y, i, static_cast<uint8_t*>(p.q), p.scales);
    if (p.ckpt) {
      quantize_part<true, true, V>(gv, at[c], p.ckpt, p.ckpt_scales);
      quantize_part<true, true, V>(uv, at[c] + p.d, p.ckpt, p.ckpt_scales);
    }
  }
}

// V codes from part i of the checkpoint times their block's scale.
template <int V>
struct Kept {
  uint32_t c[V / 4];
  float s;
};
template <int V>
__device__ __forceinline__ Kept<V> kept_load(const uint8_t* codes, const float* scales, int64_t i) {
  Kept<V> k;
  memcpy(k.c, __builtin_assume_aligned(codes + i * V, V), V);
  k.s = scales[i / (128 / V)];
  return k;
}
template <int V>
__device__ __forceinline__ void kept_values(const Kept<V>& k, float (&v)[V]) {
#pragma unroll
  for (int h = 0; h < V / 4; ++h) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)k.c[h], false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)k.c[h], true);
    v[4 * h] = a.x * k.s;
    v[4 * h + 1] = a.y * k.s;
    v[4 * h + 2] = b.x * k.s;
    v[4 * h + 3] = b.y * k.s;
  }
}
template <bool BF16>
__device__ __forceinline__ void part_store(void* base, int64_t i, const float (&v)[Part<BF16>::kValues]) {
  if constexpr (BF16) {
    store8<true>(base, i, v);
  } else {
    st_u32x4(static_cast<u32x4*>(base) + i, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                  __float_as_uint(v[2]), __float_as_uint(v[3])});
  }
}

// ROWS: 0 none, 1 MXFP4, 2 FP8.  20011 x 2176 into bf16 54 us (6.5 TB/s); 65536 x 2048
// into FP8 rows 135 us (6.1 TB/s; with the rows stored through the caches 12 more), into
// MXFP4 rows 123 us (5.6 TB/s).
template <bool BF16, int ROWS>
__global__ __launch_bounds__(kThreads) void swiglu_grad_kernel(SwigluArgs p, int64_t blk0) {
  constexpr int U = kSpan / kThreads, V = Part<BF16>::kValues;
  const int64_t i0 = ((int64_t)blockIdx.x + blk0) * kSpan;
  const int64_t row0 = i0 / p.d;
  const uint32_t part0 = (uint32_t)(i0 - row0 * p.d);
  u32x4 dy[U];
  Kept<V> g[U], u[U];
  int64_t at[U];
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const uint32_t local = c * kThreads + threadIdx.x;
    const Place o = place_of(row0, part0, local, p.d, p.magic);
    at[c] = o.row * (2 * (int64_t)p.d) + o.part;
    if (i0 + local < p.parts) {
      dy[c] = ld_u32x4(static_cast<const u32x4*>(p.x) + i0 + local);
      g[c] = kept_load<V>(p.ckpt, p.ckpt_scales, at[c]);
      u[c] = kept_load<V>(p.ckpt, p.ckpt_scales, at[c] + p.d);
    }
  }
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const int64_t i = i0 + c * kThreads + threadIdx.x;
    if (i >= p.parts) continue;
    float dv[V], gv[V], uv[V];
    part_values<BF16>(dy[c], dv);
    kept_values<V>(g[c], gv);
    kept_values<V>(u[c], uv);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float rest;
      const float d = dv[j] * sigmoid<BF16, true>(gv[j], rest), du = d * gv[j];
      gv[j] = d * uv[j] * fmaf(gv[j], rest, 1.0f);
      uv[j] = du;
    }
    if (ROWS == 0 || p.dx) {
      part_store<BF16>(p.dx, at[c], gv);
      part_store<BF16>(p.dx, at[c] + p.d, uv);
    }
    if constexpr (ROWS != 0) {
      quantize_part<ROWS == 2, true, V>(gv, at[c], static_cast<uint8_t*>(p.q), p.scales);
      quantize_part<ROWS == 2, true, V>(uv, at[c] + p.d, static_cast<uint8_t*>(p.q), p.scales);
    }
  }
}

// Bytes of the codes and scales of n values in rows of format fmt.
int64_t code_bytes(int64_t n, int fmt) { return fmt == FP4_ROWS_FP8 ? n : n / 2; }
int64_t scale_bytes(int64_t n) { return n / 32; }   // a byte for 32 values, or four for 128

bool any_overlap(const void* const* outs, const int64_t* outn, int no, const void* const* ins,
                 const int64_t* inn, int ni) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j)
      if (overlaps(outs[i], outn[i], ins[j], inn[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outn[i], outs[j], outn[j])) return true;
  }
  return false;
}

SwigluArgs swiglu_args(const void* x, int isz, int64_t rows, int64_t ffn) {
  SwigluArgs p = {};
  p.x = x;
  p.d = (uint32_t)(ffn * isz / 16);
  p.magic = (uint32_t)(((uint64_t(1) << 32) + p.d - 1) / p.d);
  p.parts = rows * p.d;
  return p;
}

}  // namespace
}  // namespace fp4mi

using namespace fp4mi;

extern "C" int swiglu_quantize(const void* x, int dtype, int64_t rows, int64_t ffn, int fmt, void* q,
                               void* scales, uint8_t* ckpt, float* ckpt_scales, void* stream) {
  const int isz = dtype_size(dtype);
  if (!isz) return FP4_EDTYPE;
  if (fmt != FP4_ROWS_MXFP4 && fmt != FP4_ROWS_FP8) return FP4_EINVAL;
  if (!ckpt != !ckpt_scales) return FP4_EINVAL;
  int64_t n, n2;
  if (ffn <= 0 || ffn >= (int64_t(1) << 20) || ffn % (fmt == FP4_ROWS_FP8 || ckpt ? 128 : 32) ||
      !checked_count(rows, ffn, &n) || !checked_count(rows, 2 * ffn, &n2))
    return FP4_ESHAPE;
  if (n == 0) return FP4_OK;
  if (!x || !q || !scales) return FP4_EINVAL;
  if (!is_aligned(x, 16) || !is_aligned(q, 16) || !is_aligned(scales, 4) || !is_aligned(ckpt, 16) ||
      !is_aligned(ckpt_scales, 4))
    return FP4_EALIGN;
  const void* outs[4] = {q, scales, ckpt, ckpt_scales};
  const int64_t outn[4] = {code_bytes(n, fmt), scale_bytes(n), n2, scale_bytes(n2)}, inn = n2 * isz;
  if (any_overlap(outs, outn, 4, &x, &inn, 1)) return FP4_EOVERLAP;
  SwigluArgs p = swiglu_args(x, isz, rows, ffn);
  p.q = q;
  p.scales = scales;
  p.ckpt = ckpt;
  p.ckpt_scales = ckpt_scales;
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const int64_t blocks = (p.parts + kSpan - 1) / kSpan;
  const bool bf16 = dtype == FP4_DTYPE_BF16, fp8 = fmt == FP4_ROWS_FP8;
  launch_1d(bf16 ? (fp8 ? swiglu_kernel<true, true> : swiglu_kernel<true, false>)
                 : (fp8 ? swiglu_kernel<false, true> : swiglu_kernel<false, false>),
            blocks, kThreads, st, p);
  return launch_status();
}

extern "C" int swiglu_backward(const void* dy, int dtype, const uint8_t* ckpt,
                               const float* ckpt_scales, int64_t rows, int64_t ffn, void* dx, int fmt,
                               void* q, void* scales, void* stream) {
  const int isz = dtype_size(dtype);
  if (!isz) return FP4_EDTYPE;
  if (q && fmt != FP4_ROWS_MXFP4 && fmt != FP4_ROWS_FP8) return FP4_EINVAL;
  if (!q != !scales) return FP4_EINVAL;
  int64_t n, n2;
  if (ffn <= 0 || ffn >= (int64_t(1) << 20) || ffn % 128 || !checked_count(rows, ffn, &n) ||
      !checked_count(rows, 2 * ffn, &n2))
    return FP4_ESHAPE;
  if (n == 0) return FP4_OK;
  if (!dy || !ckpt || !ckpt_scales || (!dx && !q)) return FP4_EINVAL;
  if (!is_aligned(dy, 16) || !is_aligned(ckpt, 16) || !is_aligned(ckpt_scales, 4) ||
      !is_aligned(dx, 16) || !is_aligned(q, 16) || !is_aligned(scales, 4))
    return FP4_EALIGN;
  const void *outs[3] = {dx, q, scales}, *ins[3] = {dy, ckpt, ckpt_scales};
  const int64_t outn[3] = {n2 * isz, code_bytes(n2, fmt), scale_bytes(n2)};
  const int64_t inn[3] = {n * isz, n2, scale_bytes(n2)};
  if (any_overlap(outs, outn, 3, ins, inn, 3)) return FP4_EOVERLAP;
  SwigluArgs p = swiglu_args(dy, isz, rows, ffn);
  p.ckpt = const_cast<uint8_t*>(ckpt);
  p.ckpt_scales = const_cast<float*>(ckpt_scales);
  p.dx = dx;
  p.q = q;
  p.scales = scales;
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const int64_t blocks = (p.parts + kSpan - 1) / kSpan;
  const bool bf16 = dtype == FP4_DTYPE_BF16;
  const int rows_fmt = !q ? 0 : (fmt == FP4_ROWS_FP8 ? 2 : 1);
  void (*kernels[2][3])(SwigluArgs, int64_t) = {
      {swiglu_grad_kernel<false, 0>, swiglu_grad_kernel<false, 1>, swiglu_grad_kernel<false, 2>},
      {swiglu_grad_kernel<true, 0>, swiglu_grad_kernel<true, 1>, swiglu_grad_kernel<true, 2>}};
  launch_1d(kernels[bf16][rows_fmt], blocks, kThreads, st, p);
  return launch_status();
}
