// SwiGLU into quantized rows with an 8-bit checkpoint, and its gradient.
#include "fp4mi_moe.h"
#include "host_common.hpp"
#include "rows_common.hpp"

namespace fp4mi {
namespace {

// s = 1 / (1 + exp(-g)), 0 where exp(-g) is past fp32, and 1 - s: for g > 0 as
// exp(-g) s, where the difference would lose what is left.
__device__ __forceinline__ float sigmoid(float g, float& rest) {
  const float e = exp_f32(-g), s = __builtin_amdgcn_rcpf(1.0f + e);
  rest = g > 0.0f ? e * s : 1.0f - s;
  return s;
}

// Row and octet of flat octet `i0 + local` of a tensor of d octets a row, from
// those of i0; local < kSpan.  i0 is the workgroup's, so its 64-bit division is
// scalar; magic = 2^32 / d rounded up is exact while (d + kSpan) d < 2^32, and a
// longer row is passed at most once.
constexpr int kSpan = 1024;
struct OctetPlace {
  int64_t row;
  int oct;
};
__device__ __forceinline__ OctetPlace place_of(int64_t row0, uint32_t oct0, uint32_t local, uint32_t d,
                                               uint32_t magic) {
  const uint32_t o = oct0 + local;
  const uint32_t q = d >= kSpan ? (o >= d ? 1u : 0u) : __umulhi(o, magic);
  return {row0 + q, (int)(o - q * d)};
}

struct SwigluArgs {
  const void* x;        // forward: [rows, 2 ffn]; backward: dy [rows, ffn]
  uint8_t* ckpt;
  float* ckpt_scales;
  void* q;
  void* scales;
  void* dx;
  int64_t octets;       // rows * ffn / 8
  uint32_t d, magic;    // ffn / 8
};

// A thread takes an octet of y: the octets of g and u, of the same row.  Lanes
// that share a block of y share blocks of g and u too.
template <bool BF16, bool FP8>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(SwigluArgs p, int64_t blk0) {
  constexpr int U = kSpan / kThreads / 2;
  const int64_t i0 = ((int64_t)blockIdx.x + blk0) * (kThreads * U);
  const int64_t row0 = i0 / p.d;
  const uint32_t oct0 = (uint32_t)(i0 - row0 * p.d);
  Octet<BF16> g[U], u[U];
  int64_t at[U];
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const uint32_t local = c * kThreads + threadIdx.x;
    const OctetPlace o = place_of(row0, oct0, local, p.d, p.magic);
    at[c] = o.row * (2 * (int64_t)p.d) + o.oct;
    if (i0 + local < p.octets) {
      g[c] = octet_load<BF16>(p.x, at[c]);
      u[c] = octet_load<BF16>(p.x, at[c] + p.d);
    }
  }
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const int64_t i = i0 + c * kThreads + threadIdx.x;
    if (i >= p.octets) continue;   // a block's lanes leave together
    float gv[8], uv[8], y[8];
    octet_values<BF16>(g[c], gv);
    octet_values<BF16>(u[c], uv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float rest;
      y[j] = gv[j] * sigmoid(gv[j], rest) * uv[j];
    }
    quantize_octet<FP8>(y, i, static_cast<uint8_t*>(p.q), p.scales);
    if (p.ckpt) {
      quantize_octet<true>(gv, at[c], p.ckpt, p.ckpt_scales);
      quantize_octet<true>(uv, at[c] + p.d, p.ckpt, p.ckpt_scales);
    }
  }
}

// Octet of codes times its block's scale.
__device__ __forceinline__ void kept_values(u32x2 c, float s, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], true);
    v[4 * h] = a.x * s;
    v[4 * h + 1] = a.y * s;
    v[4 * h + 2] = b.x * s;
    v[4 * h + 3] = b.y * s;
  }
}

// ROWS: 0 none, 1 MXFP4, 2 FP8.
template <bool BF16, int ROWS>
__global__ __launch_bounds__(kThreads) void swiglu_grad_kernel(SwigluArgs p, int64_t blk0) {
  constexpr int U = kSpan / kThreads / 2;
  const int64_t i0 = ((int64_t)blockIdx.x + blk0) * (kThreads * U);
  const int64_t row0 = i0 / p.d;
  const uint32_t oct0 = (uint32_t)(i0 - row0 * p.d);
  Octet<BF16> dy[U];
  u32x2 g[U], u[U];
  float gs[U], us[U];
  int64_t at[U];
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const uint32_t local = c * kThreads + threadIdx.x;
    const OctetPlace o = place_of(row0, oct0, local, p.d, p.magic);
    at[c] = o.row * (2 * (int64_t)p.d) + o.oct;
    if (i0 + local < p.octets) {
      dy[c] = octet_load<BF16>(p.x, i0 + local);
      g[c] = *reinterpret_cast<const u32x2*>(p.ckpt + 8 * at[c]);
      u[c] = *reinterpret_cast<const u32x2*>(p.ckpt + 8 * (at[c] + p.d));
      gs[c] = p.ckpt_scales[at[c] >> 4];
      us[c] = p.ckpt_scales[(at[c] + p.d) >> 4];
    }
  }
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const int64_t i = i0 + c * kThreads + threadIdx.x;
    if (i >= p.octets) continue;
    float dv[8], gv[8], uv[8];
    octet_values<BF16>(dy[c], dv);
    kept_values(g[c], gs[c], gv);
    kept_values(u[c], us[c], uv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float rest;
      const float s = sigmoid(gv[j], rest), du = dv[j] * gv[j] * s;
      gv[j] = dv[j] * uv[j] * s * fmaf(gv[j], rest, 1.0f);
      uv[j] = du;
    }
    if (ROWS == 0 || p.dx) {
      store8<BF16>(p.dx, at[c], gv);
      store8<BF16>(p.dx, at[c] + p.d, uv);
    }
    if constexpr (ROWS != 0) {
      quantize_octet<ROWS == 2>(gv, at[c], static_cast<uint8_t*>(p.q), p.scales);
      quantize_octet<ROWS == 2>(uv, at[c] + p.d, static_cast<uint8_t*>(p.q), p.scales);
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

SwigluArgs swiglu_args(const void* x, int64_t rows, int64_t ffn) {
  SwigluArgs p = {};
  p.x = x;
  p.d = (uint32_t)(ffn / 8);
  p.magic = (uint32_t)(((uint64_t(1) << 32) + p.d - 1) / p.d);
  p.octets = rows * (ffn / 8);
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
  SwigluArgs p = swiglu_args(x, rows, ffn);
  p.q = q;
  p.scales = scales;
  p.ckpt = ckpt;
  p.ckpt_scales = ckpt_scales;
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const int64_t blocks = (p.octets + kSpan / 2 - 1) / (kSpan / 2);
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
  SwigluArgs p = swiglu_args(dy, rows, ffn);
  p.ckpt = const_cast<uint8_t*>(ckpt);
  p.ckpt_scales = const_cast<float*>(ckpt_scales);
  p.dx = dx;
  p.q = q;
  p.scales = scales;
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const int64_t blocks = (p.octets + kSpan / 2 - 1) / (kSpan / 2);
  const bool bf16 = dtype == FP4_DTYPE_BF16;
  const int rows_fmt = !q ? 0 : (fmt == FP4_ROWS_FP8 ? 2 : 1);
  void (*kernels[2][3])(SwigluArgs, int64_t) = {
      {swiglu_grad_kernel<false, 0>, swiglu_grad_kernel<false, 1>, swiglu_grad_kernel<false, 2>},
      {swiglu_grad_kernel<true, 0>, swiglu_grad_kernel<true, 1>, swiglu_grad_kernel<true, 2>}};
  launch_1d(kernels[bf16][rows_fmt], blocks, kThreads, st, p);
  return launch_status();
}
