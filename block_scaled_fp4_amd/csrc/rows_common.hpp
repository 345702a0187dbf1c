// Shared by the kernels that write quantized rows: octets of a row, sums and
// maxima over lanes, and the codes and scales of a block.
#pragma once

#include "device_common.hpp"

namespace fp4mi {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// exp(x), 2 units in the last place: exp2 of the rounded x log2(e), corrected by
// the part of it that the rounding lost (without, the error grows with |x|).
__device__ __forceinline__ float exp_f32(float x) {
  const float t = x * 0x1.715476p+0f;
  const float lost = fmaf(x, 0x1.4ae0cp-26f, fmaf(x, 0x1.715476p+0f, -t));
  const float e = __builtin_amdgcn_exp2f(t) * fmaf(lost, 0x1.62e43p-1f, 1.0f);
  return t < -150.0f ? 0.0f : e;   // of -inf too, where `lost` is NaN
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

// The block's scale 2^k, 2^-127 where all are zero.
__device__ __forceinline__ float fp8_scale(float amax, int k) {
  return amax > 0.0f ? __uint_as_float((uint32_t)(k + 127) << 23) : 0x1p-127f;
}
// Eight E4M3 codes of z / 2^k, to nearest even.  |z| <= 448 * 2^k: nothing
// saturates; infinities and NaN become NaN codes.
__device__ __forceinline__ u32x2 fp8_codes8(const float (&z)[8], int k) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_ldexpf(z[j], -k);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  return u32x2{(uint32_t)lo, (uint32_t)hi};
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
  if constexpr (FP8) {
    const int k = fp8_block_exponent(am);
    *reinterpret_cast<u32x2*>(q + 8 * i) = fp8_codes8(z, k);
    if ((i & 15) == 0) static_cast<float*>(scales)[i >> 4] = fp8_scale(am, k);
  } else {
    const int b = max((int)(__float_as_uint(am) >> 23) - 2, 0);   // floor(log2 amax) - 2 + 127
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_ldexpf(z[j], 127 - b);
    *reinterpret_cast<uint32_t*>(q + 4 * i) = rtn8_unit(v);
    if ((i & 3) == 0) static_cast<uint8_t*>(scales)[i >> 2] = (uint8_t)b;
  }
}

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

}  // namespace fp4mi
