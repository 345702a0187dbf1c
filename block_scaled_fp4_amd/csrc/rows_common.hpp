// Shared by the kernels that write quantized rows: octets of a row, sums and
// maxima over lanes, and the codes and scales of a block.
#pragma once

#include "lane_common.hpp"

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

// Largest v >= 0 over the L lanes (4 to 32) that share a quantization block.  As
// integers: floats would each be made canonical first.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  uint32_t u = __float_as_uint(v);
  u = max(u, lane_dpp<0xB1>(u));
  u = max(u, lane_dpp<0x4E>(u));
  if constexpr (L >= 8) u = max(u, lane_dpp<0x141>(u));
  if constexpr (L >= 16) u = max(u, lane_dpp<0x140>(u));
  if constexpr (L == 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    u = max(p[0], p[1]);
  }
  return __uint_as_float(u);
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
// Four or eight E4M3 codes of z / 2^k, to nearest even.  |z| <= 448 * 2^k: nothing
// saturates; infinities and NaN become NaN codes.
__device__ __forceinline__ uint32_t fp8_codes4(const float* z, int k) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  const float scale = __uint_as_float((uint32_t)(k + 127) << 23);
  s16x2 c = {0, 0};
  c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, z[0], z[1], scale, false);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, z[2], z[3], scale, true);
  return __builtin_bit_cast(uint32_t, c);
}
__device__ __forceinline__ u32x2 fp8_codes8(const float (&z)[8], int k) {
  return u32x2{fp8_codes4(z, k), fp8_codes4(z + 4, k)};
}

// V (4 or 8) values z of a row -> their codes; the block's first lane stores the
// scale.  i: index of the V in the tensor.  NT: the codes are not read again soon.
template <bool FP8, bool NT, int V>
__device__ __forceinline__ void quantize_part(const float (&z)[V], int64_t i, uint8_t* q, void* scales) {
  constexpr int L = (FP8 ? 128 : 32) / V;   // lanes of a block
  float am = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) am = fmaxf(am, fabsf(z[j]));
  am = lanes_max<L>(am);
  auto put = [&](auto codes) {
    auto* to = reinterpret_cast<decltype(codes)*>(q + (int64_t)sizeof(codes) * i);
    if constexpr (NT) __builtin_nontemporal_store(codes, to);
    else *to = codes;
  };
  if constexpr (FP8) {
    const int k = fp8_block_exponent(am);
    if constexpr (V == 8) put(fp8_codes8(z, k));
    else put(fp8_codes4(z, k));
    if (i % L == 0) static_cast<float*>(scales)[i / L] = fp8_scale(am, k);
  } else {
    const int b = max((int)(__float_as_uint(am) >> 23) - 2, 0);   // floor(log2 amax) - 2 + 127
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = __builtin_amdgcn_ldexpf(z[j], 127 - b);
    if constexpr (V == 8) {
      put(rtn8_unit(v));
    } else {
      const uint32_t lo = cvt_fp4x2_f32<0>(0u, v[0], v[1], 1.0f);
      put((uint16_t)cvt_fp4x2_f32<1>(lo, v[2], v[3], 1.0f));
    }
    if (i % L == 0) static_cast<uint8_t*>(scales)[i / L] = (uint8_t)b;
  }
}
template <bool FP8>
__device__ __forceinline__ void quantize_octet(const float (&z)[8], int64_t i, uint8_t* q, void* scales) {
  quantize_part<FP8, false, 8>(z, i, q, scales);
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

// A thread's part of a row is 16 bytes, of which a wave's loads lie together: eight
// bf16 values or four fp32 (the octets of fp32 rows, 32 bytes a thread in two loads,
// took 107 us for 16384 x 7168).
template <bool BF16>
struct Part {
  static constexpr int kValues = BF16 ? 8 : 4, kLanes = 128 / kValues;   // values, lanes of a block
};
template <bool BF16>
__device__ __forceinline__ void part_values(u32x4 raw, float (&z)[Part<BF16>::kValues]) {
  if constexpr (BF16) {
    octet_values<true>(Octet<true>{raw, {}}, z);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = __uint_as_float(raw[j]);
  }
}
template <int N>
__device__ __forceinline__ float part_max(const float (&z)[N], float am) {
#pragma unroll
  for (int j = 0; j < N; ++j) am = fmaxf(am, fabsf(z[j]));
  return am;
}

}  // namespace fp4mi
