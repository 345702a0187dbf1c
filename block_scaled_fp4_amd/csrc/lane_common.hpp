// Shared by the operators' kernels: lanes of a row among themselves, and the bytes of
// four words.
#pragma once

#include "device_common.hpp"

namespace fp4mi {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// row_half_mirror and row_mirror: of values that are equal within each quad (each
// eight), the other quad's of the eight (the other eight's of the sixteen).
template <int CTRL>
__device__ __forceinline__ uint32_t lane_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ float other_quad(float v) { return __uint_as_float(lane_dpp<0x141>(__float_as_uint(v))); }
__device__ __forceinline__ float other_eight(float v) { return __uint_as_float(lane_dpp<0x140>(__float_as_uint(v))); }

// Byte j of four words -> word j.
__device__ __forceinline__ void transpose_bytes(const uint32_t (&w)[4], uint32_t (&t)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);
  const uint32_t b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  t[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  t[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  t[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
  t[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

}  // namespace fp4mi
