// Weight gradients per expert from FP8 columns with 128-token scale blocks.
#include <string.h>

#include "fp4mi_ops.h"
#include "host_common.hpp"
#include "mfma_common.hpp"

namespace fp4mi {
namespace {

struct WgradArgs {
  const uint8_t* a;        // E4M3 columns of dY: expert e's [M, n_e] at byte M off[e]
  const float* a_scales;   // expert e's [M, ceil(n_e/128)] at M (ceil(off[e]/128) + e)
  const uint8_t* b;        // the same of X, with N
  const float* b_scales;
  const int64_t* offsets;
  void* out;               // [E, M, N]
  int tokens, m, n;
  int m_tiles, n_tiles;
};

// 32 tokens t .. t+31 of a channel at any byte alignment; tokens past the
// shard's end count as zero and are not read.
__device__ __forceinline__ Frag<true> load_tokens(const uint8_t* ch, int t, int count) {
  Frag<true> f;
  if (t + 32 <= count) {
    memcpy(&f.lo, ch + t, 16);
    memcpy(&f.hi, ch + t + 16, 16);
  } else {
    int w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t v = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (t + 4 * i + b < count) v |= (uint32_t)ch[t + 4 * i + b] << (8 * b);
      w[i] = (int)v;
    }
    f.lo = i32x4{w[0], w[1], w[2], w[3]};
    f.hi = i32x4{w[4], w[5], w[6], w[7]};
  }
  return f;
}

// One wave per 64 x 64 tile of one expert's gradient, operands straight from
// memory.  N is operand A of the instruction, so a lane ends with four
// consecutive columns of one row of out.
struct LaneTokens {
  Frag<true> v;
  int s;
};
constexpr int kWF = 4;
template <bool BF16>
__global__ __launch_bounds__(64) void wgrad_kernel(WgradArgs p, int64_t blk0) {
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)((blk / p.n_tiles) % p.m_tiles);
  const int e = (int)(blk / ((int64_t)p.n_tiles * p.m_tiles));
  const int lane = threadIdx.x, r = lane & 15, g = lane >> 4;
  int lo, hi;
  shard_bounds(p.offsets, e, p.tokens, lo, hi);
  const int cnt = hi - lo, blocks = (cnt + 127) >> 7;
  const int64_t sblk = ((int64_t)lo + 127) / 128 + e;
  const int m0 = mt * 16 * kWF, n0 = nt * 16 * kWF;
  f32x4 acc[kWF][kWF] = {};
  for (int j = 0; j < blocks; ++j) {
    LaneTokens a[kWF], b[kWF];
#pragma unroll
    for (int f = 0; f < kWF; ++f) {
      const int n = n0 + 16 * f + r, m = m0 + 16 * f + r;
      b[f].v = load_tokens(p.b + (int64_t)p.n * lo + (int64_t)n * cnt, 128 * j + 32 * g, cnt);
      b[f].s = (int)e8m0_of(p.b_scales[sblk * p.n + (int64_t)n * blocks + j]);
      a[f].v = load_tokens(p.a + (int64_t)p.m * lo + (int64_t)m * cnt, 128 * j + 32 * g, cnt);
      a[f].s = (int)e8m0_of(p.a_scales[sblk * p.m + (int64_t)m * blocks + j]);
    }
    mfma_bf16_step(b, a, acc);
  }
#pragma unroll
  for (int x = 0; x < kWF; ++x)
#pragma unroll
    for (int y = 0; y < kWF; ++y)
      store_out4<BF16>(p.out, (int64_t)e * p.m + m0 + 16 * y + r, p.n, n0 + 16 * x + 4 * g, acc[x][y]);
}

}  // namespace
}  // namespace fp4mi

using namespace fp4mi;

extern "C" int fp8_matmul_tokblk(const uint8_t* a, const float* a_scales, const uint8_t* b,
                                 const float* b_scales, const int64_t* token_offsets,
                                 int32_t num_experts, int64_t total_tokens, int64_t M, int64_t N,
                                 void* out, int out_dtype, void* stream) {
  if (num_experts < 1) return FP4_EINVAL;
  const int osz = dtype_size(out_dtype);
  if (!osz) return FP4_EDTYPE;
  const int64_t T = total_tokens, E = num_experts;
  if (T < 0 || M < 0 || N < 0 || M % 128 || N % 128) return FP4_ESHAPE;
  if (T >= (int64_t(1) << 26) || M >= (int64_t(1) << 21) || N >= (int64_t(1) << 21) ||
      E >= (int64_t(1) << 23))
    return FP4_ESHAPE;
  int64_t n_a, n_b, n_mn, n_out;
  if (!checked_count(T, M, &n_a) || !checked_count(T, N, &n_b) || !checked_count(M, N, &n_mn) ||
      !checked_count(E, n_mn, &n_out))
    return FP4_ESHAPE;
  if (!token_offsets) return FP4_EINVAL;
  if (n_out == 0) return FP4_OK;
  if (!out || (T && (!a || !a_scales || !b || !b_scales))) return FP4_EINVAL;
  if (!is_aligned(a, 4) || !is_aligned(a_scales, 4) || !is_aligned(b, 4) ||
      !is_aligned(b_scales, 4) || !is_aligned(token_offsets, 8) || !is_aligned(out, 16))
    return FP4_EALIGN;
  const int64_t blocks = (T + 127) / 128 + E;
  const void* ins[5] = {a, a_scales, b, b_scales, token_offsets};
  const int64_t inn[5] = {n_a, T ? M * blocks * 4 : 0, n_b, T ? N * blocks * 4 : 0, (E + 1) * 8};
  for (int i = 0; i < 5; ++i)
    if (overlaps(out, n_out * osz, ins[i], inn[i])) return FP4_EOVERLAP;
  WgradArgs p = {a, a_scales, b, b_scales, token_offsets, out, (int)T, (int)M, (int)N,
                 (int)(M / (16 * kWF)), (int)(N / (16 * kWF))};
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const int64_t grid = E * p.m_tiles * p.n_tiles;
  if (out_dtype == FP4_DTYPE_BF16)
    launch_1d(wgrad_kernel<true>, grid, 64, st, p);
  else
    launch_1d(wgrad_kernel<false>, grid, 64, st, p);
  return launch_status();
}
