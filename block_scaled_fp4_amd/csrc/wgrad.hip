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

struct LaneTokens {
  Frag<true> v;
  int s;
};

// 16 tokens from t; FULL: all inside the shard.
template <bool FULL>
__device__ __forceinline__ i32x4 load_tokens16(const uint8_t* ch, int t, int count) {
  i32x4 v;
  if (FULL || t + 16 <= count) {
    memcpy(&v, ch + t, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (t + 4 * i + b < count) w |= (uint32_t)ch[t + 4 * i + b] << (8 * b);
      v[i] = (int)w;
    }
  }
  return v;
}

// See bf16_tile: channels of b are its operand A (consecutive columns of the
// output), channels of a its operand B, tokens its k.
template <bool BF16>
__global__ __launch_bounds__(256, 1) void wgrad_tiles_kernel(WgradArgs p, int64_t blk0) {
  __shared__ __align__(16) union {
    Bf16Shared<true> t;
    uint8_t out[4][quarter_bytes<4, BF16>()];
  } sh;
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)((blk / p.n_tiles) % p.m_tiles);
  const int e = (int)(blk / ((int64_t)p.n_tiles * p.m_tiles));
  int lo, hi;
  shard_bounds(p.offsets, e, p.tokens, lo, hi);
  const int cnt = hi - lo, blocks = (cnt + 127) >> 7;
  const int64_t sblk = ((int64_t)lo + 127) / 128 + e;
  const int m0 = mt * kBM, n0 = nt * kBN, nrows = p.n - n0;
  const uint8_t* a = p.a + (int64_t)p.m * lo + (int64_t)m0 * cnt;
  const uint8_t* b = p.b + (int64_t)p.n * lo + (int64_t)n0 * cnt;
  const float* as = p.a_scales + sblk * p.m + (int64_t)m0 * blocks;
  const float* bs = p.b_scales + sblk * p.n + (int64_t)n0 * blocks;
  f32x16 acc[4][2] = {};
  const bool odd = bf16_tile<true>(
      sh.t, blocks, cnt >> 7,
      [&](auto full, int s, int row, int c) {
        return load_tokens16<decltype(full)::value>(b + (int64_t)min(row, nrows - 1) * cnt, s * 128 + c * 16, cnt);
      },
      [&](auto full, int s, int row, int c) {
        return load_tokens16<decltype(full)::value>(a + (int64_t)row * cnt, s * 128 + c * 16, cnt);
      },
      [&](auto, int s, int row) { return e8m0_of(bs[(int64_t)min(row, nrows - 1) * blocks + s]); },
      [&](int s, int row) { return e8m0_of(as[(int64_t)row * blocks + s]); }, acc);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mw = m0 + (wave >> 1) * 64, nw = n0 + (wave & 1) * 128;
  const int64_t orow = (int64_t)e * p.m;
  auto lane_tokens = [&](const uint8_t* ch, const float* sc, int row, int s, int g, LaneTokens& l) {
    l.v = load_tokens(ch + (int64_t)row * cnt, 128 * s + 32 * g, cnt);
    l.s = (int)e8m0_of(sc[(int64_t)row * blocks + s]);
  };
  const auto slow = [&]() {   // whether a scale outside the window has codes to scale
    bool bad = false;
    for (int i = 0; i < 4 * blocks; ++i) {
      LaneTokens lb, la;
      lane_tokens(b, bs, min((int)threadIdx.x, nrows - 1), i >> 2, i & 3, lb);
      lane_tokens(a, as, threadIdx.x % kBM, i >> 2, i & 3, la);
      bad |= !scale_fits(lb) || !scale_fits(la);
    }
    return bad;
  };
  if (__syncthreads_or(odd) && __syncthreads_or(slow())) {
    // rare: 16 x 16 at a time, straight from memory, with every scale's range
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    if (nw >= p.n) return;
    for (int i = 0; i < 32; ++i) {
      const int m = mw + (i >> 3) * 16, n = nw + (i & 7) * 16;
      LaneTokens lb[1], la[1];
      f32x4 c[1][1] = {};
      for (int s = 0; s < blocks; ++s) {
        lane_tokens(b, bs, n - n0 + r, s, g, lb[0]);
        lane_tokens(a, as, m - m0 + r, s, g, la[0]);
        mfma_bf16_step(lb, la, c);
      }
      store_out4<BF16>(p.out, orow + m + r, p.n, n + 4 * g, c[0][0]);
    }
    return;
  }
  store_quarter<4, 2, BF16>(acc, sh.out[wave], p.out, orow + mw, orow + p.m, p.n, nw, nullptr);
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
                 (int)(M / kBM), (int)((N + kBN - 1) / kBN)};
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const int64_t grid = E * p.m_tiles * p.n_tiles;
  if (out_dtype == FP4_DTYPE_BF16)
    launch_1d(wgrad_tiles_kernel<true>, grid, 256, st, p);
  else
    launch_1d(wgrad_tiles_kernel<false>, grid, 256, st, p);
  return launch_status();
}
