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

// 16 tokens from t of a channel of `count`, at any byte alignment.  Tokens past
// the end count as zero: the load ends at the last token and is shifted down
// (drop_bytes), or, of a shard of fewer than 16, runs into the next channels and
// is masked (keep_bytes).
__device__ __forceinline__ i32x4 load_tokens16(const uint8_t* ch, uint32_t t) {
  i32x4 v;
  memcpy(&v, ch + t, 16);
  return v;
}
// v without its lowest `drop` bytes, 0 <= drop <= 16.
__device__ __forceinline__ void drop_bytes(int drop, i32x4& v) {
  uint64_t q[2];
  memcpy(q, &v, 16);
  const int d = (drop * 8) & 63;
  const uint64_t hi = q[1] >> d, lo = d ? (q[0] >> d) | (q[1] << (64 - d)) : q[0];
  const uint64_t l = drop < 8 ? lo : (drop < 16 ? hi : 0), h = drop < 8 ? hi : 0;
  v = i32x4{(int)l, (int)(l >> 32), (int)h, (int)(h >> 32)};
}
// Only the lowest `keep` bytes of v, keep <= 16 (none where it is negative).
__device__ __forceinline__ void keep_bytes(int keep, i32x4& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = keep - 4 * i;
    v[i] = k <= 0 ? 0 : (k >= 4 ? v[i] : (int)((uint32_t)v[i] & ((1u << (8 * k)) - 1u)));
  }
}
// The same for any count, byte by byte.
__device__ __forceinline__ i32x4 load_few_tokens16(const uint8_t* ch, int t, int count) {
  uint64_t q[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint64_t w = 0;
    const int n = min(count - t - 8 * h, 8);
#pragma unroll 1
    for (int b = 0; b < n; ++b) w |= (uint64_t)ch[t + 8 * h + b] << (8 * b);
    q[h] = w;
  }
  return i32x4{(int)q[0], (int)(q[0] >> 32), (int)q[1], (int)(q[1] >> 32)};
}

struct LaneTokens {
  Frag<true> v;
  int s;
};

// What the rare path of a tile needs of its shard: from channel 0 of the tile.
struct TileView {
  const uint8_t *a, *b;
  const float *as, *bs;
  int cnt, blocks, mrows, nrows;
};
__device__ __forceinline__ void lane_tokens(const uint8_t* ch, const float* sc, int row, int cnt,
                                            int blocks, int s, int g, LaneTokens& l) {
  l.v.lo = load_few_tokens16(ch + (int64_t)row * cnt, 128 * s + 32 * g, cnt);
  l.v.hi = load_few_tokens16(ch + (int64_t)row * cnt, 128 * s + 32 * g + 16, cnt);
  l.s = (int)e8m0_of(sc[(int64_t)row * blocks + s]);
}
// Whether the 128 tokens of stage s of a channel of `cnt` hold zeros alone.
__device__ __forceinline__ bool zero_tokens(const uint8_t* ch, int s, int cnt) {
  i32x4 all = {0, 0, 0, 0};
#pragma unroll 1
  for (int q = 0; q < 8; ++q) {
    const int t = 128 * s + 16 * q;
    if (t >= cnt) continue;
    i32x4 v;
    if (cnt < 16) {
      v = load_few_tokens16(ch, t, cnt);
    } else {
      v = load_tokens16(ch, (uint32_t)min(t, cnt - 16));
      drop_bytes(t - min(t, cnt - 16), v);   // tokens of the stage before
    }
    all |= v;
  }
  return ((all.x | all.y | all.z | all.w) & 0x7F7F7F7F) == 0;
}
// Whether some scale outside the bf16 window has codes to scale.  A block of
// zeros (tokens masked out of a loss) has the smallest scale, so most tiles that
// come here only hold such blocks: the scales are read again, four stages at
// once, and codes where a scale is outside (4096 x 4096 from 16384 tokens of one
// expert: 778 us, with 128 tokens masked 849).  Eight stages at once, or the
// loads of a block together, take registers that the kernel then shuffles on its
// common path too (5 x 2048 x 1024 from 1009 tokens 24.1 -> 24.8 us).
template <int BM>
__device__ __attribute__((noinline)) bool scales_need_care(TileView v) {
  const int br = min((int)threadIdx.x % kBN, v.nrows - 1), ar = min((int)threadIdx.x % BM, v.mrows - 1);
  const uint8_t *b = v.b + (int64_t)br * v.cnt, *a = v.a + (int64_t)ar * v.cnt;
  const float *bs = v.bs + (int64_t)br * v.blocks, *as = v.as + (int64_t)ar * v.blocks;
  bool bad = false;
#pragma unroll 1
  for (int s0 = 0; s0 < v.blocks; s0 += 4) {
    int sb[4], sa[4];
    uint32_t odd = 0;   // bit j: b's stage s0 + j, bit 4 + j: a's
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sb[j] = (int)e8m0_of(bs[min(s0 + j, v.blocks - 1)]);
      sa[j] = (int)e8m0_of(as[min(s0 + j, v.blocks - 1)]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bad |= sb[j] >= 228 || sa[j] >= 228;
      odd |= (scale_in_window(sb[j]) ? 0u : 1u << j) | (scale_in_window(sa[j]) ? 0u : 16u << j);
    }
#pragma unroll 1
    for (; odd; odd &= odd - 1) {
      const int j = __builtin_ctz(odd);
      bad |= !zero_tokens(j < 4 ? b : a, min(s0 + (j & 3), v.blocks - 1), v.cnt);
    }
  }
  return bad;
}
// A wave's 128 x 64 of a tile at channels mw, nw of it, 16 x 16 at a time
// straight from memory, for scales of any range and any number of tokens.  Out
// of line, like the above, so that it costs the common path no registers.
template <bool BF16>
__device__ __attribute__((noinline)) void rare_quarter(TileView v, int mw, int nw, void* out,
                                                       int64_t out_row, int n_cols, int out_col) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  if (nw >= v.nrows || mw >= v.mrows) return;   // sides are multiples of 128
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {
    const int m = mw + (i >> 3) * 16, n = nw + (i & 7) * 16;
    LaneTokens lb[1], la[1];
    f32x4 c[1][1] = {};
#pragma unroll 1
    for (int s = 0; s < v.blocks; ++s) {
      lane_tokens(v.b, v.bs, n + r, v.cnt, v.blocks, s, g, lb[0]);
      lane_tokens(v.a, v.as, m + r, v.cnt, v.blocks, s, g, la[0]);
      mfma_bf16_step(lb, la, c);
    }
    store_out4<BF16>(out, out_row + m + r, n_cols, out_col + n + 4 * g, c[0][0]);
  }
}

// See bf16_tile: channels of b are its operand A (consecutive columns of the
// output), channels of a its operand B, tokens its k.  16 x 4096 x 7168 from
// 16384 tokens in 1.09 ms, 0.88 PFLOP/s: the matrix cores are at their bf16 peak
// inside a stage, the rest is the start of the tiles (28 a compute unit, a few
// stages each) and loads whose rows begin at any byte.  One workgroup takes all
// of its expert's tokens: with few tiles most of the card stands idle (one expert
// of 256 x 256 from 16384 tokens: 300 us for 9 MB).
template <int WM, bool BF16>
__global__ __launch_bounds__(128 * WM, 1) void wgrad_tiles_kernel(WgradArgs p, int64_t blk0) {
  constexpr int kBM = 64 * WM;
  __shared__ __align__(16) union {
    Bf16Shared<true, WM> t;
    uint8_t out[2 * WM][quarter_bytes<4, BF16>()];
  } sh;
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)((blk / p.n_tiles) % p.m_tiles);
  const int e = (int)(blk / ((int64_t)p.n_tiles * p.m_tiles));
  int lo, hi;
  shard_bounds(p.offsets, e, p.tokens, lo, hi);
  const int cnt = hi - lo, blocks = (cnt + 127) >> 7;
  const int64_t sblk = ((int64_t)lo + 127) / 128 + e;
  const int m0 = mt * kBM, n0 = nt * kBN, nrows = p.n - n0, mrows = p.m - m0;
  const uint8_t* a = p.a + (int64_t)p.m * lo + (int64_t)m0 * cnt;
  const uint8_t* b = p.b + (int64_t)p.n * lo + (int64_t)n0 * cnt;
  const float* as = p.a_scales + sblk * p.m + (int64_t)m0 * blocks;
  const float* bs = p.b_scales + sblk * p.n + (int64_t)n0 * blocks;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mw = m0 + (wave >> 1) * 64, nw = n0 + (wave & 1) * 128;
  const int64_t orow = (int64_t)e * p.m;
  const TileView view = {a, b, as, bs, cnt, blocks, mrows, nrows};
  f32x16 acc[4][2] = {};
  // a thread's rows are 16 WM apart; with only 128 rows left on a side, those
  // past them are the first again
  const int ch = (threadIdx.x & 7) * 16;
  const uint32_t row_at = (threadIdx.x >> 3) * (uint32_t)cnt;
  const int64_t step = (int64_t)(16 * WM) * cnt;
  const int ia = nrows >= kBN ? 15 : 128 / (16 * WM) - 1, ib = mrows >= kBM ? 15 : 128 / (16 * WM) - 1;
  // With fewer than 16 tokens a load runs into the next channels, and at the end
  // of the operand begins `over` bytes early.
  const int64_t a_end = (int64_t)p.m * p.tokens - (a - p.a), b_end = (int64_t)p.n * p.tokens - (b - p.b);
  auto over = [&](int64_t end, int64_t row0) { return (int)max(row0 + row_at + 16 - end, (int64_t)0); };
  const bool few = cnt < 16;
  // They are one stage, so that what the loop loads ahead only has to be there.
  const uint32_t row_in = few ? 0 : row_at;
  const int last = max(cnt - 16, 0), ia_in = few ? 0 : ia, ib_in = few ? 0 : ib;
  auto load = [&](auto first, const uint8_t* ch0, int64_t end, int i, int mask, int mask_in, int s) {
    if constexpr (decltype(first)::value) {
      if (few) return load_tokens16(ch0 + (i & mask) * step - over(end, (i & mask) * step), row_at);
    }
    return load_tokens16(ch0 + (i & mask_in) * step, row_in + (uint32_t)min(s * 128 + ch, last));
  };
  auto cut = [&](int64_t end, int64_t row0, int s, i32x4& v) {
    const int t = s * 128 + ch;
    if (few) {
      drop_bytes(over(end, row0), v);
      keep_bytes(cnt - t, v);
    } else {
      drop_bytes(min(t - min(t, cnt - 16), 16), v);
    }
  };
  const bool odd = bf16_tile<true, WM>(
      sh.t, blocks, cnt >> 7,
      [&](auto first, int s, int i) { return load(first, b, b_end, i, ia, ia_in, s); },
      [&](auto first, int s, int i) { return load(first, a, a_end, i, ib, ib_in, s); },
      [&](int s, int i, i32x4& v) { cut(b_end, (i & ia) * step, s, v); },
      [&](int s, int i, i32x4& v) { cut(a_end, (i & ib) * step, s, v); },
      [&](int s, int row) { return e8m0_of(bs[(int64_t)min(row, nrows - 1) * blocks + s]); },
      [&](int s, int row) { return e8m0_of(as[(int64_t)min(row, mrows - 1) * blocks + s]); }, acc);
  if (__syncthreads_or(odd) && __syncthreads_or(scales_need_care<kBM>(view))) {
    rare_quarter<BF16>(view, mw - m0, nw - n0, p.out, orow + m0, p.n, n0);
    return;
  }
  store_quarter<4, 2, BF16>(acc, sh.out[wave], p.out, orow + mw, orow + p.m, p.n, nw, nullptr);
}

template <int WM, bool BF16>
void launch_wgrad(WgradArgs p, int64_t experts, hipStream_t st) {
  p.m_tiles = (p.m + 64 * WM - 1) / (64 * WM);
  p.n_tiles = (p.n + kBN - 1) / kBN;
  launch_1d(wgrad_tiles_kernel<WM, BF16>, experts * p.m_tiles * p.n_tiles, 128 * WM, st, p);
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
  if (T >= (int64_t(1) << 24) || M >= (int64_t(1) << 21) || N >= (int64_t(1) << 21) ||
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
  WgradArgs p = {a, a_scales, b, b_scales, token_offsets, out, (int)T, (int)M, (int)N, 0, 0};
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const bool bf16 = out_dtype == FP4_DTYPE_BF16;
  // The larger tiles read less, the smaller ones are twice as many and spread
  // better while they are few (us, 256 x 128 | 256 x 256 by the number of the
  // second): 128: 52 | 63, 256: 47 | 51, 512: 84 | 55, 1024: 232 | 160.
  if (E * ((M + 255) / 256) * ((N + 255) / 256) >= 512)
    bf16 ? launch_wgrad<4, true>(p, E, st) : launch_wgrad<4, false>(p, E, st);
  else
    bf16 ? launch_wgrad<2, true>(p, E, st) : launch_wgrad<2, false>(p, E, st);
  return launch_status();
}
