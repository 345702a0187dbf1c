// MXFP4 products, dense and grouped by expert.
#include <string.h>
#include <utility>

#include "fp4mi_ops.h"
#include "host_common.hpp"
#include "mfma_common.hpp"

namespace fp4mi {
namespace {

// --------------------------------------------------------------- few rows
// One workgroup owns 16 FN columns of W by 16 FM tokens; its W waves take the
// steps of 128 k in turn, straight from memory to registers, U steps at a time
// with the next U in flight, and add their sums through LDS.  The weights are
// read once, by as many waves as there is work for, so that all of them are in
// flight at once; splitting k inside the workgroup needs no second launch.  What
// bounds it is the number of vector loads, then memory: 4096 x 7168 by one token
// 4.8 us, 64 tokens over 32 experts of 2048 x 7168 29.1 us (4.8 TB/s).

// 4 scale bytes of a row of `bytes` >= 4 from byte `at`.  Past the row's end
// stand other bytes of the row: the codes there count as zero, and a NaN scale
// among them makes the same outputs NaN by itself.  FULL: there are none.
template <bool FULL>
__device__ __forceinline__ uint32_t load_scales4(const uint8_t* row, int at, int bytes) {
  const int have = FULL ? at : min(at, bytes - 4);
  uint32_t w;
  memcpy(&w, row + have, 4);
  return FULL ? w : w >> (8 * min(at - have, 3));
}

// The U words of scale bytes (four blocks of 32, or one fp32 scale, a word) of
// steps st .. st + U - 1 of a row, in one load where the row has them all.
template <int U>
__device__ __forceinline__ void load_scale_words(const uint8_t* row, int st, int bytes,
                                                 uint32_t (&v)[U]) {
  if (4 * (st + U) <= bytes) {
    memcpy(v, row + 4 * st, 4 * U);
  } else if (bytes >= 4) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load_scales4<false>(row, 4 * (st + u), bytes);
  } else {   // K < 128
    uint32_t w = 0;
    for (int i = 0; i < bytes; ++i) w |= (uint32_t)row[i] << (8 * i);
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = w;
  }
}

template <bool A8, bool KT, int FN, int FM, int W, int U, bool BF16>
__global__ __launch_bounds__(64 * W) void product_rows_kernel(ProductArgs p, int64_t blk0) {
  __shared__ f32x4 red[W][FN * FM][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)(blk / p.n_tiles);
  int e = 0, row0 = p.offsets ? 0 : mt * (16 * FM), row_end = (int)p.tokens;
  if (p.offsets) {
    if (!locate_tile<16 * FM>(p.offsets, p.experts, (int)p.tokens, mt, e, row0, row_end)) return;
  }
  const int r = lane & 15, g = lane >> 4, n0 = nt * (16 * FN);
  const uint8_t* w = p.w + (int64_t)e * p.n * (p.k >> 1);
  const uint8_t* ws = p.w_scales + (int64_t)e * p.n * (p.k >> 5);
  int wn[FN], am[FM];
#pragma unroll
  for (int f = 0; f < FN; ++f) wn[f] = min(n0 + 16 * f + r, p.n - 1);
#pragma unroll
  for (int f = 0; f < FM; ++f) am[f] = min(row0 + 16 * f + r, row_end - 1);

  f32x4 acc[FN][FM] = {};
  const int steps = (p.k + 127) >> 7;
  struct Batch {
    LaneStep<false> w[U][FN];
    LaneStep<A8> a[U][FM];
  } even = {}, odd = {};   // in turn, so that no load is waited for before its use
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int f = 0; f < FM; ++f)
      if (A8) even.a[u][f].s = odd.a[u][f].s = 127;   // of lanes without a token: inside the window
  // Loads are counted here, not bytes: one instruction takes the scales of U
  // steps, and with few tokens lanes past the last load nothing.
  const int kb = p.k >> 1, ksb = p.k >> 5;
  auto load = [&](int c, Batch& b) {
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      uint32_t sc[U];
      load_scale_words<U>(ws + (int64_t)wn[f] * ksb, c, ksb, sc);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kk = min(c + u, steps - 1) * 128 + 32 * g;
        const bool in = !KT || kk < p.k;
        b.w[u][f].v.lo = *reinterpret_cast<const i32x4*>(w + (int64_t)wn[f] * kb + ((in ? kk : 0) >> 1));
        if (KT && !in) b.w[u][f].v.lo = i32x4{0, 0, 0, 0};   // past K codes count as zero
        b.w[u][f].s = (int)((sc[u] >> (8 * g)) & 0xFFu);
      }
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      if (FM <= 2 && row0 + 16 * f + r >= row_end) continue;
      uint32_t sc[U];
      load_scale_words<U>(static_cast<const uint8_t*>(p.a_scales) + (int64_t)am[f] * (A8 ? p.k >> 5 : ksb),
                          c, ksb, sc);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int kk = min(c + u, steps - 1) * 128 + 32 * g, at = !KT || kk < p.k ? kk : 0;
        if constexpr (A8) {
          const i32x4* q = reinterpret_cast<const i32x4*>(p.a + (int64_t)am[f] * p.k + at);
          b.a[u][f].v.lo = q[0];
          b.a[u][f].v.hi = q[1];
          b.a[u][f].s = (int)((sc[u] >> 23) & 0xFFu);
        } else {
          b.a[u][f].v.lo = *reinterpret_cast<const i32x4*>(p.a + (int64_t)am[f] * kb + (at >> 1));
          b.a[u][f].s = (int)((sc[u] >> (8 * g)) & 0xFFu);
        }
      }
    }
  };
  auto multiply = [&](int c, const Batch& b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u >= steps) continue;
      if constexpr (A8) {
        mfma_bf16_step(b.w[u], b.a[u], acc);
      } else {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j)
            acc[i][j] = mfma_scaled<0, 0>(b.w[u][i].v, b.a[u][j].v, acc[i][j], b.w[u][i].s, b.a[u][j].s);
      }
    }
  };
  int c = wave * U;
  constexpr int S = W * U;
  if (c < steps) load(c, even);
  for (; c < steps; c += 2 * S) {
    if (c + S < steps) load(c + S, odd);
    multiply(c, even);
    if (c + S >= steps) break;
    if (c + 2 * S < steps) load(c + 2 * S, even);
    multiply(c + S, odd);
  }
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) red[wave][i * FM + j][lane] = acc[i][j];
  __syncthreads();
  for (int s = threadIdx.x; s < FN * FM * 64; s += 64 * W) {
    const int f = s >> 6, l = s & 63;
    f32x4 v = red[0][f][l];
#pragma unroll
    for (int q = 1; q < W; ++q) v += red[q][f][l];
    const int m = row0 + 16 * (f % FM) + (l & 15), n = n0 + 16 * (f / FM) + 4 * (l >> 4);
    if (m < row_end && n < p.n) {
      if (p.a_row_scale) v *= p.a_row_scale[m];
      store_out4<BF16>(p.out, m, p.n, n, v);
    }
  }
}

template <bool A8, bool KT, int FN, int FM, int W, int U>
void launch_rows(ProductArgs p, int out_dtype, hipStream_t st) {
  p.n_tiles = (p.n + 16 * FN - 1) / (16 * FN);
  const int64_t blocks =
      p.n_tiles * max_row_tiles(p.tokens, p.experts, 16 * FM, p.offsets != nullptr);
  if (out_dtype == FP4_DTYPE_BF16)
    launch_1d(product_rows_kernel<A8, KT, FN, FM, W, U, true>, blocks, 64 * W, st, p);
  else
    launch_1d(product_rows_kernel<A8, KT, FN, FM, W, U, false>, blocks, 64 * W, st, p);
}

// --------------------------------------------------------------- many rows
// MXFP4 by MXFP4: one workgroup of four waves owns 64 FN columns of W by 64 FM
// tokens, each wave a 32 FN x 32 FM quarter in 32 x 32 x 64 instructions (lane
// l: row l % 32, the 32 k of group l / 32; D's lane l: column l % 32, rows
// 8 (i / 4) + 4 (l / 32) + i % 4).  A stage is 256 k: 128 bytes of every row go
// to LDS with direct loads, two stages in turn, one barrier each.  A row's
// eight 16-byte chunks lie at position chunk ^ (row / 2 % 8), so that neither the
// line-wide direct loads nor the 32-row fragment reads meet a bank twice (16
// lanes of a read take all 64 banks: row parity picks the half, row / 2 the
// place in it).
// 8192^3 in 255 us, 4.3 PFLOP/s.  The matrix cores are busy 55% of the cycles,
// at the 1.8 GHz that the card holds under this load; each of a compute unit's 4
// tiles has 10 us of start and output around it, and with the LDS reads, direct
// loads and scales left out the rest takes 183 us in place of 255.
template <int SA, int SB>
__device__ __forceinline__ f32x16 mfma_scaled32(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
  const i32x8 x = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, y = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, kE2M1, kE2M1, SA, sa, SB, sb);
}

template <int FN, int FM>
struct TileShared {
  uint8_t w[2][64 * FN * 128];
  uint8_t x[2][64 * FM * 128];
  // Scales of two pairs of stages: [pair][k group][half of the rows][row % 32],
  // a word of the bytes of rows r, r + 32, r + 64, r + 96, the fragments of one
  // wave (of both, where a wave has two).
  uint32_t ws[2][16][2][32];
  uint32_t xs[2][16][FM / 2][32];
};

template <int FN, int FM, bool BF16>
__global__ __launch_bounds__(256, 1) void product_tiles_kernel(ProductArgs p, int64_t blk0) {
  static_assert(FN == 4 && (FM == 4 || FM == 2), "scale words");
  constexpr int BN = 64 * FN, BM = 64 * FM;
  __shared__ __align__(16) union {
    TileShared<FN, FM> t;
    uint8_t out[4][quarter_bytes<FN, BF16>()];
  } sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)(blk / p.n_tiles);
  int e = 0, row0 = p.offsets ? 0 : mt * BM, row_end = (int)p.tokens;
  if (p.offsets) {
    if (!locate_tile<BM>(p.offsets, p.experts, (int)p.tokens, mt, e, row0, row_end)) return;
  }
  const int n0 = nt * BN, kb = p.k >> 1, ksb = p.k >> 5;
  const uint8_t* w = p.w + ((int64_t)e * p.n) * kb;
  const uint8_t* ws = p.w_scales + (int64_t)e * p.n * ksb;
  const int wn = wave & 1, wm = wave >> 1;   // this wave's quarter
  const int stages = (p.k + 255) >> 8;

  // Direct loads: instruction i of this wave covers 8 rows; lane l is row
  // l / 8, position l % 8, which holds chunk (l % 8) ^ (row / 2 % 8).
  auto ch = [&](int i) { return (lane & 7) ^ (((i & 1) << 2) | (lane >> 4)); };
  const uint8_t* xa = p.a + (int64_t)row0 * kb;
  w += (int64_t)n0 * kb;
  ws += (int64_t)n0 * ksb;
  const int wrows = p.n - n0, xrows = row_end - row0;
  uint32_t wo[2 * FN], xo[2 * FM];
#pragma unroll
  for (int i = 0; i < 2 * FN; ++i)
    wo[i] = (uint32_t)min(8 * (wave * 2 * FN + i) + (lane >> 3), wrows - 1) * (uint32_t)kb + ch(i) * 16;
#pragma unroll
  for (int i = 0; i < 2 * FM; ++i)
    xo[i] = (uint32_t)min(8 * (wave * 2 * FM + i) + (lane >> 3), xrows - 1) * (uint32_t)kb + ch(i) * 16;
  const buffer_t wb = buffer_of(w, (int64_t)min(wrows, BN) * kb);
  const buffer_t xb = buffer_of(xa, (int64_t)min(xrows, BM) * kb);
  // Stage s into buffer B.  In a last stage that reaches past K, the chunks
  // there are other bytes of the tile: mask() has them count as zero.
  constexpr int kLoads = 2 * FN + 2 * FM;
  auto fetch_one = [&](auto b, auto full, int s, int i) {
    constexpr int B = decltype(b)::value;
    const bool isw = i < 2 * FN;
    const int j = isw ? i : i - 2 * FN;
    uint32_t v = isw ? wo[j] : xo[j], so = s * 128;
    if (!decltype(full)::value && s * 256 + 256 > p.k) {
      v += so - (uint32_t)max(s * 128 + ch(j) * 16 + 16 - kb, 0);
      so = 0;
    }
    if (isw) load_to_lds(wb, v, so, &sh.t.w[B][(wave * 2 * FN + j) * 1024]);
    else load_to_lds(xb, v, so, &sh.t.x[B][(wave * 2 * FM + j) * 1024]);
  };
  auto fetch = [&](auto b, auto full, int s, int from, int to) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (i >= from && i < to) fetch_one(b, full, s, i);
  };
  // Scales: a thread loads 4 bytes (4 of a pair of stages' 16 k groups) of four
  // rows and writes them as four words, one a k group.
  const int seg = tid & 3, sr = (tid >> 2) & 31, sh2 = tid >> 7;
  uint32_t wso[4], xso[4];
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    wso[f] = (uint32_t)min(sh2 * 128 + f * 32 + sr, wrows - 1) * (uint32_t)ksb;
    xso[f] = (uint32_t)min((FM == 4 ? sh2 * 128 : 0) + f * 32 + sr, xrows - 1) * (uint32_t)ksb;
  }
  const uint8_t* xsc = static_cast<const uint8_t*>(p.a_scales) + (int64_t)row0 * ksb;
  uint32_t wq[4], xq[4];
  auto fetch_scales = [&](auto full, int s) {   // of stages s and s + 1
    constexpr bool FULL = decltype(full)::value;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      wq[f] = load_scales4<FULL>(ws + wso[f], s * 8 + seg * 4, ksb);
      xq[f] = load_scales4<FULL>(xsc + xso[f], s * 8 + seg * 4, ksb);
    }
  };
  auto put_scales = [&](int s) {
    uint32_t t[4];
    const int pair = (s >> 1) & 1;
    transpose_bytes(wq, t);
#pragma unroll
    for (int j = 0; j < 4; ++j) sh.t.ws[pair][seg * 4 + j][sh2][sr] = t[j];
    transpose_bytes(xq, t);
#pragma unroll
    for (int j = 0; j < 4; ++j) sh.t.xs[pair][seg * 4 + j][FM == 4 ? sh2 : 0][sr] = t[j];
  };

  const int r = lane & 31, g = lane >> 5;
  struct Step {
    i32x4 w[FN], x[FM];
    int ws, xs;
  };
  const uint8_t *wl[4], *xl[4];   // this lane's chunk of its first fragment, for each 64 k
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const int c = ((2 * ks + g) ^ ((r >> 1) & 7)) * 16;
    wl[ks] = &sh.t.w[0][(wn * FN * 32 + r) * 128 + c];
    xl[ks] = &sh.t.x[0][(wm * FM * 32 + r) * 128 + c];
  }
  // Of 64 k of stage s, the scales (i = 0) or fragment i - 1 of both operands.
  auto read_part = [&](auto b, int s, int ks, int i, Step& o) {
    constexpr int B = decltype(b)::value;
    if (i == 0) {
      const int pair = (s >> 1) & 1;
      o.ws = (int)sh.t.ws[pair][B * 8 + 2 * ks + g][wn][r];
      o.xs = FM == 4 ? (int)sh.t.xs[pair][B * 8 + 2 * ks + g][wm][r]
                     : (int)(sh.t.xs[pair][B * 8 + 2 * ks + g][0][r] >> (16 * wm));
      return;
    }
    const int f = i - 1;
    o.w[f] = *reinterpret_cast<const i32x4*>(wl[ks] + (B * BN + f * 32) * 128);
    if (f < FM) o.x[f] = *reinterpret_cast<const i32x4*>(xl[ks] + (B * BM + f * 32) * 128);
  };
  f32x16 acc[FN][FM] = {};
  // The FN FM products of a step, between(i) after product i; both stay where
  // they are written.
  auto multiply = [&](const Step& o, auto between) {
    unrolled<FN * FM>([&](auto idx) {
      constexpr int I = decltype(idx)::value / FM, J = decltype(idx)::value % FM;
      acc[I][J] = mfma_scaled32<I, J>(o.w[I], o.x[J], acc[I][J], o.ws, o.xs);
      between(idx);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // Past K in the last stage W's codes count as zero.
  auto mask = [&](int s, int ks, Step& o) {
    if (s * 256 + ks * 64 + 32 * g >= p.k) {
#pragma unroll
      for (int f = 0; f < FN; ++f) o.w[f] = i32x4{0, 0, 0, 0};
    }
  };
  auto landed = [&]() {   // this wave's direct loads are in LDS, then everyone's
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    __syncthreads();
  };

  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  fetch_scales(no, 0);
  fetch(first, no, 0, 0, kLoads);
  put_scales(0);
  if (stages > 2) fetch_scales(no, 2);
  landed();
  Step even, odd;
#pragma unroll
  for (int i = 0; i <= FN; ++i) read_part(first, 0, 0, i, even);
  if (stages > 1) fetch(second, no, 1, 0, kLoads / 2);
  // Stage s in buffer b, the next in nb.  MID: stages s + 1 and s + 2 follow and
  // end inside K; where b is the first, so do the scales of s + 4 and s + 5;
  // then nothing here branches.
  // The direct loads of a stage are spread over the 16 products that follow the
  // barrier and the 16 after those: issued together they would hold the wave up.
  constexpr int kAll = FN * FM;
  auto stage = [&](auto b, auto nb, auto mid, int s) {
    constexpr bool MID = decltype(mid)::value;
    const bool more = MID || s + 1 < stages, more2 = MID || s + 2 < stages;
    auto reads = [&](auto bb, int st, int ks, Step& o, int i) {
      if (i <= FN) read_part(bb, st, ks, i, o);
    };
    auto loads = [&](auto bb, int st, int half, int i) {   // one of half the loads every other product
      constexpr int every = 2 * kAll / kLoads > 1 ? 2 * kAll / kLoads : 1;
      if (i % every == every - 1 && i / every < kLoads / 2) fetch_one(bb, mid, st, half * (kLoads / 2) + i / every);
    };
    if (!MID) mask(s, 0, even);
    multiply(even, [&](auto i) {
      reads(b, s, 1, odd, i);
      if (more) loads(nb, s + 1, 1, i);
    });
    if (!MID) mask(s, 1, odd);
    multiply(odd, [&](auto i) {
      reads(b, s, 2, even, i);
      if (decltype(b)::value == 0 && i == kAll - 2 && more2) put_scales(s + 2);
    });
    if (!MID) mask(s, 2, even);
    multiply(even, [&](auto i) {
      reads(b, s, 3, odd, i);
      if (decltype(b)::value == 0 && i == FN + 1 && (MID || s + 4 < stages)) fetch_scales(mid, s + 4);
    });
    landed();   // stage s + 1; and everyone has read stage s
    if (!MID) mask(s, 3, odd);
    multiply(odd, [&](auto i) {
      if (more) reads(nb, s + 1, 0, even, i);
      if (more2) loads(b, s + 2, 0, i);
    });
  };
  int s = 0;
  for (; s + 6 <= (p.k >> 8); s += 2) {
    stage(first, second, yes, s);
    stage(second, first, yes, s + 1);
  }
  for (; s < stages; s += 2) {
    stage(first, second, no, s);
    if (s + 1 < stages) stage(second, first, no, s + 1);
  }

  __syncthreads();
  store_quarter<FN, FM, BF16>(acc, sh.out[wave], p.out, row0 + wm * FM * 32, row_end, p.n,
                              n0 + wn * FN * 32, p.a_row_scale);
}

template <int FN, int FM>
void launch_tiles(ProductArgs p, int out_dtype, hipStream_t st) {
  p.n_tiles = (p.n + 64 * FN - 1) / (64 * FN);
  const int64_t blocks =
      p.n_tiles * max_row_tiles(p.tokens, p.experts, 64 * FM, p.offsets != nullptr);
  if (out_dtype == FP4_DTYPE_BF16)
    launch_1d(product_tiles_kernel<FN, FM, true>, blocks, 256, st, p);
  else
    launch_1d(product_tiles_kernel<FN, FM, false>, blocks, 256, st, p);
}

// What the rare path of a tile needs, from the tile's first rows.
struct Fp8TileView {
  const uint8_t* x;
  const float* xs;
  const uint8_t *w, *ws;
  int k, xrows, wrows;
};
// Whether some scale outside the bf16 window has codes to scale.  A block of
// zeros has the smallest scale, so most tiles that come here only hold such
// blocks: the scales are read again, eight stages at once, and codes where a
// scale is outside (4096^3: 135 us, with one row in 100 of zeros 163).
__device__ __attribute__((noinline)) bool scales_need_care(Fp8TileView v) {
  const int wr = min((int)threadIdx.x % kBN, v.wrows - 1), xr = min((int)threadIdx.x % 128, v.xrows - 1);
  const int stages = v.k >> 7;
  const uint8_t* w = v.w + (int64_t)wr * (v.k >> 1);
  const uint8_t* x = v.x + (int64_t)xr * v.k;
  const uint32_t* ws = reinterpret_cast<const uint32_t*>(v.ws + (int64_t)wr * (v.k >> 5));
  const float* xs = v.xs + (int64_t)xr * stages;
  bool bad = false;
#pragma unroll 1
  for (int s0 = 0; s0 < stages; s0 += 8) {
    uint32_t sw[8], sx[8], odd_w = 0, odd_x = 0;   // bit 4 j + q: block q of stage s0 + j; bit j
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sw[j] = ws[min(s0 + j, stages - 1)];
      sx[j] = e8m0_of(xs[min(s0 + j, stages - 1)]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int b = (int)((sw[j] >> (8 * q)) & 0xFFu);
        bad |= b >= 228;
        odd_w |= scale_in_window(b) ? 0u : 1u << (4 * j + q);
      }
      bad |= sx[j] >= 228;
      odd_x |= scale_in_window((int)sx[j]) ? 0u : 1u << j;
    }
#pragma unroll 1
    for (; odd_w; odd_w &= odd_w - 1) {
      const int s = min(s0 + __builtin_ctz(odd_w) / 4, stages - 1), q = __builtin_ctz(odd_w) & 3;
      bad |= !zero_codes(Frag<false>{*reinterpret_cast<const i32x4*>(w + s * 64 + q * 16)});
    }
#pragma unroll 1
    for (; odd_x; odd_x &= odd_x - 1) {
      const i32x4* c = reinterpret_cast<const i32x4*>(x + min(s0 + __builtin_ctz(odd_x), stages - 1) * 128);
#pragma unroll
      for (int q = 0; q < 4; ++q) bad |= !zero_codes(Frag<true>{c[2 * q], c[2 * q + 1]});
    }
  }
  return bad;
}
// A wave's 128 x 64 of a tile, 16 x 16 at a time straight from memory, for scales
// of any range.  Out of line, like the above, so that it costs the common path no
// registers.
template <bool BF16>
__device__ __attribute__((noinline)) void rare_quarter(Fp8TileView v, int mw, int nw, void* out,
                                                       int64_t out_row, int n_cols, int out_col,
                                                       const float* row_scale) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {
    const int m = mw + (i >> 3) * 16, n = nw + (i & 7) * 16;
    LaneStep<false> lw[1];
    LaneStep<true> lx[1];
    f32x4 c[1][1] = {};
#pragma unroll 1
    for (int s = 0; s < v.k >> 7; ++s) {
      load_lane<false>(v.w, v.ws, min(n + r, v.wrows - 1), v.k, s, g, lw[0]);
      load_lane<true>(v.x, v.xs, min(m + r, v.xrows - 1), v.k, s, g, lx[0]);
      mfma_bf16_step(lw, lx, c);
    }
    if (m + r < v.xrows) {
      if (row_scale) c[0][0] *= row_scale[out_row + m + r];
      store_out4<BF16>(out, out_row + m + r, n_cols, out_col + n + 4 * g, c[0][0]);
    }
  }
}

// FP8 rows by MXFP4, see bf16_tile.  Two workgroups a compute unit hide each
// other's starts and barriers (one: 225 us, two: 159 for 5001 tokens over 13
// experts of 7168 x 2048, 0.9 PFLOP/s).
constexpr int kBM = 128;
template <bool BF16>
__global__ __launch_bounds__(256, 2) void product_fp8_tiles_kernel(ProductArgs p, int64_t blk0) {
  __shared__ __align__(16) union {
    Bf16Shared<false, 2> t;
    uint8_t out[4][quarter_bytes<4, BF16>()];
  } sh;
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)(blk / p.n_tiles);
  int e = 0, row0 = p.offsets ? 0 : mt * kBM, row_end = (int)p.tokens;
  if (p.offsets) {
    if (!locate_tile<kBM>(p.offsets, p.experts, (int)p.tokens, mt, e, row0, row_end)) return;
  }
  const int n0 = nt * kBN, kb = p.k >> 1, ksb = p.k >> 5, kx = p.k >> 7;
  const int wrows = p.n - n0, xrows = row_end - row0;
  const uint8_t* w = p.w + ((int64_t)e * p.n + n0) * kb;
  const uint8_t* ws = p.w_scales + ((int64_t)e * p.n + n0) * ksb;
  const uint8_t* x = p.a + (int64_t)row0 * p.k;
  const float* xs = static_cast<const float*>(p.a_scales) + (int64_t)row0 * kx;
  uint32_t wo[4], xo[4];
  const int tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wo[i] = (uint32_t)min((tid >> 2) + 64 * i, wrows - 1) * (uint32_t)kb + (tid & 3) * 16;
    xo[i] = (uint32_t)min((tid >> 3) + 32 * i, xrows - 1) * (uint32_t)p.k + (tid & 7) * 16;
  }
  f32x16 acc[4][2] = {};
  const bool odd = bf16_tile<false, 2>(
      sh.t, kx, kx,
      [&](auto, int s, int i) { return *reinterpret_cast<const i32x4*>(w + s * 64 + wo[i]); },
      [&](auto, int s, int i) { return *reinterpret_cast<const i32x4*>(x + s * 128 + xo[i]); },
      [](int, int, i32x4&) {}, [](int, int, i32x4&) {},
      [&](int s, int row) {
        return *reinterpret_cast<const uint32_t*>(ws + (int64_t)min(row, wrows - 1) * ksb + s * 4);
      },
      [&](int s, int row) { return e8m0_of(xs[(int64_t)min(row, xrows - 1) * kx + s]); }, acc);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = row0 + (wave >> 1) * 64, nw = n0 + (wave & 1) * 128;
  const Fp8TileView view = {x, xs, w, ws, p.k, xrows, wrows};
  if (__syncthreads_or(odd) && __syncthreads_or(scales_need_care(view))) {
    rare_quarter<BF16>(view, m0 - row0, nw - n0, p.out, row0, p.n, n0, p.a_row_scale);
    return;
  }
  store_quarter<4, 2, BF16>(acc, sh.out[wave], p.out, m0, row_end, p.n, nw, p.a_row_scale);
}

void launch_fp8_tiles(ProductArgs p, int out_dtype, hipStream_t st) {
  p.n_tiles = (p.n + kBN - 1) / kBN;
  const int64_t blocks = p.n_tiles * max_row_tiles(p.tokens, p.experts, kBM, p.offsets != nullptr);
  if (out_dtype == FP4_DTYPE_BF16)
    launch_1d(product_fp8_tiles_kernel<true>, blocks, 256, st, p);
  else
    launch_1d(product_fp8_tiles_kernel<false>, blocks, 256, st, p);
}

// Which kernel.  The few-row kernels' time follows the number of workgroups; that
// of the tiles hardly depends on it before the card is full.  So a plain product
// goes by the number of 32 x 32 workgroups it would take (k = 4096; us, 32 x 32 |
// tiles):
//   MXFP4 512: 13.5 | 20.4, 1024: 24.1 | 22.2, 2048: 45.0 | 22.6;
//   FP8 1024: 44.6 | 68, 2048: 87 | 68.
// The count does not tell tokens from columns, and a wide weight takes tiles for
// one token too (129280 x 7168; us, few-row | tiles): MXFP4 1 token 95 | 126, 32
// tokens 139 | 130; FP8 213 | 194 and 272 | 201.
// Below the tiles, up to 16 tokens take 16 x 16 a workgroup, the most workgroups
// (4096 x 7168 by one token: 4.8 us, 6.8 us with 32 x 32).
// Grouped, where weights are read once a row tile, by the mean of tokens a shard
// (32 Zipf shards, 2048 x 4096): MXFP4 32: 69 | 53; FP8 32: 133 | 100, 128: 393 |
// 112 (64 tokens by 2048 x 7168: 59 | 106).
// Of the MXFP4 tiles, 256 x 128 keeps more compute units busy and 256 x 256 feeds
// the matrix cores better (4096 x 4096; us, first | second): 2048 tokens, 256 tiles
// of the first, 27.4 | 32.1; 4096 tokens 49.8 | 38.8.  With shards under 256 tokens
// the second's rows stand empty (64 a shard: 86 | 102, 512 a shard: 261 | 209).
template <bool A8, bool KT>
void launch_product(const ProductArgs& p, int out_dtype, hipStream_t st) {
  const int64_t per = p.tokens / p.experts;
  const bool grouped = p.offsets != nullptr;
  const int64_t small = (int64_t)((p.n + 31) / 32) * ((p.tokens + 31) / 32);
  const bool tiles = p.k >= 128 && (grouped ? per >= (A8 ? 40 : 24) : small > (A8 ? 1600 : 768));
  if (!tiles) {
    if (p.tokens <= 16) launch_rows<A8, KT, 1, 1, 8, 4>(p, out_dtype, st);
    else launch_rows<A8, KT, 2, 2, 8, 2>(p, out_dtype, st);
  } else if constexpr (A8) {
    launch_fp8_tiles(p, out_dtype, st);
  } else {
    const int64_t wide = (int64_t)((p.n + 255) / 256) * max_row_tiles(p.tokens, p.experts, 128, grouped);
    if (wide > 256 && (!grouped || per >= 256)) launch_tiles<4, 4>(p, out_dtype, st);
    else launch_tiles<4, 2>(p, out_dtype, st);
  }
}

// Checks shared by both products; experts == 0 stands for the plain one.
int product(const void* a, int a_fmt, const void* a_scales, const float* a_row_scale,
            const uint8_t* w, const uint8_t* w_scales, const int64_t* offsets, int32_t experts,
            int64_t T, int64_t N, int64_t K, void* out, int out_dtype, void* stream) {
  if (a_fmt != FP4_ROWS_MXFP4 && a_fmt != FP4_ROWS_FP8) return FP4_EINVAL;
  const int osz = dtype_size(out_dtype);
  if (!osz) return FP4_EDTYPE;
  const int64_t E = experts ? experts : 1;
  if (T < 0 || N < 0 || K <= 0 || K % (a_fmt == FP4_ROWS_FP8 ? 128 : 32)) return FP4_ESHAPE;
  if (T >= (int64_t(1) << 26) || N >= (int64_t(1) << 26) || K >= (int64_t(1) << 21) ||
      E >= (int64_t(1) << 23))
    return FP4_ESHAPE;
  int64_t n_out, n_a, n_row, n_w;
  if (!checked_count(T, N, &n_out) || !checked_count(T, K, &n_a) || !checked_count(N, K, &n_row) ||
      !checked_count(E, n_row, &n_w))
    return FP4_ESHAPE;
  if (experts && !offsets) return FP4_EINVAL;
  if (n_out == 0) return FP4_OK;
  if (!a || !a_scales || !w || !w_scales || !out) return FP4_EINVAL;
  if (!is_aligned(a, 16) || !is_aligned(a_scales, 4) || !is_aligned(a_row_scale, 4) ||
      !is_aligned(w, 16) || !is_aligned(w_scales, 4) || !is_aligned(offsets, 8) ||
      !is_aligned(out, 16))
    return FP4_EALIGN;
  const bool a8 = a_fmt == FP4_ROWS_FP8;
  const void* ins[6] = {a, a_scales, a_row_scale, w, w_scales, offsets};
  const int64_t inn[6] = {a8 ? n_a : n_a / 2, a8 ? n_a / 128 * 4 : n_a / 32, T * 4,
                          n_w / 2,            n_w / 32,                      (E + 1) * 8};
  for (int i = 0; i < 6; ++i)
    if (overlaps(out, n_out * osz, ins[i], inn[i])) return FP4_EOVERLAP;
  ProductArgs p = {static_cast<const uint8_t*>(a), a_scales, a_row_scale, w, w_scales, offsets,
                   out, T, (int)E, (int)N, (int)K, 0};
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  if (a8)
    launch_product<true, false>(p, out_dtype, st);
  else if (K % 128)
    launch_product<false, true>(p, out_dtype, st);
  else
    launch_product<false, false>(p, out_dtype, st);
  return launch_status();
}

}  // namespace
}  // namespace fp4mi

using namespace fp4mi;

extern "C" int mxfp4_matmul(const void* a, int a_fmt, const void* a_scales,
                            const float* a_row_scale, const uint8_t* b, const uint8_t* b_scales,
                            int64_t M, int64_t N, int64_t K, void* out, int out_dtype,
                            void* stream) {
  return product(a, a_fmt, a_scales, a_row_scale, b, b_scales, nullptr, 0, M, N, K, out, out_dtype,
                 stream);
}

extern "C" int mxfp4_matmul_grouped(const void* a, int a_fmt, const void* a_scales,
                                    const float* a_row_scale, const uint8_t* w,
                                    const uint8_t* w_scales, const int64_t* token_offsets,
                                    int32_t num_experts, int64_t total_tokens, int64_t N,
                                    int64_t K, void* out, int out_dtype, void* stream) {
  if (num_experts < 1) return FP4_EINVAL;
  return product(a, a_fmt, a_scales, a_row_scale, w, w_scales, token_offsets, num_experts,
                 total_tokens, N, K, out, out_dtype, stream);
}
