// MXFP4 products, dense and grouped by expert.
#include <string.h>

#include "fp4mi_ops.h"
#include "host_common.hpp"
#include "mfma_common.hpp"

namespace fp4mi {
namespace {

// --------------------------------------------------------------- few rows
// One workgroup owns 16 FN columns of W by 16 FM tokens; its W waves take the
// steps of 128 k in turn, straight from memory to registers, U steps at a time
// with the next U in flight, and add their sums through LDS.
template <bool A8>
struct LaneStep {   // one lane's part of one 16-row operand at one step
  Frag<A8> v;
  int s;
};

// Row `row` of an operand at step `st`, group g.  KT: the last step may be
// short, and what lies past K counts as zero (and is not read).
template <bool A8, bool KT>
__device__ __forceinline__ void load_lane(const uint8_t* base, const void* scales, int64_t row,
                                          int k, int st, int g, LaneStep<A8>& o) {
  const int kk = st * 128 + 32 * g;
  const bool in = !KT || kk < k;
  const int at = in ? kk : 0;
  if constexpr (A8) {
    const i32x4* p = reinterpret_cast<const i32x4*>(base + row * k + at);
    o.v.lo = p[0];
    o.v.hi = p[1];
    o.s = (int)e8m0_of(static_cast<const float*>(scales)[row * (k >> 7) + (at >> 7)]);
  } else {
    o.v.lo = *reinterpret_cast<const i32x4*>(base + row * (k >> 1) + (at >> 1));
    o.s = static_cast<const uint8_t*>(scales)[row * (k >> 5) + (at >> 5)];
    if (KT && !in) {
      o.v.lo = i32x4{0, 0, 0, 0};
      o.s = 127;
    }
  }
}

template <bool A8, bool KT, int FN, int FM, int W, int U, bool BF16>
__global__ __launch_bounds__(64 * W) void product_rows_kernel(ProductArgs p, int64_t blk0) {
  __shared__ f32x4 red[W][FN * FM][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)(blk / p.n_tiles);
  int e = 0, row0 = mt * (16 * FM), row_end = (int)p.tokens;
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
  LaneStep<false> wc[U][FN], wx[U][FN];
  LaneStep<A8> ac[U][FM], ax[U][FM];
  auto load = [&](int c, LaneStep<false>(&lw)[U][FN], LaneStep<A8>(&la)[U][FM]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int st = min(c + u, steps - 1);
#pragma unroll
      for (int f = 0; f < FN; ++f) load_lane<false, KT>(w, ws, wn[f], p.k, st, g, lw[u][f]);
#pragma unroll
      for (int f = 0; f < FM; ++f) load_lane<A8, KT>(p.a, p.a_scales, am[f], p.k, st, g, la[u][f]);
    }
  };
  int c = wave * U;
  if (c < steps) load(c, wc, ac);
  for (; c < steps; c += W * U) {
    if (c + W * U < steps) load(c + W * U, wx, ax);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u >= steps) continue;
      if constexpr (A8) {
        mfma_bf16_step(wc[u], ac[u], acc);
      } else {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j)
            acc[i][j] = mfma_scaled<0, 0>(wc[u][i].v, ac[u][j].v, acc[i][j], wc[u][i].s,
                                                     ac[u][j].s);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int f = 0; f < FN; ++f) wc[u][f] = wx[u][f];
#pragma unroll
      for (int f = 0; f < FM; ++f) ac[u][f] = ax[u][f];
    }
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
// eight 16-byte chunks lie at position chunk ^ (row % 8), so that neither the
// line-wide direct loads nor the 32-row fragment reads meet a bank twice.
typedef float f32x16 __attribute__((ext_vector_type(16)));

typedef __amdgpu_buffer_rsrc_t buffer_t;
__device__ __forceinline__ buffer_t buffer_of(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
// 16 bytes a lane from base + v + s to l + 16 lane; l is the wave's.
__device__ __forceinline__ void load_to_lds(buffer_t b, uint32_t v, uint32_t s, void* l) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)l, 16, (int)v,
                                           (int)s, 0, 0);
}

template <int SA, int SB>
__device__ __forceinline__ f32x16 mfma_scaled32(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
  const i32x8 x = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, y = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, kE2M1, kE2M1, SA, sa, SB, sb);
}

// 16 scale bytes of a row of `bytes` >= 4 from byte `at`.  Past the row's end
// stand other bytes of the row: the codes there count as zero, and a NaN scale
// among them makes the same outputs NaN by itself.  FULL: there are none.
template <bool FULL>
__device__ __forceinline__ i32x4 load_scales16(const uint8_t* row, int at, int bytes) {
  i32x4 v;
  if (FULL || at + 16 <= bytes) {
    memcpy(&v, row + at, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int want = at + 4 * i, have = min(want, bytes - 4);
      uint32_t w;
      memcpy(&w, row + have, 4);
      v[i] = (int)(w >> (8 * min(want - have, 3)));
    }
  }
  return v;
}

template <int FN, int FM>
struct TileShared {
  uint8_t w[2][64 * FN * 128];
  uint8_t x[2][64 * FM * 128];
  // [k group][half of the rows][row % 32][row / 32 % F]: a lane's scale bytes
  // of its wave's fragments are one word
  uint8_t ws[2][8][2][32][FN];
  uint8_t xs[2][8][2][32][FM];
};

template <int FN, int FM, bool BF16>
__global__ __launch_bounds__(256, 1) void product_tiles_kernel(ProductArgs p, int64_t blk0) {
  static_assert(FN == 4 && (FM == 4 || FM == 2), "scale words");
  constexpr int BN = 64 * FN, BM = 64 * FM;
  __shared__ __align__(16) union {
    TileShared<FN, FM> t;
    uint8_t out[4][32 * (32 * FN * 4 + 16)];
  } sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)(blk / p.n_tiles);
  int e = 0, row0 = mt * BM, row_end = (int)p.tokens;
  if (p.offsets) {
    if (!locate_tile<BM>(p.offsets, p.experts, (int)p.tokens, mt, e, row0, row_end)) return;
  }
  const int n0 = nt * BN, kb = p.k >> 1, ksb = p.k >> 5;
  const uint8_t* w = p.w + ((int64_t)e * p.n) * kb;
  const uint8_t* ws = p.w_scales + (int64_t)e * p.n * ksb;
  const int wn = wave & 1, wm = wave >> 1;   // this wave's quarter
  const int stages = (p.k + 255) >> 8;

  // Direct loads: instruction i of this wave covers 8 rows; lane l is row
  // l / 8, position l % 8, which holds chunk (l % 8) ^ (row % 8).
  const int ch = (lane & 7) ^ (lane >> 3);
  const uint8_t* xa = p.a + (int64_t)row0 * kb;
  w += (int64_t)n0 * kb;
  ws += (int64_t)n0 * ksb;
  const int wrows = p.n - n0, xrows = row_end - row0;
  uint32_t wo[2 * FN], xo[2 * FM];
#pragma unroll
  for (int i = 0; i < 2 * FN; ++i)
    wo[i] = (uint32_t)min(8 * (wave * 2 * FN + i) + (lane >> 3), wrows - 1) * (uint32_t)kb + ch * 16;
#pragma unroll
  for (int i = 0; i < 2 * FM; ++i)
    xo[i] = (uint32_t)min(8 * (wave * 2 * FM + i) + (lane >> 3), xrows - 1) * (uint32_t)kb + ch * 16;
  const buffer_t wb = buffer_of(w, (int64_t)min(wrows, BN) * kb);
  const buffer_t xb = buffer_of(xa, (int64_t)min(xrows, BM) * kb);
  // Stage s into buffer B.  In a last stage that reaches past K, the chunks
  // there are other bytes of the tile: mask() has them count as zero.
  auto fetch = [&](auto b, auto full, int s) {
    constexpr int B = decltype(b)::value;
    if (decltype(full)::value || s * 256 + 256 <= p.k) {
#pragma unroll
      for (int i = 0; i < 2 * FN; ++i) load_to_lds(wb, wo[i], s * 128, &sh.t.w[B][(wave * 2 * FN + i) * 1024]);
#pragma unroll
      for (int i = 0; i < 2 * FM; ++i) load_to_lds(xb, xo[i], s * 128, &sh.t.x[B][(wave * 2 * FM + i) * 1024]);
    } else {
      const uint32_t past = (uint32_t)max(s * 128 + ch * 16 + 16 - kb, 0);
#pragma unroll
      for (int i = 0; i < 2 * FN; ++i) load_to_lds(wb, wo[i] + s * 128 - past, 0, &sh.t.w[B][(wave * 2 * FN + i) * 1024]);
#pragma unroll
      for (int i = 0; i < 2 * FM; ++i) load_to_lds(xb, xo[i] + s * 128 - past, 0, &sh.t.x[B][(wave * 2 * FM + i) * 1024]);
    }
  };
  // Scales: thread t owns row t of W's tile and row t % BM of X's; 16 bytes
  // serve two stages.
  const uint8_t* wsp = ws + (int64_t)min(tid, wrows - 1) * ksb;
  const uint8_t* xsp = static_cast<const uint8_t*>(p.a_scales) +
                       (int64_t)(row0 + min(tid % BM, xrows - 1)) * ksb;
  i32x4 wsc, xsc;
  auto fetch_scales = [&](auto full, int s) {
    wsc = load_scales16<decltype(full)::value>(wsp, s * 8, ksb);
    xsc = load_scales16<decltype(full)::value>(xsp, s * 8, ksb);
  };
  // of the pair's first or second stage; with half as many X rows, thread t
  // and t + BM write half of row t's bytes each
  uint8_t* wput = &sh.t.ws[0][0][tid / (32 * FN)][tid & 31][(tid >> 5) % FN];
  const int xr = tid % BM, xj = tid / BM * (8 * BM / 256);
  uint8_t* xput = &sh.t.xs[0][xj][xr / (32 * FM)][xr & 31][(xr >> 5) % FM];
  auto put_scales = [&](auto b) {
    constexpr int B = decltype(b)::value;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      wput[(B * 8 + j) * 64 * FN] = (uint8_t)((uint32_t)wsc[2 * B + (j >> 2)] >> (8 * (j & 3)));
    if constexpr (FM == 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        xput[(B * 8 + j) * 64 * FM] = (uint8_t)((uint32_t)xsc[2 * B + (j >> 2)] >> (8 * (j & 3)));
    } else {
        const uint32_t v = (uint32_t)(tid < BM ? xsc[2 * B] : xsc[2 * B + 1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) xput[(B * 8 + j) * 64 * FM] = (uint8_t)(v >> (8 * j));
    }
  };

  const int r = lane & 31, g = lane >> 5;
  struct Step {
    i32x4 w[FN], x[FM];
    int ws, xs;
  };
  const uint8_t *wl[4], *xl[4];   // this lane's chunk of its first fragment, for each 64 k
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const int c = ((2 * ks + g) ^ (r & 7)) * 16;
    wl[ks] = &sh.t.w[0][(wn * FN * 32 + r) * 128 + c];
    xl[ks] = &sh.t.x[0][(wm * FM * 32 + r) * 128 + c];
  }
  const uint8_t *wsl = &sh.t.ws[0][g][wn][r][0], *xsl = &sh.t.xs[0][g][wm][r][0];
  auto read = [&](auto b, int ks, Step& o) {   // 64 k of a stage
    constexpr int B = decltype(b)::value;
#pragma unroll
    for (int f = 0; f < FN; ++f)
      o.w[f] = *reinterpret_cast<const i32x4*>(wl[ks] + (B * BN + f * 32) * 128);
#pragma unroll
    for (int f = 0; f < FM; ++f)
      o.x[f] = *reinterpret_cast<const i32x4*>(xl[ks] + (B * BM + f * 32) * 128);
    o.ws = *reinterpret_cast<const int*>(wsl + (B * 8 + 2 * ks) * 64 * FN);
    if constexpr (FM == 4)
      o.xs = *reinterpret_cast<const int*>(xsl + (B * 8 + 2 * ks) * 64 * FM);
    else
      o.xs = *reinterpret_cast<const uint16_t*>(xsl + (B * 8 + 2 * ks) * 64 * FM);
  };
  f32x16 acc[FN][FM] = {};
  auto multiply = [&](const Step& o) {
#define FP4MI_ROW(I)                                                                   \
  acc[I][0] = mfma_scaled32<I, 0>(o.w[I], o.x[0], acc[I][0], o.ws, o.xs);              \
  acc[I][1] = mfma_scaled32<I, 1>(o.w[I], o.x[1], acc[I][1], o.ws, o.xs);              \
  if constexpr (FM == 4) {                                                             \
    acc[I][FM - 2] = mfma_scaled32<I, 2>(o.w[I], o.x[FM - 2], acc[I][FM - 2], o.ws, o.xs); \
    acc[I][FM - 1] = mfma_scaled32<I, 3>(o.w[I], o.x[FM - 1], acc[I][FM - 1], o.ws, o.xs); \
  }
    FP4MI_ROW(0) FP4MI_ROW(1) FP4MI_ROW(2) FP4MI_ROW(3)
#undef FP4MI_ROW
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
  fetch(first, no, 0);
  put_scales(first);
  landed();
  Step even, odd;
  read(first, 0, even);
  if (stages > 1) fetch(second, no, 1);
  // Stage s in buffer b, the next in nb.  MID: stages s + 1, s + 2 and, where b
  // is the first, s + 3 follow and end inside K; then nothing here branches, and
  // the loads, reads and products stay in the order written.
  auto stage = [&](auto b, auto nb, auto mid, int s) {
    constexpr bool MID = decltype(mid)::value;
    const bool more = MID || s + 1 < stages;
    read(b, 1, odd);
    if (!MID) mask(s, 0, even);
    multiply(even);
    __builtin_amdgcn_sched_barrier(0);
    read(b, 2, even);
    if (more) put_scales(nb);
    if (decltype(b)::value == 0 && (MID || s + 2 < stages)) fetch_scales(mid, s + 2);
    if (!MID) mask(s, 1, odd);
    multiply(odd);
    __builtin_amdgcn_sched_barrier(0);
    read(b, 3, odd);
    if (!MID) mask(s, 2, even);
    multiply(even);
    __builtin_amdgcn_sched_barrier(0);
    landed();   // stage s + 1; and everyone has read stage s
    if (more) read(nb, 0, even);
    if (MID || s + 2 < stages) fetch(b, mid, s + 2);
    if (!MID) mask(s, 3, odd);
    multiply(odd);
    __builtin_amdgcn_sched_barrier(0);
  };
  int s = 0;
  for (; s + 4 <= (p.k >> 8); s += 2) {
    stage(first, second, yes, s);
    stage(second, first, yes, s + 1);
  }
  for (; s < stages; s += 2) {
    stage(first, second, no, s);
    if (s + 1 < stages) stage(second, first, no, s + 1);
  }

  // Each wave turns its quarter through LDS, 32 tokens at a time, so that a
  // token's columns leave as whole lines.
  constexpr int kRow = 32 * FN * (BF16 ? 2 : 4) + 16;
  uint8_t* buf = sh.out[wave];
  const int nw = n0 + wn * 32 * FN;
  __syncthreads();
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    const int mbase = row0 + (wm * FM + fm) * 32;
    const float rs = p.a_row_scale ? p.a_row_scale[min(mbase + r, row_end - 1)] : 1.0f;
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = fn * 32 + 8 * q + 4 * g;
        const f32x16& c = acc[fn][fm];
        const f32x4 v = {c[4 * q] * rs, c[4 * q + 1] * rs, c[4 * q + 2] * rs, c[4 * q + 3] * rs};
        if constexpr (BF16)
          *reinterpret_cast<u32x2*>(buf + r * kRow + n * 2) =
              u32x2{pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
        else
          *reinterpret_cast<f32x4*>(buf + r * kRow + n * 4) = v;
      }
    __builtin_amdgcn_wave_barrier();
    constexpr int kLanes = 32 * FN * (BF16 ? 2 : 4) / 16;   // lanes a row takes
    constexpr int kEl = BF16 ? 8 : 4;
#pragma unroll
    for (int it = 0; it < 32 * kLanes / 64; ++it) {
      const int m = it * (64 / kLanes) + lane / kLanes, n = (lane % kLanes) * kEl;
      if (mbase + m < row_end)
        store_chunk<BF16>(p.out, mbase + m, p.n, nw + n, buf + m * kRow + (lane % kLanes) * 16);
    }
    __builtin_amdgcn_wave_barrier();
  }
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

template <bool A8, bool KT>
void launch_product(const ProductArgs& p, int out_dtype, hipStream_t st) {
  if constexpr (!A8) {
    const int64_t per = p.tokens / p.experts;
    if (per >= 512) return launch_tiles<4, 4>(p, out_dtype, st);
    if (per >= 128) return launch_tiles<4, 2>(p, out_dtype, st);
  }
  launch_rows<A8, KT, 2, 2, 4, 2>(p, out_dtype, st);
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
