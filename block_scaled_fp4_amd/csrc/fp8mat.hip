// Products of FP8 rows with FP8 weights, dense and grouped by expert.
#include <string.h>

#include "fp4mi_moe.h"
#include "host_common.hpp"
#include "mfma_common.hpp"

namespace fp4mi {
namespace {

// Operands of C[t, :] = A[t, :] . W[e]^T, rows t of shard e.  offsets is null for
// a plain product (one shard of `tokens` rows).
struct Fp8Args {
  const uint8_t* a;          // E4M3 [T, K]
  const float* a_scales;     // [T, K/128]
  const float* a_row_scale;  // [T] or null
  const uint8_t* w;          // E4M3 [E, N, K]
  const float* w_scales;     // [E, scale_rows, K/128]
  const int64_t* offsets;    // [E + 1] or null
  void* out;                 // [T, N]
  int64_t tokens;
  int experts;
  int n, k;
  int scale_shift;           // row n's scales are row n >> scale_shift of w_scales
  int scale_rows;
  int n_tiles;               // tiles along N
  int64_t m_tiles;           // row tiles, or a bound on them
  bool tall;                 // row tiles of 256 with 128 for what is left, or of 128
};

// Tile of workgroup blk.  Workgroups go to the 8 XCDs in turn and an XCD runs 32 of
// these at a time, so of every 256 each XCD gets 32 that lie together: kPanel row
// tiles by 32 / kPanel column tiles, which share their operands in its cache.
constexpr int kPanel = 4;
__device__ __forceinline__ void place_tile(const Fp8Args& p, int64_t blk, int& mt, int& nt) {
  const int64_t total = p.m_tiles * p.n_tiles, base = blk & ~int64_t(255);
  const int count = (int)min(total - base, (int64_t)256), i = (int)(blk - base), x = i & 7;
  const int64_t id = base + x * (count >> 3) + min(x, count & 7) + (i >> 3);
  const int64_t panel = id / (kPanel * p.n_tiles);
  const int in = (int)(id - panel * kPanel * p.n_tiles), high = (int)min(p.m_tiles - panel * kPanel, (int64_t)kPanel);
  nt = in / high;
  mt = (int)(panel * kPanel) + in % high;
}

// Row tile mt: the shard, its first row and the shard's end; `half`: it has 128 rows
// and not 256.  Whole tiles of all shards (tall: a rest over 128 rows is one) come
// first, then the halves, which even out the end of the launch.  False past the
// last tile.  The result is the same in every lane.
__device__ __forceinline__ bool locate_mixed(const Fp8Args& p, int mt, int& e, int& row0, int& row_end, bool& half) {
  const int lane = threadIdx.x & 63, experts = p.offsets ? p.experts : 1;
  half = false;
#pragma unroll 1
  for (int pass = p.tall ? 0 : 1; pass < 2; ++pass) {
    int base = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < experts; e0 += 64) {
      int lo = 0, hi = 0;
      if (e0 + lane < experts) {
        if (p.offsets) shard_bounds(p.offsets, e0 + lane, (int)p.tokens, lo, hi);
        else hi = (int)p.tokens;
      }
      const int n = hi - lo, whole = (n + 127) >> 8;   // of 256 rows, a rest over 128 among them
      const int own = pass == 0 ? whole : (p.tall ? (n > whole << 8 ? 1 : 0) : (n + 127) >> 7);
      int sum = own;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(sum, d);
        if (lane >= d) sum += v;
      }
      const int total = __builtin_amdgcn_readlane(sum, 63);
      if (mt < base + total) {
        const int src = __builtin_ctzll(__ballot(base + sum > mt));
        const int nth = mt - base - __builtin_amdgcn_readlane(sum, src) + __builtin_amdgcn_readlane(own, src);
        e = e0 + src;
        half = pass == 1;
        row0 = __builtin_amdgcn_readlane(lo, src);
        row0 += half ? (p.tall ? __builtin_amdgcn_readlane(whole, src) << 8 : nth << 7) : nth << 8;
        row_end = __builtin_amdgcn_readlane(hi, src);
        return true;
      }
      base += total;
    }
    mt -= base;
  }
  return false;
}

constexpr int kE4M3 = 0;   // the scaled instruction's operand format field

__device__ __forceinline__ i32x8 words(const Frag<true>& f) {
  return i32x8{f.lo.x, f.lo.y, f.lo.z, f.lo.w, f.hi.x, f.hi.y, f.hi.z, f.hi.w};
}

// --------------------------------------------------------------- few rows
// One workgroup owns 16 FN columns of W by 16 FM tokens; its W waves take the
// steps of 128 k in turn, straight from memory to registers, U steps at a time
// with the next U in flight, and add their sums through LDS.
template <int FN, int FM, int W, int U, bool BF16>
__global__ __launch_bounds__(64 * W) void fp8_rows_product_kernel(Fp8Args p, int64_t blk0) {
  __shared__ f32x4 red[W][FN * FM][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)(blk / p.n_tiles);
  int e = 0, row0 = p.offsets ? 0 : mt * (16 * FM), row_end = (int)p.tokens;
  if (p.offsets) {
    if (!locate_tile<16 * FM>(p.offsets, p.experts, (int)p.tokens, mt, e, row0, row_end)) return;
  }
  const int r = lane & 15, g = lane >> 4, n0 = nt * (16 * FN), steps = p.k >> 7;
  const uint8_t* w = p.w + (int64_t)e * p.n * p.k + 32 * g;
  const float* ws = p.w_scales + (int64_t)e * p.scale_rows * steps;
  int wn[FN], am[FM];
#pragma unroll
  for (int f = 0; f < FN; ++f) wn[f] = min(n0 + 16 * f + r, p.n - 1);
#pragma unroll
  for (int f = 0; f < FM; ++f) am[f] = min(row0 + 16 * f + r, row_end - 1);

  f32x4 acc[FN][FM] = {};
  struct Batch {
    LaneStep<true> w[U][FN], a[U][FM];
  } even = {}, odd = {};   // in turn, so that no load is waited for before its use
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int f = 0; f < FM; ++f) even.a[u][f].s = odd.a[u][f].s = 127;   // of lanes without a token
  // U scales of a row from step c in one load where the row has them all
  auto load_scales = [&](const float* row, int c, uint32_t (&s)[U]) {
    if (c + U <= steps) {
      memcpy(s, row + c, 4 * U);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = __float_as_uint(row[min(c + u, steps - 1)]);
    }
  };
  auto load = [&](int c, Batch& b) {
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      uint32_t sc[U];
      load_scales(ws + (int64_t)(wn[f] >> p.scale_shift) * steps, c, sc);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const i32x4* q = reinterpret_cast<const i32x4*>(w + (int64_t)wn[f] * p.k + min(c + u, steps - 1) * 128);
        b.w[u][f].v.lo = q[0];
        b.w[u][f].v.hi = q[1];
        b.w[u][f].s = (int)((sc[u] >> 23) & 0xFFu);
      }
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      if (FM <= 2 && row0 + 16 * f + r >= row_end) continue;
      uint32_t sc[U];
      load_scales(p.a_scales + (int64_t)am[f] * steps, c, sc);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const i32x4* q = reinterpret_cast<const i32x4*>(p.a + (int64_t)am[f] * p.k + min(c + u, steps - 1) * 128 + 32 * g);
        b.a[u][f].v.lo = q[0];
        b.a[u][f].v.hi = q[1];
        b.a[u][f].s = (int)((sc[u] >> 23) & 0xFFu);
      }
    }
  };
  auto multiply = [&](int c, const Batch& b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u >= steps) continue;
      if constexpr (!BF16) {
        mfma_bf16_step(b.w[u], b.a[u], acc);
      } else {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                words(b.w[u][i].v), words(b.a[u][j].v), acc[i][j], kE4M3, kE4M3, 0, b.w[u][i].s, 0, b.a[u][j].s);
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

template <int FN, int FM, int W, int U>
void launch_rows(Fp8Args p, int out_dtype, hipStream_t st) {
  p.n_tiles = (p.n + 16 * FN - 1) / (16 * FN);
  const int64_t blocks = p.n_tiles * max_row_tiles(p.tokens, p.experts, 16 * FM, p.offsets != nullptr);
  if (out_dtype == FP4_DTYPE_BF16)
    launch_1d(fp8_rows_product_kernel<FN, FM, W, U, true>, blocks, 64 * W, st, p);
  else
    launch_1d(fp8_rows_product_kernel<FN, FM, W, U, false>, blocks, 64 * W, st, p);
}

// ---------------------------------------------- many rows, exact products
// What the rare path of a tile needs, from the tile's first rows.
struct Fp8View {
  const uint8_t *x, *w;
  const float *xs, *ws;   // ws: of the expert's first row
  int k, xrows, wrows, n0, shift;
};
__device__ __forceinline__ const float* weight_scales(const Fp8View& v, int row) {
  return v.ws + (int64_t)((v.n0 + row) >> v.shift) * (v.k >> 7);
}
// Whether some scale outside the bf16 window has codes to scale (a block of
// zeros has the smallest scale): the scales are read again, and codes where a
// scale is outside.
template <int BM>
__device__ __attribute__((noinline)) bool scales_need_care(Fp8View v) {
  const int wr = min((int)threadIdx.x % kBN, v.wrows - 1), xr = min((int)threadIdx.x % BM, v.xrows - 1);
  const int stages = v.k >> 7;
  const uint8_t *w = v.w + (int64_t)wr * v.k, *x = v.x + (int64_t)xr * v.k;
  const float *ws = weight_scales(v, wr), *xs = v.xs + (int64_t)xr * stages;
  auto zeros = [](const uint8_t* c) {
    const i32x4* q = reinterpret_cast<const i32x4*>(c);
    bool z = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) z &= zero_codes(Frag<true>{q[2 * i], q[2 * i + 1]});
    return z;
  };
  bool bad = false;
#pragma unroll 1
  for (int s0 = 0; s0 < stages; s0 += 8) {
    uint32_t sw[8], sx[8], odd = 0;   // bit j: w's stage s0 + j, bit 8 + j: x's
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sw[j] = e8m0_of(ws[min(s0 + j, stages - 1)]);
      sx[j] = e8m0_of(xs[min(s0 + j, stages - 1)]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bad |= sw[j] >= 228 || sx[j] >= 228;
      odd |= (scale_in_window((int)sw[j]) ? 0u : 1u << j) | (scale_in_window((int)sx[j]) ? 0u : 256u << j);
    }
#pragma unroll 1
    for (; odd; odd &= odd - 1) {
      const int j = __builtin_ctz(odd);
      bad |= !zeros((j < 8 ? w : x) + min(s0 + (j & 7), stages - 1) * 128);
    }
  }
  return bad;
}
__device__ __forceinline__ void load_step(const uint8_t* row, const float* scales, int s, int g,
                                          LaneStep<true>& o) {
  const i32x4* q = reinterpret_cast<const i32x4*>(row + s * 128 + 32 * g);
  o.v.lo = q[0];
  o.v.hi = q[1];
  o.s = (int)e8m0_of(scales[s]);
}
// A wave's 128 x 64 of a tile, 16 x 16 at a time straight from memory, for scales
// of any range.  Out of line, like the above, so that it costs the common path no
// registers.
template <bool BF16>
__device__ __attribute__((noinline)) void rare_quarter(Fp8View v, int mw, int nw, void* out,
                                                       int64_t out_row, int n_cols, const float* row_scale) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {
    const int m = mw + (i >> 3) * 16, n = nw + (i & 7) * 16;
    const int wr = min(n + r, v.wrows - 1), xr = min(m + r, v.xrows - 1);
    LaneStep<true> lw[1], lx[1];
    f32x4 c[1][1] = {};
#pragma unroll 1
    for (int s = 0; s < v.k >> 7; ++s) {
      load_step(v.w + (int64_t)wr * v.k, weight_scales(v, wr), s, g, lw[0]);
      load_step(v.x + (int64_t)xr * v.k, v.xs + (int64_t)xr * (v.k >> 7), s, g, lx[0]);
      mfma_bf16_step(lw, lx, c);
    }
    if (m + r < v.xrows) {
      if (row_scale) c[0][0] *= row_scale[out_row + m + r];
      store_out4<BF16>(out, out_row + m + r, n_cols, v.n0 + n + 4 * g, c[0][0]);
    }
  }
}

// See bf16_tile: W's rows are its operand A.
template <int WM, bool BF16>
__global__ __launch_bounds__(128 * WM, 1) void fp8_exact_tiles_kernel(Fp8Args p, int64_t blk0) {
  constexpr int kBM = 64 * WM, T = 128 * WM;
  __shared__ __align__(16) union {
    Bf16Shared<true, WM> t;
    uint8_t out[2 * WM][quarter_bytes<4, BF16>()];
  } sh;
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)(blk / p.n_tiles);
  int e = 0, row0 = p.offsets ? 0 : mt * kBM, row_end = (int)p.tokens;
  if (p.offsets) {
    if (!locate_tile<kBM>(p.offsets, p.experts, (int)p.tokens, mt, e, row0, row_end)) return;
  }
  const int n0 = nt * kBN, kx = p.k >> 7;
  const Fp8View v = {p.a + (int64_t)row0 * p.k, p.w + ((int64_t)e * p.n + n0) * p.k,
                     p.a_scales + (int64_t)row0 * kx, p.w_scales + (int64_t)e * p.scale_rows * kx,
                     p.k, row_end - row0, p.n - n0, n0, p.scale_shift};
  constexpr int kLW = kBN * 8 / T, kLX = kBM * 8 / T;
  uint32_t wo[kLW], xo[kLX];
  const int tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < kLW; ++i)
    wo[i] = (uint32_t)min((tid >> 3) + T / 8 * i, v.wrows - 1) * (uint32_t)p.k + (tid & 7) * 16;
#pragma unroll
  for (int i = 0; i < kLX; ++i)
    xo[i] = (uint32_t)min((tid >> 3) + T / 8 * i, v.xrows - 1) * (uint32_t)p.k + (tid & 7) * 16;
  f32x16 acc[4][2] = {};
  const bool odd = bf16_tile<true, WM>(
      sh.t, kx, kx,
      [&](auto, int s, int i) { return *reinterpret_cast<const i32x4*>(v.w + s * 128 + wo[i]); },
      [&](auto, int s, int i) { return *reinterpret_cast<const i32x4*>(v.x + s * 128 + xo[i]); },
      [](int, int, i32x4&) {}, [](int, int, i32x4&) {},
      [&](int s, int row) { return e8m0_of(weight_scales(v, min(row, v.wrows - 1))[s]); },
      [&](int s, int row) { return e8m0_of(v.xs[(int64_t)min(row, v.xrows - 1) * kx + s]); }, acc);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), mw = (wave >> 1) * 64, nw = (wave & 1) * 128;
  if (__syncthreads_or(odd) && __syncthreads_or(scales_need_care<kBM>(v))) {
    rare_quarter<BF16>(v, mw, nw, p.out, row0, p.n, p.a_row_scale);
    return;
  }
  store_quarter<4, 2, BF16>(acc, sh.out[wave], p.out, row0 + mw, row_end, p.n, n0 + nw, p.a_row_scale);
}

template <int WM>
void launch_exact_tiles(Fp8Args p, int out_dtype, hipStream_t st) {
  p.n_tiles = (p.n + kBN - 1) / kBN;
  const int64_t blocks = p.n_tiles * max_row_tiles(p.tokens, p.experts, 64 * WM, p.offsets != nullptr);
  if (out_dtype == FP4_DTYPE_BF16)
    launch_1d(fp8_exact_tiles_kernel<WM, true>, blocks, 128 * WM, st, p);
  else
    launch_1d(fp8_exact_tiles_kernel<WM, false>, blocks, 128 * WM, st, p);
}

// ------------------------------------------------ many rows, bf16 outputs
// One workgroup of four waves owns 256 columns of W by 64 FM tokens, each wave 128
// by 32 FM in 32 x 32 x 64 scaled instructions (lane l: row l % 32, the 32 k of
// group l / 32; D's lane l: column l % 32, rows 8 (i / 4) + 4 (l / 32) + i % 4).
// A stage is a scale block of 128 k: whole lines of 128 bytes of every row go to
// LDS with direct loads, kBuffers stages in turn.  While one half of a stage is
// multiplied from registers the next half's fragments are read; once a stage's
// second half is read, the waves meet, and a later stage is asked for into its
// buffer.
// A row's eight 16-byte chunks lie at position chunk ^ (row / 2 % 8): 16 rows of a
// fragment read take every bank once.
template <int FM>
struct Fp8TileShared {
  static constexpr int kBuffers = FM == 4 ? 2 : 3, kStage = (256 + 64 * FM) * 128;
  uint8_t rows[kBuffers][kStage];   // W's, then A's
  // scales of eight stages: bytes of rows r, r + 32, .. of a wave's half
  uint32_t ws[8][2][32], xs[8][2][32];
};

template <int SA, int SB>
__device__ __forceinline__ f32x16 mfma_fp8(const Frag<true>& a, const Frag<true>& b, f32x16 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(words(a), words(b), c, kE4M3, kE4M3, SA, sa, SB, sb);
}

template <int FM>
union Fp8TileMemory {
  Fp8TileShared<FM> t;
  uint8_t out[4][quarter_bytes<4, true>()];
};
template <int FM>
__device__ __forceinline__ void fp8_tile(const Fp8Args& p, Fp8TileMemory<FM>& sh, int e, int row0, int row_end,
                                         int nt) {
  constexpr int FN = 4, BM = 64 * FM, kAll = FN * FM, kLoads = 2 * (FN + FM);
  constexpr int kBuffers = Fp8TileShared<FM>::kBuffers, kStage = Fp8TileShared<FM>::kStage;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = nt * 256, stages = p.k >> 7;
  const int wrows = p.n - n0, xrows = row_end - row0;
  const uint8_t* w = p.w + ((int64_t)e * p.n + n0) * p.k;
  const uint8_t* x = p.a + (int64_t)row0 * p.k;
  const int wn = wave & 1, wm = wave >> 1;   // this wave's quarter

  // Direct loads: an instruction covers 8 rows; lane l is row l / 8, position l % 8.
  auto ch = [&](int i) { return (lane & 7) ^ (((i & 1) << 2) | (lane >> 4)); };
  uint32_t wo[2 * FN], xo[2 * FM];
#pragma unroll
  for (int i = 0; i < 2 * FN; ++i)
    wo[i] = (uint32_t)min(8 * (wave * 2 * FN + i) + (lane >> 3), wrows - 1) * (uint32_t)p.k + ch(i) * 16;
#pragma unroll
  for (int i = 0; i < 2 * FM; ++i)
    xo[i] = (uint32_t)min(8 * (wave * 2 * FM + i) + (lane >> 3), xrows - 1) * (uint32_t)p.k + ch(i) * 16;
  const buffer_t wb = buffer_of(w, (int64_t)min(wrows, 256) * p.k);
  const buffer_t xb = buffer_of(x, (int64_t)min(xrows, BM) * p.k);
  auto fetch = [&](int at, int s, int i) {   // into buffer at; past the end the last stage again, which nobody reads
    const uint32_t so = (uint32_t)min(s, stages - 1) * 128;
    uint8_t* to = sh.t.rows[0] + at * kStage;
    if (i < 2 * FN) load_to_lds(wb, wo[i < 2 * FN ? i : 0], so, to + (wave * 2 * FN + i) * 1024);
    else load_to_lds(xb, xo[i < 2 * FN ? 0 : i - 2 * FN], so, to + 256 * 128 + (wave * 2 * FM + i - 2 * FN) * 1024);
  };
  // Scales, four stages at a time: thread t those of row t of either operand.
  const float* ws = p.w_scales + ((int64_t)e * p.scale_rows + ((n0 + min(tid, wrows - 1)) >> p.scale_shift)) * stages;
  const float* xs = p.a_scales + (int64_t)(row0 + min(tid % BM, xrows - 1)) * stages;
  u32x4 wq, xq;
  auto fetch_scales = [&](int s) {   // of four stages or more, the last four where s + 3 is past the end
    const int at = min(s, stages - 4);
    memcpy(&wq, ws + at, 16);
    memcpy(&xq, xs + at, 16);
  };
  auto put_scales = [&](int s) {
    const int past = min(max(s - max(stages - 4, 0), 0), 3);   // stages past the end get any scale
    const auto pack = [&](u32x4& v) {
      asm volatile("" : "+v"(v));   // else each is loaded as its upper half alone
      const uint32_t lo = (v[0] >> 23 & 0xFFu) | (v[1] >> 15 & 0xFF00u);
      const uint32_t all = lo | (v[2] >> 7 & 0xFF0000u) | (v[3] << 1 & 0xFF000000u);
      return all >> (8 * past);
    };
    const uint32_t wb4 = pack(wq), xb4 = pack(xq);
    const int wat = (tid >> 7) * 128 + (tid & 31) * 4 + ((tid >> 5) & 3);
    const int xat = tid % BM / (32 * FM) * 128 + (tid & 31) * 4 + (tid >> 5) % FM;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      reinterpret_cast<uint8_t*>(sh.t.ws)[((s + j) & 7) * 256 + wat] = (uint8_t)(wb4 >> (8 * j));
      reinterpret_cast<uint8_t*>(sh.t.xs)[((s + j) & 7) * 256 + xat] = (uint8_t)(xb4 >> (8 * j));
    }
  };

  const int r = lane & 31, g = lane >> 5;
  struct Step {
    Frag<true> w[FN], x[FM];
  };
  Step step[2];
  int wsc, xsc, wsn, xsn;   // scale words of this stage and the next
  const uint8_t *wl[2], *xl[2];   // this lane's first chunk of its first fragment, for either half
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    const int c = ((4 * ks + 2 * g) ^ ((r >> 1) & 7)) * 16;
    wl[ks] = sh.t.rows[0] + (wn * 128 + r) * 128 + c;
    xl[ks] = sh.t.rows[0] + (256 + wm * 32 * FM + r) * 128 + c;
  }
  // Piece i of the fragments of half ks of the stage in buffer at: chunk i % 2 of
  // fragment i / 2.  The second chunk is the first's neighbour, at position ^ 1.
  const int flip = ((r >> 1) & 1) ? -16 : 16;
  auto read = [&](int at, int ks, int i, Step& o) {
    const int f = i >> 1, c = ((i & 1) ? flip : 0) + at * kStage;
    i32x4& to = f < FN ? ((i & 1) ? o.w[f < FN ? f : 0].hi : o.w[f < FN ? f : 0].lo)
                       : ((i & 1) ? o.x[f < FN ? 0 : f - FN].hi : o.x[f < FN ? 0 : f - FN].lo);
    to = f < FN ? *reinterpret_cast<const i32x4*>(wl[ks] + c + f * 32 * 128)
                : *reinterpret_cast<const i32x4*>(xl[ks] + c + (f - FN) * 32 * 128);
  };
  auto read_scales = [&](int s) {
    wsn = (int)sh.t.ws[s & 7][wn][r];
    xsn = (int)sh.t.xs[s & 7][wm][r];
  };
  f32x16 acc[FN][FM] = {};

  // Of the 2 kAll products of a stage: the second half's 2 (FN + FM) pieces are read
  // behind kRead of them; behind product kMeet the waves have all read this stage,
  // and the loads into its buffer follow, kLoadPer a product; behind product kLand
  // the next stage has landed, and its first half is read.
  constexpr int kPieces = 2 * (FN + FM), kRead = kAll == 16 ? 8 : 4, kPer = (kPieces + kRead - 1) / kRead;
  constexpr int kMeet = kAll == 16 ? 11 : 6, kLoadPer = kAll == 16 ? 1 : 2, kLand = kAll == 16 ? 17 : 8;
  int now = 0;   // the buffer of stage s
  // Stage s, s % 4 = Q; SCALES: its share of bringing the next four stages' scales.
  auto stage = [&](auto q, auto scales, int s) {
    constexpr int Q = decltype(q)::value;
    const int here = now;
    now = now + 1 == kBuffers ? 0 : now + 1;
    wsc = wsn;
    xsc = xsn;
    unrolled<2 * kAll>([&](auto idx) {
      constexpr int i = decltype(idx)::value, I = i % kAll / FM, J = i % FM, ks = i / kAll;
      acc[I][J] = mfma_fp8<I, J>(step[ks].w[I], step[ks].x[J], acc[I][J], wsc, xsc);
      if constexpr (i < kRead) {
#pragma unroll
        for (int c = i * kPer; c < (i + 1) * kPer; ++c)
          if (c < kPieces) read(here, 1, c, step[1]);
      }
      if constexpr (i > kLand && i <= kLand + kRead) {
#pragma unroll
        for (int c = (i - kLand - 1) * kPer; c < (i - kLand) * kPer; ++c)
          if (c < kPieces) read(now, 0, c, step[0]);
      }
      if constexpr (i == kLand + kRead) read_scales(s + 1);
      if constexpr (decltype(scales)::value && Q == 0 && i == kLand + 1) fetch_scales(s + 4);
      if constexpr (decltype(scales)::value && Q == 2 && i == kRead) put_scales(s + 2);
      if constexpr (i == kMeet) {
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
      }
      if constexpr (i == kLand) {
        constexpr int kNew = (kLand - kMeet - 1) * kLoadPer;
        constexpr int kBehind = (kBuffers - 2) * kLoads + (kNew < kLoads ? kNew : kLoads);
        __builtin_amdgcn_s_waitcnt(0x0F70 | (kBehind & 15) | (kBehind >> 4) << 14);   // vmcnt
        __builtin_amdgcn_s_barrier();
      }
      if constexpr (i > kMeet) {
#pragma unroll
        for (int c = (i - kMeet - 1) * kLoadPer; c < (i - kMeet) * kLoadPer; ++c)
          if (c < kLoads) fetch(here, s + kBuffers, c);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    // the sums are made here: left to itself the compiler moves the products past
    // every branch that follows, to the end of the loop
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) asm volatile("" : "+a"(acc[i][j]));
  };

  constexpr std::integral_constant<int, 0> q0{};
  constexpr std::integral_constant<int, 1> q1{};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    wq[j] = __float_as_uint(ws[min(j, stages - 1)]);
    xq[j] = __float_as_uint(xs[min(j, stages - 1)]);
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) fetch(0, 0, i);
  put_scales(0);
#pragma unroll
  for (int b = 1; b < kBuffers; ++b)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) fetch(b, b, i);
  constexpr int kBehind = (kBuffers - 1) * kLoads;
  __builtin_amdgcn_s_waitcnt(0x0070 | (kBehind & 15) | (kBehind >> 4) << 14);   // stage 0 has landed
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) read(0, 0, i, step[0]);
  read_scales(0);
  int s = 0;
  for (; s + 4 <= stages; s += 4) unrolled<4>([&](auto q) { stage(q, std::true_type(), s + decltype(q)::value); });
  for (; s < stages; s += 2) {
    stage(q0, std::false_type(), s);
    if (s + 1 >= stages) break;
    stage(q1, std::false_type(), s + 1);
  }
  __builtin_amdgcn_s_waitcnt(0x0070);   // what was asked for past the end has landed too
  __syncthreads();
  store_quarter<FN, FM, true>(acc, sh.out[wave], p.out, row0 + wm * 32 * FM, row_end, p.n, n0 + wn * 128,
                              p.a_row_scale);
}

__global__ __launch_bounds__(256, 1) void fp8_tiles_kernel(Fp8Args p, int64_t blk0) {
  __shared__ __align__(16) union {
    Fp8TileMemory<4> whole;
    Fp8TileMemory<2> half;
  } sh;
  int nt, mt, e, row0, row_end;
  bool half;
  place_tile(p, (int64_t)blockIdx.x + blk0, mt, nt);
  if (!locate_mixed(p, mt, e, row0, row_end, half)) return;
  if (half) fp8_tile<2>(p, sh.half, e, row0, row_end, nt);
  else fp8_tile<4>(p, sh.whole, e, row0, row_end, nt);
}

void launch_tiles(Fp8Args p, hipStream_t st) {
  const bool grouped = p.offsets != nullptr;
  p.n_tiles = (p.n + 255) / 256;
  p.m_tiles = max_row_tiles(p.tokens, p.experts, 256, grouped);
  p.tall = p.m_tiles * p.n_tiles > 192;
  if (!p.tall) p.m_tiles = max_row_tiles(p.tokens, p.experts, 128, grouped);
  launch_1d(fp8_tiles_kernel, p.n_tiles * p.m_tiles, 256, st, p);
}

void launch_product(const Fp8Args& p, int out_dtype, hipStream_t st) {
  const int64_t per = p.tokens / p.experts;
  const bool grouped = p.offsets != nullptr;
  const int64_t small = (int64_t)((p.n + 31) / 32) * ((p.tokens + 31) / 32);
  const bool tiles = grouped ? per >= 40 : small > 1600;
  if (!tiles) {
    if (p.tokens <= 16) launch_rows<1, 1, 8, 4>(p, out_dtype, st);
    else launch_rows<2, 2, 8, 2>(p, out_dtype, st);
  } else if (out_dtype == FP4_DTYPE_BF16) {
    launch_tiles(p, st);
  } else {
    launch_exact_tiles<2>(p, out_dtype, st);
  }
}

// Checks shared by both products; experts == 0 stands for the plain one.
int product(const uint8_t* a, const float* a_scales, const float* a_row_scale, const uint8_t* w,
            const float* w_scales, int block_rows, const int64_t* offsets, int32_t experts, int64_t T,
            int64_t N, int64_t K, void* out, int out_dtype, void* stream) {
  if (block_rows != 1 && block_rows != 128) return FP4_EINVAL;
  const int osz = dtype_size(out_dtype);
  if (!osz) return FP4_EDTYPE;
  const int64_t E = experts ? experts : 1;
  if (T < 0 || N < 0 || K <= 0 || K % 128) return FP4_ESHAPE;
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
      !is_aligned(w, 16) || !is_aligned(w_scales, 4) || !is_aligned(offsets, 8) || !is_aligned(out, 16))
    return FP4_EALIGN;
  const int64_t scale_rows = block_rows == 1 ? N : (N + 127) / 128;
  const void* ins[6] = {a, a_scales, a_row_scale, w, w_scales, offsets};
  const int64_t inn[6] = {n_a, n_a / 32, T * 4, n_w, E * scale_rows * (K / 128) * 4, (E + 1) * 8};
  for (int i = 0; i < 6; ++i)
    if (overlaps(out, n_out * osz, ins[i], inn[i])) return FP4_EOVERLAP;
  Fp8Args p = {a, a_scales, a_row_scale, w, w_scales, offsets, out, T, (int)E, (int)N, (int)K,
               block_rows == 1 ? 0 : 7, (int)scale_rows, 0, 0, false};
  clear_stale_error();
  launch_product(p, out_dtype, as_stream(stream));
  return launch_status();
}

}  // namespace
}  // namespace fp4mi

using namespace fp4mi;

extern "C" int fp8_matmul(const uint8_t* a, const float* a_scales, const float* a_row_scale,
                          const uint8_t* b, const float* b_scales, int b_block_rows, int64_t M,
                          int64_t N, int64_t K, void* out, int out_dtype, void* stream) {
  return product(a, a_scales, a_row_scale, b, b_scales, b_block_rows, nullptr, 0, M, N, K, out,
                 out_dtype, stream);
}

extern "C" int fp8_matmul_grouped(const uint8_t* a, const float* a_scales, const float* a_row_scale,
                                  const uint8_t* w, const float* w_scales, int w_block_rows,
                                  const int64_t* token_offsets, int32_t num_experts,
                                  int64_t total_tokens, int64_t N, int64_t K, void* out,
                                  int out_dtype, void* stream) {
  if (num_experts < 1) return FP4_EINVAL;
  return product(a, a_scales, a_row_scale, w, w_scales, w_block_rows, token_offsets, num_experts,
                 total_tokens, N, K, out, out_dtype, stream);
}
