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
// One workgroup owns 16 FN columns of W by 16 FM tokens; each of its waves takes a
// run of the steps of 128 k, and their sums meet in LDS.  A wave's rows come by
// direct loads, a line of 128 bytes each, into NB buffers of its own, so it waits
// for nobody.  (Straight to registers 16 lanes read 16 rows, and each costs the
// cache a look-up: 64 tokens by 4096 x 4096 12.1 us so, 8.6 by way of LDS, 256 tokens
// 42.6 and 13.4.)  Bound by memory where the weights are large: 64 tokens over 32
// experts of 2048 x 7168 48 us, 5.5 TB/s; one token by 4096 x 7168 5.3 us.
// EXACT: products of bf16 values, added in fp32, in place of the scaled instruction,
// which drops the lowest bits of 8 products that it adds together.  One token 5.9 us,
// 64 over the 32 experts 47.8 for 47.3, 256 by 4096 x 4096 19.2 for 13.0.
template <int FN, int FM, int W, int NB, bool BF16, bool EXACT>
__global__ __launch_bounds__(64 * W) void fp8_rows_product_kernel(Fp8Args p, int64_t blk0) {
  static_assert(8 % NB == 0, "eight steps end where they began");
  constexpr int kLoads = 2 * (FN + FM), kStep = 16 * (FN + FM) * 128;
  __shared__ __align__(16) union {
    uint8_t rows[W][NB][kStep];   // W's, then A's; chunks placed as in the tiles below
    f32x4 red[W][FN * FM][64];
  } sh;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t blk = (int64_t)blockIdx.x + blk0;
  const int nt = (int)(blk % p.n_tiles), mt = (int)(blk / p.n_tiles);
  int e = 0, row0 = p.offsets ? 0 : mt * (16 * FM), row_end = (int)p.tokens;
  if (p.offsets) {
    if (!locate_tile<16 * FM>(p.offsets, p.experts, (int)p.tokens, mt, e, row0, row_end)) return;
  }
  const int r = lane & 15, g = lane >> 4, n0 = nt * (16 * FN), steps = p.k >> 7;
  const int wrows = min(p.n - n0, 16 * FN), xrows = min(row_end - row0, 16 * FM);
  const buffer_t wb = buffer_of(p.w + ((int64_t)e * p.n + n0) * p.k, (int64_t)wrows * p.k);
  const buffer_t xb = buffer_of(p.a + (int64_t)row0 * p.k, (int64_t)xrows * p.k);
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = 8 * (i < 2 * FN ? i : i - 2 * FN) + (lane >> 3);
    off[i] = (uint32_t)min(row, (i < 2 * FN ? wrows : xrows) - 1) * (uint32_t)p.k +
             (((lane & 7) ^ (((i & 1) << 2) | (lane >> 4))) << 4);
  }
  auto fetch = [&](int b, int c) {   // past the end the last step again, which nobody reads
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      load_to_lds(i < 2 * FN ? wb : xb, off[i], (uint32_t)min(c, steps - 1) * 128, &sh.rows[wave][b][i * 1024]);
  };
  // The scales of eight steps of each fragment's row, as bytes.  The compiler loads the upper
  // half of each word by itself, fragment after fragment, and waits for all there is
  // in flight: FN + FM times every eight steps.
  const float *ws[FN], *xs[FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
    ws[f] = p.w_scales + ((int64_t)e * p.scale_rows + ((n0 + min(16 * f + r, wrows - 1)) >> p.scale_shift)) * steps;
#pragma unroll
  for (int f = 0; f < FM; ++f) xs[f] = p.a_scales + (int64_t)(row0 + min(16 * f + r, xrows - 1)) * steps;
  auto scales8 = [&](const float* row, int c, uint32_t (&out)[2]) {
    uint32_t v[8];
    const int at = min(c, steps - 8), past = c - at;
    if (steps >= 8) {
      memcpy(v, row + at, 32);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(row[min(c + j, steps - 1)]);
    }
    uint64_t all = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) all |= (uint64_t)((v[j] >> 23) & 0xFFu) << (8 * j);
    if (steps >= 8) all >>= 8 * min(past, 7);
    out[0] = (uint32_t)all;
    out[1] = (uint32_t)(all >> 32);
  };

  f32x4 acc[FN][FM] = {};
  const uint8_t* mine = &sh.rows[wave][0][r * 128 + (((2 * g) ^ (r >> 1)) << 4)];
  const int flip = (r & 2) ? -16 : 16;
  const int c0 = wave * steps / W, c1 = (wave + 1) * steps / W;
  if (c0 < c1) {
#pragma unroll
    for (int b = 0; b < NB; ++b) fetch(b, c0 + b);
  }
  for (int c = c0; c < c1; c += 8) {
    uint32_t wq[FN][2], xq[FM][2];
#pragma unroll
    for (int f = 0; f < FN; ++f) scales8(ws[f], c, wq[f]);
#pragma unroll
    for (int f = 0; f < FM; ++f) scales8(xs[f], c, xq[f]);
    unrolled<8>([&](auto step) {
      constexpr int S = decltype(step)::value, B = S % NB;
      if (c + S >= c1) return;
      constexpr int kBehind = (NB - 1) * kLoads;
      __builtin_amdgcn_s_waitcnt(0x0F70 | (kBehind & 15) | (kBehind >> 4) << 14);   // vmcnt: this step has landed
      __builtin_amdgcn_wave_barrier();
      LaneStep<true> w[FN], x[FM];
      auto read = [&](int i, Frag<true>& v) {
        v.lo = *reinterpret_cast<const i32x4*>(mine + B * kStep + i * 16 * 128);
        v.hi = *reinterpret_cast<const i32x4*>(mine + flip + B * kStep + i * 16 * 128);
      };
#pragma unroll
      for (int f = 0; f < FN; ++f) read(f, w[f].v);
#pragma unroll
      for (int f = 0; f < FM; ++f) read(FN + f, x[f].v);
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): read, and free for the next
      __builtin_amdgcn_wave_barrier();
      fetch(B, c + S + NB);
      if constexpr (!EXACT) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                words(w[i].v), words(x[j].v), acc[i][j], kE4M3, kE4M3, S & 3, (int)wq[i][S >> 2], S & 3, (int)xq[j][S >> 2]);
      } else {
#pragma unroll
        for (int f = 0; f < FN; ++f) w[f].s = (int)((wq[f][S >> 2] >> (8 * (S & 3))) & 0xFFu);
#pragma unroll
        for (int f = 0; f < FM; ++f) x[f].s = (int)((xq[f][S >> 2] >> (8 * (S & 3))) & 0xFFu);
        mfma_bf16_step(w, x, acc);
      }
    });
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // what was asked for past the end has landed too
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) sh.red[wave][i * FM + j][lane] = acc[i][j];
  __syncthreads();
  for (int s = threadIdx.x; s < FN * FM * 64; s += 64 * W) {
    const int f = s >> 6, l = s & 63;
    f32x4 v = sh.red[0][f][l];
#pragma unroll
    for (int q = 1; q < W; ++q) v += sh.red[q][f][l];
    const int m = row0 + 16 * (f % FM) + (l & 15), n = n0 + 16 * (f / FM) + 4 * (l >> 4);
    if (m < row_end && n < p.n) {
      if (p.a_row_scale) v *= p.a_row_scale[m];
      store_out4<BF16>(p.out, m, p.n, n, v);
    }
  }
}

template <int FN, int FM, int W, int NB, bool BF16, bool EXACT>
void launch_rows(Fp8Args p, hipStream_t st) {
  p.n_tiles = (p.n + 16 * FN - 1) / (16 * FN);
  const int64_t blocks = p.n_tiles * max_row_tiles(p.tokens, p.experts, 16 * FM, p.offsets != nullptr);
  launch_1d(fp8_rows_product_kernel<FN, FM, W, NB, BF16, EXACT>, blocks, 64 * W, st, p);
}

// ------------------------------------------------------------- many rows
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
// 128 columns by `rows` tokens of a tile, 16 x 16 at a time straight from memory, for
// scales of any range.  Out of line, like the above, so that it costs the common
// path no registers.
template <bool BF16>
__device__ __attribute__((noinline)) void rare_quarter(Fp8View v, int mw, int rows, int nw, void* out,
                                                       int64_t out_row, int n_cols, const float* row_scale) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll 1
  for (int i = 0; i < rows / 2; ++i) {
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
// 8192^3 in 381 to 422 us from card to card, 2.6 to 2.9 PFLOP/s: the matrix cores are busy 73% of the cycles, at
// the 1.8 GHz that the card holds under this load; with loads and reads left out the
// products take 280.  Half blocks of k in four buffers, requests of 64 bytes and twice
// the barriers, took 431; touching the lines of later stages ahead made it slower
// (428), as the touch is waited for in its turn.  Where weights come from memory a
// stage waits for them (16384 tokens, 512 each for 32 experts of 4096 x 7168 420 us, the
// same product with one weight 343).
// Exact products (EXACT: fp32 outputs, or bf16 ones where the caller asks for them) are
// four 32 x 32 x 16 products of bf16 values, which hold code times scale exactly, in
// the place of a scaled one.  Their time is that of the products (twice the scaled
// one's) and of the conversions, which do not run beside them (16 cycles each, as many
// for two products as one takes; spread evenly between the products they cost the
// same): 8192^3 1018 to 1033 us, into bf16 1000.  32 and 48 vector registers are spilled
// there, behind the stages' loop and ahead of the output.
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

template <int FM, bool BF16>
union Fp8TileMemory {
  Fp8TileShared<FM> t;
  uint8_t out[4][quarter_bytes<4, BF16>()];
};
template <int FM, bool BF16, bool EXACT>
__device__ __forceinline__ void fp8_tile(const Fp8Args& p, Fp8TileMemory<FM, BF16>& sh, int e, int row0, int row_end,
                                         int nt) {
  constexpr int FN = 4, BM = 64 * FM, kAll = FN * FM, kLoads = 2 * (FN + FM);
  constexpr int kBuffers = Fp8TileShared<FM>::kBuffers, kStage = Fp8TileShared<FM>::kStage;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = nt * 256, stages = p.k >> 7;
  const int wrows = p.n - n0, xrows = row_end - row0;
  const uint8_t* w = p.w + ((int64_t)e * p.n + n0) * p.k;
  const uint8_t* x = p.a + (int64_t)row0 * p.k;
  const int wn = wave & 1, wm = wave >> 1;   // this wave's quarter

  // Direct loads: an instruction covers 8 rows; lane l is row l / 8, position l % 8,
  // which holds chunk position ^ (row / 2 % 8): of two kinds, by the instruction's parity.
  // A row's place is made up for each load; sixteen kept ones cost registers (fp32
  // outputs, 16383 tokens over 32 experts of 4096 x 7168 1451 us, 1470 with them kept).
  const uint32_t k8 = (uint32_t)p.k * 8u;
  const uint32_t own = (uint32_t)(lane >> 3) * (uint32_t)p.k;
  const uint32_t even = ((lane & 7) ^ (lane >> 4)) * 16u;
  const uint32_t wend = (uint32_t)(min(wrows, 256) - 1) * (uint32_t)p.k, xend = (uint32_t)(min(xrows, BM) - 1) * (uint32_t)p.k;
  const buffer_t wb = buffer_of(w, (int64_t)min(wrows, 256) * p.k);
  const buffer_t xb = buffer_of(x, (int64_t)min(xrows, BM) * p.k);
  auto fetch = [&](int at, int s, int i) {   // into buffer at; past the end the last stage again, which nobody reads
    const uint32_t so = (uint32_t)min(s, stages - 1) * 128;
    uint8_t* to = sh.t.rows[0] + at * kStage;
    const bool isw = i < 2 * FN;
    const int j = isw ? wave * 2 * FN + i : wave * 2 * FM + i - 2 * FN;
    const uint32_t v = min(own + (uint32_t)j * k8, isw ? wend : xend) + ((i & 1) ? even ^ 64u : even);
    load_to_lds(isw ? wb : xb, v, so, to + (isw ? 0 : 256 * 128) + j * 1024);
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
  bool odd = false;   // some scale is outside the bf16 window
  auto put_scales = [&](int s) {
    const int past = min(max(s - max(stages - 4, 0), 0), 3);   // stages past the end get any scale
    const auto pack = [&](u32x4& v) {
      asm volatile("" : "+v"(v));   // else each is loaded as its upper half alone
      if constexpr (EXACT) {
#pragma unroll
        for (int j = 0; j < 4; ++j) odd |= !scale_in_window((int)(v[j] >> 23 & 0xFFu));
      }
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
  // Exact products, four in the place of one scaled: place i of a half has quarter
  // i / FM, and of its FN FM products number 4 (i % FM) to + 3.  y: A's operands of
  // this quarter and the next, v: W's of this place and the next.
  constexpr int kOwn = 4 / FM;
  bf16x8_t y[2][FM], v[2][kOwn];
  auto scale_byte = [](int word, int f) { return scale_of((word >> (8 * f)) & 0xFF); };
  auto to_y = [&](auto quarter, int f, const Step& o, int scales) {
    constexpr int Q4 = decltype(quarter)::value;
    y[Q4 & 1][f] = bf16_of<Q4>(o.x[f], scale_byte(scales, f));
  };
  auto to_v = [&](auto place, const Step& o, int scales) {
    constexpr int i = decltype(place)::value;
#pragma unroll
    for (int d = 0; d < kOwn; ++d)
      v[i & 1][d] = bf16_of<i / FM>(o.w[i % FM * kOwn + d], scale_byte(scales, i % FM * kOwn + d));
  };
  // Stage s, s % 4 = Q; SCALES: its share of bringing the next four stages' scales.
  auto stage = [&](auto q, auto scales, int s) {
    constexpr int Q = decltype(q)::value;
    const int here = now;
    now = now + 1 == kBuffers ? 0 : now + 1;
    wsc = wsn;
    xsc = xsn;
    unrolled<2 * kAll>([&](auto idx) {
      constexpr int i = decltype(idx)::value, ks = i / kAll, j = i % kAll;
      if constexpr (!EXACT) {
        constexpr int I = j / FM, J = j % FM;
        acc[I][J] = mfma_fp8<I, J>(step[ks].w[I], step[ks].x[J], acc[I][J], wsc, xsc);
      } else {
        constexpr int q4 = j / FM, t = j % FM, next = (j + 1) % kAll;
        constexpr bool later = i == 2 * kAll - 1;   // the next place is the next stage's
        constexpr bool turn = q4 == 3;              // the next quarter is the next half's
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int I = (4 * t + c) / FM, J = (4 * t + c) % FM;
          acc[I][J] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[j & 1][I - t * kOwn], y[q4 & 1][J], acc[I][J], 0, 0, 0);
        }
        to_v(std::integral_constant<int, next>(), step[j + 1 == kAll ? 1 - ks : ks], later ? wsn : wsc);
        to_y(std::integral_constant<int, (q4 + 1) & 3>(), t, step[turn ? 1 - ks : ks], turn && ks == 1 ? xsn : xsc);
      }
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
  if constexpr (EXACT) {
#pragma unroll
    for (int f = 0; f < FM; ++f) to_y(std::integral_constant<int, 0>(), f, step[0], xsn);
    to_v(std::integral_constant<int, 0>(), step[0], wsn);
  }
  int s = 0;
  for (; s + 4 <= stages; s += 4) unrolled<4>([&](auto q) { stage(q, std::true_type(), s + decltype(q)::value); });
  for (; s < stages; s += 2) {
    stage(q0, std::false_type(), s);
    if (s + 1 >= stages) break;
    stage(q1, std::false_type(), s + 1);
  }
  __builtin_amdgcn_s_waitcnt(0x0070);   // what was asked for past the end has landed too
  __syncthreads();
  if constexpr (EXACT) {
    const Fp8View view = {x, w, p.a_scales + (int64_t)row0 * stages,
                          p.w_scales + (int64_t)e * p.scale_rows * stages, p.k, min(xrows, BM), wrows, n0, p.scale_shift};
    if (__syncthreads_or(odd) && __syncthreads_or(scales_need_care<BM>(view))) {
      rare_quarter<BF16>(view, wm * 32 * FM, 32 * FM, wn * 128, p.out, row0, p.n, p.a_row_scale);
      return;
    }
  }
  store_quarter<FN, FM, BF16>(acc, sh.out[wave], p.out, row0 + wm * 32 * FM, row_end, p.n, n0 + wn * 128,
                              p.a_row_scale);
}

template <bool BF16, bool EXACT>
__global__ __launch_bounds__(256, 1) void fp8_tiles_kernel(Fp8Args p, int64_t blk0) {
  __shared__ __align__(16) union {
    Fp8TileMemory<4, BF16> whole;
    Fp8TileMemory<2, BF16> half;
  } sh;
  int nt, mt, e, row0, row_end;
  bool half;
  place_tile(p, (int64_t)blockIdx.x + blk0, mt, nt);
  if (!locate_mixed(p, mt, e, row0, row_end, half)) return;
  if (half) fp8_tile<2, BF16, EXACT>(p, sh.half, e, row0, row_end, nt);
  else fp8_tile<4, BF16, EXACT>(p, sh.whole, e, row0, row_end, nt);
}

template <bool BF16, bool EXACT>
void launch_tiles(Fp8Args p, hipStream_t st) {
  const bool grouped = p.offsets != nullptr;
  p.n_tiles = (p.n + 255) / 256;
  p.m_tiles = max_row_tiles(p.tokens, p.experts, 256, grouped);
  p.tall = p.m_tiles * p.n_tiles > 192;
  if (!p.tall) p.m_tiles = max_row_tiles(p.tokens, p.experts, 128, grouped);
  launch_1d(fp8_tiles_kernel<BF16, EXACT>, p.n_tiles * p.m_tiles, 256, st, p);
}

// Which kernel.  A few-row kernel's time hardly changes while each of its workgroups
// has a compute unit to itself, and then grows with their number; the tiles' grows
// with theirs only from there.  So the smallest few-row tile with 256 workgroups or
// fewer is taken (4096 x 4096; us by columns x tokens of a workgroup, and tiles):
//   1 token    16 x 16 4.5, 32 x 16 5.4, 32 x 32 6.3, 64 x 32 7.5, 64 x 64 9.5, tiles 24
//   64 tokens  17.3, 13.6, 8.6, 8.7, 12.2, 25;  256 tokens  57, 46, 28, 16.6, 13.4, 25.
// With more workgroups than that, weights are read once a row tile, so the tile's
// tokens follow the tokens that there are, of a shard on average: up to a few 64 x 16
// (16 tokens by 16384 x 4096 13.7, 64 x 32 14.9, 32 x 16 17.6; 64 tokens over 32
// experts of 2048 x 4096 30.0, 33.5, 36.7), then 64 x 32 (256 tokens over the 32 46.8, 64 x
// 64 51.8, tiles 43), 64 x 64 (1024 tokens 68.6, 64 x 32 72.9, tiles 76) and the tiles
// (2048 tokens 87, 64 x 64 99).  Few experts leave the tiles few too, and 64 x 64 stays
// ahead (448 tokens over 5 of 1393 x 3328: 264 workgroups 15.4, tiles 24.2; 2000 over 16
// of 512 x 1024: 376 18.3, 11.4; dense 512 by 4096 x 4096: 512 25.8, 27.1, 1000 by 2000 x
// 2048: 512 20.6, 16.4).  With exact products the tiles take longer (fp32 outputs: 512
// tokens by 4096 x 4096: 64 x 64 38, tiles 67, 1024 tokens 75 both; 4096 tokens over the
// 32: 191, 273, 8192 tokens 349, 295).  The average is all that the host knows: where one shard of
// many experts has all the tokens, its weights are read once for each 16 to 64 of them
// (4096 tokens of 1024 experts of 512 x 1024 142 us, spread evenly 240, as one product 12).
template <bool BF16, bool EXACT>
void launch_product(const Fp8Args& p, hipStream_t st) {
  const int64_t per = p.tokens / p.experts;
  const bool grouped = p.offsets != nullptr;
  auto count = [&](int cols, int rows) {
    return (int64_t)((p.n + cols - 1) / cols) * max_row_tiles(p.tokens, p.experts, rows, grouped);
  };
  if (count(16, 16) <= 256) return launch_rows<1, 1, 8, 2, BF16, EXACT>(p, st);
  if (count(32, 16) <= 256) return launch_rows<2, 1, 8, 2, BF16, EXACT>(p, st);
  if (grouped ? per <= 4 : p.tokens <= 16) return launch_rows<4, 1, 4, 2, BF16, EXACT>(p, st);
  if (count(32, 32) <= 256) return launch_rows<2, 2, 4, 4, BF16, EXACT>(p, st);
  if (count(64, 32) <= 256 || (grouped && per <= 24)) return launch_rows<4, 2, 4, 2, BF16, EXACT>(p, st);
  if (count(64, 64) <= (EXACT ? 1024 : (grouped ? 288 : 384)) || (grouped && per <= (EXACT ? 160 : 40)))
    return launch_rows<4, 4, 4, 2, BF16, EXACT>(p, st);
  launch_tiles<BF16, EXACT>(p, st);
}

// Checks shared by both products; experts == 0 stands for the plain one.
int product(const uint8_t* a, const float* a_scales, const float* a_row_scale, const uint8_t* w,
            const float* w_scales, int block_rows, const int64_t* offsets, int32_t experts, int64_t T,
            int64_t N, int64_t K, void* out, int out_dtype, void* stream) {
  if (block_rows != 1 && block_rows != 128) return FP4_EINVAL;
  const bool exact = (out_dtype & FP4_EXACT) != 0;
  out_dtype &= ~FP4_EXACT;
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
  if (out_dtype == FP4_DTYPE_F32) launch_product<false, true>(p, as_stream(stream));
  else if (exact) launch_product<true, true>(p, as_stream(stream));
  else launch_product<true, false>(p, as_stream(stream));
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
