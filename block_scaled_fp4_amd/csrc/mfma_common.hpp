// Shared by the matrix-product kernels: the scaled matrix instruction, E8M0
// helpers, expert shards and the output epilogue.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 computes D[i][j] += sum_k A[i][k] 2^(sa-127)
// B[j][k] 2^(sb-127) over 128 values of k.  Lane l holds, of either operand,
// row l % 16 and the 32 consecutive k from 32 g, g = l / 16 -- 16 bytes of E2M1
// codes, one MX block, so each lane supplies the E8M0 byte of its own block.
// D's lane l holds column l % 16 and rows 4 g .. 4 g + 3.
// The weights are operand A throughout, so a lane ends with four consecutive
// output columns of one token and stores them as one vector.
#pragma once

#include <type_traits>
#include <utility>

#include "lane_common.hpp"

namespace fp4mi {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kE2M1 = 4;   // the instruction's operand format field

// The 16 or 32 bytes one lane holds of an operand.
template <bool F8>
struct Frag {
  i32x4 lo;
};
template <>
struct Frag<true> {
  i32x4 lo, hi;
};

// SA, SB: which byte of the scale words sa, sb this instruction uses.
template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma_scaled(const Frag<false>& a, const Frag<false>& b, f32x4 c,
                                             int sa, int sb) {
  const i32x8 x = {a.lo.x, a.lo.y, a.lo.z, a.lo.w, 0, 0, 0, 0};
  const i32x8 y = {b.lo.x, b.lo.y, b.lo.z, b.lo.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, kE2M1, kE2M1, SA, sa, SB, sb);
}

// Products with an FP8 operand.  The scaled instruction lines the products of
// adjacent k up with the largest of them and drops what lies 14 bits or more
// below it; over E4M3's 18 binades that costs about 2e-5 of a sum (measured on
// Gaussian rows), which is not a sum in fp32.  E2M1 by E2M1 spans 8 bits within
// a block and loses nothing, whatever the other blocks' scales are (of a block
// that cancels 2^0 to 2^40 above its neighbour the rest is 0.2 of fp32's last
// place at most).  E4M3 goes through bf16 products, which are exact and are
// added in fp32 (6e-8 measured), at half the scaled instruction's rate: with
// MXFP4 weights, in the weight gradient, and of FP8 by FP8 wherever the output is
// fp32 or the caller asks for exact products; other bf16 outputs of FP8 by FP8
// take the scaled instruction, as their entry points state.  A lane then holds the 32 consecutive k from 32 g of both operands, and
// instruction q of four takes its 8 from 8 q.
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ bf16x8_t join(bf16x2_t a, bf16x2_t b, bf16x2_t c, bf16x2_t d) {
  return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
template <int Q>
__device__ __forceinline__ bf16x8_t bf16_of(const Frag<false>& f, float scale) {
  const uint32_t w = (uint32_t)f.lo[Q];
  return join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0),
              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1),
              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2),
              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
}
template <int Q>
__device__ __forceinline__ bf16x8_t bf16_of(const Frag<true>& f, float scale) {
  const uint32_t a = (uint32_t)(Q < 2 ? f.lo[(2 * Q) & 3] : f.hi[(2 * Q) & 3]);
  const uint32_t b = (uint32_t)(Q < 2 ? f.lo[(2 * Q + 1) & 3] : f.hi[(2 * Q + 1) & 3]);
  return join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false),
              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true),
              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false),
              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true));
}
// 2^(byte - 127) as the converters' scale operand.
__device__ __forceinline__ float scale_of(int byte) { return __uint_as_float((uint32_t)byte << 23); }

// Scales 2^-100 .. 2^100: code times scale is then a normal bf16 value.
__device__ __forceinline__ bool scale_in_window(int byte) { return (unsigned)(byte - 27) <= 200u; }
// So does any scale but NaN over codes that are all zero (a block of zeros has
// byte 0).
__device__ __forceinline__ bool zero_codes(const Frag<false>& f) {
  return ((f.lo.x | f.lo.y | f.lo.z | f.lo.w) & 0x77777777) == 0;
}
__device__ __forceinline__ bool zero_codes(const Frag<true>& f) {
  return ((f.lo.x | f.lo.y | f.lo.z | f.lo.w | f.hi.x | f.hi.y | f.hi.z | f.hi.w) & 0x7F7F7F7F) == 0;
}
template <typename L>
__device__ __forceinline__ bool scale_fits(const L& f) {
  return scale_in_window(f.s) || (f.s < 228 && zero_codes(f.v));
}

// The four instructions of a step, with scale(i) for row fragment i.
template <int N, int M, typename LA, typename LB, typename SA, typename SB>
__device__ __forceinline__ void bf16_quarters(const LA (&a)[N], const LB (&b)[M], SA sa, SB sb,
                                              f32x4 (&acc)[N][M]) {
  auto quarter = [&](auto q) {
    bf16x8_t x[N], y[M];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = bf16_of<decltype(q)::value>(a[i].v, sa(i));
#pragma unroll
    for (int j = 0; j < M; ++j) y[j] = bf16_of<decltype(q)::value>(b[j].v, sb(j));
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < M; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y[j], acc[i][j], 0, 0, 0);
  };
  quarter(std::integral_constant<int, 0>());
  quarter(std::integral_constant<int, 1>());
  quarter(std::integral_constant<int, 2>());
  quarter(std::integral_constant<int, 3>());
}

// 16 x 16 x 128 of the above: N row fragments of A by M of B, fragments with
// their scale byte (.v, .s).  If any lane's scale is outside the window (a NaN
// scale included), the step's four blocks of 32 run one by one on the bare
// codes, and the two scales multiply each block's sum in fp32.
template <int N, int M, typename LA, typename LB>
__device__ __forceinline__ void mfma_bf16_step(const LA (&a)[N], const LB (&b)[M], f32x4 (&acc)[N][M]) {
  bool fine = true;
#pragma unroll
  for (int i = 0; i < N; ++i) fine &= scale_in_window(a[i].s);
#pragma unroll
  for (int j = 0; j < M; ++j) fine &= scale_in_window(b[j].s);
  if (!__all(fine)) {
    fine = true;
#pragma unroll
    for (int i = 0; i < N; ++i) fine &= scale_fits(a[i]);
#pragma unroll
    for (int j = 0; j < M; ++j) fine &= scale_fits(b[j]);
  }
  if (__all(fine)) {
    bf16_quarters(a, b, [&](int i) { return scale_of(a[i].s); },
                  [&](int j) { return scale_of(b[j].s); }, acc);
    return;
  }
  const int g = (threadIdx.x & 63) >> 4, r = threadIdx.x & 15;
#pragma unroll 1
  for (int blk = 0; blk < 4; ++blk) {
    LA one[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      one[i] = a[i];
      if (g != blk) one[i].v = {};
    }
    f32x4 part[N][M] = {};
    bf16_quarters(one, b, [](int) { return 1.0f; }, [](int) { return 1.0f; }, part);
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int sb = __shfl(b[j].s, 16 * blk + r);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int sa = __shfl(a[i].s, 16 * blk + 4 * g + c);
          acc[i][j][c] += (sa == 255 || sb == 255) ? __builtin_nanf("")
                                                   : ldexpf(part[i][j][c], sa + sb - 254);
        }
    }
  }
}

// A power-of-two fp32 scale as its E8M0 byte (2^-127, an fp32 subnormal, is
// byte 0); sign and fraction bits are not read.
__device__ __forceinline__ uint32_t e8m0_of(float s) {
  return (__float_as_uint(s) >> 23) & 0xFFu;
}

template <bool A8>
struct LaneStep {   // one lane's part of one 16-row operand at one step
  Frag<A8> v;
  int s;
};

// Row `row` of an operand at step `st`, group g.
template <bool A8>
__device__ __forceinline__ void load_lane(const uint8_t* base, const void* scales, int64_t row,
                                          int k, int st, int g, LaneStep<A8>& o) {
  const int at = st * 128 + 32 * g;
  if constexpr (A8) {
    const i32x4* p = reinterpret_cast<const i32x4*>(base + row * k + at);
    o.v.lo = p[0];
    o.v.hi = p[1];
    o.s = (int)e8m0_of(static_cast<const float*>(scales)[row * (k >> 7) + st]);
  } else {
    o.v.lo = *reinterpret_cast<const i32x4*>(base + row * (k >> 1) + (at >> 1));
    o.s = static_cast<const uint8_t*>(scales)[row * (k >> 5) + (at >> 5)];
  }
}

// ------------------------------------------------------ direct loads to LDS
typedef __amdgpu_buffer_rsrc_t buffer_t;
__device__ __forceinline__ buffer_t buffer_of(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
// 16 bytes a lane from base + v + s to l + 16 lane; l is the wave's.
__device__ __forceinline__ void load_to_lds(buffer_t b, uint32_t v, uint32_t s, void* l) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)l, 16, (int)v,
                                           (int)s, 0, 0);
}

// Operands of C[t, :] = A[t, :] . W[e]^T, rows t of shard e.  offsets is
// null for a plain product (one shard of `tokens` rows).
struct ProductArgs {
  const uint8_t* a;          // MXFP4 [T, K/2] or E4M3 [T, K]
  const void* a_scales;      // UE8M0 [T, K/32] or fp32 [T, K/128]
  const float* a_row_scale;  // fp32 [T] or null
  const uint8_t* w;          // [E, N, K/2]
  const uint8_t* w_scales;   // [E, N, K/32]
  const int64_t* offsets;    // [E + 1] or null
  void* out;                 // [T, N]
  int64_t tokens;
  int experts;
  int n, k;
  int n_tiles;               // tiles along N
};

// Rows [lo, hi) of `tokens` that shard e owns; malformed offsets are clamped,
// so that whatever they hold every access stays inside the buffers.
__device__ __forceinline__ void shard_bounds(const int64_t* off, int e, int tokens, int& lo,
                                             int& hi) {
  const int64_t a = off[e], b = off[e + 1];
  lo = (int)(a < 0 ? 0 : (a > tokens ? tokens : a));
  hi = (int)(b < lo ? lo : (b > tokens ? tokens : b));
}

// The shard and first row of row tile `mt`, tiles counted shard by shard with
// ceil(n_e / BM) each.  A wave looks at 64 shards at a time: each lane counts
// its shard's tiles and a prefix sum finds the one that holds mt.  False past
// the last tile.  The result is the same in every lane.
template <int BM>
__device__ __forceinline__ bool locate_tile(const int64_t* off, int experts, int tokens, int mt,
                                            int& e, int& row0, int& row_end) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < experts; e0 += 64) {
    int lo = 0, hi = 0;
    if (e0 + lane < experts) shard_bounds(off, e0 + lane, tokens, lo, hi);
    const int own = (hi - lo + BM - 1) / BM;
    int sum = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    const int total = __builtin_amdgcn_readlane(sum, 63);
    if (mt < base + total) {
      const int src = __builtin_ctzll(__ballot(base + sum > mt));
      const int before = base + __builtin_amdgcn_readlane(sum, src) - __builtin_amdgcn_readlane(own, src);
      e = e0 + src;
      row0 = __builtin_amdgcn_readlane(lo, src) + (mt - before) * BM;
      row_end = __builtin_amdgcn_readlane(hi, src);
      return true;
    }
    base += total;
  }
  return false;
}

// Row tiles of at most this many exist: sum ceil(n_e / bm) over non-empty shards.
inline int64_t max_row_tiles(int64_t tokens, int64_t experts, int bm, bool grouped) {
  return grouped ? tokens / bm + (experts < tokens ? experts : tokens) : (tokens + bm - 1) / bm;
}

// Four consecutive columns n .. n+3 of one output row, rounded once to the
// output type (fp32 sums to here); columns past the row's end are dropped.  A row
// may begin at any element: whole vectors are stored at any alignment of it.
template <bool BF16>
__device__ __forceinline__ void store_out4(void* out, int64_t row, int n_cols, int n, f32x4 v) {
  if constexpr (BF16) {
    uint16_t* p = static_cast<uint16_t*>(out) + row * n_cols + n;
    const u32x2 w = {pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
    if (n + 4 <= n_cols) {
      __builtin_memcpy(p, &w, 8);
    } else {
      if (n < n_cols) p[0] = (uint16_t)w.x;
      if (n + 1 < n_cols) p[1] = (uint16_t)(w.x >> 16);
      if (n + 2 < n_cols) p[2] = (uint16_t)w.y;
    }
  } else {
    float* p = static_cast<float*>(out) + row * n_cols + n;
    if (n + 4 <= n_cols) {
      __builtin_memcpy(p, &v, 16);
    } else {
      if (n < n_cols) p[0] = v.x;
      if (n + 1 < n_cols) p[1] = v.y;
      if (n + 2 < n_cols) p[2] = v.z;
    }
  }
}

// 16 bytes at `src`: eight bf16 or four fp32 consecutive columns from n of one
// output row, which may begin at any element; columns past its end are dropped (6061
// tokens by 5668 x 768 in FP8: 72 us element by element).  Nontemporal: outputs of
// whole tiles would push the operands out of the caches (plain stores against
// these: the gradient of 16 x 4096 x 7168 1100 | 1072 us, 5001 tokens by 13 x
// 7168 x 2048 170 | 159 us, 8192^3 in MXFP4 260 | 256 us).
template <bool BF16>
__device__ __forceinline__ void store_chunk(void* out, int64_t row, int n_cols, int n,
                                            const uint8_t* src) {
  constexpr int kEl = BF16 ? 8 : 4;
  uint8_t* dst = static_cast<uint8_t*>(out) + (row * n_cols + n) * (16 / kEl);
  if (n + kEl <= n_cols) {
    typedef u32x4 anywhere __attribute__((aligned(2)));
    __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(src), reinterpret_cast<anywhere*>(dst));
  } else {
#pragma unroll 1
    for (int j = 0; j < min(kEl, n_cols - n); ++j) {
      if constexpr (BF16)
        reinterpret_cast<uint16_t*>(dst)[j] = reinterpret_cast<const uint16_t*>(src)[j];
      else
        reinterpret_cast<uint32_t*>(dst)[j] = reinterpret_cast<const uint32_t*>(src)[j];
    }
  }
}

// f(integral_constant<int, 0>) .. f(integral_constant<int, N - 1>)
template <typename F, int... I>
__device__ __forceinline__ void unrolled_seq(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unrolled(F f) {
  unrolled_seq(f, std::make_integer_sequence<int, N>());
}

// A wave's quarter of a tile, 32 FN columns from `n0` by 32 FM tokens from
// `m0`, in 32 x 32 fragments (D's lane l: column l % 32 = the token, rows
// 8 (i / 4) + 4 (l / 32) + i % 4 = the columns of the output).  32 tokens at a
// time are turned through `buf`, so that a token's columns leave as whole lines
// and not as 16 bytes each; the padding keeps the rows on different banks.
template <int FN, bool BF16>
constexpr int quarter_bytes() {
  return 32 * (32 * FN * (BF16 ? 2 : 4) + 16);
}
template <int FN, int FM, bool BF16>
__device__ __forceinline__ void store_quarter(const f32x16 (&acc)[FN][FM], uint8_t* buf, void* out,
                                              int64_t m0, int64_t row_end, int n_cols, int n0,
                                              const float* row_scale) {
  constexpr int kRow = quarter_bytes<FN, BF16>() / 32;
  constexpr int kLanes = 32 * FN * (BF16 ? 2 : 4) / 16, kEl = BF16 ? 8 : 4;   // lanes a row takes
  const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
  float scale[FM];
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    const int64_t m = m0 + fm * 32 + r;
    scale[fm] = row_scale ? row_scale[m < row_end ? m : row_end - 1] : 1.0f;
  }
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    const int64_t mbase = m0 + fm * 32;
    const float rs = scale[fm];
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
#pragma unroll
    for (int it = 0; it < 32 * kLanes / 64; ++it) {
      const int t = it * (64 / kLanes) + lane / kLanes, n = (lane % kLanes) * kEl;
      if (mbase + t < row_end)
        store_chunk<BF16>(out, mbase + t, n_cols, n0 + n, buf + t * kRow + (lane % kLanes) * 16);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ------------------------------------------------ tiles of bf16 products
// The E4M3 products at size: one workgroup of 2 WM waves owns 256 rows of
// operand A (the output's columns) by 64 WM of operand B, each wave 128 x 64 of
// them in 32 x 32 x 16 instructions.  A stage is 128 k.  Codes are staged
// through registers into LDS as they are, two stages in turn with one barrier
// each, and become bf16 values on their way to the instructions; each wave
// converts 12 operand rows' worth for 64 instructions' time.
//
// E4M3 rows are 8 chunks of 16 bytes, chunk c at position c ^ (row / 2 % 8); E2M1
// rows are 4 chunks, c at c ^ (row / 4 % 4): 16 consecutive rows then touch
// every bank once.  Scales lie beside for 8 stages at a time, one byte a row and
// stage (E4M3, one block of 128) or four (E2M1): a stage's own few bytes of
// each row would cost as many cache lines as its codes.
constexpr int kBN = 256;

template <bool A8, int WM>
struct Bf16Shared {
  static constexpr int kA = A8 ? 128 : 64;   // bytes of a row of A
  static constexpr int kBM = 64 * WM;
  uint8_t a[2][kBN * kA];
  uint8_t b[2][kBM * 128];
  uint8_t as[8][kBN * (A8 ? 1 : 4)];
  uint8_t bs[8][kBM];
};

// load_a(first, s, i), load_b: a thread's i-th 16 bytes of stage s (the first
// stage, where `first` says so), chunk tid % C of row tid / C + i (threads / C),
// C chunks a row; from stage full_stages on, cut_a(s, i, v), cut_b make of them
// what counts, once they are there.  scale_a(s, row): the row's word of four bytes (E2M1) or its byte
// (E4M3), scale_b(s, row): its byte.  Returns whether some scale that this
// thread loaded was outside the window.
template <bool A8, int WM, typename LA, typename LB, typename CA, typename CB, typename SA,
          typename SB>
__device__ __forceinline__ bool bf16_tile(Bf16Shared<A8, WM>& sh, int stages, int full_stages,
                                          LA load_a, LB load_b, CA cut_a, CB cut_b, SA scale_a, SB scale_b,
                                          f32x16 (&acc)[4][2]) {
  constexpr int T = 128 * WM, kBM = 64 * WM;
  constexpr int kPerA = Bf16Shared<A8, WM>::kA / 16, kLA = kBN * kPerA / T, kLB = kBM * 8 / T;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1, r = lane & 31, g = lane >> 5;
  i32x4 ra[kLA], rb[kLB];
  bool odd_scale = false;
  auto fetch_some = [&](auto first, int s, int from, int to) {
#pragma unroll
    for (int i = 0; i < kLA + kLB; ++i) {
      if (i < from || i >= to) continue;
      if (i < kLA) ra[i < kLA ? i : 0] = load_a(first, s, i);
      else rb[i < kLA ? 0 : i - kLA] = load_b(first, s, i - kLA);
    }
  };
  // T / C is a multiple of 16, so a thread's rows share their place in the pattern
  const int put8 = (tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 4) & 7)) << 4);
  const int put4 = (tid >> 2) * 64 + (((tid & 3) ^ ((tid >> 4) & 3)) << 4);
  auto put = [&](int s) {
    const int b = s & 1;
    if (s >= full_stages) {
#pragma unroll
      for (int i = 0; i < kLA; ++i) cut_a(s, i, ra[i]);
#pragma unroll
      for (int i = 0; i < kLB; ++i) cut_b(s, i, rb[i]);
    }
#pragma unroll
    for (int i = 0; i < kLA; ++i)
      *reinterpret_cast<i32x4*>(&sh.a[b][(A8 ? put8 : put4) + i * T * 16]) = ra[i];
#pragma unroll
    for (int i = 0; i < kLB; ++i) *reinterpret_cast<i32x4*>(&sh.b[b][put8 + i * T * 16]) = rb[i];
  };
  // the scales of stages 8 grp .. 8 grp + 7
  auto put_scales = [&](int grp) {
    uint32_t va[8], vb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = min(8 * grp + j, stages - 1);
      va[j] = scale_a(s, tid % kBN);
      vb[j] = scale_b(s, tid % kBM);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (A8) {
        sh.as[j][tid % kBN] = (uint8_t)va[j];
        odd_scale |= !scale_in_window((int)va[j]);
      } else {
        reinterpret_cast<uint32_t*>(sh.as[j])[tid % kBN] = va[j];
#pragma unroll
        for (int q = 0; q < 4; ++q) odd_scale |= !scale_in_window((int)((va[j] >> (8 * q)) & 0xFFu));
      }
      sh.bs[j][tid % kBM] = (uint8_t)vb[j];
      odd_scale |= !scale_in_window((int)vb[j]);
    }
  };
  const int rb0 = (wm * 64 + r) * 128, ra0 = (wn * 128 + r) * Bf16Shared<A8, WM>::kA;
  // Fragment f of A, and both of B, for the ks-th 64 k of stage s, as codes.
  auto read_a = [&](int s, int ks, int f, Frag<A8>& v, float& sc) {
    const int b = s & 1, sj = s & 7;
    const int c0 = ((4 * ks + 2 * g) ^ ((r >> 1) & 7)) << 4, c4 = ((2 * ks + g) ^ ((r >> 2) & 3)) << 4;
    if constexpr (A8) {
      v.lo = *reinterpret_cast<const i32x4*>(&sh.a[b][ra0 + f * 32 * 128 + c0]);
      v.hi = *reinterpret_cast<const i32x4*>(&sh.a[b][ra0 + f * 32 * 128 + (c0 ^ 16)]);
      sc = scale_of(sh.as[sj][wn * 128 + f * 32 + r]);
    } else {
      v.lo = *reinterpret_cast<const i32x4*>(&sh.a[b][ra0 + f * 32 * 64 + c4]);
      sc = scale_of(sh.as[sj][(wn * 128 + f * 32 + r) * 4 + 2 * ks + g]);
    }
  };
  auto read_b = [&](int s, int ks, Frag<true> (&v)[2], float (&sc)[2]) {
    const int b = s & 1, sj = s & 7, c0 = ((4 * ks + 2 * g) ^ ((r >> 1) & 7)) << 4;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      v[f].lo = *reinterpret_cast<const i32x4*>(&sh.b[b][rb0 + f * 32 * 128 + c0]);
      v[f].hi = *reinterpret_cast<const i32x4*>(&sh.b[b][rb0 + f * 32 * 128 + (c0 ^ 16)]);
      sc[f] = scale_of(sh.bs[sj][wm * 64 + f * 32 + r]);
    }
  };
  // before(i), i = 0 .. 7: ahead of the i-th eighth.  With E4M3 on both sides each
  // eighth's fragments are read an eighth earlier (16 x 4096 x 7168: 1072 us, read
  // in place 1086); with E2M1 two workgroups share the registers and cover the
  // reads, and the registers that this takes cost more (5001 tokens by 13 x 7168 x
  // 2048: in place 159 us, earlier 166).
  auto compute = [&](int s, auto before) {
    Frag<A8> va[2];
    Frag<true> vb[2];
    float sa[2], sb[2];
    if constexpr (A8) {
      read_b(s, 0, vb, sb);
      read_a(s, 0, 0, va[0], sa[0]);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      bf16x8_t y[2][4];
      if constexpr (!A8) read_b(s, ks, vb, sb);
#pragma unroll
      for (int f = 0; f < 2; ++f)
        unrolled<4>([&](auto q) { y[f][q] = bf16_of<decltype(q)::value>(vb[f], sb[f]); });
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int i = ks * 4 + f;
        __builtin_amdgcn_sched_barrier(0);
        before(i);
        if constexpr (A8) {
          if (i < 7) read_a(s, (i + 1) >> 2, (i + 1) & 3, va[(i + 1) & 1], sa[(i + 1) & 1]);
          if (i == 3) read_b(s, 1, vb, sb);
          __builtin_amdgcn_sched_barrier(0);
        } else {
          read_a(s, ks, f, va[i & 1], sa[i & 1]);
        }
        unrolled<4>([&](auto q) {
          const bf16x8_t x = bf16_of<decltype(q)::value>(va[i & 1], sa[i & 1]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[f][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y[j][q], acc[f][j], 0, 0, 0);
        });
      }
    }
  };
  if (stages == 0) return false;
  fetch_some(std::true_type(), 0, 0, kLA + kLB);
  put_scales(0);
  put(0);
  __syncthreads();
  for (int s = 0; s < stages; ++s) {
    // the next stage's loads go out an eighth at a time: issued together they
    // would hold the products up until the last is taken
    const int next = min(s + 1, stages - 1);
    compute(s, [&](int i) {
      fetch_some(std::false_type(), next, i * (kLA + kLB) / 8, (i + 1) * (kLA + kLB) / 8);
    });
    // the products stay before what follows: sums left for later would be
    // moved past the branches to the end of the loop
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(acc[f][j]));
    put(s + 1);
    __syncthreads();
    if ((s & 7) == 7) {   // past the barrier all have read these eight
      put_scales(s / 8 + 1);
      __syncthreads();
    }
  }
  return odd_scale;
}

}  // namespace fp4mi
