// MXFP4 products, dense and grouped by expert.
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

template <bool A8, bool KT>
void launch_product(const ProductArgs& p, int out_dtype, hipStream_t st) {
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
