// The router's balance loss, the tokens of each expert, and the loss' gradient.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "fp4mi_moe.h"
#include "host_common.hpp"
#include "rows_common.hpp"

namespace fp4mi {
namespace {

constexpr int kMaxExperts = 4096;

// Four elements from element i, at any alignment of their type.
template <bool BF16>
__device__ __forceinline__ f32x4 load4(const void* base, int64_t i) {
  if constexpr (BF16) {
    u32x2 w;
    memcpy(&w, static_cast<const uint16_t*>(base) + i, 8);
    return f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
  } else {
    f32x4 v;
    memcpy(&v, static_cast<const float*>(base) + i, 16);
    return v;
  }
}
template <bool BF16>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
  if constexpr (BF16) return bf16_lo(static_cast<const uint16_t*>(base)[i]);
  else return static_cast<const float*>(base)[i];
}
template <bool BF16>
__device__ __forceinline__ void store4(void* base, int64_t i, f32x4 v) {
  if constexpr (BF16) {
    const u32x2 w = {pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
    memcpy(static_cast<uint16_t*>(base) + i, &w, 8);
  } else {
    memcpy(static_cast<float*>(base) + i, &v, 16);
  }
}
template <bool BF16>
__device__ __forceinline__ void store1(void* base, int64_t i, float v) {
  if constexpr (BF16) static_cast<uint16_t*>(base)[i] = (uint16_t)pack_bf16x2(v, v);
  else static_cast<float*>(base)[i] = v;
}

// A row of E values over L lanes, 4 CH of them a lane: chunk c of lane l holds
// columns 4 (c L + l) .. + 3, `fill` past the row's end.
template <bool BF16, int L, int CH>
__device__ __forceinline__ void load_row(const void* base, int64_t row, int experts, int l, float fill,
                                         f32x4 (&v)[CH]) {
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = 4 * (c * L + l);
    if (e + 4 <= experts) {
      v[c] = load4<BF16>(base, row * experts + e);
    } else {
      v[c] = f32x4{fill, fill, fill, fill};
      for (int j = 0; j < 3; ++j)
        if (e + j < experts) v[c][j] = load1<BF16>(base, row * experts + e + j);
    }
  }
}

// f over the L lanes of a row, in every one of them, without LDS.
template <int L, typename F>
__device__ __forceinline__ float over_lanes(float v, F f) {
  v = f(v, lane_xor1(v));
  v = f(v, lane_xor2(v));
  v = f(v, other_quad(v));
  if constexpr (L >= 16) v = f(v, other_eight(v));
  if constexpr (L >= 32) {   // both halves of the pair, each in both
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  if constexpr (L >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  return v;
}

// exp(x - max) of a row in place; returns the factor that makes them its softmax.  The
// maximum is subtracted before log2(e) is multiplied in: times it, a type's lowest
// value is infinite, and a maximum past 2^30 is rounded by more than the exponent
// holds.  A row of -inf alone becomes zeros; NaN and +inf make the factor NaN.
// exp2's argument is rounded once more than the difference x - max itself, and as much
// (half of fp32's last place each), so p is off by 2.1e-7 (relative, root mean
// square) where exp of the difference gives 1.5e-7; exp_f32 in its place took 65536 x 256
// from 26 to 29 us, its gradient in bf16 from 22 to 25.
template <int L, int CH>
__device__ __forceinline__ float softmax_row(f32x4 (&v)[CH]) {
  float top = -INFINITY;
#pragma unroll
  for (int c = 0; c < CH; ++c) top = fmaxf(fmaxf(fmaxf(v[c].x, v[c].y), fmaxf(v[c].z, v[c].w)), top);
  top = over_lanes<L>(top, [](float a, float b) { return fmaxf(a, b); });
  constexpr float kLog2e = 0x1.715476p+0f;
  const float from = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[c][j] = __builtin_amdgcn_exp2f((v[c][j] - from) * kLog2e);
      sum += v[c][j];
    }
  }
  sum = over_lanes<L>(sum, [](float a, float b) { return a + b; });
  return sum == 0.0f ? 0.0f : 1.0f / sum;
}

struct BalanceArgs {
  const void* x;
  const void* idx;
  const uint8_t* mask;
  int64_t tokens;
  int64_t slots;       // tokens * k
  int experts, k;
  float coef;
  float* loss;
  int32_t* counts;
  int64_t* offsets;
  float* grad;
  float* part_p;       // [blocks, E]
  int32_t* part_c;     // [blocks, E]
  int32_t* part_n;     // [blocks]
  double* part_loss;   // [join blocks]
  uint32_t* joined;    // join blocks that are done
  int blocks;
};

// The sums of the counts before each expert, by one wave.
template <typename F>
__device__ __forceinline__ void write_offsets(const BalanceArgs& p, int lane, F count) {
  int64_t base = 0;
  for (int e0 = 0; e0 < p.experts; e0 += 64) {
    const int own = e0 + lane < p.experts ? count(e0 + lane) : 0;
    int sum = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(sum, d);
      if (lane >= d) sum += v;
    }
    if (e0 + lane < p.experts) p.offsets[e0 + lane] = base + sum - own;
    base += __builtin_amdgcn_readlane(sum, 63);
  }
  if (lane == 0) p.offsets[p.experts] = base;
}

// A workgroup adds its rows' p in registers, row after row, its waves' sums in the
// order of the waves, and leaves them, its counts and its number of counted tokens in
// the workspace.  A call of one workgroup ends here.
// The rows asked for ahead are on their way in fp32.  bf16 is unpacked inside load_row's
// branch, which waits for each load there: 65536 x 256 28 us, in fp32 26; 20000 x 2500 133
// and 89.
constexpr int kRowsAhead = 2;
template <bool BF16, bool IDX64, int L, int CH, int W>
__global__ __launch_bounds__(64 * W) void balance_kernel(BalanceArgs p) {
  constexpr int R = 64 / L, kWide = L * CH * 4;   // rows a wave takes at once, columns
  __shared__ f32x4 sums[W][kWide / 4];
  __shared__ int hist[kWide];
  __shared__ int counted[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & (L - 1), sub = lane / L;
  for (int e = tid; e < kWide; e += 64 * W) hist[e] = 0;
  if (blockIdx.x == 0 && tid == 0) *p.joined = 0;
  __syncthreads();
  constexpr int D = CH <= 2 ? kRowsAhead : 1;
  f32x4 acc[CH] = {}, ahead[D][CH];
  int n = 0, in[D];
  const int64_t step = (int64_t)p.blocks * W * R;
  int64_t row = ((int64_t)blockIdx.x * W + wave) * R + sub;
  auto fetch = [&](int64_t at, int d) {
    in[d] = 1;
    if (at >= p.tokens) return;
    load_row<BF16, L, CH>(p.x, at, p.experts, l, -INFINITY, ahead[d]);
    if (p.mask) in[d] = p.mask[at];
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(row + d * step, d);
  for (; row < p.tokens;) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (row >= p.tokens) continue;
      f32x4 cur[CH];
      const int counts = in[d];
#pragma unroll
      for (int c = 0; c < CH; ++c) cur[c] = ahead[d][c];
      fetch(row + D * step, d);
      const float inv = softmax_row<L, CH>(cur);
      if (counts) {   // not p times 0: a row that is not counted may hold anything
        ++n;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[c][j] = fmaf(cur[c][j], inv, acc[c][j]);
      }
      row += step;
    }
  }
  for (int64_t s = (int64_t)blockIdx.x * (64 * W) + tid; s < p.slots; s += (int64_t)p.blocks * (64 * W)) {
    const uint64_t e = IDX64 ? (uint64_t)static_cast<const int64_t*>(p.idx)[s]
                             : (uint64_t)(int64_t)static_cast<const int32_t*>(p.idx)[s];
    if (e < (uint64_t)p.experts && (!p.mask || p.mask[(uint32_t)s / (uint32_t)p.k])) atomicAdd(&hist[e], 1);
  }
#pragma unroll
  for (int d = L; d < 64; d <<= 1) {   // rows of a wave
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[c][j] += __shfl_xor(acc[c][j], d);
    n += __shfl_xor(n, d);
  }
  if (lane == 0) counted[wave] = n;
  if (sub == 0) {
#pragma unroll
    for (int c = 0; c < CH; ++c) sums[wave][c * L + l] = acc[c];
  }
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) total += counted[w];
  const bool whole = p.blocks == 1;
  const double share = whole && total > 0 ? (double)p.coef * p.experts / ((double)p.k * total * total) : 0.0;
  double loss = 0.0;
  for (int e = tid; e < p.experts; e += 64 * W) {
    const float* column = reinterpret_cast<const float*>(sums) + e;
    float v = column[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += column[w * kWide];
    if (whole) {
      p.counts[e] = hist[e];
      p.grad[e] = (float)(share * hist[e]);
      if (total > 0) loss += share * hist[e] * (double)v;
    } else {
      p.part_p[(int64_t)blockIdx.x * p.experts + e] = v;
      p.part_c[(int64_t)blockIdx.x * p.experts + e] = hist[e];
    }
  }
  if (!whole) {
    if (tid == 0) p.part_n[blockIdx.x] = total;
    return;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) loss += __shfl_xor(loss, d);
  __syncthreads();   // the columns are read
  if (lane == 0) reinterpret_cast<double*>(sums)[wave] = loss;
  __syncthreads();
  if (wave) return;
  if (lane == 0) {
    for (int w = 1; w < W; ++w) loss += reinterpret_cast<double*>(sums)[w];
    *p.loss = (float)loss;
  }
  write_offsets(p, lane, [&](int i) { return hist[i]; });
}

// Adds the workgroups' parts, in fp64 and in a fixed order: a workgroup those of
// kJoin experts.  The last to be done (all of them count themselves) writes what
// takes every expert: the loss and the offsets.
constexpr int kJoin = 16;
__global__ __launch_bounds__(1024) void balance_join_kernel(BalanceArgs p) {
  __shared__ double dsum[16][kJoin];
  __shared__ int isum[16][kJoin];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x * kJoin + lane % kJoin;
  int n = 0, c = 0;
  double s = 0.0;
  for (int b = lane; b < p.blocks; b += 64) n += p.part_n[b];   // every wave for itself
  if (e < p.experts) {
#pragma unroll 4
    for (int b = wave * 4 + lane / kJoin; b < p.blocks; b += 64) {
      s += (double)p.part_p[(int64_t)b * p.experts + e];
      c += p.part_c[(int64_t)b * p.experts + e];
    }
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    n += __shfl_xor(n, d);
    if (d >= kJoin) {
      s += __shfl_xor(s, d);
      c += __shfl_xor(c, d);
    }
  }
  if (lane < kJoin) {
    dsum[wave][lane] = s;
    isum[wave][lane] = c;
  }
  __syncthreads();
  if (wave == 0) {
    const double share = n > 0 ? (double)p.coef * p.experts / ((double)p.k * n * n) : 0.0;
    s = 0.0;
    c = 0;
    if (lane < kJoin) {
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        s += dsum[w][lane];
        c += isum[w][lane];
      }
      if (e < p.experts) {
        p.counts[e] = c;
        p.grad[e] = (float)(share * c);
      }
    }
    double loss = n > 0 ? share * c * s : 0.0;   // of nobody s may be anything, c is 0 past E
#pragma unroll
    for (int d = kJoin / 2; d; d >>= 1) loss += __shfl_xor(loss, d);
    if (lane == 0) {
      p.part_loss[blockIdx.x] = loss;
      __threadfence();
      last = atomicAdd(p.joined, 1u) + 1 == gridDim.x;
    }
  }
  __syncthreads();
  if (!last || wave) return;
  __threadfence();
  double loss = 0.0;
  int64_t base = 0;
  for (unsigned b = lane; b < gridDim.x; b += 64)
    loss += __hip_atomic_load(&p.part_loss[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int d = 32; d; d >>= 1) loss += __shfl_xor(loss, d);
  if (lane == 0) *p.loss = (float)loss;
  write_offsets(p, lane, [&](int i) { return __hip_atomic_load(&p.counts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); });
}

struct BalanceGradArgs {
  const void* x;
  const float* v;
  const float* dloss;
  const uint8_t* mask;
  const void* add;
  void* out;
  int64_t tokens;
  int experts;
  int blocks;
};

template <bool BF16, int L, int CH, int W>
__global__ __launch_bounds__(64 * W) void balance_grad_kernel(BalanceGradArgs p) {
  constexpr int R = 64 / L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & (L - 1), sub = lane / L;
  // The next row is asked for ahead but where a lane has 16 chunks, on the measurement alone
  // (20000 rows of 2500: bf16 154 us, 282 with it, fp32 117, 161; of 4096: 216, 379 and 184,
  // 173; no registers are spilled either way).  bf16 rows, of half the bytes, take longer than
  // fp32 there: load_row unpacks them in its branch and so waits for chunk after chunk.
  constexpr bool kAhead = CH <= 8;
  f32x4 v[CH], cur[CH], next[CH];
  load_row<false, L, CH>(p.v, 0, p.experts, l, 0.0f, v);
  const float dl = p.dloss ? *p.dloss : 1.0f;
  const int64_t step = (int64_t)p.blocks * W * R;
  int64_t row = ((int64_t)blockIdx.x * W + wave) * R + sub;
  if (kAhead && row < p.tokens) load_row<BF16, L, CH>(p.x, row, p.experts, l, -INFINITY, next);
  for (; row < p.tokens; row += step) {
    if constexpr (kAhead) {
#pragma unroll
      for (int c = 0; c < CH; ++c) cur[c] = next[c];
    } else {
      load_row<BF16, L, CH>(p.x, row, p.experts, l, -INFINITY, cur);
    }
    const bool in = !p.mask || p.mask[row];
    f32x4 add[CH] = {};
    if (p.add) load_row<BF16, L, CH>(p.add, row, p.experts, l, 0.0f, add);
    if (kAhead && row + step < p.tokens) load_row<BF16, L, CH>(p.x, row + step, p.experts, l, -INFINITY, next);
    const float inv = softmax_row<L, CH>(cur);
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) dot = fmaf(cur[c][j], v[c][j], dot);
    dot = over_lanes<L>(dot, [](float a, float b) { return a + b; }) * inv;
    const float scale = dl * inv;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int e = 4 * (c * L + l);
      f32x4 d = add[c];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (in) d[j] = fmaf(scale * cur[c][j], v[c][j] - dot, d[j]);
      if (e + 4 <= p.experts) {
        store4<BF16>(p.out, row * p.experts + e, d);
      } else {
        for (int j = 0; j < 3; ++j)
          if (e + j < p.experts) store1<BF16>(p.out, row * p.experts + e + j, d[j]);
      }
    }
  }
}

// Lanes of a row and its chunks a lane: the fewest lanes that hold it in one
// chunk, then more chunks.  Places past a row's end cost what the others do: 20000 x
// 1500 fp32 in 8 chunks 45 us and its gradient 69, in 16 80 and 160.
// f(integral constants L, CH, W).
template <int N>
using Int = std::integral_constant<int, N>;
template <typename F>
void by_width(int experts, F f) {
  if (experts <= 32) f(Int<8>(), Int<1>(), Int<16>());
  else if (experts <= 64) f(Int<16>(), Int<1>(), Int<16>());
  else if (experts <= 128) f(Int<32>(), Int<1>(), Int<16>());
  else if (experts <= 256) f(Int<64>(), Int<1>(), Int<16>());
  else if (experts <= 512) f(Int<64>(), Int<2>(), Int<16>());
  else if (experts <= 1024) f(Int<64>(), Int<4>(), Int<8>());
  else if (experts <= 2048) f(Int<64>(), Int<8>(), Int<8>());
  else f(Int<64>(), Int<16>(), Int<4>());
}

constexpr int kBalanceBlocks = 256;
// Rounds that one workgroup takes alone: eight take about 1 us more on the card than two
// launches do, and the second launch costs the caller 3.5 us (512 tokens of 64 experts: 10.2
// us, in two 9.2; a call with its allocations 14.4 us of the caller's time, in two 18).
constexpr int kOneBlock = 8;
// Rows that a lane adds up in fp32; the workgroups' sums are added in fp64.  Rows alike,
// as of a router that starts with zeros, are rounded alike: 4096 rows of 1 / 160 are
// off by 4e-5 of their sum, 128 by 1e-6.  The workgroups that this takes past 256 cost
// nothing (2^20 x 256 in bf16 304 us in 256 workgroups, 230 in 512; 2^18 x 4096 2158, 2175).
constexpr int kLaneRows = 128;
int balance_blocks(int64_t tokens, int experts) {
  int64_t blocks = 0;
  by_width(experts, [&](auto l, auto, auto w) {
    constexpr int rows = 64 / decltype(l)::value * decltype(w)::value;
    const int64_t rounds = (tokens + rows - 1) / rows, least = (rounds + kLaneRows - 1) / kLaneRows;
    blocks = rounds <= kOneBlock ? 1 : std::min(rounds, std::max<int64_t>(kBalanceBlocks, least));
  });
  return (int)blocks;
}

int64_t join_blocks(int experts) { return (experts + kJoin - 1) / kJoin; }

}  // namespace
}  // namespace fp4mi

using namespace fp4mi;

extern "C" int64_t router_balance_workspace(int64_t tokens, int32_t num_experts) {
  if (tokens < 0 || tokens >= (int64_t(1) << 31) || num_experts < 1 || num_experts > kMaxExperts) return 0;
  return 16 + 8 * join_blocks(num_experts) + (int64_t)balance_blocks(tokens, num_experts) * (8 * num_experts + 4);
}

extern "C" int router_balance(const void* logits, int dtype, const void* experts, int index_size,
                              const uint8_t* mask, int64_t tokens, int32_t num_experts, int32_t k,
                              float coef, float* loss, int32_t* counts, int64_t* offsets,
                              float* prob_grad, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  const int isz = dtype_size(dtype);
  if (!isz) return FP4_EDTYPE;
  if ((index_size != 4 && index_size != 8) || !(fabsf(coef) < INFINITY)) return FP4_EINVAL;
  if (tokens < 0 || tokens >= (int64_t(1) << 31) || num_experts < 1 || num_experts > kMaxExperts ||
      k < 1 || (tokens && k > ((int64_t(1) << 31) - 1) / tokens))
    return FP4_ESHAPE;
  const int64_t need = router_balance_workspace(tokens, num_experts), slots = tokens * k;
  if (workspace_bytes < need) return FP4_ESHAPE;
  if ((tokens && (!logits || !experts)) || !loss || !counts || !offsets || !prob_grad || !workspace)
    return FP4_EINVAL;
  if (!is_aligned(logits, isz) || !is_aligned(experts, index_size) || !is_aligned(loss, 4) ||
      !is_aligned(counts, 4) || !is_aligned(offsets, 8) || !is_aligned(prob_grad, 4) ||
      !is_aligned(workspace, 16))
    return FP4_EALIGN;
  const void* outs[5] = {loss, counts, offsets, prob_grad, workspace};
  const int64_t outn[5] = {4, 4 * (int64_t)num_experts, 8 * ((int64_t)num_experts + 1),
                           4 * (int64_t)num_experts, need};
  const void* ins[3] = {logits, experts, mask};
  const int64_t inn[3] = {tokens * num_experts * isz, slots * index_size, tokens};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 3; ++j)
      if (overlaps(outs[i], outn[i], ins[j], inn[j])) return FP4_EOVERLAP;
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outn[i], outs[j], outn[j])) return FP4_EOVERLAP;
  }
  BalanceArgs p = {logits, experts, mask, tokens, slots, num_experts, k, coef, loss, counts, offsets, prob_grad};
  p.blocks = balance_blocks(tokens, num_experts);
  const int64_t joins = join_blocks(num_experts);
  p.joined = static_cast<uint32_t*>(workspace);
  p.part_loss = reinterpret_cast<double*>(p.joined + 4);
  p.part_p = reinterpret_cast<float*>(p.part_loss + joins);
  p.part_c = reinterpret_cast<int32_t*>(p.part_p + (int64_t)p.blocks * num_experts);
  p.part_n = p.part_c + (int64_t)p.blocks * num_experts;
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  const bool bf16 = dtype == FP4_DTYPE_BF16, wide = index_size == 8;
  by_width(num_experts, [&](auto l, auto ch, auto w) {
    constexpr int L = decltype(l)::value, CH = decltype(ch)::value, W = decltype(w)::value;
    hipLaunchKernelGGL((bf16 ? (wide ? balance_kernel<true, true, L, CH, W> : balance_kernel<true, false, L, CH, W>)
                             : (wide ? balance_kernel<false, true, L, CH, W> : balance_kernel<false, false, L, CH, W>)),
                       dim3(p.blocks), dim3(64 * W), 0, st, p);
  });
  if (p.blocks > 1) hipLaunchKernelGGL(balance_join_kernel, dim3((unsigned)joins), dim3(1024), 0, st, p);
  return launch_status();
}

extern "C" int router_balance_backward(const void* logits, int dtype, const float* prob_grad,
                                       const float* dloss, const uint8_t* mask, const void* add,
                                       int64_t tokens, int32_t num_experts, void* dlogits,
                                       void* stream) {
  const int isz = dtype_size(dtype);
  if (!isz) return FP4_EDTYPE;
  if (tokens < 0 || tokens >= (int64_t(1) << 31) || num_experts < 1 || num_experts > kMaxExperts)
    return FP4_ESHAPE;
  if (tokens == 0) return FP4_OK;
  if (!logits || !prob_grad || !dlogits) return FP4_EINVAL;
  if (!is_aligned(logits, isz) || !is_aligned(prob_grad, 4) || !is_aligned(dloss, 4) ||
      !is_aligned(add, isz) || !is_aligned(dlogits, isz))
    return FP4_EALIGN;
  const int64_t n = tokens * num_experts * isz;
  if ((dlogits != logits && overlaps(dlogits, n, logits, n)) ||
      (dlogits != add && overlaps(dlogits, n, add, n)) ||
      overlaps(dlogits, n, prob_grad, 4 * (int64_t)num_experts) || overlaps(dlogits, n, dloss, 4) ||
      overlaps(dlogits, n, mask, tokens))
    return FP4_EOVERLAP;
  BalanceGradArgs p = {logits, prob_grad, dloss, mask, add, dlogits, tokens, num_experts, 0};
  clear_stale_error();
  hipStream_t st = as_stream(stream);
  by_width(num_experts, [&](auto l, auto ch, auto) {
    constexpr int L = decltype(l)::value, CH = decltype(ch)::value, W = 4, rows = 64 / L * W;
    const int64_t blocks = (tokens + rows - 1) / rows;
    p.blocks = (int)(blocks < 2048 ? blocks : 2048);
    hipLaunchKernelGGL((dtype == FP4_DTYPE_BF16 ? balance_grad_kernel<true, L, CH, W>
                                                : balance_grad_kernel<false, L, CH, W>),
                       dim3(p.blocks), dim3(64 * W), 0, st, p);
  });
  return launch_status();
}
