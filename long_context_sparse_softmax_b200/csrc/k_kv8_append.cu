// kv8_append: new key / value rows into the 8-bit cache (E4M3 codes, one E8M0 scale per block
// of bt tokens and head).
//
// One CTA per (sequence, block it touches, head, keys | values): the block's new rows stay in
// registers, as they came, between the maximum and the rounding, so they are read once.  Memory's
// latency bounds it (a CTA lives for a few accesses), so the rows are fetched before the block's id
// is known, and little is held per thread: six CTAs on a multiprocessor.  16384 BF16 tokens of 8 heads of
// 128 dims: 18.9 us in a graph of such calls, 5.3 TB/s (82 % of the measured copy rate), 20.7 us as a call among
// others (38.9 us with the id first and wide divisions); a token for each of 32 sequences 3.2 us in a graph, 5.8 as
// a call: a launch and three latencies.  The scale is the
// smallest 2^e that covers them (exact integer arithmetic on the exponent), kept at or above the
// scale of a block that already holds tokens; where that grows, the block's older codes are
// rounded again from their exact values.  Everything is exact but the final roundings, so the
// result does not depend on the launch shape.
#include "lc_e4m3.cuh"
#include "lc_internal.h"

namespace lc {

namespace {

constexpr int kThreads = 256;
constexpr int kEMin = -32, kEMax = 31;

__device__ __forceinline__ int scale_exp(uint8_t byte) { return min(max(static_cast<int>(byte) - 127, kEMin), kEMax); }

// 8 values as they lie in memory
template <bool kF32>
struct Raw {
  uint4 w[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int j = 0; j < (kF32 ? 2 : 1); ++j) w[j] = __ldcs(reinterpret_cast<const uint4*>(p) + j);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[kF32].x, w[kF32].y, w[kF32].z, w[kF32].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kF32) {
        v[2 * j] = __uint_as_float(u[2 * j]);
        v[2 * j + 1] = __uint_as_float(u[2 * j + 1]);
      } else {
        v[2 * j] = __uint_as_float(u[j] << 16);
        v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
  }
};

}  // namespace

// kV groups of 8 values per thread: bt * D / 8 <= kThreads * kV
template <bool kF32, int kV>
__global__ void __launch_bounds__(kThreads) k_kv8_append(lc_kv8_append_args a, uint32_t max_blk) {
  __shared__ float s_max[kThreads / 32];
  const lc_kv8_cache& c = a.cache;
  // blockIdx.x = ((s * max_blk + j) * 2 + values) * H_kv + h
  uint32_t u = blockIdx.x;
  const int h = static_cast<int>(u % static_cast<uint32_t>(c.H_kv));
  u /= static_cast<uint32_t>(c.H_kv);
  const bool val = u & 1;
  u >>= 1;
  const int j = static_cast<int>(u % max_blk);
  const int s = static_cast<int>(u / max_blk);
  const int t0 = __ldg(a.tok_start + s), t1 = __ldg(a.tok_start + s + 1), p0 = __ldg(a.pos0 + s);
  const int n = min(t1 - t0, a.max_tok);
  const int bt_log = __ffs(c.bt) - 1, per_log = __ffs(c.D) - 4;  // groups per row: D / 8
  const int col = (p0 >> bt_log) + j;
  const int64_t first = static_cast<int64_t>(col) << bt_log;  // position of the block's row 0
  if (n <= 0 || p0 < 0 || first >= static_cast<int64_t>(p0) + n) return;
  const int r_lo = static_cast<int>(max(static_cast<int64_t>(p0) - first, int64_t{0}));  // new rows [r_lo, r_hi)
  const int r_hi = static_cast<int>(min(static_cast<int64_t>(p0) + n - first, static_cast<int64_t>(c.bt)));
  const int blk = col < c.table_cols ? __ldg(c.table + static_cast<int64_t>(s) * c.table_cols + col) : -1;
  const int64_t dense = static_cast<int64_t>(c.H_kv) * c.D;
  const int64_t stride = val ? (a.v_stride ? a.v_stride : dense) : (a.k_stride ? a.k_stride : dense);
  constexpr int kEsz = kF32 ? 4 : 2;
  // group g0 + i * kThreads: rows kThreads / (D / 8) apart, the same columns
  const int g0 = (r_lo << per_log) + threadIdx.x, g_end = r_hi << per_log;
  const char* x = static_cast<const char*>(val ? a.v : a.k) +
                  ((t0 + (first - p0) + (g0 >> per_log)) * stride + static_cast<int64_t>(h) * c.D + (g0 & ((1 << per_log) - 1)) * 8) * kEsz;
  const int64_t x_step = (kThreads >> per_log) * stride * kEsz;

  Raw<kF32> v[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (g0 + i * kThreads < g_end) v[i].load(x + i * x_step);
  if (blk < 0 || blk >= c.n_blocks) {
    if (threadIdx.x == 0) set_status(a.status, LC_DEV_BAD_BLOCK);
    return;
  }
  const int64_t slot = static_cast<int64_t>(blk) * c.H_kv + h;
  uint8_t* codes = (val ? c.v : c.k) + slot * c.bt * c.D;
  uint8_t* scale = (val ? c.v_scale : c.k_scale) + slot;
  const int e_old = r_lo > 0 ? scale_exp(*scale) : kEMin;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    if (g0 + i * kThreads >= g_end) continue;
    float y[8];
    v[i].values(y);
#pragma unroll
    for (int q = 0; q < 8; ++q) amax = fmaxf(amax, fabsf(y[q]));  // passes over NaN
  }
  // an infinity among the values: the largest finite one, then
  if (__syncthreads_or(amax == INFINITY)) {
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if (g0 + i * kThreads >= g_end) continue;
      float y[8];
      v[i].values(y);
#pragma unroll
      for (int q = 0; q < 8; ++q) amax = fmaxf(amax, finite_abs(y[q]));
    }
  }
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();  // every thread has read the old scale, too
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  int e = amax > 0.f ? min(max(e4m3_scale_exp(amax), kEMin), kEMax) : kEMin;
  e = max(e, e_old);
  if (r_lo > 0 && e > e_old) {
    // the older codes, rounded again: code * 2^(e_old - e) is exact before the rounding
    const float f = pow2f(e_old - e);
    for (int g = threadIdx.x; g < r_lo << per_log; g += kThreads) {
      uint2* p = reinterpret_cast<uint2*>(codes) + g;
      const uint2 w = *p;
      const float2 a0 = e4m3x2_to_f32x2(static_cast<uint16_t>(w.x & 0xffffu));
      const float2 a1 = e4m3x2_to_f32x2(static_cast<uint16_t>(w.x >> 16));
      const float2 a2 = e4m3x2_to_f32x2(static_cast<uint16_t>(w.y & 0xffffu));
      const float2 a3 = e4m3x2_to_f32x2(static_cast<uint16_t>(w.y >> 16));
      *p = make_uint2(e4m3x4(a0.x * f, a0.y * f, a1.x * f, a1.y * f), e4m3x4(a2.x * f, a2.y * f, a3.x * f, a3.y * f));
    }
  }
  const float f = pow2f(-e);
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int g = g0 + i * kThreads;
    if (g >= g_end) continue;
    float y[8];
    v[i].values(y);
    reinterpret_cast<uint2*>(codes)[g] = make_uint2(e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f), e4m3x4(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
  }
  if (threadIdx.x == 0) *scale = static_cast<uint8_t>(e + 127);
}

namespace {

template <bool kF32>
cudaError_t launch(const lc_kv8_append_args& a, unsigned grid, uint32_t max_blk, cudaStream_t st) {
  auto go = [&](auto kernel) { return launch_ex(kernel, dim3(grid), dim3(kThreads), 0, st, false, 1, a, max_blk); };  // nothing to set up ahead
  const int groups = a.cache.bt * a.cache.D / 8;  // 128 .. 2048
  if (groups <= kThreads) return go(k_kv8_append<kF32, 1>);
  if (groups <= 2 * kThreads) return go(k_kv8_append<kF32, 2>);
  if (groups <= 4 * kThreads) return go(k_kv8_append<kF32, 4>);
  return go(k_kv8_append<kF32, 8>);
}

}  // namespace

cudaError_t launch_kv8_append(const lc_kv8_append_args& a, cudaStream_t st) {
  // max_tok tokens touch at most 1 + (max_tok - 1 + bt - 1) / bt blocks, wherever the first lies
  const int bt = a.cache.bt;
  const int64_t max_blk = 1 + (static_cast<int64_t>(a.max_tok) + bt - 2) / bt;
  if (2.0 * max_blk * a.num_seqs * a.cache.H_kv > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int64_t grid = max_blk * 2 * a.num_seqs * a.cache.H_kv;
  if (a.in_fmt == LC_FMT_F32) return launch<true>(a, static_cast<unsigned>(grid), static_cast<uint32_t>(max_blk), st);
  return launch<false>(a, static_cast<unsigned>(grid), static_cast<uint32_t>(max_blk), st);
}

}  // namespace lc
