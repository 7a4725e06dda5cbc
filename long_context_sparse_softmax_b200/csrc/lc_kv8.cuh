// What the kernels that read the 8-bit cache share: the key range of a tile of query rows, its
// splits, the scale bytes, and the joining of partial softmax results.
//
// A partial result over some keys is (O, R, l): with x_t = log2(e) scale <q, k_t> and value
// exponents ev_t (the value of token t is code_t 2^ev_t),
//   w_t = 2^(x_t + ev_t - R),  O = sum w_t code_t,  l = sum w_t 2^-ev_t,
// so o = O / l and lse = ln 2 (R + log2 l).  The reference R follows the largest x_t + ev_t, not
// the largest logit: the weights that multiply the codes then stay in F16's range whatever the
// blocks' scales are.  Exponents within [-32, 31] keep l in FP32's range.
#pragma once

#include "lc_internal.h"
#include "lc_ptx_dense.cuh"

namespace lc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kKv8EMin = -32, kKv8EMax = 31;

__device__ __forceinline__ int kv8_exp(uint8_t byte) { return min(max(static_cast<int>(byte) - 127, kKv8EMin), kKv8EMax); }

// 2^(a - b) for references that may both be the same infinity
__device__ __forceinline__ float ref_factor(float a, float b) { return a == b ? 1.f : ex2(a - b); }

// Keys that the rows [row0, row0 + n_row) of one sequence and shared head can see: [lo, hi); row r
// is query r / g.  lo16 is lo rounded down to 16 (a 16-key step lies in one block).  Positions may be
// anywhere below 2^31, a window behind the cache or a query before its first token: lo16 <= lo <= kv and
// lo16 <= hi <= kv all the same, so what starts at lo16 neither leaves the table nor 32 bits.
struct Kv8Range {
  int lo, hi, lo16;
};
__device__ __forceinline__ Kv8Range kv8_range(int kv, int W, int p_first, int p_last) {
  Kv8Range r;
  r.hi = p_last < kv ? p_last + 1 : kv;
  r.lo = min(W > 0 && p_first >= W ? p_first - (W - 1) : 0, kv);  // W up to the type's last value
  r.lo16 = r.lo & ~15;
  if (r.hi <= r.lo) r.hi = r.lo16;
  return r;
}

// Split of n keys over CTAs: `len` keys each.  A function of the row's own key count and of the
// shared heads alone, so a sequence's result does not depend on the batch it is in.  256 keys where
// a sequence is short and its latency counts, 512 above 4096 keys, 1024 above 8192 (what a CTA does
// besides its keys, and the partial rows, cost as much as 200 keys), and from most_splits * 1024
// keys on as many as fill the device with one sequence (576 CTAs: 4 on each multiprocessor), up to
// 8192 keys each.
constexpr int kKv8MaxSplit = 8192;
__host__ __device__ __forceinline__ int kv8_most_splits(int H_kv) { return H_kv >= 8 ? 72 : H_kv >= 2 ? 576 / H_kv : 512; }
__host__ __device__ __forceinline__ int kv8_split_len(int n, int H_kv) {
  const int most = kv8_most_splits(H_kv);
  const int want = ((n + most - 1) / most + 63) / 64 * 64, least = n <= 4096 ? 256 : n <= 8192 ? 512 : 1024;
  return want < least ? least : want > kKv8MaxSplit ? kKv8MaxSplit : want;
}
__host__ __device__ __forceinline__ int kv8_n_split(int n, int H_kv) {
  const int len = kv8_split_len(n, H_kv);
  return n <= len ? 1 : static_cast<int>((static_cast<int64_t>(n) + len - 1) / len);
}
// the most splits of any row with up to n keys
inline int kv8_split_bound(int n, int H_kv) {
  if (n <= 4096) return kv8_n_split(n, H_kv);
  const int most = kv8_most_splits(H_kv), s = kv8_n_split(n, H_kv);
  const int low = n <= 1024 * most ? 16 : most;  // 16: at 4096 and at 8192 keys
  return s > low ? s : low;
}

// A query's weight on a key it does not see is 0, but 0 times the E4M3 NaN is a NaN.  In the steps
// where rows of a tile see different keys the kernels replace NaN value codes by 0 (nan_bytes) and
// note it; the rows that do see such a code are then found by reading the codes again (rare).

// 0xff in each byte of v that holds an E4M3 NaN
__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) {
  const uint32_t m = ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return m | (m - (m >> 7));
}
// which of the value codes of dims d .. d + 3 are NaN for some token of [lo, hi): bytes 0xff
__device__ __forceinline__ uint32_t kv8_value_nans(const lc_kv8_cache& c, int s, int h, int lo, int hi, int d) {
  uint32_t m = 0;
  for (int t = lo; t < hi; ++t) {
    const int blk = __ldg(c.table + static_cast<int64_t>(s) * c.table_cols + t / c.bt);
    if (blk < 0 || blk >= c.n_blocks) continue;
    m |= nan_bytes(__ldg(reinterpret_cast<const uint32_t*>(
        c.v + ((static_cast<int64_t>(blk) * c.H_kv + h) * c.bt + t % c.bt) * c.D + d)));
  }
  return m;
}

// four E4M3 codes -> two pairs of F16 values (exact)
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& a, uint32_t& b) {
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.rn.f16x2.e4m3x2 %0, lo;\ncvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
      : "=r"(a), "=r"(b)
      : "r"(v));
}

// How a call's rows and keys are spread over CTAs.
struct Kv8Geom {
  int g;          // query heads per shared head
  int row_tiles;  // row tiles per (sequence, shared head)
  int n_split;    // CTAs per row tile (1: no split); of k_kv8_attn an upper bound
  int rows;       // rows per row tile
  int tc;         // k_kv8_attn_tc: every row has n_split partial results
  int decode;     // query s belongs to sequence s
};

// rows of a CTA of k_kv8_attn_tc
inline int kv8_tc_rows(int D) { return D == 128 ? 256 : 128; }
cudaError_t launch_kv8_attn_tc(const lc_kv8_attn_args& a, const Kv8Geom& geo, unsigned grid, float* ws_o, float2* ws_ml,
                               cudaStream_t st);

// The output of one row from its joined partial result: the factor on O, and lse.
__device__ __forceinline__ float kv8_finish(float R, float l, const float* sink, int head, float* lse) {
  if (!sink) {
    if (R == -INFINITY && l == 0.f) {
      *lse = -INFINITY;
      return 0.f;
    }
    *lse = R * kLn2 + logf(l);
    return 1.f / l;
  }
  const float s2 = __ldg(sink + head) * kLog2e;
  if (R == -INFINITY && l == 0.f) {
    *lse = __ldg(sink + head);
    return 0.f;
  }
  const float M = fmaxf(R, s2);
  const float fr = ref_factor(R, M);
  const float Z = l * fr + ref_factor(s2, M);
  *lse = M * kLn2 + logf(Z);
  return fr / Z;
}

}  // namespace lc
