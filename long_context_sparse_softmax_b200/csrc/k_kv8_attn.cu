// kv8_attn: attention over the 8-bit cache (E4M3 codes, one E8M0 scale per block and head).
//
// Bulk copies bring 16 keys and their values at a time into a ring of two steps that each warp has for
// itself; from there they go into the registers that the matrix instruction reads.  The products are written transposed, keys (then
// dims) on the 16-row side and 8 query rows on the other, so 8 heads that share a cache head fill
// the instruction:
//   S^T[16 keys, 8 rows] = K Q^T      (A = K, B = Q),
//   O^T[16 dims, 8 rows] += V^T P^T   (A = V^T, B = P).
// The order of the summed dims is free as long as both operands agree, so a thread's A registers
// of a key are D / 4 consecutive bytes of its row (four summed dims per step and thread), read 16 at a
// time; the copies' swizzle puts what eight lanes read, of keys and of values, into different banks.  V^T needs two keys' codes of one dim side by side: the thread
// that holds dims 16 g .. 16 g + 15 of keys 2t, 2t + 1 interleaves their bytes (one prmt per four)
// and widens them.  E4M3 is a subset of F16, so widening is exact.
//
// Queries are scaled per row by a power of two into F16's range (exact down to 2^-39 of the row's
// largest value); K's block scale multiplies the logits, V's joins the softmax exponent (see
// lc_kv8.cuh).  P is rounded to F16 (11 bits), the operand that the codes widen to exactly; l sums the
// unrounded weights.  That rounding is 1.4e-4 of o (2-norm), a tenth of o's own to BF16 (1.65e-3 with it or
// without); a second F16 term for the rest of P would double the products with V.  The reference R moves
// only when a weight would pass 2^8, so the lanes meet once per 16 keys, in a vote.
//
// Warps of a CTA take 16-key steps in turn and join through shared memory; the keys of a row
// tile are split over CTAs, joined by k_kv8_combine.
//
// HBM bounds it: a step of a warp is 4 KB (128 dims).  One context of 262144 tokens, 8 shared heads, 64
// queries' heads: 95 us, 5.7 TB/s (87 % of the measured copy rate; the join is 5 us of it).  32 contexts up
// to 16384: 100 us in a graph of such calls, 5.6 TB/s (86 %), 111 us as a call among others (78 %): here a
// CTA has 16 steps a warp, and what it does besides (about 1100 instructions a warp, one after another) costs
// as much as 100 keys; the join is 5 us.  What brought it there:
// two conversions per instruction pair and no divisions by the block size (209 -> 157 us for the batch),
// block ids before the queries, 32-bit index arithmetic (143), splits of 1024 keys (127), the ring (119 -> 106:
// loads of 16 bytes a lane straight into registers kept L1 75 % busy, 99 % for one context; that one lost 94 ->
// 97), a join without bank conflicts and one pass over a split's block ids (102), two warps a
// joined row instead of four (100); splits that fill the device once and a join by a CTA per row
// (135 -> 100 us for the one).  Three steps in the ring: 109 us and 101; five CTAs a multiprocessor: 114 and 124;
// three, of a ring of four: 110 and 119; eight, of two warps: 110 and 117; the block ids asked for before the
// lengths were known, so that a start waits once less: no difference.
#include "lc_e4m3.cuh"
#include "lc_kv8.cuh"
#include "lc_tma.h"

namespace lc {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxPages = kKv8MaxSplit / 16 + 1;  // block ids and scales of a split sit in shared memory
constexpr long kSpin = 1L << 20;              // a few seconds
constexpr float kHeadroom = 8.f;              // log2 of the largest weight before R moves

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint4 lds16(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
  return v;
}

// A 16-key step of one warp.  k: keys g and g + 8, D / 4 bytes at (D / 4) t;
// v: keys 2t, 2t + 1, 2t + 8, 2t + 9, D / 8 bytes at (D / 8) g.
template <int D>
struct Step {
  uint32_t k[2][D / 16];
  uint32_t v[4][D / 32];
};

}  // namespace

// A warp's steps in flight, in shared memory: its own ring, so that no other warp is waited for.  After
// the last step the warp's sums lie in the same place.
template <int D>
struct Kv8Ring {
  static constexpr int kStages = 2;
  static constexpr int kHalf = 16 * D, kStage = 2 * kHalf;  // keys | values
  static constexpr int kWarp = kStages * kStage, kBytes = kWarps * kWarp + 1024;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 3)
    k_kv8_attn(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, lc_kv8_attn_args a, Kv8Geom geo, float* __restrict__ ws_o, float2* __restrict__ ws_ml) {
  constexpr int kRows = 8 * NT;
  constexpr int kKS = D / 16;   // summed steps of S
  constexpr int kMT = D / 16;   // 16-dim tiles of O^T
  constexpr int kVB = D / 8;    // bytes of V per key and thread
  __shared__ int s_page[kMaxPages];
  __shared__ float s_kf[kMaxPages], s_ev[kMaxPages];
  __shared__ float2 s_ml[kWarps][kRows];
  using Ring = Kv8Ring<D>;
  constexpr int kStages = Ring::kStages;
  __shared__ __align__(8) uint64_t s_bar[kWarps][kStages];
  extern __shared__ uint8_t smem_raw[];
  static_assert(kRows * D * 4 <= Ring::kWarp, "the sums' place");

  const lc_kv8_cache& c = a.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  const int bt_log = __ffs(c.bt) - 1;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)) + warp * Ring::kWarp;
  const uint32_t ring_at = su32(ring), bar_at = su32(s_bar[warp]);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bar_at + 8 * i, 1);
    fence_mbar_init();
    if (a.max_kv > 0 && c.n_blocks > 0) {  // else the host made no maps
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_v);
    }
  }
  pdl_wait();
  pdl_trigger();
  // 32-bit divisions: what a CTA does besides its keys counts when a split has 512 of them
  uint32_t u = blockIdx.x;
  const int split = static_cast<int>(u % static_cast<uint32_t>(geo.n_split));
  u /= static_cast<uint32_t>(geo.n_split);
  const int rt = static_cast<int>(u % static_cast<uint32_t>(geo.row_tiles));
  u /= static_cast<uint32_t>(geo.row_tiles);
  const int h = static_cast<int>(u % static_cast<uint32_t>(c.H_kv));
  const int s = static_cast<int>(u / static_cast<uint32_t>(c.H_kv));

  const int q0 = __ldg(a.q_start + s);
  const int nq = min(__ldg(a.q_start + s + 1) - q0, a.max_q);
  const uint32_t row0 = rt * kRows, g_heads = geo.g;
  const uint32_t all_rows = nq > 0 ? nq * g_heads : 0;  // the host keeps max_q * g below 2^31
  if (row0 >= all_rows) return;
  const int n_row = static_cast<int>(min(static_cast<uint32_t>(kRows), all_rows - row0));
  // query of a row of the tile (the first one where there is one, and for the tile's rows past n_row)
  auto query = [&](int r) -> int { return nq == 1 ? 0 : static_cast<int>((row0 + r) / g_heads); };
  const int p0 = __ldg(a.q_pos0 + s);
  const int kv_all = __ldg(a.kv_len + s);
  const int kv = min(min(kv_all, a.max_kv), c.table_cols * c.bt);
  if (kv < min(kv_all, a.max_kv) && tid == 0) set_status(a.status, LC_DEV_BAD_BLOCK);
  const int q_first = query(0), q_last = query(n_row - 1);
  const Kv8Range rg = kv8_range(kv, a.W, p0 + q_first, p0 + q_last);
  const int n = rg.hi - rg.lo16;
  const int len = geo.n_split > 1 ? kv8_split_len(n, c.H_kv) : n;
  const int n_split = geo.n_split > 1 ? kv8_n_split(n, c.H_kv) : 1;
  if (split >= n_split) return;
  const int k_begin = rg.lo16 + split * len;
  const int k_end = min(rg.hi, k_begin + len);

  // visible keys of this thread's rows
  int r_lo[NT][2], r_hi[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int rr = i * 8 + 2 * t4 + j;
      const int p = p0 + query(rr);
      const Kv8Range x = kv8_range(kv, a.W, p, p);
      r_lo[i][j] = x.lo;
      r_hi[i][j] = rr < n_row ? x.hi : 0;
    }
  // keys that every row sees: [all_lo, all_hi)
  const Kv8Range first = kv8_range(kv, a.W, p0 + q_first, p0 + q_first);
  const Kv8Range last = kv8_range(kv, a.W, p0 + q_last, p0 + q_last);
  const int all_lo = last.lo, all_hi = first.hi;

  float o[NT][kMT][4];
  float R[NT][2], l[NT][2];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][m][j] = 0.f;
    R[i][0] = R[i][1] = -INFINITY;
    l[i][0] = l[i][1] = 0.f;
  }

  uint32_t qf[NT][kKS][2];
  float f_row[NT][2];  // rows 2 t4, 2 t4 + 1: log2(e) scale 2^eq
  bool nan_seen = false;  // NaN value codes replaced in an edge step
  // blocks of [k_begin, k_end): at most kKv8MaxSplit keys (without splits the host saw 256 or fewer)
  const int pg0 = k_begin >> bt_log, n_pg = k_end > k_begin ? ((k_end - 1) >> bt_log) - pg0 + 1 : 0;
  auto stage_pages = [&]() {
    for (int i = tid; i < n_pg; i += kThreads) {
      int blk = __ldg(c.table + static_cast<int64_t>(s) * c.table_cols + pg0 + i);
      if (blk < 0 || blk >= c.n_blocks) {
        blk = -1;
        set_status(a.status, LC_DEV_BAD_BLOCK);
      }
      s_page[i] = blk;
    }
  };
  auto stage_scales = [&]() {
    for (int i = tid; i < n_pg; i += kThreads) {
      const int blk = s_page[i];
      const int64_t slot = static_cast<int64_t>(blk < 0 ? 0 : blk) * c.H_kv + h;
      s_kf[i] = blk < 0 ? 0.f : pow2f(kv8_exp(__ldg(c.k_scale + slot)));
      s_ev[i] = blk < 0 ? 0.f : static_cast<float>(kv8_exp(__ldg(c.v_scale + slot)));
    }
  };
  // The warp's turns: turn i (key t) uses place i % kStages.  Sent by one lane, a step of a block that is
  // skipped without copies.
  int sent = 0, place_in = 0;
  auto send = [&](int t) {
    if (t >= k_end) return;
    if (lane == 0) {
      const int pg = s_page[(t >> bt_log) - pg0];
      const uint32_t bar = bar_at + 8 * place_in, dst = ring_at + place_in * Ring::kStage;
      if (pg < 0) {
        mbar_arrive(bar);
      } else {
        mbar_expect_tx(bar, Ring::kStage);
        tma_tile3d(dst, &map_k, 0, t & (c.bt - 1), pg * c.H_kv + h, bar);
        tma_tile3d(dst + Ring::kHalf, &map_v, 0, t & (c.bt - 1), pg * c.H_kv + h, bar);
      }
    }
    ++sent;
    if (++place_in == kStages) place_in = 0;
  };
  // where the swizzled copy put a thread's bytes: 16-byte piece x of row r at piece x ^ r (128 dims), or, with two
  // rows to 128 bytes, at x ^ (r / 2)
  const uint32_t at_k = D == 128 ? g8 * 128 + ((2 * t4) ^ g8) * 16 : g8 * 64 + (t4 ^ (g8 >> 1)) * 16;
  const uint32_t at_v = D == 128 ? t4 * 256 + (g8 ^ (2 * t4)) * 16 : t4 * 128 + ((g8 >> 1) ^ t4) * 16 + (g8 & 1) * 8;
  auto take = [&](int place, Step<D>& st) {
    const uint32_t k = ring_at + place * Ring::kStage + at_k, v = ring_at + place * Ring::kStage + Ring::kHalf + at_v;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        const uint4 w = lds16((k + r * 8 * D) ^ (x * 16));
        st.k[r][4 * x] = w.x;
        st.k[r][4 * x + 1] = w.y;
        st.k[r][4 * x + 2] = w.z;
        st.k[r][4 * x + 3] = w.w;
      }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // key 2 t + (r & 1) + 8 (r / 2)
      if constexpr (D == 128) {
        const uint4 w = lds16((v + (r & 1) * 128 + (r >> 1) * 1024) ^ ((r & 1) * 16));
        st.v[r][0] = w.x;
        st.v[r][1] = w.y;
        st.v[r][2] = w.z;
        st.v[r][3] = w.w;
      } else {
        const uint2 w = lds8(v + (r & 1) * 64 + (r >> 1) * 512);
        st.v[r][0] = w.x;
        st.v[r][1] = w.y;
      }
    }
  };
  auto step = [&](int t0, Step<D>& cur) {
    const int ip = (t0 >> bt_log) - pg0;
    if (s_page[ip] >= 0) {
      const float kf = s_kf[ip], ev = s_ev[ip];
      const float un_ev = pow2f(-static_cast<int>(ev));
      const bool edge = t0 < all_lo || t0 + 16 > all_hi;
      float x[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
      for (int k = 0; k < kKS; ++k) {
        uint32_t a0, a1, a2, a3;
        widen4(cur.k[0][k], a0, a2);
        widen4(cur.k[1][k], a1, a3);
#pragma unroll
        for (int i = 0; i < NT; ++i) mma16816(x[i], a0, a1, a2, a3, qf[i][k][0], qf[i][k][1]);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = fmaf(x[i][j], f_row[i][j & 1] * kf, ev);
      if (edge) {
        const int ka = t0 + g8, kb = ka + 8;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (ka < r_lo[i][j] || ka >= r_hi[i][j]) x[i][j] = -INFINITY;
            if (kb < r_lo[i][j] || kb >= r_hi[i][j]) x[i][2 + j] = -INFINITY;
          }
        // rows of the block that nobody sees may hold anything: their weight 0 must not meet a NaN
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int key = t0 + 2 * t4 + (r & 1) + (r >> 1) * 8;
          const bool out = key < rg.lo || key >= rg.hi;
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            const uint32_t m = out ? 0xffffffffu : nan_bytes(cur.v[r][q]);
            nan_seen |= !out && m != 0;
            cur.v[r][q] &= ~m;
          }
        }
      }
      bool up = false;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) up |= fmaxf(x[i][j], x[i][2 + j]) > R[i][j] + kHeadroom;
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float m = fmaxf(x[i][j], x[i][2 + j]);
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            m = fmaxf(m, R[i][j]);
            const float al = ref_factor(R[i][j], m);
            R[i][j] = m;
            l[i][j] *= al;
#pragma unroll
            for (int d = 0; d < kMT; ++d) {
              o[i][d][j] *= al;
              o[i][d][2 + j] *= al;
            }
          }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float ra = R[i][0] == -INFINITY ? 0.f : R[i][0], rb = R[i][1] == -INFINITY ? 0.f : R[i][1];
        const float w0 = ex2(x[i][0] - ra), w1 = ex2(x[i][1] - rb), w2 = ex2(x[i][2] - ra), w3 = ex2(x[i][3] - rb);
        l[i][0] = fmaf(w0 + w2, un_ev, l[i][0]);
        l[i][1] = fmaf(w1 + w3, un_ev, l[i][1]);
        const __half2 ha = __floats2half2_rn(w0, w1), hb = __floats2half2_rn(w2, w3);
        pf[i][0] = movm(*reinterpret_cast<const uint32_t*>(&ha));
        pf[i][1] = movm(*reinterpret_cast<const uint32_t*>(&hb));
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        // bytes 4q .. 4q + 3 of the thread's dims: tiles 2q, 2q + 1
        const uint32_t lo0 = __byte_perm(cur.v[0][q], cur.v[1][q], 0x5140), lo1 = __byte_perm(cur.v[0][q], cur.v[1][q], 0x7362);
        const uint32_t hi0 = __byte_perm(cur.v[2][q], cur.v[3][q], 0x5140), hi1 = __byte_perm(cur.v[2][q], cur.v[3][q], 0x7362);
        uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
        widen4(lo0, a0, a1);
        widen4(hi0, a2, a3);
        widen4(lo1, b0, b1);
        widen4(hi1, b2, b3);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          mma16816(o[i][2 * q], a0, a1, a2, a3, pf[i][0], pf[i][1]);
          mma16816(o[i][2 * q + 1], b0, b1, b2, b3, pf[i][0], pf[i][1]);
        }
      }
    }
  };

  // The chain of dependent accesses before the first keys is what a short split waits for: block ids
  // first, then the first keys, and the queries while those travel
  constexpr int kTurn = 16 * kWarps;  // keys that the warps take in one turn
  stage_pages();
  __syncthreads();
  for (int i = 0; i < kStages; ++i) send(k_begin + warp * 16 + i * kTurn);
  stage_scales();
  // queries: B operand, row g8 of each 8-row tile; the row's power of two goes to the logits
  const int64_t q_stride = a.q_stride ? a.q_stride : static_cast<int64_t>(a.H) * D;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const bool on = i * 8 + g8 < n_row;
    const int qi = query(i * 8 + g8);
    uint32_t w[kKS][2], mb = 0;
    const uint16_t* qr = static_cast<const uint16_t*>(a.q) + (q0 + qi) * q_stride +
                         (static_cast<int64_t>(h) * geo.g + (static_cast<int>(row0) + i * 8 + g8 - qi * geo.g)) * D;
#pragma unroll
    for (int k = 0; k < kKS; k += 2) {
      // dims (D / 4) t + 4 k .. + 7
      uint4 v = make_uint4(0, 0, 0, 0);
      if (on) v = __ldg(reinterpret_cast<const uint4*>(qr + (D / 4) * t4 + 4 * k));
      w[k][0] = v.x;
      w[k][1] = v.y;
      w[k + 1][0] = v.z;
      w[k + 1][1] = v.w;
      mb = max_u16x2(mb, max_u16x2(max_u16x2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), max_u16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
    // the largest magnitude as BF16 bits; only where that is not finite the largest finite one
    mb = max_u16x2(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
    mb = max_u16x2(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
    float amax = __uint_as_float(max(mb & 0xffffu, mb >> 16) << 16);
    if (__any_sync(0xffffffffu, !(amax < INFINITY))) {
      amax = 0.f;
#pragma unroll
      for (int k = 0; k < kKS; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          amax = fmaxf(amax, fmaxf(finite_abs(__uint_as_float(w[k][j] << 16)), finite_abs(__uint_as_float(w[k][j] & 0xffff0000u))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    }
    // largest value into [2^14, 2^15)
    const int eq = amax > 0.f ? max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -100) : 0;
    const float dn = pow2f(-eq);
#pragma unroll
    for (int k = 0; k < kKS; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __half2 hv = __floats2half2_rn(__uint_as_float(w[k][j] << 16) * dn, __uint_as_float(w[k][j] & 0xffff0000u) * dn);
        qf[i][k][j] = *reinterpret_cast<const uint32_t*>(&hv);
      }
    const float f = a.scale * kLog2e * pow2f(eq);
    f_row[i][0] = __shfl_sync(0xffffffffu, f, 8 * t4);
    f_row[i][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
  }
  __syncthreads();
  int place = 0;
  uint32_t parity = 0;
  bool ok = true;
  auto arrived = [&](int at, uint32_t par) -> bool {
    for (long it = 0; it < kSpin; ++it)
      if (mbar_test(bar_at + 8 * at, par)) return true;
    set_status(a.status, LC_DEV_TIMEOUT);
    return false;
  };
  for (int t0 = k_begin + warp * 16; t0 < k_end; t0 += kTurn) {
    ok = __all_sync(0xffffffffu, arrived(place, parity));
    if (!ok) break;
    Step<D> cur;
    take(place, cur);
    __syncwarp();
    send(t0 + kStages * kTurn);
    step(t0, cur);
    if (++place == kStages) {
      place = 0;
      parity ^= 1;
    }
  }
  // after a wait that ran out: what is still on its way lands (or runs out, too) before the CTA ends
  if (!ok)
    for (int i = max(0, sent - kStages); i < sent; ++i)
      for (long it = 0; it < kSpin && !mbar_test(bar_at + 8 * (i % kStages), (i / kStages) & 1); ++it) {
      }
  __syncwarp();

  // join the warps.  A pair of dims of a row lies at its index ^ pair_key, so that the 16 lanes of a store, four
  // rows of the same few dims, meet 16 banks
  auto pair_key = [](int r, int d) { return D == 128 ? (d >> 5 & 1) | (r & 6) : r >> 1 & 3; };
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      l[i][j] += __shfl_xor_sync(0xffffffffu, l[i][j], 4);
      l[i][j] += __shfl_xor_sync(0xffffffffu, l[i][j], 8);
      l[i][j] += __shfl_xor_sync(0xffffffffu, l[i][j], 16);
      const int r = i * 8 + 2 * t4 + j;
      if (g8 == 0) s_ml[warp][r] = make_float2(R[i][j], l[i][j]);
#pragma unroll
      for (int m = 0; m < kMT; ++m)
        reinterpret_cast<float2*>(ring)[r * (D / 2) + ((kVB / 2 * g8 + m) ^ pair_key(r, kVB * g8))] = make_float2(o[i][m][j], o[i][m][2 + j]);
    }
  const bool nans = __syncthreads_or(nan_seen);
  for (int i = tid; i < n_row * (D / 4); i += kThreads) {
    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
    float M = s_ml[0][r].x;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_ml[w][r].x);
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int key = pair_key(r, d);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ref_factor(s_ml[w][r].x, M);
      L = fmaf(s_ml[w][r].y, f, L);
      float4 v = reinterpret_cast<const float4*>(ring + (w - warp) * Ring::kWarp)[r * (D / 4) + (d / 4 ^ key >> 1)];
      if (key & 1) v = make_float4(v.z, v.w, v.x, v.y);
      acc.x = fmaf(v.x, f, acc.x);
      acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z);
      acc.w = fmaf(v.w, f, acc.w);
    }
    const int qi = query(r);
    if (nans) {
      // the edge steps that this row sees: below all_lo, and from the step of all_hi on
      const Kv8Range x = kv8_range(kv, a.W, p0 + qi, p0 + qi);
      const int lo = max(x.lo, k_begin), hi = min(x.hi, k_end);
      const uint32_t m = kv8_value_nans(c, s, h, lo, min(hi, (all_lo + 15) & ~15), d) |
                         kv8_value_nans(c, s, h, max(lo, all_hi & ~15), hi, d);
      if (m & 0xffu) acc.x = NAN;
      if (m & 0xff00u) acc.y = NAN;
      if (m & 0xff0000u) acc.z = NAN;
      if (m & 0xff000000u) acc.w = NAN;
    }
    const int head = h * geo.g + (static_cast<int>(row0) + r - qi * geo.g);
    const int64_t orow = static_cast<int64_t>(q0 + qi) * a.H + head;
    if (n_split > 1) {
      *reinterpret_cast<float4*>(ws_o + (orow * geo.n_split + split) * D + d) = acc;
      if (d == 0) ws_ml[orow * geo.n_split + split] = make_float2(M, L);
    } else {
      float lse;
      const float f = kv8_finish(M, L, a.sink, head, &lse);
      const uint32_t w0 = static_cast<uint32_t>(f32_to_bf16_bits(acc.x * f)) |
                          (static_cast<uint32_t>(f32_to_bf16_bits(acc.y * f)) << 16);
      const uint32_t w1 = static_cast<uint32_t>(f32_to_bf16_bits(acc.z * f)) |
                          (static_cast<uint32_t>(f32_to_bf16_bits(acc.w * f)) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + d) = make_uint2(w0, w1);
      if (a.lse && d == 0) a.lse[orow] = lse;
    }
  }
}

// Joins the splits of each row: a CTA per (query, head), its warps take splits in turn (eight at a
// time in flight) and meet in shared memory.  What a warp does besides its splits counts: with two of them the join
// of 2048 rows of up to 16 splits takes 5 us of a call's 100 (four: 7, eight: 14), of 64 rows of 72 splits 5 of 96
// (one of 16: 4).
constexpr int kCombineWarps = 2;

template <int D>
__global__ void __launch_bounds__(32 * kCombineWarps) k_kv8_combine(lc_kv8_attn_args a, Kv8Geom geo, const float* __restrict__ ws_o,
                                                                    const float2* __restrict__ ws_ml) {
  constexpr int kE = D / 32;
  __shared__ float s_m[kCombineWarps], s_l[kCombineWarps];
  __shared__ float s_o[kCombineWarps][D];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t orow = blockIdx.x;
  const int q = static_cast<int>(blockIdx.x / static_cast<uint32_t>(a.H)), head = static_cast<int>(blockIdx.x % static_cast<uint32_t>(a.H));
  if (!geo.decode && (q < __ldg(a.q_start) || q >= __ldg(a.q_start + a.num_seqs))) return;
  const int s = geo.decode ? q : seq_of_query(a.q_start, a.num_seqs, q);
  const int q0 = __ldg(a.q_start + s), p0 = __ldg(a.q_pos0 + s);
  const int nq = min(__ldg(a.q_start + s + 1) - q0, a.max_q);
  if (q - q0 >= nq) return;
  int n_split = geo.n_split;
  if (!geo.tc) {
    // the range of the row tile that held this row
    const uint32_t rr = (q - q0) * geo.g + static_cast<uint32_t>(head) % static_cast<uint32_t>(geo.g);
    const uint32_t row0 = rr / static_cast<uint32_t>(geo.rows) * geo.rows;
    const uint32_t row1 = min(row0 + geo.rows, static_cast<uint32_t>(nq) * geo.g) - 1;
    const int kv = min(min(__ldg(a.kv_len + s), a.max_kv), a.cache.table_cols * a.cache.bt);
    const Kv8Range rg = nq == 1 ? kv8_range(kv, a.W, p0, p0)
                                : kv8_range(kv, a.W, p0 + static_cast<int>(row0 / static_cast<uint32_t>(geo.g)), p0 + static_cast<int>(row1 / static_cast<uint32_t>(geo.g)));
    n_split = kv8_n_split(rg.hi - rg.lo16, a.cache.H_kv);
  }
  if (n_split <= 1) return;
  const float2* ml = ws_ml + orow * geo.n_split;
  const float* po = ws_o + orow * geo.n_split * D + lane * kE;
  // each warp on its own first: it needs no one else's maximum
  float M = -INFINITY, L = 0.f, acc[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) acc[e] = 0.f;
  for (int i0 = warp; i0 < n_split; i0 += 8 * kCombineWarps) {
    float2 x[8];
    float v[8][kE];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * kCombineWarps;
      x[j] = make_float2(-INFINITY, 0.f);
      if (i < n_split) {
        x[j] = ml[i];
        if constexpr (kE == 4) {
          const float4 t = *reinterpret_cast<const float4*>(po + static_cast<int64_t>(i) * D);
          v[j][0] = t.x; v[j][1] = t.y; v[j][2] = t.z; v[j][3] = t.w;
        } else {
          const float2 t = *reinterpret_cast<const float2*>(po + static_cast<int64_t>(i) * D);
          v[j][0] = t.x; v[j][1] = t.y;
        }
      }
    }
    float m = M;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, x[j].x);
    const float f0 = ref_factor(M, m);
    M = m;
    L *= f0;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] *= f0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (x[j].x == -INFINITY && x[j].y == 0.f) continue;  // saw no key
      const float f = ref_factor(x[j].x, M);
      L = fmaf(x[j].y, f, L);
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[e] = fmaf(v[j][e], f, acc[e]);
    }
  }
  if (lane == 0) {
    s_m[warp] = M;
    s_l[warp] = L;
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) s_o[warp][lane * kE + e] = acc[e];
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  M = s_m[0];
#pragma unroll
  for (int w = 1; w < kCombineWarps; ++w) M = fmaxf(M, s_m[w]);
  L = 0.f;
  float o0 = 0.f, o1 = 0.f;
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) {
    if (s_m[w] == -INFINITY && s_l[w] == 0.f) continue;
    const float f = ref_factor(s_m[w], M);
    L = fmaf(s_l[w], f, L);
    const float2 t = *reinterpret_cast<const float2*>(&s_o[w][2 * threadIdx.x]);
    o0 = fmaf(t.x, f, o0);
    o1 = fmaf(t.y, f, o1);
  }
  float lse;
  const float f = kv8_finish(M, L, a.sink, head, &lse);
  reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + orow * D)[threadIdx.x] =
      static_cast<uint32_t>(f32_to_bf16_bits(o0 * f)) | (static_cast<uint32_t>(f32_to_bf16_bits(o1 * f)) << 16);
  if (a.lse && threadIdx.x == 0) a.lse[orow] = lse;
}

namespace {

// From this many rows per (sequence, shared head) on, a call takes the tensor-memory kernel: its tiles have
// 128 rows whether they are full or not, k_kv8_attn reads the keys again for every 8 (or 16) rows.
// Measured (us, k_kv8_attn / k_kv8_attn_tc), 8 heads of 128 dims, 8 query heads each: one sequence of 8192
// tokens 16.5 / 17.3 at 16 rows, 19.9 / 18.1 at 32, 32 / 19 at 64; of 65536 49 / 68, 87 / 66, 161 / 70; eight of
// 8192 35 / 70, 63 / 71, 116 / 74.  8 heads of 64 dims, 4 query heads each, eight of 8192: 48 / 44 at 32, 66 / 46 at 64.
// The rule looks at the rows of one sequence alone: for several sequences of 32 rows (four queries, 8 heads
// each) it takes the slower kernel, by an eighth in the table above.
constexpr int kTcRows = 32;

// Splits that any row tile of the call can have.
Kv8Geom geometry(const lc_kv8_attn_args& a, bool decode) {
  Kv8Geom geo;
  geo.g = a.H / a.cache.H_kv;
  const int64_t all = static_cast<int64_t>(a.max_q) * geo.g;
  geo.decode = decode;
  geo.tc = !decode && all >= kTcRows;
  geo.rows = geo.tc ? kv8_tc_rows(a.cache.D) : geo.g <= 8 ? 8 : 16;
  geo.row_tiles = static_cast<int>((all + geo.rows - 1) / geo.rows);
  geo.n_split = 1;
  // keys of a row tile: as the kernels cut them, and of the window with its start rounded down
  int64_t keys = min(a.max_kv, a.cache.table_cols * a.cache.bt);
  if (a.W > 0) keys = min(keys, static_cast<int64_t>(a.W) + a.max_q - 1 + 16);
  const int n = static_cast<int>(keys);
  if (geo.tc) {
    // fewer CTAs than the device holds at once: split the keys, at least 4 tiles of 128 each
    const int64_t ctas = static_cast<int64_t>(geo.row_tiles) * a.cache.H_kv * a.num_seqs;
    const int64_t fill = sm_count() * (a.cache.D == 128 ? 1 : 2) / ctas;
    geo.n_split = static_cast<int>(max(int64_t{1}, min(fill, static_cast<int64_t>(n) / 512)));
  } else {
    geo.n_split = kv8_split_bound(n, a.cache.H_kv);
  }
  return geo;
}

size_t align16(size_t n) { return (n + 15) & ~size_t{15}; }

template <int D, int NT>
cudaError_t launch_few(const lc_kv8_attn_args& a, const Kv8Geom& geo, unsigned grid, float* ws_o, float2* ws_ml, cudaStream_t st) {
  CUtensorMap map_k = {}, map_v = {};
  const int64_t slots = static_cast<int64_t>(a.cache.n_blocks) * a.cache.H_kv;
  if (a.max_kv > 0 && slots > 0) {  // else there is nothing to copy, and the kernel does not touch the maps
    constexpr CUtensorMapSwizzle swizzle = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!encode_bytes()) return cudaErrorNotSupported;
    if (!byte_map3(&map_k, a.cache.k, slots, a.cache.bt, D, 16, swizzle) || !byte_map3(&map_v, a.cache.v, slots, a.cache.bt, D, 16, swizzle))
      return cudaErrorInvalidValue;
  }
  constexpr size_t smem = Kv8Ring<D>::kBytes;
  return launch_big<k_kv8_attn<D, NT>>(smem, dim3(grid), dim3(kThreads), smem, st, 1, map_k, map_v, a, geo, ws_o, ws_ml);
}

template <int D>
cudaError_t launch(const lc_kv8_attn_args& a, const Kv8Geom& geo, cudaStream_t st) {
  if (1.0 * geo.n_split * geo.row_tiles * a.cache.H_kv * a.num_seqs > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int64_t grid = static_cast<int64_t>(geo.n_split) * geo.row_tiles * a.cache.H_kv * a.num_seqs;
  const size_t rows = static_cast<size_t>(a.n_q) * a.H;
  float* ws_o = static_cast<float*>(a.workspace);
  float2* ws_ml = reinterpret_cast<float2*>(static_cast<char*>(a.workspace) + align16(rows * geo.n_split * D * 4));
  const cudaError_t e = geo.tc ? launch_kv8_attn_tc(a, geo, static_cast<unsigned>(grid), ws_o, ws_ml, st)
                        : geo.rows == 8 ? launch_few<D, 1>(a, geo, static_cast<unsigned>(grid), ws_o, ws_ml, st)
                                        : launch_few<D, 2>(a, geo, static_cast<unsigned>(grid), ws_o, ws_ml, st);
  if (e != cudaSuccess || geo.n_split == 1) return e;
  return launch_ex(k_kv8_combine<D>, dim3(static_cast<unsigned>(rows)), dim3(32 * kCombineWarps), 0, st, true, 1, a, geo,
                   static_cast<const float*>(ws_o), static_cast<const float2*>(ws_ml));
}

}  // namespace

size_t kv8_attn_workspace(const lc_kv8_attn_args& a, bool decode) {
  const Kv8Geom geo = geometry(a, decode);
  if (geo.n_split == 1) return 0;
  const size_t rows = static_cast<size_t>(a.n_q) * a.H;
  return align16(rows * geo.n_split * a.cache.D * 4) + rows * geo.n_split * sizeof(float2);
}

cudaError_t launch_kv8_attn(const lc_kv8_attn_args& a, bool decode, cudaStream_t st) {
  const Kv8Geom geo = geometry(a, decode);
  return a.cache.D == 128 ? launch<128>(a, geo, st) : launch<64>(a, geo, st);
}

}  // namespace lc
