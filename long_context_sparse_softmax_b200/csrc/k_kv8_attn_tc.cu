// kv8_attn for many query rows (prefill) on the 5th-generation tensor cores (tcgen05, F16 operands,
// FP32 accumulators in tensor memory).  The same arithmetic as k_kv8_attn.cu: see lc_kv8.cuh.
//
// A CTA holds one or two tiles (kT) of 128 rows of one sequence and shared head (row r: query r / g,
// head r % g of the group), which share every key tile of 128 tokens:
//   S_i = Q_i K^T   M = 128 rows, N = 64 keys (half tiles, two of them per row tile), both K-major in
//                   shared memory;
//   P_i             F16 weights (11 bits: see k_kv8_attn.cu), written over S_i's columns of tensor memory;
//   O_i += P_i V    A = P_i in tensor memory, B = V (keys x dims, dims contiguous: MN-major).
// The codes are widened to F16 (exact) once per CTA, and the row's softmax keeps the precision that
// it has with few rows.  S of a half tile is computed while the softmax works on the half before, and
// one row tile's (or CTA's) softmax runs while the tensor core works on the other's products.
//
// Warps 0 .. 4 kT - 1: softmax, a thread per row (its sums need no shuffles).  The next 4: fetch codes
// into registers a tile ahead, widen them into the two-stage rings of K and V.  The next kT: one lane
// issues the products of a row tile.  (The others only complete their warpgroup.)
// A softmax thread computes its half tile's weights with the reference R it has; only when their sum
// passes 2^12 does R move to the largest logit, O is rescaled in tensor memory and the weights are computed again (the
// first half tile, and rarely after it).  Half tiles whose keys every row sees skip the mask.
// Every wait on an mbarrier is bounded (LC_DEV_TIMEOUT).
//
// What bounds it: the exponentials (16 a cycle on a multiprocessor: 2048 cycles per 256 x 128 tile, as
// many as its products take) and the latency of each softmax step; a tile takes about 4000 cycles, 2950
// of them for the weights.
// 2048 queries at the end of 8192 tokens, 64 / 8 heads of 128 dims: 501 us in a graph of such calls, 960
// TFLOP/s (56 % of the measured F16 rate; 512 CTAs are 3.46 rounds of 148, run as 4), 521 us as a call among
// others.  On the way there: a mma.sync kernel with
// 8 rows a tile 4960 us; 256 rows on tcgen05 1190; packed FP32 pairs and a uniform issuing warp 734; half
// tiles ahead of the softmax 545; cheaper widening and masks 520.
#include "lc_e4m3.cuh"
#include "lc_kv8.cuh"

namespace lc {

namespace {

constexpr int kTK = 128;                 // keys per tile
constexpr int kHK = 64;                  // keys per product with Q and per softmax step
constexpr int kRT = 128;                 // rows per row tile
constexpr float kMaxSum = 4096.f;         // of a half tile's weights before R moves
constexpr long kSpin = 1L << 20;         // a few seconds
constexpr int kHalf = kTK * 128;         // bytes of 128 rows x 64 F16 values (SWIZZLE_128B)

struct Bars {
  uint64_t qfull[2];   // Q_i in shared memory (128 arrivals)
  uint64_t fin[2];     // a role that gave up: its products are complete (commit)
  uint64_t kfull[2], vfull[2];    // stage written (128)
  uint64_t kempty[2], vempty[2];  // stage read by every row tile (commits)
  uint64_t sfull[2][2];  // S_i of a half tile computed (commit), its scales in shared memory (the issuer's arrival)
  uint64_t pfull[2][2];  // P_i written, O_i rescaled (128)
  uint64_t ofull[2][2];  // O_i updated (commit)
};

// D += A B with A (128 rows x 16 F16 values) in tensor memory
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}

// shared-memory loads that stay where they are written: hoisted, a tile's scales would take registers
__device__ __forceinline__ float2 ld_shared2(const void* p) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(su32(p)) : "memory");
  return v;
}
__device__ __forceinline__ float ld_shared1(const void* p) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(su32(p)) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// offset of chunk j (8 values) of half hf of row r in a tile of 128 rows
__device__ __forceinline__ uint32_t tile_off(int r, int hf, int j) { return hf * kHalf + sw128_off(r, j); }

// Row tiles of a CTA.  128 dims: two (tensor memory is full with S and O of both).  64 dims: one, and
// two CTAs a multiprocessor: each starts and ends while the other computes (ragged windowed prefill of
// 28 / 4 heads, 10 key tiles a CTA: 92 us with two row tiles a CTA, 83 us with one, 80 us without a maximum
// per key).
template <int D>
struct Shape {
  static constexpr int kT = D == 128 ? 2 : 1;
  static constexpr int kSoft = 4 * kT;                     // softmax warps, then 4 that widen, then the issuing ones
  static constexpr int kThreads = 32 * (kSoft + 8);
  static constexpr int kPerSm = kT == 1 ? 2 : 1;
  // registers a thread at launch, and by role: together what the CTA was launched with
  static constexpr int kLaunch = kT == 2 ? 128 : 80, kRegSoft = kT == 2 ? 192 : 144, kRegWiden = kT == 2 ? 96 : 64, kRegIssue = 32;
  static_assert(32 * kSoft * kRegSoft + 128 * (kRegWiden + kRegIssue) <= kThreads * kLaunch, "registers");
  static constexpr uint32_t kColO = 128 * kT, kCols = 256 * kT;  // S_i at 128 i (two half tiles), O_i behind them
  static constexpr size_t kSmem = (kT + 4) * static_cast<size_t>(kHalf) * (D / 64) + 1024;
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, Shape<D>::kPerSm)
    k_kv8_attn_tc(lc_kv8_attn_args a, Kv8Geom geo, float* __restrict__ ws_o, float2* __restrict__ ws_ml) {
  constexpr int kTile = kHalf * (D / 64);  // bytes of a 128 x D F16 tile
  constexpr int kPR = D / 16;              // 16-code pieces per row
  constexpr int kIt = kTK * kPR / 128;     // pieces per converter thread
  constexpr int kT = Shape<D>::kT, kSoft = Shape<D>::kSoft, kThreads = Shape<D>::kThreads;
  constexpr uint32_t kColO = Shape<D>::kColO;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* Qs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* Ks = Qs + kT * kTile;
  uint8_t* Vs = Ks + 2 * kTile;
  __shared__ float4 s_sc[4][8];  // per 16 keys of a tile: 2^ek, ev, 2^-ev (ring of 4 tiles)
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_nan;
  __shared__ __align__(8) Bars bars;

  pdl_wait();
  pdl_trigger();
  const lc_kv8_cache& c = a.cache;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  int64_t u = blockIdx.x;
  const int split = static_cast<int>(u % geo.n_split);
  u /= geo.n_split;
  const int h = static_cast<int>(u % c.H_kv);
  u /= c.H_kv;
  const int s = static_cast<int>(u % a.num_seqs);
  // the last rows of a sequence see the most keys: they start first
  const int rt = geo.row_tiles - 1 - static_cast<int>(u / a.num_seqs);

  const int q0 = __ldg(a.q_start + s);
  const int nq = min(__ldg(a.q_start + s + 1) - q0, a.max_q);
  const int64_t row0 = static_cast<int64_t>(rt) * (kT * kRT);
  const int64_t all_rows = static_cast<int64_t>(nq) * geo.g;
  if (nq <= 0 || row0 >= all_rows) return;
  const int n_row = static_cast<int>(min(static_cast<int64_t>(kT * kRT), all_rows - row0));
  const int n_act = n_row > kRT ? 2 : 1;
  const int p0 = __ldg(a.q_pos0 + s);
  const int kv_all = __ldg(a.kv_len + s);
  const int kv = min(min(kv_all, a.max_kv), c.table_cols * c.bt);
  if (kv < min(kv_all, a.max_kv) && tid == 0) set_status(a.status, LC_DEV_BAD_BLOCK);
  auto pos = [&](int r) { return p0 + static_cast<int>((row0 + r) / geo.g); };
  const Kv8Range rg = kv8_range(kv, a.W, pos(0), pos(n_row - 1));
  const int kb0 = rg.lo16 & ~(kTK - 1);
  const int all_tiles = rg.hi > rg.lo16 ? (rg.hi - kb0 + kTK - 1) / kTK : 0;
  const int tile0 = static_cast<int>(static_cast<int64_t>(all_tiles) * split / geo.n_split);
  const int n_tiles = static_cast<int>(static_cast<int64_t>(all_tiles) * (split + 1) / geo.n_split) - tile0;
  const int k0 = kb0 + tile0 * kTK;                      // first key of the CTA
  const int k_end = min(rg.hi, k0 + n_tiles * kTK);

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const uint32_t addr = su32(bar);
    for (long it = 0; it < kSpin; ++it) {
      if (mbar_test(addr, parity)) return true;
      if ((it & 1023) == 1023 && *reinterpret_cast<volatile int*>(&s_abort)) return false;
    }
    set_status(a.status, LC_DEV_TIMEOUT);
    atomicExch(&s_abort, 1);
    return false;
  };

  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };

  if (warp == kSoft + 4) tmem_alloc(su32(&s_tmem), Shape<D>::kCols);
  if (tid == 0) {
    s_abort = s_nan = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(su32(&bars.qfull[i]), 128);
      mbar_init(su32(&bars.fin[i]), 1);
      mbar_init(su32(&bars.kfull[i]), 128);
      mbar_init(su32(&bars.vfull[i]), 128);
      mbar_init(su32(&bars.kempty[i]), n_act);
      mbar_init(su32(&bars.vempty[i]), n_act);
      for (int b = 0; b < 2; ++b) {
        mbar_init(su32(&bars.sfull[i][b]), 2);
        mbar_init(su32(&bars.pfull[i][b]), 128);
        mbar_init(su32(&bars.ofull[i][b]), 1);
      }
    }
    fence_mbar_init();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = s_tmem;

  const int i = warp < kSoft ? warp >> 2 : warp - (kSoft + 4);  // row tile of a softmax or issuing warp
  const int r = tid;                               // softmax: row of the CTA
  float R = -INFINITY, l = 0.f;
  bool good = true;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;

  if (warp < kSoft) {
    regs_inc<Shape<D>::kRegSoft>();
    if (i < n_act) {
      // ---------------- Q: the row, scaled by a power of two into F16's range (k_kv8_attn.cu)
      float f_row;
      {
        const int64_t q_stride = a.q_stride ? a.q_stride : static_cast<int64_t>(a.H) * D;
        const int64_t rr = row0 + r;
        const uint4* qr = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (q0 + rr / geo.g) * q_stride +
                                                         (static_cast<int64_t>(h) * geo.g + rr % geo.g) * D);
        uint4 v[D / 8];
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) v[k] = r < n_row ? __ldg(qr + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, fmaxf(finite_abs(__uint_as_float(w[j] << 16)), finite_abs(__uint_as_float(w[j] & 0xffff0000u))));
        }
        const int eq = amax > 0.f ? max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -100) : 0;
        const float dn = pow2f(-eq);
        f_row = a.scale * kLog2e * pow2f(eq);
        uint8_t* qt = Qs + i * kTile;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __half2 hv = __floats2half2_rn(__uint_as_float(w[j] << 16) * dn, __uint_as_float(w[j] & 0xffff0000u) * dn);
            o[j] = *reinterpret_cast<const uint32_t*>(&hv);
          }
          *reinterpret_cast<uint4*>(qt + tile_off(r & (kRT - 1), k / 8, k % 8)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_async_smem();
        mbar_arrive(su32(&bars.qfull[i]));
      }
      // visible keys of the row, and those that every row of the tile sees
      const Kv8Range me = kv8_range(kv, a.W, pos(r), pos(r));
      const int r_lo = me.lo, r_hi = r < n_row ? me.hi : 0;
      const int last_r = min(n_row, (i + 1) * kRT) - 1;
      const int all_hi = kv8_range(kv, a.W, pos(i * kRT), pos(i * kRT)).hi;
      const int all_lo = kv8_range(kv, a.W, pos(last_r), pos(last_r)).lo;
      const uint32_t ts = tm + lane_off + i * kTK, to = tm + lane_off + kColO + i * 128;

      for (int hh = 0; hh < 2 * n_tiles; ++hh) {
        const int t = hh >> 1, bf = hh & 1;
        const int t0 = k0 + hh * kHK;
        const bool edge = t0 < all_lo || t0 + kHK > all_hi;
        const bool ok = wait(&bars.sfull[i][bf], t & 1);
        if (!__all_sync(0xffffffffu, ok)) {
          good = false;
          break;
        }
        fence_after();
        uint32_t y[2][32];
        tmem_ld32(ts + bf * kHK, y[0]);
        tmem_ld32(ts + bf * kHK + 32, y[1]);
        tmem_wait_ld();
        // y = x + ev - R
        const float Ru = R == -INFINITY ? 0.f : R;
#pragma unroll
        for (int g = 0; g < kHK / 16; ++g) {
          const float2 sc = ld_shared2(&s_sc[t & 3][bf * 4 + g]);
          const uint64_t fk = pack2(f_row * sc.x, f_row * sc.x), off = pack2(sc.y - Ru, sc.y - Ru);
          uint32_t* v = y[g / 2] + (g & 1) * 16;
#pragma unroll
          for (int j = 0; j < 16; j += 2) fma2_regs(v[j], v[j + 1], fk, off);
        }
        bool sees = r < n_row;  // a key of the half tile
        if (edge) {
          const int d_lo = r_lo - t0, d_hi = r_hi - t0;  // the row's keys within the half tile
          sees = d_lo < kHK && d_hi > 0 && d_lo < d_hi;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // bit j: the row sees key 32 x + j of the half tile
            const int lo = min(max(d_lo - 32 * x, 0), 32), hi = min(max(d_hi - 32 * x, 0), 32);
            const uint32_t below = hi < 32 ? (1u << hi) - 1 : 0xffffffffu, from = lo < 32 ? 0xffffffffu << lo : 0u;
            const uint32_t see = below & from;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(see & (1u << j))) y[x][j] = 0xff800000u;
          }
        }
        // the weights 2^y, their sum, and the part of l that is theirs
        uint32_t pk[kHK / 2];
        float ls, al = 1.f;
        bool again = false;
        do {
          const bool second = again;
          float sum = 0.f;
          ls = 0.f;
#pragma unroll
          for (int g = 0; g < kHK / 16; ++g) {
            const uint32_t* v = y[g / 2] + (g & 1) * 16;
            uint64_t gs = 0;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float w0 = ex2(__uint_as_float(v[j])), w1 = ex2(__uint_as_float(v[j + 1]));
              gs = add2(gs, pack2(w0, w1));
              const __half2 hv = __floats2half2_rn(w0, w1);
              pk[g * 8 + j / 2] = *reinterpret_cast<const uint32_t*>(&hv);
            }
            const float s16 = sum2(gs);
            sum += s16;
            ls = fmaf(s16, ld_shared1(&s_sc[t & 3][bf * 4 + g].z), ls);
          }
          // R is the largest logit when it is set; a sum says whether a weight has come near F16's end since
          const bool need = !second && (R == -INFINITY ? sees : sum > kMaxSum);
          again = __any_sync(0xffffffffu, need);
          if (again) {
            float ymax = -INFINITY;
#pragma unroll
            for (int j = 0; j < kHK; ++j) ymax = fmaxf(ymax, __uint_as_float(y[j / 32][j % 32]));
            const float up = need && ymax > -INFINITY ? ymax : 0.f;
            if (need && ymax > -INFINITY) {
              al = ref_factor(R, Ru + up);
              R = Ru + up;
            }
#pragma unroll
            for (int j = 0; j < kHK; ++j) y[j / 32][j % 32] = __float_as_uint(__uint_as_float(y[j / 32][j % 32]) - up);
          }
        } while (again);
        if (__any_sync(0xffffffffu, al != 1.f) && hh > 0) {
          if (!__all_sync(0xffffffffu, wait(&bars.ofull[i][bf ^ 1], ((hh - 1) >> 1) & 1))) {
            good = false;
            break;
          }
          fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 16) {
            uint32_t ov[16];
            tmem_ld16(to + d, ov);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * al);
            tmem_st16(to + d, ov);
          }
        }
        l = fmaf(l, al, ls);
        tmem_st32(ts + bf * kHK, pk);
        tmem_wait_st();
        fence_before();
        mbar_arrive(su32(&bars.pfull[i][bf]));
      }
      if (good && n_tiles > 0) good = __all_sync(0xffffffffu, wait(&bars.ofull[i][1], (n_tiles - 1) & 1));
    }
    named_bar(1, kThreads);
    // ---------------- output: a thread per row
    if (i < n_act) {
      fence_after();
      const int64_t rr = row0 + r;
      const int head = h * geo.g + static_cast<int>(rr % geo.g);
      const int64_t orow = static_cast<int64_t>(q0 + rr / geo.g) * a.H + head;
      const bool store = good && r < n_row;
      const int p = pos(r);
      float lse = 0.f, f = 1.f;
      if (geo.n_split == 1) {
        f = store ? kv8_finish(R, l, a.sink, head, &lse) : 0.f;
        if (store && a.lse) a.lse[orow] = lse;
      } else if (store) {
        ws_ml[orow * geo.n_split + split] = make_float2(R, l);
      }
  #pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t ov[32];
        if (n_tiles > 0) {
          tmem_ld32(tm + lane_off + kColO + i * 128 + d, ov);
          tmem_wait_ld();
        } else {
  #pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = 0;
        }
        if (s_nan && store) {
          // value codes that were replaced: those of the row's keys make its outputs NaN.  They lie in the
          // tiles that not every row of the CTA sees whole, below last.lo and from the tile of first.hi on
          // (elsewhere a NaN has reached O by itself): a few tiles, however long the cache is
          const Kv8Range me = kv8_range(kv, a.W, p, p);
          const Kv8Range first = kv8_range(kv, a.W, pos(0), pos(0)), last = kv8_range(kv, a.W, pos(n_row - 1), pos(n_row - 1));
          const int lo = max(me.lo, k0), hi = min(me.hi, k_end);
          const int below = min(hi, (last.lo + kTK - 1) & ~(kTK - 1)), from = max(lo, first.hi & ~(kTK - 1));
  #pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const uint32_t m = kv8_value_nans(c, s, h, lo, below, d + j) | kv8_value_nans(c, s, h, from, hi, d + j);
  #pragma unroll
            for (int b = 0; b < 4; ++b)
              if (m >> (8 * b) & 0xffu) ov[j + b] = 0x7fffffffu;
          }
        }
        if (!store) continue;
        if (geo.n_split > 1) {
          float* o = ws_o + (orow * geo.n_split + split) * D + d;
  #pragma unroll
          for (int j = 0; j < 32; j += 4) *reinterpret_cast<uint4*>(o + j) = make_uint4(ov[j], ov[j + 1], ov[j + 2], ov[j + 3]);
        } else {
          uint16_t* o = static_cast<uint16_t*>(a.out) + orow * D + d;
          uint32_t w[16];
  #pragma unroll
          for (int j = 0; j < 16; ++j)
            w[j] = static_cast<uint32_t>(f32_to_bf16_bits(__uint_as_float(ov[2 * j]) * f)) |
                   (static_cast<uint32_t>(f32_to_bf16_bits(__uint_as_float(ov[2 * j + 1]) * f)) << 16);
  #pragma unroll
          for (int j = 0; j < 16; j += 4) *reinterpret_cast<uint4*>(o + 2 * j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
        }
      }
      fence_before();
    }
  } else if (warp < kSoft + 4) {
    // ---------------- codes -> F16 tiles
    regs_dec<Shape<D>::kRegWiden>();
    const int cw = warp - kSoft;
    // a warp's 32 pieces are whole rows (512 bytes); the eight lanes of a 16-byte store phase take four
    // pieces of two neighbouring rows, whose chunks fall into different banks
    const int piece = D == 128 ? (lane & 3) | (lane >> 1 & 4) : lane & 3;
    const int rsub = D == 128 ? cw * 4 + (lane >> 2 & 1) + (lane >> 4) * 2 : cw * 8 + (lane >> 2);
    constexpr int kRStep = 128 / kPR;             // rows rsub + it * kRStep
    const int all_lo = kv8_range(kv, a.W, pos(n_row - 1), pos(n_row - 1)).lo;  // keys that every row sees
    const int all_hi = kv8_range(kv, a.W, pos(0), pos(0)).hi;
    bool nan_seen = false, ok = true;
    const int bt_log = __ffs(c.bt) - 1;
    const int64_t slot_bytes = static_cast<int64_t>(D) << bt_log;
    // block * H_kv + h of the tile's 16-key group lane % 8, -1: none
    auto slot = [&](int t) -> int {
      const int key = k0 + t * kTK + (lane & 7) * 16;
      if (t >= n_tiles || key >= k_end) return -1;
      const int blk = __ldg(c.table + static_cast<int64_t>(s) * c.table_cols + (key >> bt_log));
      if (blk >= 0 && blk < c.n_blocks) return blk * c.H_kv + h;
      if (key + 16 > rg.lo) set_status(a.status, LC_DEV_BAD_BLOCK);
      return -1;
    };
    // tiles start at multiples of 128, of every block size: a row's place in its block is the same in each
    auto fetch = [&](const uint8_t* base, int sl, uint4 (&v)[kIt]) {
      const bool whole = __all_sync(0xffffffffu, sl >= 0);
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const int row = rsub + it * kRStep;
        const int sr = __shfl_sync(0xffffffffu, sl, row >> 4);
        const uint8_t* p = base + sr * slot_bytes + (row & (c.bt - 1)) * D + piece * 16;
        if (!whole) v[it] = make_uint4(0, 0, 0, 0);
        if (whole || sr >= 0) v[it] = __ldg(reinterpret_cast<const uint4*>(p));
      }
    };
    auto widen = [&](uint32_t tile, const uint4 (&v)[kIt]) {
      const uint32_t lo = tile + tile_off(rsub, piece >> 2, (piece & 3) * 2), hi = tile + tile_off(rsub, piece >> 2, (piece & 3) * 2 + 1);
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        uint32_t o[8];
        widen4(v[it].x, o[0], o[1]);
        widen4(v[it].y, o[2], o[3]);
        widen4(v[it].z, o[4], o[5]);
        widen4(v[it].w, o[6], o[7]);
        // rows 16 (or 32) apart have the same place in the swizzle
        st_shared4(lo + it * kRStep * 128, o[0], o[1], o[2], o[3]);
        st_shared4(hi + it * kRStep * 128, o[4], o[5], o[6], o[7]);
      }
    };
    uint4 kr[kIt], vr[kIt];
    int sl = slot(0), sl_next = slot(1);
    fetch(c.k, sl, kr);
    fetch(c.v, sl, vr);
    for (int t = 0; t < n_tiles; ++t) {
      const int st = t & 1;
      uint8_t bk = 127, bv = 127;
      if (cw == 0 && lane < 8 && sl >= 0) {
        bk = __ldg(c.k_scale + sl);
        bv = __ldg(c.v_scale + sl);
      }
      if (t >= 2) ok = wait(&bars.kempty[st], ((t >> 1) - 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (cw == 0 && lane < 8)
        s_sc[t & 3][lane] = sl < 0 ? make_float4(0.f, -INFINITY, 0.f, 0.f)
                                   : make_float4(pow2f(kv8_exp(bk)), static_cast<float>(kv8_exp(bv)), pow2f(-kv8_exp(bv)), 0.f);
      widen(su32(Ks + st * kTile), kr);
      fence_async_smem();
      mbar_arrive(su32(&bars.kfull[st]));
      fetch(c.k, sl_next, kr);
      if (t >= 2) ok = wait(&bars.vempty[st], ((t >> 1) - 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int t0 = k0 + t * kTK;
      if (t0 < all_lo || t0 + kTK > all_hi) {
        // rows that nobody sees may hold anything, and not every row of the CTA sees the others
#pragma unroll
        for (int it = 0; it < kIt; ++it) {
          const int key = t0 + rsub + it * kRStep;
          const bool out = key < rg.lo || key >= rg.hi;
          uint32_t* w = reinterpret_cast<uint32_t*>(&vr[it]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t m = out ? 0xffffffffu : nan_bytes(w[j]);
            nan_seen |= !out && m != 0;
            w[j] &= ~m;
          }
        }
      }
      widen(su32(Vs + st * kTile), vr);
      fence_async_smem();
      mbar_arrive(su32(&bars.vfull[st]));
      fetch(c.v, sl_next, vr);
      sl = sl_next;
      sl_next = slot(t + 2);
    }
    if (nan_seen) s_nan = 1;
    named_bar(1, kThreads);
  } else {
    // ---------------- products of row tile i
    regs_dec<Shape<D>::kRegIssue>();
    if (i < n_act) {
      const bool one = elect_one();
      const uint32_t id_s = (1u << 4) | (static_cast<uint32_t>(kHK >> 3) << 17) | (static_cast<uint32_t>(kRT >> 4) << 24);
      const uint32_t id_o = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (static_cast<uint32_t>(kRT >> 4) << 24);
      const uint64_t qd = sw128_desc(su32(Qs + i * kTile));  // the address field counts 16 bytes
      const uint32_t ts = tm + i * kTK, to = tm + kColO + i * 128;
      const int n_half = 2 * n_tiles;
      // S of half tile hh; its columns hold P of hh - 2 until that is used up
      auto issue_s = [&](int hh) -> bool {
        const int t = hh >> 1, st = t & 1, bf = hh & 1;
        if (!wait_all(&bars.kfull[st], (t >> 1) & 1) || (hh >= 2 && !wait_all(&bars.ofull[i][bf], (t - 1) & 1))) return false;
        fence_after();
        const uint64_t kd = sw128_desc(su32(Ks + st * kTile)) + bf * (kHK * 128 / 16);
        if (one) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = ((k / 4) * kHalf + (k % 4) * 32) / 16;
            mma_f16(ts + bf * kHK, qd + at, kd + at, id_s, k > 0);
          }
          mma_commit(su32(&bars.sfull[i][bf]));
          mbar_arrive(su32(&bars.sfull[i][bf]));
          if (bf) mma_commit(su32(&bars.kempty[st]));
        }
        return true;
      };
      bool ok = n_tiles == 0 || (wait_all(&bars.qfull[i], 0) && issue_s(0) && issue_s(1));
      for (int hh = 0; ok && hh < n_half; ++hh) {
        const int t = hh >> 1, st = t & 1, bf = hh & 1;
        ok = wait_all(&bars.vfull[st], (t >> 1) & 1) && wait_all(&bars.pfull[i][bf], t & 1);
        if (!ok) break;
        fence_after();
        const uint64_t vd = sw128_mn_desc(su32(Vs + st * kTile), kHalf) + bf * (kHK * 128 / 16);
        if (one) {
#pragma unroll
          for (int k = 0; k < kHK / 16; ++k)
            mma_f16_ts(to, ts + bf * kHK + k * 8, vd + k * (2048 / 16), id_o, hh > 0 || k > 0);
          mma_commit(su32(&bars.ofull[i][bf]));
          if (bf) mma_commit(su32(&bars.vempty[st]));
        }
        if (hh + 2 < n_half) ok = issue_s(hh + 2);
      }
      // a role that gave up: its products complete before tensor memory is released
      if (!ok && one) {
        mma_commit(su32(&bars.fin[i]));
        for (long it = 0; it < kSpin && !mbar_test(su32(&bars.fin[i]), 0); ++it) {
        }
      }
    }
    __syncwarp();
    named_bar(1, kThreads);
  }
  __syncthreads();
  if (warp == kSoft + 4) tmem_dealloc(tm, Shape<D>::kCols);
}

template <int D>
static cudaError_t launch_d(const lc_kv8_attn_args& a, const Kv8Geom& geo, unsigned grid, float* ws_o, float2* ws_ml, cudaStream_t st) {
  constexpr size_t smem = Shape<D>::kSmem;
  return launch_big<k_kv8_attn_tc<D>>(smem, dim3(grid), dim3(Shape<D>::kThreads), smem, st, 1, a, geo, ws_o, ws_ml);
}

cudaError_t launch_kv8_attn_tc(const lc_kv8_attn_args& a, const Kv8Geom& geo, unsigned grid, float* ws_o, float2* ws_ml,
                               cudaStream_t st) {
  return a.cache.D == 128 ? launch_d<128>(a, geo, grid, ws_o, ws_ml, st) : launch_d<64>(a, geo, grid, ws_o, ws_ml, st);
}

}  // namespace lc
