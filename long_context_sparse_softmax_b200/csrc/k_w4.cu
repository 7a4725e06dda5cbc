// w4_proj: y[n, g d_g + c] = sum_k x[n, g K + k] W_g[c, k] for a few rows x, W in MXFP4 (E2M1 codes,
// one E8M0 scale per 32), x in BF16 or MXFP8.
//
// The weights bound it (17/32 byte each, read once); widening them on the CUDA cores would cost
// about as much issue time as their transfer takes.  So they go to the tensor core as they are:
// tcgen05 kind::mxf8f6f4 takes A = 128 outputs x 32 inputs of E2M1 and B = N columns x 32 inputs of
// E4M3 with their E8M0 scales, and accumulates in FP32 in tensor memory.  A BF16 row becomes two
// columns of B: with X the row's scale for a block of 32, hi = e4m3(x / X) and lo = e4m3(16 (x / X
// - hi)) at the scale X / 16.  An E4M3 value keeps 4 significant bits, the rest of a BF16 value
// fits the other 4.  The block's largest value is above 224 X and lo's step is 2^-13 X: hi + lo is x
// exactly from 2^-6 X on, that is from 1 / 14336 of the largest value (2^-13.8) on, and within 2^-14 X,
// 2^-21.8 of the largest value, below.
//
// A CTA holds one tile of 128 outputs of a group and a range of its inputs, in steps of 128:
//   * warps 24 and 25: one thread each copies codes (pairs of steps: 128 bytes of a row) and x into
//     shared memory as they lie (bulk tensor copies; what is past an end reads as 0);
//   * warps 0-23 bring them into the tensor core's layouts: 16 codes into the first 8 bytes of each
//     16-byte slot (it reads 4-bit operands with 8 bytes of padding behind every 16 values), rows of
//     x into B's columns, scales into scale blocks; then they run the epilogue;
//   * warps 26 and 27: one lane each copies a step's scales into tensor memory and issues its four
//     K = 32 MMAs; each warp has its own sums.
// A cluster of `split` CTAs shares a tile's inputs when there are fewer tiles than
// multiprocessors; each sends its partial sums to the CTA that adds up the row of x, which adds
// them in rank order, so the result does not depend on timing.  Every mbarrier wait is bounded
// (LC_DEV_TIMEOUT).
//
// What bounds it is the chain through these roles, not memory: one row through 7168 x 4096 takes
// 9.1 us in a graph, 8.2 as a call among others (2.4 us of weights at 6.47 TB/s): 2 us to the first full stage, 3.5 us for 14
// steps (scales -> MMAs -> stage free), 1.4 us to join 4 CTAs, the rest is the start of the next
// cluster.  32 rows through 8 groups of 4096 x 1024: 14.9 us, of which widening x (16 conversions per
// 8 values, in every CTA that shares them) took 850 cycles a step when the whole took 15.3; 17 rows of MXFP8 through
// 7168 x 7000: 14.3 us.
// The rows of a prompt read and lay out the weights for every 32 (64 of MXFP8) of them: 2048 rows through
// 7168 x 4096 take 446 us (200), 270 TFLOP/s (600).
// Tried: cp.async in place of the bulk copies (50 cycles of issue each: 12.7 and 18.4 us), one x
// block per thread (1000 cycles a step), two steps per round of the issuing warps (11.0 and 16.7, when
// this took 10.7 and 16.4), BF16 weights by table lookup for the warps' own matrix instruction (9.5 us
// for one row, then 10.7 here, and 18.4: bound by the integer pipe).
#include <cuda.h>

#include <type_traits>

#include "lc_e4m3.cuh"
#include "lc_internal.h"
#include "lc_ptx_dense.cuh"
#include "lc_tma.h"

namespace lc {

namespace {

constexpr int kM = 128;                 // outputs per tile
constexpr int kK = 128;                 // inputs per step
constexpr int kTileA = kM * kK;         // bytes of A in shared memory (padded codes)
constexpr int kSf = 512;                // bytes of a 128-row scale block: 32 rows of 4 words
// 24 warps bring operands into the tensor core's layouts, in groups of 4 that take steps in turn
constexpr int kWarpCopy = 24, kWarpMma = kWarpCopy + 2;
constexpr int kTurns = 2;               // issuing warps, in turn
constexpr int kThreads = 32 * (kWarpMma + kTurns);
constexpr long kSpin = 1L << 20;  // a few seconds

// shared memory for N columns of B: kRawW steps of codes and scale words as they come from memory,
// kRawX steps of x, and kStages steps in the tensor core's layout
template <int N, bool kMx>
struct W4Smem {
  static constexpr int kTok = kMx ? N : N / 2;
  static constexpr int kUnits = kTok * (kMx ? 8 : 16);    // 16-byte units of x per step
  // turns for the codes (128 threads each) and for x (kXT threads each; what is enough for a few rows or
  // for MXFP8 would hold up 16 or 32 rows of BF16)
  static constexpr bool kWide = !kMx && N >= 32;
  static constexpr int kTurnsW = kWide ? 2 : 4, kTurnsX = 4, kXT = kWide ? 128 : 64;
  static_assert(4 * kTurnsW + kXT / 32 * kTurnsX == kWarpCopy, "warps");
  static constexpr int kStages = 4;
  static constexpr int kRawX = N <= 32 ? 8 : 4;
  static constexpr int kRawW = N <= 16 ? 6 : N <= 32 ? 4 : kMx ? 2 : 3;  // of two steps each: a row's 128 bytes
  // Every place always has the same turns, so that no barrier is waited for a round too early
  static_assert(kStages % kTurnsW == 0 && kStages % kTurnsX == 0 && kStages % kTurns == 0, "turns");
  static_assert(2 * kRawW % kTurnsW == 0 && kRawX % kTurnsX == 0, "turns");
  static constexpr int kStage = kTileA + N * kK + 2 * kSf;
  static constexpr int kRawWBytes = kM * kK, kRawXBytes = kUnits * 16;
  static constexpr int kRing = kStages * kStage, kW = kRawW * kRawWBytes, kX = kRawX * kRawXBytes;
  // a CTA's share of the joined rows: (n_tok + split - 1) / split rows of `split` partial sums
  static constexpr int kPart = (kTok + 7) * kM * 4;
  static constexpr int kBytes = kRing + kW + kX + kPart + 1024;
};

__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void st_shared8(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1,%2};\n" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void st_shared4(uint32_t a, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ void st_shared1(uint32_t a, uint32_t x) {
  asm volatile("st.shared.b8 [%0], %1;\n" ::"r"(a), "r"(x) : "memory");
}

// scale block (32 rows x 16 bytes) -> 4 columns of tensor memory, every lane quadrant
__device__ __forceinline__ void tmem_scales(uint32_t taddr, const void* smem) {
  uint64_t d = static_cast<uint64_t>((su32(smem) >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(16 >> 4) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(d));
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// byte of row r, 32-value block b of a scale block
__device__ __forceinline__ int sf_off(int r, int b) { return (r & 31) * 16 + (r >> 5) * 4 + b; }

__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(__half2 v) {
  return __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 e4m3x2_to_f16x2(uint16_t v) { return __half2(__nv_cvt_fp8x2_to_halfraw2(v, __NV_E4M3)); }

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, uint32_t rank, float v) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(r), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }

}  // namespace

// N: columns of B (a multiple of 16: 2 per BF16 row, 1 per MXFP8 row)
template <int N, bool kMx>
__global__ void __launch_bounds__(kThreads, 1)
    k_w4_proj(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, lc_w4_proj_args a, int split, int tiles_g) {
  using L = W4Smem<N, kMx>;
  constexpr int kStages = L::kStages, kTok = L::kTok, kTurnsW = L::kTurnsW, kTurnsX = L::kTurnsX;
  constexpr int kWarpX = 4 * kTurnsW, kXT = L::kXT;  // first warp that widens x
  constexpr int kAcc = N + 16;                    // tensor-memory columns of an issuing warp: sums, scales
  constexpr uint32_t kCols = kTurns * kAcc <= 64 ? 64 : kTurns * kAcc <= 128 ? 128 : kTurns * kAcc <= 256 ? 256 : 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* As = smem;                              // [kStages][kTileA]
  uint8_t* Bs = As + kStages * kTileA;             // [kStages][N * kK]
  uint8_t* SFa = Bs + kStages * N * kK;            // [kStages][kSf]
  uint8_t* SFb = SFa + kStages * kSf;              // [kStages][kSf]
  uint8_t* Wr = SFb + kStages * kSf;               // [kRawW][kRawWBytes], in multiples of 1024 bytes so far
  uint8_t* Xr = Wr + L::kW;                        // [kRawX][kRawXBytes]
  // partial sums of a cluster: the row's place in the share of the CTA that adds it up, rank, output
  float* part = reinterpret_cast<float*>(Xr + L::kX);
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], done;
  __shared__ __align__(8) uint64_t wfull[L::kRawW], wempty[L::kRawW], xfull[L::kRawX], xempty[L::kRawX];

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x) % split;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int g = tile / tiles_g;
  const int c0 = (tile % tiles_g) * kM;                    // first output of the tile within the group
  const int n0 = static_cast<int>(blockIdx.y) * kTok;      // first row of x
  const int n_tok = min(kTok, a.n_q - n0);
  const int n_sub = (a.K + kK - 1) / kK;
  // this rank's steps: whole pairs (a pair of steps is 128 bytes of a row of codes)
  const int n_pair = (n_sub + 1) / 2;
  const int s_begin = 2 * static_cast<int>(static_cast<int64_t>(n_pair) * rank / split);
  const int n_step = min(n_sub, 2 * static_cast<int>(static_cast<int64_t>(n_pair) * (rank + 1) / split)) - s_begin;
  const int rows = min(kM, a.d_g - c0);

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

  if (warp == kWarpMma) tmem_alloc(su32(&s_tmem), kCols);
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(su32(&full[i]), 128 + kXT);
      mbar_init(su32(&empty[i]), 1);
    }
    for (int i = 0; i < L::kRawW; ++i) {
      mbar_init(su32(&wfull[i]), 1);
      mbar_init(su32(&wempty[i]), 256);
    }
    for (int i = 0; i < L::kRawX; ++i) {
      mbar_init(su32(&xfull[i]), 1);
      mbar_init(su32(&xempty[i]), kXT);
    }
    mbar_init(su32(&done), kTurns);
    fence_mbar_init();
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_x);
  }
  // columns of B without a row of x stay zero (scale 2^0) in every stage
  for (int i = tid; i < kStages * N * kK / 16; i += kThreads) reinterpret_cast<uint4*>(Bs)[i] = make_uint4(0, 0, 0, 0);
  for (int i = tid; i < kStages * kSf / 4; i += kThreads) reinterpret_cast<uint32_t*>(SFb)[i] = 0x7f7f7f7fu;
  fence_async_smem();
  fence_before();
  // what was set up so far overlapped the kernel before; its results are there now, and all before it
  // (only then may the next kernel start: it can rely on this one's inputs, too)
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  fence_after();
  const uint32_t tm = s_tmem;
  if (split > 1) cluster_arrive();  // this CTA runs: its peers can write to its shared memory (they wait below)

  const bool words = a.K % 128 == 0;  // a row's four scale bytes of a step are one aligned word
  if (warp == kWarpCopy || warp == kWarpCopy + 1) {
    // ---------------- copies: one thread for the codes, one for x.  Rows of 128 bytes: with 64 (a step at
    // a time) the copies of a step took 650 cycles, whoever made them
    if (lane == 0) {
      const bool codes = warp == kWarpCopy;
      const int n = codes ? (n_step + 1) / 2 : n_step, ring = codes ? L::kRawW : L::kRawX;
      uint64_t *full_b = codes ? wfull : xfull, *empty_b = codes ? wempty : xempty;
      const uint32_t dst = su32(codes ? Wr : Xr), bytes = codes ? L::kRawWBytes : L::kRawXBytes;
      const CUtensorMap* map = codes ? &map_w : &map_x;
      const int row = codes ? g * a.d_g + c0 : n0, step = codes ? kK : kK * (kMx ? 1 : 2);
      int col = codes ? s_begin * (kK / 2) : (g * a.K + s_begin * kK) * (kMx ? 1 : 2);
      int i = 0;
      for (; i < n; ++i, col += step) {
        const int slot = i % ring;
        if (i >= ring && !wait(&empty_b[slot], ((i / ring) - 1) & 1)) break;
        mbar_expect_tx(su32(&full_b[slot]), bytes);
        tma_tile2d(dst + slot * bytes, map, col, row, su32(&full_b[slot]));
      }
      // a role that gave up leaves copies in flight: they land (in bounded time) before the CTA ends
      if (i < n)
        for (int q = max(0, i - ring); q < i; ++q)
          for (long it = 0; it < kSpin && !mbar_test(su32(&full_b[q % ring]), (q / ring) & 1); ++it) {
          }
    }
  } else if (warp < kWarpX) {
    // ---------------- the weights into A's layout (8-byte copies would land there by themselves, but ran
    // at a third of the rate): codes 32 seg .. + 15 and + 16 .. + 31 of a row are the first 8 bytes of
    // slots 2 seg and 2 seg + 1
    // four lanes a row, rows r and r ^ 5 side by side: in the 128-byte swizzles of both layouts their
    // pieces fall into different banks
    const int wt = tid & 127, seg = wt & 3, r0 = (wt & ~31) / 4 + ((lane >> 3) ^ (lane & 4 ? 5 : 0));
    const uint32_t raw = su32(Wr) + sw128_off(r0, (warp >> 2 & 1) * 4 + seg);  // even steps have the first half of each pair
    const uint32_t d0 = su32(As) + sw128_off(r0, 2 * seg), d1 = su32(As) + sw128_off(r0, 2 * seg + 1);
    const uint32_t ds = su32(SFa) + sf_off(wt, 0);
    // the row's scales of a step, a turn ahead
    const uint8_t* sp = a.w_scale + (static_cast<int64_t>(g) * a.d_g + c0 + wt) * (a.K / 32) + s_begin * 4;
    auto scale_word = [&](int i) -> uint32_t {
      if (wt >= rows || i >= n_step) return 0x7f7f7f7fu;
      if (words) return __ldg(reinterpret_cast<const uint32_t*>(sp + i * 4));
      uint32_t w = 0x7f7f7f7fu;
      const int nb = a.K / 32 - (s_begin + i) * 4;  // scale bytes left in the row
      for (int b = 0; b < min(nb, 4); ++b) w ^= (0x7fu ^ __ldg(sp + i * 4 + b)) << (8 * b);
      return w;
    };
    uint32_t sw = scale_word(warp >> 2);
#pragma unroll 1
    for (int i = warp >> 2; i < n_step; i += kTurnsW) {
      const int st = i % kStages, slot = i / 2 % L::kRawW;
      if (!wait(&wfull[slot], (i / 2 / L::kRawW) & 1) || (i >= kStages && !wait(&empty[st], ((i / kStages) - 1) & 1))) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 v = ld_shared16(raw + slot * L::kRawWBytes + j * 4096);
        st_shared8(d0 + st * kTileA + j * 4096, v.x, v.y);
        st_shared8(d1 + st * kTileA + j * 4096, v.z, v.w);
      }
      st_shared4(ds + st * kSf, sw);
      sw = scale_word(i + kTurnsW);
      mbar_arrive(su32(&wempty[slot]));
      fence_async_smem();
      mbar_arrive(su32(&full[st]));
    }
  } else if (warp < kWarpCopy) {
    // ---------------- x into B's columns.  Four lanes share a 32-value block of a BF16 row (8 values each),
    // two a block of MXFP8 codes
    constexpr int kLpr = kMx ? 8 : 16, kXTok = kXT / kLpr;
    const int xt = (tid - 32 * kWarpX) % kXT, xc = xt % kLpr, xb = xc / (kLpr / 4), t0 = xt / kLpr;
    const bool scaler = xc % (kLpr / 4) == 0;
    const uint32_t raw = su32(Xr) + xt * 16;
    constexpr int kU = (kTok + kXTok - 1) / kXTok;
    // MXFP8: a block's scale byte, a turn ahead
    const int64_t ld_s = static_cast<int64_t>(a.G) * (a.K / 32);
    const uint8_t* sp = kMx ? a.x_scale + (n0 + t0) * ld_s + static_cast<int64_t>(g) * (a.K / 32) + s_begin * 4 + xb : nullptr;
    uint8_t sc[kU];
    auto scale_bytes = [&](int i) {
      const bool in = i < n_step && scaler && (s_begin + i) * 4 + xb < a.K / 32;
#pragma unroll
      for (int m = 0; m < kU; ++m)
        sc[m] = in && t0 + kXTok * m < n_tok ? __ldg(sp + i * 4 + m * kXTok * ld_s) : static_cast<uint8_t>(127);
    };
    const int first = (warp - kWarpX) / (kXT / 32);
    if constexpr (kMx) scale_bytes(first);
#pragma unroll 1
    for (int i = first; i < n_step; i += kTurnsX) {
      const int st = i % kStages, slot = i % L::kRawX;
      // the warp leaves together: its lanes meet in shuffles and votes below
      const bool ready = wait(&xfull[slot], (i / L::kRawX) & 1) && (i < kStages || wait(&empty[st], ((i / kStages) - 1) & 1));
      if (!__all_sync(0xffffffffu, ready)) break;
      const uint32_t Bt = su32(Bs) + st * N * kK, sf = su32(SFb) + st * kSf;
      const bool in = (s_begin + i) * 4 + xb < a.K / 32;  // else the next group's values
      // Lays out the rows; a block whose largest value is near BF16's end, or not finite, once more with `end`
      // (what can go wrong there is looked at in that pass alone: in the other it cost 0.2 us of 15)
      auto lay_out = [&](auto pass) -> bool {
        constexpr bool end = pass.value;
        bool again = false;
#pragma unroll
        for (int m = 0; m < kU; ++m) {
          const int t = t0 + kXTok * m;
          if (t - (lane / kLpr) >= n_tok) break;  // the same for every lane
          uint4 v = ld_shared16(raw + slot * L::kRawXBytes + m * (kXT * 16));
          if (!in) v = make_uint4(0, 0, 0, 0);
          if constexpr (kMx) {
            if (t >= n_tok) continue;
            st_shared16(Bt + sw128_off(t, xc), v);
            if (scaler) st_shared1(sf + sf_off(t, xb), sc[m]);
          } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            // the block's largest magnitude as BF16 bits (an infinity's or a NaN's are larger still)
            uint32_t mb = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
            mb = max_u16x2(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
            mb = max_u16x2(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
            mb = max(mb & 0xffffu, mb >> 16);
            again |= mb >= 0x7f78u;  // 248 2^120
            bool inf = false;
            if constexpr (end) {  // the largest finite value
              float amax = 0.f;
              for (int j = 0; j < 4; ++j) {
                amax = fmaxf(amax, fmaxf(finite_abs(__uint_as_float(w[j] << 16)), finite_abs(__uint_as_float(w[j] & 0xffff0000u))));
                inf |= ((w[j] & 0x7f80u) == 0x7f80u) | ((w[j] & 0x7f800000u) == 0x7f800000u);
              }
              amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
              amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
              mb = __float_as_uint(amax) >> 16;
            }
            // from -123, where X / 16 is the least E8M0 value (BF16's subnormals are exact from there), to 120, the
            // exponent of the largest BF16 value
            const int e = mb > 0 ? max(e4m3_scale_exp(__uint_as_float(mb << 16)), -123) : 0;
            const float f = pow2f(-e);
            // 248 X and more would round up to 256 X, which is 2^128 under the largest X: there hi takes 240 X and lo
            // the rest (8 X .. 15 X, exact), so that no term passes FP32's range by itself
            const __half2 most = __float2half2_rn(e > 119 ? 240.f : 448.f);
            uint16_t h8[4], l8[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // x / X in F16: exact, or below 2^-17, where both terms are 0 anyway
              const __half2 y = __floats2half2_rn(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xffff0000u) * f);
              h8[j] = f16x2_to_e4m3x2(end ? __hmin2_nan(__hmax2_nan(y, __hneg2(most)), most) : y);
              l8[j] = f16x2_to_e4m3x2(__hmul2(__hsub2(y, e4m3x2_to_f16x2(h8[j])), __float2half2_rn(16.f)));  // exact before the rounding
            }
            if (t >= n_tok) continue;
            uint32_t h0 = h8[0] | static_cast<uint32_t>(h8[1]) << 16;
            if (inf) h0 |= 0x7fu;  // an infinity has no E4M3 code; like a NaN it makes the outputs NaN
            const uint32_t off = sw128_off(t, xc >> 1) + (xc & 1) * 8;
            st_shared8(Bt + off, h0, h8[2] | static_cast<uint32_t>(h8[3]) << 16);
            st_shared8(Bt + off + kTok * 128, l8[0] | static_cast<uint32_t>(l8[1]) << 16, l8[2] | static_cast<uint32_t>(l8[3]) << 16);
            if (scaler) {
              st_shared1(sf + sf_off(t, xb), e + 127);
              st_shared1(sf + sf_off(kTok + t, xb), e - 4 + 127);
            }
          }
        }
        return again;
      };
      const bool again = lay_out(std::false_type{});
      if constexpr (!kMx) {
        if (__any_sync(0xffffffffu, again)) lay_out(std::true_type{});
      }
      mbar_arrive(su32(&xempty[slot]));
      if constexpr (kMx) scale_bytes(i + kTurnsX);
      fence_async_smem();
      mbar_arrive(su32(&full[st]));
    }
  } else {
    // ---------------- MMAs: E2M1 x E4M3, E8M0 scales, FP32 accumulate.  Each issuing warp has its own sums
    // (one thread issues an instruction about every 55 cycles, seven a step); the warp stays together and
    // one lane issues, which keeps the descriptors in uniform registers
    const int me = warp - kWarpMma;
    const uint32_t acc = tm + me * kAcc;
    const bool one = elect_one();
    const uint32_t idesc0 = (5u << 7) | (0u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
                            (static_cast<uint32_t>(kM >> 4) << 24);
    bool ok = true;
#pragma unroll 1
    for (int i = me; i < n_step; i += kTurns) {
      const int st = i % kStages;
      ok = __all_sync(0xffffffffu, wait(&full[st], (i / kStages) & 1));
      if (!ok) break;
      fence_after();
      const uint32_t sfa = acc + N + 4u * ((i / kTurns) & 1), sfb = acc + N + 8 + 4u * ((i / kTurns) & 1);
      const uint64_t ad = sw128_desc(su32(As + st * kTileA)), bd = sw128_desc(su32(Bs + st * N * kK));
      if (one) {
        tmem_scales(sfa, SFa + st * kSf);
        tmem_scales(sfb, SFb + st * kSf);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
          const uint32_t idesc = idesc0 | (k << 29) | (k << 4);
          asm volatile(
              "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
              "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(acc),
              "l"(ad + k * 2), "l"(bd + k * 2), "r"(idesc), "r"(static_cast<uint32_t>(i > me || k > 0)),
              "r"(sfa | (k << 30)), "r"(sfb | (k << 30)));
        }
        mma_commit(su32(&empty[st]));
      }
    }
    if (one) {
      mma_commit(su32(&done));
      // every MMA complete before shared and tensor memory are used again (finite on the hardware)
      if (!ok)
        for (long it = 0; it < kSpin && !mbar_test(su32(&done), 0); ++it) {
        }
    }
  }
  __syncwarp();

  // ---------------- epilogue: warps 0 .. 23, four take 8 rows of x at a time; lane r of their 128 holds
  // output c0 + r
  const bool ok = __all_sync(0xffffffffu, wait(&done, 0));
  auto store = [&](int t, int r, float v) {
    const int64_t at = static_cast<int64_t>(n0 + t) * a.G * a.d_g + static_cast<int64_t>(g) * a.d_g + c0 + r;
    if (a.out_fmt == LC_FMT_F32) static_cast<float*>(a.y)[at] = v;
    else static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_bits(v);
  };
  if (split > 1) cluster_wait();
  fence_after();
  if (warp < kWarpCopy) {
    const int r = (warp & 3) * 32 + lane;
#pragma unroll 1
    for (int t0 = (warp >> 2) * 8; t0 < n_tok; t0 += 8 * (kWarpCopy / 4)) {
      // an issuing warp that had no step left its sums unwritten
      constexpr int kSum = kMx ? kTurns : 2 * kTurns;
      uint32_t v[kSum][8];
#pragma unroll
      for (int q = 0; q < kSum; ++q)
        tmem_ld8(tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (kMx ? q : q / 2) * kAcc + (kMx ? 0 : (q & 1) * kTok) + t0, v[q]);
      tmem_wait_ld();
      int own = t0 % split, place = t0 / split * split + rank;  // of row t: the CTA that adds it up, the place there
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = t0 + j;
        float y = __uint_as_float(v[0][j]);
#pragma unroll
        for (int q = 1; q < kSum; ++q)
          if ((kMx ? q : q / 2) < n_step) y += __uint_as_float(v[q][j]);
        if (t >= n_tok || !ok) break;
        if (split > 1) {
          st_cluster_f32(su32(part + place * kM + r), own, y);
          if (++own == split) {
            own = 0;
            place += split;
          }
        } else if (r < rows) {
          store(t, r, y);
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kWarpMma) tmem_dealloc(tm, kCols);
  if (split > 1) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();  // every partial sum is in place
    // this CTA's share of the rows of x (t % split == rank), added in the order of ranks
    const int items = (n_tok - rank + split - 1) / split * kM;
    for (int u = tid; u < items; u += kThreads) {
      const int q = u / kM, r = u % kM;
      const float* p = part + q * split * kM + r;
      float y = p[0];
      for (int k = 1; k < split; ++k) y += p[k * kM];
      if (ok && r < rows) store(q * split + rank, r, y);
    }
  }
}

namespace {

template <int N, bool kMx>
cudaError_t launch_w4(const lc_w4_proj_args& a, int split, int tiles_g, cudaStream_t st) {
  constexpr int kTok = kMx ? N : N / 2;
  constexpr size_t smem = W4Smem<N, kMx>::kBytes;
  static_assert(smem <= 227 * 1024 - 512, "shared memory");
  CUtensorMap map_w, map_x;
  if (!encode_bytes()) return cudaErrorNotSupported;
  if (!byte_map(&map_w, a.w, static_cast<int64_t>(a.G) * a.d_g, a.K / 2, kK, kM, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !byte_map(&map_x, a.x, a.n_q, static_cast<int64_t>(a.G) * a.K * (kMx ? 1 : 2), kK * (kMx ? 1 : 2), kTok, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(a.G * tiles_g * split), static_cast<unsigned>((a.n_q + kTok - 1) / kTok));
  return launch_big<k_w4_proj<N, kMx>>(smem, grid, dim3(kThreads), smem, st, split, map_w, map_x, a, split, tiles_g);
}

}  // namespace

cudaError_t launch_w4_proj(const lc_w4_proj_args& a, cudaStream_t st) {
  const int tiles_g = (a.d_g + kM - 1) / kM;
  const int64_t tiles = static_cast<int64_t>(a.G) * tiles_g;
  const int n_sub = (a.K + kK - 1) / kK;
  // CTAs that share a tile's inputs (up to 8, at least 2 steps each): the number whose rounds of CTAs
  // cost least, where a CTA takes as long to start and end as kFixed steps, and kJoin more in a cluster
  constexpr int kFixed = 10, kJoin = 6;
  const int max_tok = a.in_fmt == LC_FMT_MXFP8 ? 64 : 32;  // rows of x per CTA
  const int64_t rows_y = (a.n_q + max_tok - 1) / max_tok;
  int split = 1;
  int64_t best = INT64_MAX;
  for (int s = 1; s <= 8 && (s == 1 || n_sub >= 2 * s); ++s) {
    const int64_t waves = (tiles * rows_y * s + sm_count() - 1) / sm_count();
    const int64_t cost = waves * (kFixed + (s > 1 ? kJoin : 0) + (n_sub + s - 1) / s);
    if (cost < best) {
      best = cost;
      split = s;
    }
  }
  if (a.in_fmt == LC_FMT_MXFP8) {
    if (a.n_q <= 16) return launch_w4<16, true>(a, split, tiles_g, st);
    if (a.n_q <= 32) return launch_w4<32, true>(a, split, tiles_g, st);
    return launch_w4<64, true>(a, split, tiles_g, st);
  }
  if (a.n_q <= 8) return launch_w4<16, false>(a, split, tiles_g, st);
  if (a.n_q <= 16) return launch_w4<32, false>(a, split, tiles_g, st);
  return launch_w4<64, false>(a, split, tiles_g, st);
}

}  // namespace lc
