// w4_proj: y[n, g d_g + c] = sum_k x[n, g K + k] W_g[c, k] for a few rows x, W in MXFP4 (E2M1 codes,
// one E8M0 scale per 32), x in BF16 or MXFP8.
//
// The weights bound it (17/32 byte each, read once); widening them on the CUDA cores would cost
// about as much issue time as their transfer takes.  So they go to the tensor core as they are:
// tcgen05 kind::mxf8f6f4 takes A = 128 outputs x 32 inputs of E2M1 and B = N columns x 32 inputs of
// E4M3 with their E8M0 scales, and accumulates in FP32 in tensor memory.  A BF16 row becomes two
// columns of B: with X the row's scale for a block of 32, hi = e4m3(x / X) and lo = e4m3(16 (x / X
// - hi)) at the scale X / 16.  An E4M3 value keeps 4 significant bits, the rest of a BF16 value
// fits the other 4: hi + lo is x exactly down to 2^-15 of the block's largest value.
//
// A CTA holds one tile of 128 outputs of a group and a range of its inputs, in steps of 128:
//   * warps 0-3 copy the codes (cp.async, 8 bytes = 16 codes into each 16-byte slot of the
//     SWIZZLE_128B layout: the tensor core reads 4-bit operands with 8 bytes of padding behind
//     every 16 values) and the scale words, kAhead steps ahead, and run the epilogue;
//   * warps 4-7 turn x into B's columns and scales;
//   * lane 0 of warp 8 copies a step's scales into tensor memory and issues its four K = 32 MMAs.
// A cluster of `split` CTAs shares a tile's inputs when there are fewer tiles than
// multiprocessors; the partial tiles meet in distributed shared memory and are added in rank
// order, so the result does not depend on timing.  Every mbarrier wait is bounded
// (LC_DEV_TIMEOUT).
#include "lc_e4m3.cuh"
#include "lc_internal.h"
#include "lc_ptx.cuh"

namespace lc {

namespace {

constexpr int kM = 128;                 // outputs per tile
constexpr int kK = 128;                 // inputs per step
constexpr int kTileA = kM * kK;         // bytes of A in shared memory (padded codes)
constexpr int kSf = 512;                // bytes of a 128-row scale block: 32 rows of 4 words
constexpr int kThreads = 288;
constexpr long kSpin = 1L << 20;  // a few seconds
constexpr int kMaxTok = 64;             // rows of x per CTA

// stages of the ring for N columns of B
template <int N>
struct W4Ring {
  static constexpr int kBytes = kTileA + N * kK + 2 * kSf;  // of a stage
  static constexpr int kFit = 212 * 1024 / kBytes;
  static constexpr int kStages = kFit < 10 ? kFit : 10;
};

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(valid ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}

// scale block (32 rows x 16 bytes) -> 4 columns of tensor memory, every lane quadrant
__device__ __forceinline__ void tmem_scales(uint32_t taddr, const void* smem) {
  uint64_t d = static_cast<uint64_t>((su32(smem) >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(16 >> 4) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(d));
}

// byte of row r, 32-value block b of a scale block
__device__ __forceinline__ int sf_off(int r, int b) { return (r & 31) * 16 + (r >> 5) * 4 + b; }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
  uint32_t r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(r) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

}  // namespace

// N: columns of B (a multiple of 16: 2 per BF16 row, 1 per MXFP8 row)
template <int N, bool kMx>
__global__ void __launch_bounds__(kThreads, 1) k_w4_proj(lc_w4_proj_args a, int split, int tiles_g) {
  constexpr int kStages = W4Ring<N>::kStages;
  constexpr int kAhead = kStages - 1;
  constexpr int kTok = kMx ? N : N / 2;
  constexpr uint32_t kCols = N + 16 <= 32 ? 32 : N + 16 <= 64 ? 64 : N + 16 <= 128 ? 128 : 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* As = smem;                              // [kStages][kTileA]
  uint8_t* Bs = As + kStages * kTileA;             // [kStages][N * kK]
  uint8_t* SFa = Bs + kStages * N * kK;            // [kStages][kSf]
  uint8_t* SFb = SFa + kStages * kSf;              // [kStages][kSf]
  float* part = reinterpret_cast<float*>(smem);    // after the last MMA: [kTok][kM]
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], done;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.x) % split;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int g = tile / tiles_g;
  const int c0 = (tile % tiles_g) * kM;                    // first output of the tile within the group
  const int n0 = static_cast<int>(blockIdx.y) * kTok;      // first row of x
  const int n_tok = min(kTok, a.n_q - n0);
  const int n_sub = (a.K + kK - 1) / kK;
  const int s_begin = static_cast<int>(static_cast<int64_t>(n_sub) * rank / split);
  const int n_step = static_cast<int>(static_cast<int64_t>(n_sub) * (rank + 1) / split) - s_begin;
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

  if (warp == 8) tmem_alloc(su32(&s_tmem), kCols);
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(su32(&full[i]), 256);
      mbar_init(su32(&empty[i]), 1);
    }
    mbar_init(su32(&done), 1);
    fence_mbar_init();
  }
  // columns of B without a row of x stay zero (scale 2^0) in every stage
  for (int i = tid; i < kStages * N * kK / 16; i += kThreads) reinterpret_cast<uint4*>(Bs)[i] = make_uint4(0, 0, 0, 0);
  for (int i = tid; i < kStages * kSf / 4; i += kThreads) reinterpret_cast<uint32_t*>(SFb)[i] = 0x7f7f7f7fu;
  fence_async_smem();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = s_tmem;

  if (warp < 4) {
    // ---------------- the weights
    const int64_t row_g = static_cast<int64_t>(g) * a.d_g + c0;
    const int piece = lane & 7;
    const bool words = a.K % 128 == 0;  // a row's four scale bytes of a step are one aligned word
    bool ok = true;
    for (int i = 0; ok && i < n_step + kAhead; ++i) {
      if (i < n_step) {
        const int st = i % kStages;
        if (i >= kStages) ok = wait(&empty[st], ((i / kStages) - 1) & 1);
        if (!ok) break;
        const int k = (s_begin + i) * kK + piece * 16;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = j * 16 + warp * 4 + (lane >> 3);
          const bool v = r < rows && k < a.K;
          const uint8_t* src = a.w + (v ? (row_g + r) * (a.K / 2) + k / 2 : 0);
          cp_async8(su32(As + st * kTileA) + sw128_off(r, piece), src, v);
        }
        uint8_t* sf = SFa + st * kSf + sf_off(tid, 0);
        const int b0 = (s_begin + i) * 4;
        if (words && tid < rows) {
          cp_async4(su32(sf), a.w_scale + (row_g + tid) * (a.K / 32) + b0);
        } else {
          uint32_t w = 0x7f7f7f7fu;
          if (tid < rows) {
            const uint8_t* src = a.w_scale + (row_g + tid) * (a.K / 32) + b0;
            w = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) w |= (b0 + b < a.K / 32 ? static_cast<uint32_t>(__ldg(src + b)) : 0x7fu) << (8 * b);
          }
          *reinterpret_cast<uint32_t*>(sf) = w;
        }
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kAhead) : "memory");
      if (i >= kAhead) {
        fence_async_smem();
        mbar_arrive(su32(&full[(i - kAhead) % kStages]));
      }
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
  } else if (warp < 8) {
    // ---------------- x: B's columns
    const int xt = tid - 128;
    const int64_t ldx = static_cast<int64_t>(a.G) * a.K;
    bool ok = true;
    for (int i = 0; ok && i < n_step; ++i) {
      const int st = i % kStages;
      if (i >= kStages) ok = wait(&empty[st], ((i / kStages) - 1) & 1);
      if (!ok) break;
      uint8_t* Bt = Bs + st * N * kK;
      uint8_t* sf = SFb + st * kSf;
      const int kb = (s_begin + i) * 4;  // first 32-block of the step
      for (int u = xt; u < n_tok * 4; u += 128) {
        const int t = u >> 2, b = u & 3;
        const bool in = kb + b < a.K / 32;
        const int64_t at = (n0 + t) * ldx + static_cast<int64_t>(g) * a.K + (kb + b) * 32;
        if constexpr (kMx) {
          uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
          uint8_t sc = 127;
          if (in) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.x) + at);
            v0 = __ldg(p);
            v1 = __ldg(p + 1);
            sc = __ldg(a.x_scale + at / 32);
          }
          *reinterpret_cast<uint4*>(Bt + sw128_off(t, 2 * b)) = v0;
          *reinterpret_cast<uint4*>(Bt + sw128_off(t, 2 * b + 1)) = v1;
          sf[sf_off(t, b)] = sc;
        } else {
          uint32_t w[16];
          float amax = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + at) + j);
            w[4 * j] = v.x;
            w[4 * j + 1] = v.y;
            w[4 * j + 2] = v.z;
            w[4 * j + 3] = v.w;
          }
          bool inf = false;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
            amax = fmaxf(amax, fmaxf(finite_abs(lo), finite_abs(hi)));
            inf |= !(fabsf(lo) < INFINITY) | !(fabsf(hi) < INFINITY);
          }
          // 16 / X's exponent has to fit E8M0 too, and 2^-e FP32
          const int e = amax > 0.f ? min(max(e4m3_scale_exp(amax), -120), 119) : 0;
          const float f = pow2f(-e);
          uint32_t hi4[8], lo4[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float v[4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              v[2 * q] = __uint_as_float(w[2 * j + q] << 16) * f;
              v[2 * q + 1] = __uint_as_float(w[2 * j + q] & 0xffff0000u) * f;
            }
            hi4[j] = e4m3x4(v[0], v[1], v[2], v[3]);
            const float2 h0 = e4m3x2_to_f32x2(static_cast<uint16_t>(hi4[j] & 0xffffu));
            const float2 h1 = e4m3x2_to_f32x2(static_cast<uint16_t>(hi4[j] >> 16));
            lo4[j] = e4m3x4((v[0] - h0.x) * 16.f, (v[1] - h0.y) * 16.f, (v[2] - h1.x) * 16.f, (v[3] - h1.y) * 16.f);
          }
          // an infinity has no E4M3 code; like a NaN it makes the outputs NaN
          if (inf) hi4[0] |= 0x7fu;
          *reinterpret_cast<uint4*>(Bt + sw128_off(t, 2 * b)) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
          *reinterpret_cast<uint4*>(Bt + sw128_off(t, 2 * b + 1)) = make_uint4(hi4[4], hi4[5], hi4[6], hi4[7]);
          const int t2 = kTok + t;
          *reinterpret_cast<uint4*>(Bt + sw128_off(t2, 2 * b)) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
          *reinterpret_cast<uint4*>(Bt + sw128_off(t2, 2 * b + 1)) = make_uint4(lo4[4], lo4[5], lo4[6], lo4[7]);
          sf[sf_off(t, b)] = static_cast<uint8_t>(e + 127);
          sf[sf_off(t2, b)] = static_cast<uint8_t>(e - 4 + 127);
        }
      }
      fence_async_smem();
      mbar_arrive(su32(&full[st]));
    }
  } else if (lane == 0) {
    // ---------------- MMAs: E2M1 x E4M3, E8M0 scales, FP32 accumulate
    const uint32_t idesc0 = (5u << 7) | (0u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
                            (static_cast<uint32_t>(kM >> 4) << 24);
    bool ok = true;
    for (int i = 0; i < n_step; ++i) {
      const int st = i % kStages;
      ok = wait(&full[st], (i / kStages) & 1);
      if (!ok) break;
      fence_after();
      const uint32_t sfa = tm + N + 4u * (i & 1), sfb = tm + N + 8 + 4u * (i & 1);
      tmem_scales(sfa, SFa + st * kSf);
      tmem_scales(sfb, SFb + st * kSf);
      const uint32_t ab = su32(As + st * kTileA), bb = su32(Bs + st * N * kK);
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        const uint32_t idesc = idesc0 | (k << 29) | (k << 4);
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(tm),
            "l"(sw128_desc(ab + k * 32)), "l"(sw128_desc(bb + k * 32)), "r"(idesc), "r"(static_cast<uint32_t>(i > 0 || k > 0)),
            "r"(sfa | (k << 30)), "r"(sfb | (k << 30)));
      }
      mma_commit(su32(&empty[st]));
    }
    mma_commit(su32(&done));
    // every MMA complete before shared and tensor memory are used again (finite on the hardware)
    if (!ok)
      for (long it = 0; it < kSpin && !mbar_test(su32(&done), 0); ++it) {
      }
  }
  __syncwarp();

  // ---------------- epilogue: thread r of warps 0-3 holds output c0 + r for every column
  const bool ok = warp < 4 ? __all_sync(0xffffffffu, wait(&done, 0)) : true;
  const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
  auto store = [&](int t, int r, float v) {
    const int64_t at = static_cast<int64_t>(n0 + t) * a.G * a.d_g + static_cast<int64_t>(g) * a.d_g + c0 + r;
    if (a.out_fmt == LC_FMT_F32) static_cast<float*>(a.y)[at] = v;
    else static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_bits(v);
  };
  if (warp < 4) {
    fence_after();
#pragma unroll
    for (int t0 = 0; t0 < kTok; t0 += 8) {
      uint32_t v[8], w[8];
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                   : "r"(tm + lane_off + t0));
      if constexpr (!kMx)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "r"(tm + lane_off + kTok + t0));
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = t0 + j;
        float y = __uint_as_float(v[j]);
        if constexpr (!kMx) y += __uint_as_float(w[j]);
        if (split > 1) part[t * kM + tid] = y;
        else if (ok && t < n_tok && tid < rows) store(t, tid, y);
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tm, kCols);
  if (split > 1) {
    cluster_sync();  // every partial tile is written
    // this CTA's share of the rows of x, summed over the ranks in order
    for (int u = tid; u < n_tok * kM; u += kThreads) {
      const int t = u / kM, r = u % kM;
      if (t % split != rank || r >= rows) continue;
      float y = 0.f;
      for (int p = 0; p < split; ++p) y += ld_cluster_f32(su32(part + u), p);
      store(t, r, y);
    }
    cluster_sync();  // and read by its peers before it goes
  }
}

namespace {

template <int N, bool kMx>
cudaError_t launch_w4(const lc_w4_proj_args& a, int split, int tiles_g, cudaStream_t st) {
  constexpr int kTok = kMx ? N : N / 2;
  constexpr size_t smem = static_cast<size_t>(W4Ring<N>::kStages) * W4Ring<N>::kBytes + 1024;
  static_assert(smem <= 227 * 1024 - 512 && static_cast<size_t>(kTok) * kM * 4 <= smem, "shared memory");
  const dim3 grid(static_cast<unsigned>(a.G * tiles_g * split), static_cast<unsigned>((a.n_q + kTok - 1) / kTok));
  const cudaError_t e = cudaFuncSetAttribute(k_w4_proj<N, kMx>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const cudaError_t r = launch_ex(k_w4_proj<N, kMx>, grid, dim3(kThreads), smem, st, false, split, a, split, tiles_g);
  return r != cudaSuccess ? r : cudaGetLastError();
}

}  // namespace

cudaError_t launch_w4_proj(const lc_w4_proj_args& a, cudaStream_t st) {
  const int tiles_g = (a.d_g + kM - 1) / kM;
  const int64_t tiles = static_cast<int64_t>(a.G) * tiles_g;
  const int n_sub = (a.K + kK - 1) / kK;
  // CTAs that share a tile's inputs: the power of two (up to 8, at least 2 steps each) that leaves
  // the fewest rounds of whole tiles on the multiprocessors
  int split = 1;
  double best = 1e30;
  for (int s = 1; s <= 8 && (s == 1 || n_sub >= 2 * s); s *= 2) {
    const double cost = static_cast<double>((tiles * s + sm_count() - 1) / sm_count()) / s + 0.01 * s;
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
  if (a.n_q <= 32) return launch_w4<64, false>(a, split, tiles_g, st);
  return launch_w4<128, false>(a, split, tiles_g, st);
}

}  // namespace lc
