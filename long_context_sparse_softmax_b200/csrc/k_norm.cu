// add_rms_norm: r = x + res; res_out = r; y = r / sqrt(mean(r^2) + eps) * w, y in FP32, BF16 or
// MXFP8 (E4M3 codes + one E8M0 scale per 32 values: the operand of w4_proj).
//
// HBM bounds it: 7 bytes a value for BF16 streams and an MXFP8 output, each input read once and
// each output written once.  What it takes to keep HBM busy is enough copies in flight while rows
// are worked on (a row per CTA, loaded, summed and stored in turn, reached half the bandwidth):
// CTAs stay for many tiles of rows, one warp copies the next tiles into a ring in shared memory
// (one bulk copy each for x and res: rows are contiguous), 8 warps take a tile into registers,
// give its place free, and compute.  A thread's columns, and so its weights, stay the same.
// 16384 rows of 7168, BF16 with residual, MXFP8 out: 131 us in a graph of such calls, 6.3 TB/s (97 % of the
// measured copy rate), 148 us as a call among others (86 %); before the ring 232 us.  A decode batch of 32 rows
// takes 3.8 us in a graph, 5.0 as a call: a launch and two memory latencies.
// Sums and products go in pairs (f32x2); a block's scale comes from its largest magnitude, looked
// at again only where that is not finite.
//
// The sum is a fixed tree in FP32 (thread, warp, warps in order): the same bits every call.  r w
// is rounded once (not at all for most BF16 values), 1 / sqrt to nearest: an 8-bit code next to a
// tie seldom falls the wrong way.
// An MXFP8 block is 4 neighbouring lanes' values (two shuffles for its maximum).
#include "lc_e4m3.cuh"
#include "lc_internal.h"
#include "lc_ptx_dense.cuh"

namespace lc {

namespace {

// 8 values as 4 pairs
struct Pairs {
  uint64_t p[4];
};

__device__ __forceinline__ Pairs widen_pairs(uint4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Pairs r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r.p[j] = pack2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
  return r;
}
// 8 values of a row in shared memory
template <bool kF32>
__device__ __forceinline__ Pairs load_pairs(const uint8_t* row, int d) {
  if constexpr (kF32) {
    const ulonglong2* q = reinterpret_cast<const ulonglong2*>(row + d * 4);
    const ulonglong2 a = q[0], b = q[1];
    return Pairs{{a.x, a.y, b.x, b.y}};
  } else {
    return widen_pairs(*reinterpret_cast<const uint4*>(row + d * 2));
  }
}
__device__ __forceinline__ uint32_t bf16x2(uint64_t p) {
  const float2 v = unpack2(p);
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kF32>
__device__ __forceinline__ void store_pairs(void* row, int64_t d, const Pairs& v) {
  if constexpr (kF32) {
    ulonglong2* q = reinterpret_cast<ulonglong2*>(static_cast<float*>(row) + d);
    q[0] = make_ulonglong2(v.p[0], v.p[1]);
    q[1] = make_ulonglong2(v.p[2], v.p[3]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + d) = make_uint4(bf16x2(v.p[0]), bf16x2(v.p[1]), bf16x2(v.p[2]), bf16x2(v.p[3]));
  }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

constexpr int kWarps = 8;                   // that compute; one more copies
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxStages = 4;
constexpr long kSpin = 1L << 20;            // a few seconds

// Rows are spread over the computing warps: wpr (a power of two) warps a row, so a tile is
// kWarps / wpr rows; kV groups of 8 values a thread.
struct NormGeom {
  int wpr_log, stages, n_tiles;
};

}  // namespace

// Group i of thread t (of the row's 32 wpr): values 8 (t + 32 wpr i) ..
template <bool kF32, int kV, int kOut>
__global__ void __launch_bounds__(kThreads, kV <= 4 ? 3 : 1) k_add_rms_norm(lc_add_rms_norm_args a, NormGeom geo) {
  extern __shared__ __align__(128) uint8_t smem_raw[];  // weights, [stages][x | res][tile]
  __shared__ float s_part[2][kWarps];
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], wfull;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wpr = 1 << geo.wpr_log, tile_rows = kWarps >> geo.wpr_log;
  const uint32_t esz = kF32 ? 4 : 2, row_bytes = a.d * esz, tile_bytes = row_bytes * tile_rows;
  const uint32_t stage_bytes = tile_bytes * (a.res ? 2 : 1);
  const uint32_t w_bytes = a.w ? a.d * (a.w_fmt == LC_FMT_F32 ? 4 : 2) : 0;
  uint8_t* smem = smem_raw + w_bytes;
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
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < geo.stages; ++i) {
      mbar_init(su32(&full[i]), 1);
      mbar_init(su32(&empty[i]), kWarps);
    }
    mbar_init(su32(&wfull), 1);
    fence_mbar_init();
  }
  // what was set up so far overlapped the kernel before; its results are there now, and all before it
  // (only then may the next kernel start: it can rely on this one's inputs, too)
  pdl_wait();
  pdl_trigger();
  __syncthreads();

  if (warp == kWarps) {
    // ---------------- copies
    if (lane != 0) return;
    if (a.w) {
      mbar_expect_tx(su32(&wfull), w_bytes);
      bulk_load(su32(smem_raw), a.w, w_bytes, su32(&wfull));
    }
    int st = 0, round = 0;
    for (int tile = blockIdx.x; tile < geo.n_tiles; tile += gridDim.x) {
      if (round > 0 && !wait(&empty[st], (round - 1) & 1)) break;
      const int64_t row0 = static_cast<int64_t>(tile) * tile_rows;
      const uint32_t bytes = static_cast<uint32_t>(min(static_cast<int64_t>(tile_rows), a.n_rows - row0)) * row_bytes;
      const uint32_t bar = su32(&full[st]), dst = su32(smem) + st * stage_bytes;
      mbar_expect_tx(bar, a.res ? 2 * bytes : bytes);
      bulk_load(dst, static_cast<const char*>(a.x) + row0 * row_bytes, bytes, bar);
      if (a.res) bulk_load(dst + tile_bytes, static_cast<const char*>(a.res) + row0 * row_bytes, bytes, bar);
      if (++st == geo.stages) {
        st = 0;
        ++round;
      }
    }
    // every copy has landed before the CTA can end: the computing warps waited for each, or gave up (then
    // the copies in flight end by themselves, from valid memory)
    const int n = round * geo.stages + st;
    for (int i = n > geo.stages ? n - geo.stages : 0; i < n; ++i)
      for (long it = 0; it < kSpin && !mbar_test(su32(&full[i % geo.stages]), (i / geo.stages) & 1); ++it) {
      }
    return;
  }

  const int rw = warp & (wpr - 1);            // warp within the row
  const int r_in = warp >> geo.wpr_log;       // row within the tile
  const int n8 = a.d / 8, t = rw * 32 + lane, step = 32 * wpr;
  const bool ok = !a.w || wait(&wfull, 0);
  int st = 0, round = 0, par = 0;
  for (int tile = blockIdx.x; tile < geo.n_tiles; tile += gridDim.x) {
    const int64_t row = static_cast<int64_t>(tile) * tile_rows + r_in;
    const int64_t at = row * a.d;
    bool live = row < a.n_rows;    // uniform over a row's warps
    if (!__all_sync(0xffffffffu, ok && wait(&full[st], round & 1))) live = false;
    Pairs r[kV];
    uint64_t ss2 = 0;
    const uint8_t* src = smem + st * stage_bytes + r_in * row_bytes;
    if (live) {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int c = t + step * i;
        if (c < n8) r[i] = load_pairs<kF32>(src, 8 * c);
      }
      if (a.res) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int c = t + step * i;
          if (c >= n8) continue;
          const Pairs s = load_pairs<kF32>(src + tile_bytes, 8 * c);
#pragma unroll
          for (int j = 0; j < 4; ++j) r[i].p[j] = add2(r[i].p[j], s.p[j]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(su32(&empty[st]));
    if (++st == geo.stages) {
      st = 0;
      ++round;
    }
    if (live) {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int c = t + step * i;
        if (c >= n8) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) ss2 = fma2(r[i].p[j], r[i].p[j], ss2);
        if (a.res_out) store_pairs<kF32>(a.res_out, at + 8 * c, r[i]);
      }
    }
    float ss = warp_sum(sum2(ss2));
    if (wpr > 1) {
      // the exchange's place alternates: a warp writes the next row's part while others read this one's
      if (lane == 0) s_part[par][warp] = ss;
      named_bar(1 + r_in, step);
      ss = 0.f;
      for (int q = 0; q < wpr; ++q) ss += s_part[par][(r_in << geo.wpr_log) + q];
      par ^= 1;
    }
    if (!live) continue;
    // 1 / sqrt(v): one Newton step in FP64 on the FP32 approximation, rounded once
    const double v = static_cast<double>(ss) / a.d + static_cast<double>(a.eps);
    const float seed = rsqrtf(static_cast<float>(v));
    const double y0 = seed;
    // no finite root, or a NaN: the seed says it
    const float rstd = seed > 0.f && seed < INFINITY ? static_cast<float>(y0 + 0.5 * y0 * (1.0 - v * y0 * y0)) : seed;
    const uint64_t rstd2 = pack2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = t + step * i;
      if (c >= n8) continue;
      if (a.w) {
        const Pairs w = a.w_fmt == LC_FMT_F32 ? load_pairs<true>(smem_raw, 8 * c) : load_pairs<false>(smem_raw, 8 * c);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i].p[j] = mul2(r[i].p[j], w.p[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i].p[j] = mul2(r[i].p[j], rstd2);
    }
    if constexpr (kOut == LC_FMT_MXFP8) {
      // d is a multiple of 32, so the 4 lanes of a block agree on c < n8
      float amax[kV];
      auto block_max = [&](auto mag) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          amax[i] = 0.f;
          if (t + step * i >= n8) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 q = unpack2(r[i].p[j]);
            amax[i] = fmaxf(amax[i], fmaxf(mag(q.x), mag(q.y)));
          }
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 1));
#pragma unroll
        for (int i = 0; i < kV; ++i) amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 2));
      };
      block_max([](float q) { return fabsf(q); });  // passes over NaN
      bool inf = false;
#pragma unroll
      for (int i = 0; i < kV; ++i) inf |= amax[i] == INFINITY;
      if (__any_sync(0xffffffffu, inf)) block_max([](float q) { return finite_abs(q); });
      uint8_t* codes = static_cast<uint8_t*>(a.y) + at;
      uint8_t* scales = a.y_scale + row * (a.d / 32);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int c = t + step * i;
        if (c >= n8) continue;
        const int e = amax[i] > 0.f ? min(max(e4m3_scale_exp(amax[i]), -127), 127) : 0;
        const float f = e < 127 ? pow2f(-e) : __uint_as_float(0x00400000u);  // 2^-127 is subnormal, and exact too
        float q[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 z = unpack2(mul2(r[i].p[j], pack2(f, f)));
          q[2 * j] = z.x;
          q[2 * j + 1] = z.y;
        }
        *reinterpret_cast<uint2*>(codes + 8 * c) = make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
        if ((lane & 3) == 0) scales[c / 4] = static_cast<uint8_t>(e + 127);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (t + step * i < n8) store_pairs<kOut == LC_FMT_F32>(a.y, at + 8 * (t + step * i), r[i]);
    }
  }
}

namespace {

constexpr size_t kRoom = 216 * 1024;  // dynamic shared memory of a multiprocessor that the CTAs share

template <auto kKernel>
cudaError_t launch_one(const lc_add_rms_norm_args& a, const NormGeom& geo, unsigned grid, size_t smem, cudaStream_t st) {
  if (smem > 46 * 1024) return launch_big<kKernel>(kRoom, dim3(grid), dim3(kThreads), smem, st, 1, a, geo);
  return launch_ex(kKernel, dim3(grid), dim3(kThreads), smem, st, true, 1, a, geo);  // 48 KB with the static part need no asking
}

template <bool kF32, int kV>
cudaError_t launch_norm(const lc_add_rms_norm_args& a, const NormGeom& geo, unsigned grid, size_t smem, cudaStream_t st) {
  if (a.out_fmt == LC_FMT_F32) return launch_one<k_add_rms_norm<kF32, kV, LC_FMT_F32>>(a, geo, grid, smem, st);
  if (a.out_fmt == LC_FMT_BF16) return launch_one<k_add_rms_norm<kF32, kV, LC_FMT_BF16>>(a, geo, grid, smem, st);
  return launch_one<k_add_rms_norm<kF32, kV, LC_FMT_MXFP8>>(a, geo, grid, smem, st);
}

template <bool kF32>
cudaError_t launch_norm_v(int v, const lc_add_rms_norm_args& a, const NormGeom& geo, unsigned grid, size_t smem, cudaStream_t st) {
  if (v <= 1) return launch_norm<kF32, 1>(a, geo, grid, smem, st);
  if (v <= 2) return launch_norm<kF32, 2>(a, geo, grid, smem, st);
  if (v <= 4) return launch_norm<kF32, 4>(a, geo, grid, smem, st);
  return launch_norm<kF32, 8>(a, geo, grid, smem, st);
}

}  // namespace

cudaError_t launch_add_rms_norm(const lc_add_rms_norm_args& a, cudaStream_t st) {
  // the fewest warps a row that leave at most 4 groups a thread (8 for the widest rows) and a tile of
  // at most 16 KB
  const int n8 = a.d / 8;  // <= 2048
  const size_t row = static_cast<size_t>(a.d) * (a.in_fmt == LC_FMT_F32 ? 4 : 2);
  NormGeom geo;
  geo.wpr_log = 0;
  while (geo.wpr_log < 3 && (n8 > (128 << geo.wpr_log) || row * (kWarps >> geo.wpr_log) > 16 * 1024)) ++geo.wpr_log;
  const int step = 32 << geo.wpr_log, v = (n8 + step - 1) / step;
  const int tile_rows = kWarps >> geo.wpr_log;
  geo.n_tiles = static_cast<int>((a.n_rows + tile_rows - 1) / tile_rows);
  // as many CTAs per multiprocessor as keep two stages each, then as many stages as fit
  const size_t stage = row * tile_rows * (a.res ? 2 : 1);
  const size_t w = a.w ? static_cast<size_t>(a.d) * (a.w_fmt == LC_FMT_F32 ? 4 : 2) : 0;
  size_t per_sm = 3;
  while (per_sm > 1 && per_sm * (w + 2 * stage) > kRoom) --per_sm;
  const size_t fit = (kRoom / per_sm - w) / stage;
  const int64_t most = static_cast<int64_t>(per_sm) * sm_count();
  const unsigned grid = static_cast<unsigned>(geo.n_tiles < most ? geo.n_tiles : most);
  const size_t tiles = (geo.n_tiles + grid - 1) / grid;  // of a CTA
  geo.stages = static_cast<int>(min(min(fit, tiles), static_cast<size_t>(kMaxStages)));
  const size_t smem = w + stage * geo.stages;
  return a.in_fmt == LC_FMT_F32 ? launch_norm_v<true>(v, a, geo, grid, smem, st) : launch_norm_v<false>(v, a, geo, grid, smem, st);
}

}  // namespace lc
