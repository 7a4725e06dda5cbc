// add_rms_norm: r = x + res; res_out = r; y = r / sqrt(mean(r^2) + eps) * w, y in FP32, BF16 or
// MXFP8 (E4M3 codes + one E8M0 scale per 32 values: the operand of w4_proj).
//
// One pass: a row lives in the registers of its threads (kV groups of 8 values each), the sum
// of squares is reduced over the row's warps (shuffles, then one shared-memory exchange) and y
// follows from the registers, so each input is read once and each output written once.  HBM
// bounds it: 7 bytes a value for BF16 streams and an MXFP8 output.
//
// The sum is a fixed tree in FP32 (thread, warp, warps in order): the same bits every call.
// An MXFP8 block is 4 neighbouring lanes' values (two shuffles for its maximum).
#include "lc_e4m3.cuh"
#include "lc_internal.h"

namespace lc {

// kV groups of 8 values per thread; a row takes wpr warps of the CTA, blockDim.x / 32 / wpr rows
// per CTA.  Group i of thread t (of the row's 32 wpr): values 8 (t + 32 wpr i) ..
template <bool kF32, int kV, int kOut>
__global__ void __launch_bounds__(1024 / (kV >= 4 ? 2 : 1)) k_add_rms_norm(lc_add_rms_norm_args a, int wpr) {
  __shared__ float s_part[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rw = warp % wpr;           // warp within the row
  const int r_in = warp / wpr;         // row within the CTA
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32 / wpr) + r_in;
  const bool live = row < a.n_rows;    // uniform over a warp
  const int n8 = a.d / 8, t = rw * 32 + lane, step = 32 * wpr;
  const int64_t at = row * a.d;
  const size_t esz = kF32 ? 4 : 2;
  Vec8 r[kV];
  float ss = 0.f;
  if (live) {
    const char* xr = static_cast<const char*>(a.x) + at * esz;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = t + step * i;
      if (c < n8) r[i] = load8_stream<kF32>(xr, 8 * c);
    }
    if (a.res) {
      const char* rr = static_cast<const char*>(a.res) + at * esz;
      Vec8 s[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int c = t + step * i;
        if (c < n8) s[i] = load8_stream<kF32>(rr, 8 * c);
      }
#pragma unroll
      for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i].v[j] += s[i].v[j];
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = t + step * i;
      if (c >= n8) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(r[i].v[j], r[i].v[j], ss);
      if (a.res_out) {
        const lc_rows o = {a.in_fmt, 0, a.res_out, nullptr};
        store8(o, row, a.d, 0, 8 * c, r[i]);
      }
    }
  }
  ss = warp_sum(ss);
  if (wpr > 1) {
    if (lane == 0) s_part[warp] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < wpr; ++w) ss += s_part[r_in * wpr + w];
  }
  if (!live) return;
  const float rstd = 1.f / sqrtf(ss / static_cast<float>(a.d) + a.eps);
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = t + step * i;
    const bool on = c < n8;  // MXFP8: d is a multiple of 32, so the 4 lanes of a block agree
    Vec8 y;
    if (on) {
      Vec8 w;
      if (a.w) w = a.w_fmt == LC_FMT_F32 ? load8<true>(a.w, 8 * c) : load8<false>(a.w, 8 * c);
#pragma unroll
      for (int j = 0; j < 8; ++j) y.v[j] = r[i].v[j] * rstd * (a.w ? w.v[j] : 1.f);
    }
    if constexpr (kOut == LC_FMT_MXFP8) {
      float amax = 0.f;
      if (on) {
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(y.v[j]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      if (!on) continue;
      const int e = amax > 0.f ? min(max(e4m3_scale_exp(amax), -127), 127) : 0;
      // 2^-e in two exact factors: its exponent alone can leave FP32's range
      const int e1 = e / 2;
      const float f1 = pow2f(-e1), f2 = pow2f(-(e - e1));
#pragma unroll
      for (int j = 0; j < 8; ++j) y.v[j] = y.v[j] * f1 * f2;
      reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + at)[c] =
          make_uint2(e4m3x4(y.v[0], y.v[1], y.v[2], y.v[3]), e4m3x4(y.v[4], y.v[5], y.v[6], y.v[7]));
      if ((lane & 3) == 0) a.y_scale[row * (a.d / 32) + c / 4] = static_cast<uint8_t>(e + 127);
    } else if (on) {
      const lc_rows o = {kOut, 0, a.y, nullptr};
      store8(o, row, a.d, 0, 8 * c, y);
    }
  }
}

namespace {

template <bool kF32, int kV>
void launch_norm(const lc_add_rms_norm_args& a, unsigned grid, int threads, int wpr, cudaStream_t st) {
  if (a.out_fmt == LC_FMT_F32) k_add_rms_norm<kF32, kV, LC_FMT_F32><<<grid, threads, 0, st>>>(a, wpr);
  else if (a.out_fmt == LC_FMT_BF16) k_add_rms_norm<kF32, kV, LC_FMT_BF16><<<grid, threads, 0, st>>>(a, wpr);
  else k_add_rms_norm<kF32, kV, LC_FMT_MXFP8><<<grid, threads, 0, st>>>(a, wpr);
}

}  // namespace

cudaError_t launch_add_rms_norm(const lc_add_rms_norm_args& a, cudaStream_t st) {
  const int n8 = a.d / 8;  // <= 2048
  const int v = n8 <= 1024 ? 2 : 4;
  const int wpr = (n8 + 32 * v - 1) / (32 * v);  // <= 16 warps
  const int rpc = wpr >= 4 ? 1 : 4 / wpr;        // rows per CTA: 4 warps or one row
  const int threads = 32 * wpr * rpc;
  const unsigned grid = static_cast<unsigned>((a.n_rows + rpc - 1) / rpc);
  if (a.in_fmt == LC_FMT_F32) {
    if (v == 2) launch_norm<true, 2>(a, grid, threads, wpr, st);
    else launch_norm<true, 4>(a, grid, threads, wpr, st);
  } else {
    if (v == 2) launch_norm<false, 2>(a, grid, threads, wpr, st);
    else launch_norm<false, 4>(a, grid, threads, wpr, st);
  }
  return cudaGetLastError();
}

}  // namespace lc
