// Inline-PTX wrappers that the dense layer's kernels use besides those of lc_ptx.cuh: 3-D bulk tensor
// copies, an elected lane, pairs of FP32 values.  A header of its own: what is measured of the other kernels
// is kept with their sources' hashes, lc_ptx.cuh's among them.
#pragma once

#include "lc_ptx.cuh"

namespace lc {

// 3-D tiled bulk tensor copy global -> shared, completing on an mbarrier (no multicast)
__device__ __forceinline__ void tma_tile3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// true in one lane of the (converged) warp; a branch on it leaves the other registers warp-uniform
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// the larger of each pair of 16-bit numbers
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// pairs of FP32 values (one instruction for two products or sums)
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1,%2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void fma2_regs(uint32_t& x, uint32_t& y, uint64_t m, uint64_t c) {
  asm("{\n.reg .b64 t;\nmov.b64 t, {%0,%1};\nfma.rn.f32x2 t, t, %2, %3;\nmov.b64 {%0,%1}, t;\n}\n" : "+r"(x), "+r"(y) : "l"(m), "l"(c));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t a) {
  float2 v;
  asm("mov.b64 {%0,%1}, %2;\n" : "=f"(v.x), "=f"(v.y) : "l"(a));
  return v;
}
__device__ __forceinline__ float sum2(uint64_t a) {
  float x, y;
  asm("mov.b64 {%0,%1}, %2;\n" : "=f"(x), "=f"(y) : "l"(a));
  return x + y;
}

}  // namespace lc
