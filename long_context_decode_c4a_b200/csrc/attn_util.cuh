// attn_util.cuh -- small device helpers shared by the attention kernels and the caches in pages.
#pragma once

#include <cstdint>

namespace csa {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// 2^x by the MUFU.EX2 unit (ex2.approx: about 2 ulp, 2^-inf = 0); its error is far below the
// precision to which the attention kernels keep P.
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger magnitude of two bf16 pairs, the sign undefined; NaN wins.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace csa
