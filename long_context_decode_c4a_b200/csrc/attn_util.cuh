// attn_util.cuh -- small device helpers shared by the attention kernels.
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

}  // namespace csa
