// silu.cuh -- g / (1 + e^-g) * u of one value over all of binary32, shared by the gate kernels
// and the gated product.
#pragma once

#include <cuda_runtime.h>

namespace nvfp4 {

// 2^k, k in [-149, 127]
__device__ __forceinline__ float exp2_float(int k) {
  return __int_as_float(k >= -126 ? (k + 127) << 23 : 1 << (k + 149));
}

// With h = e^(-|g| / 2): g / (1 + h^2) u for g >= 0, (g h) / (1 + h^2) (u h) below, where e^g alone may have
// no binary32 that a large u would bring back.  IEEE operations; infinities and NaN follow the formula.
__device__ __forceinline__ float silu_times(float g, float u) {
  const float h = expf(-0.5f * fabsf(g)), d = __fmaf_rn(h, h, 1.0f);
  const bool below = g < 0.0f;
  return __fmul_rn(__fdiv_rn(below ? __fmul_rn(g, h) : g, d), below ? __fmul_rn(u, h) : u);
}

}  // namespace nvfp4
