// silu.cuh -- g / (1 + e^-g) * u of one value over all of binary32, shared by the gate kernels
// and the gated product.
#pragma once

#include <cuda_runtime.h>

namespace nvfp4 {

// 2^k, k in [-149, 127]
__device__ __forceinline__ float exp2_float(int k) {
  return __int_as_float(k >= -126 ? (k + 127) << 23 : 1 << (k + 149));
}

// By IEEE operations; infinities and NaN follow the formula.  Below -80, where 1 + e^-g nears
// binary32's end and 1 + e^g is 1, it is g e^g u with e^g = 2^n e^f, n = RN(g log2 e) and f = g - n ln 2
// by two words of ln 2 (Cody and Waite's reduction): the power of two goes half to u and half to
// the product, so that a large u still meets a g whose e^g alone is too small for binary32.
__device__ __forceinline__ float silu_times(float g, float u) {
  if (!(g < -80.0f)) return __fmul_rn(__fdiv_rn(g, __fadd_rn(1.0f, expf(-g))), u);
  const float n = fmaxf(rintf(g * 1.44269502f), -290.0f);  // 2^-290: 0, whatever u is
  const float f = __fmaf_rn(n, 1.90465421e-9f, __fmaf_rn(n, -0.693147182f, g));
  const int k = static_cast<int>(n) / 2;
  return __fmul_rn(__fmul_rn(__fmul_rn(g, expf(f)), __fmul_rn(u, exp2_float(k))),
                   exp2_float(static_cast<int>(n) - k));
}

// The same without a branch and in a third of the code, for kernels that hold many copies beside much
// else (the gated product; in the gate kernels, which are short, it costs registers: 8192 x 21504 to
// MXFP8 139 us instead of 136).  With h = e^(-|g| / 2): g / (1 + h^2) u for g >= 0, (g h) / (1 + h^2) (u h)
// below; off by 2^-21 at most.
__device__ __forceinline__ float silu_times_short(float g, float u) {
  const float h = expf(-0.5f * fabsf(g)), d = __fmaf_rn(h, h, 1.0f);
  const bool below = g < 0.0f;
  return __fmul_rn(__fdiv_rn(below ? __fmul_rn(g, h) : g, d), below ? __fmul_rn(u, h) : u);
}

}  // namespace nvfp4
