// row_ops.cu -- the operators around a layer's products, with the quantizer fused in:
//   rms_norm: h = BF16(x + residual) (kept as the new residual stream),
//             v = h (w + offset) r, r = 1/sqrt(mean(h^2) + eps), rounded once where w + offset has
//             16 bits or fewer;
//   silu_mul: v = g / (1 + e^-g) * u;
// and v leaves as BF16, MXFP8, MXFP4 or NVFP4.  The block scales and codes are taken
// from v in binary32, not from a BF16 copy of it, so a block format rounds once.
//
// Formats (per block of the row, all binary32 round-to-nearest-even):
//   MXFP8 / MXFP4 (OCP Microscaling Formats v1.0): 32 values, shared exponent
//     floor(log2 amax) - 8 (E4M3 elements) or - 2 (E2M1), clamped to [-127, 127], -127 for
//     an all-zero block; scale byte 255 (NaN) for a block that holds a NaN;
//   NVFP4: the absmax rule of the quantizer: s_b = E4M3(amax_b / (6 s_g)), codes
//     E2M1(v * RN(1 / (s_b s_g))), s_g given or amax / 2688 over the whole output
//     (1 for an all-zero one).  A block that holds a NaN has a NaN scale.
//
// One thread owns 16 consecutive values (a 32-byte load): an NVFP4 block, or half
// an MX block (the pair of lanes shares its maximum with one shuffle).
#include <cuda_runtime.h>

#include "../../include/nvfp4.h"
#include "layer_ops.h"
#include "ptx.cuh"
#include "quant_block.cuh"
#include "silu.cuh"

namespace nvfp4 {

namespace {

constexpr int kUnit = 16;       // values per thread step
constexpr int kCluster = 8;     // CTAs that share one amax through distributed shared memory
// Values of a gate that one cluster handles, amax and all, instead of a memset and two
// launches (8.2 us): 4.1 us for 14336 or 28672, 8.4 us for 114688.
constexpr int64_t kClusterMax = 128 * 1024;
constexpr int64_t kMaxFlat = int64_t{1} << 34;  // values of a gate handled as one row (its units fit an int)
// Threads per row and units per thread of norm_kernel: U = 1 up to 1024 threads, U = 2,
// 4, 8 up to 512 (64 or 128 registers each); the longest row is 8 x 512 units.
constexpr int norm_threads(int U) { return U == 1 ? 1024 : 512; }
constexpr int64_t kNormMaxCols = 8 * 512 * kUnit;

// The phases of an operator whose NVFP4 tensor scale is computed from its own output.
enum Phase {
  kOnePass,  // the scale is given, or the format has none
  kCluster1, // one cluster: amax through distributed shared memory, then the output
  kAmax,     // first of two launches: (residual stream and) amax
  kFormat    // second launch: the output, under the amax word of the first
};

__device__ __forceinline__ uint4 ld_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// two floats -> BF16 pair, a in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}

// two floats -> E4M3 pair (saturating, NaN kept), a in the low byte
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
  return d;
}

// A unit is one 32-byte access where every row starts at a multiple of 32 bytes (`wide`),
// else two of 16 (8192 x 5376 to MXFP8 47.7 against 50.7 us).
__device__ __forceinline__ void load_unit(const uint16_t* p, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.L2::256B.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = ld_v4(p), b = ld_v4(p + 8);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

__device__ __forceinline__ void store_unit(uint16_t* p, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// max(|a|, |b|, |c|), NaN if one is
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float amax16(const float (&v)[16]) {
  float m = max3_abs(v[0], v[1], v[2]);
#pragma unroll
  for (int i = 3; i < 15; i += 2) m = max3_abs(m, v[i], v[i + 1]);
  return max_nan(m, fabsf(v[15]));
}

// s_g of an output whose largest magnitude is amax (a division in binary64 instead of the product,
// which is off by 2^-52 before the rounding to a float: 8192 x 5376, two launches, 84.0 us, not 82.8)
__device__ __forceinline__ float tensor_scale(double amax) {
  return amax == 0.0 ? 1.0f : static_cast<float>(amax * (1.0 / 2688.0));
}

// amax >= 0 or NaN: the bit patterns order like the values, NaN above all
__device__ __forceinline__ unsigned long long amax_bits(double amax) {
  return static_cast<unsigned long long>(__double_as_longlong(amax)) & 0x7FFFFFFFFFFFFFFFull;
}

__device__ __forceinline__ void publish_amax(double amax, unsigned long long* word) {
  if (amax_bits(amax) != 0u) atomicMax(word, amax_bits(amax));
}

// shared exponent of an MX block: floor(log2 amax) - emax, clamped (amax = 0: -127)
__device__ __forceinline__ int mx_exponent(float amax, int emax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23);
  const int lg = e > 0 ? e - 127 : (31 - __clz(static_cast<int>(bits))) - 149;
  return bits == 0u ? -127 : max(-127, min(127, lg - emax));
}

__device__ __forceinline__ float exp2_int(int k) {  // k in [-127, 127]
  return k >= -126 ? __uint_as_float(static_cast<uint32_t>(k + 127) << 23) : __uint_as_float(0x00400000u);
}

// The words again, for the compiler unknown ones: it keeps them, not the floats they were widened
// to before (twice the registers; 8192 x 5375: 84 us instead of 72).
template <int N>
__device__ __forceinline__ void as_words(uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(w[i]));
}

// Writes unit u (values 16 u .. 16 u + 15) of row r.  Every lane of the warp calls it
// with u = a multiple of 32 + lane; `active`: u is inside the row.
template <int FMT>
__device__ __forceinline__ void emit(const float (&v)[16], int64_t r, int64_t u, bool active, int64_t cols, float sg,
                                     const RowOutput& o) {
  if constexpr (FMT == NVFP4_OUT_BF16) {
    if (!active) return;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    store_unit(static_cast<uint16_t*>(o.out) + r * o.ld_out + u * kUnit, o.wide, w);
  } else {
    const int lane = threadIdx.x & 31;
    constexpr int kLanes = FMT == NVFP4_OUT_NVFP4 ? 1 : 2;  // lanes per block
    const int64_t nblk = cols / (kUnit * kLanes);
    float amax = active ? amax16(v) : 0.0f;
    uint32_t sbyte = 0;
    if constexpr (FMT == NVFP4_OUT_NVFP4) {
      sbyte = cvt_e4m3_satfinite(__fdiv_rn(amax, __fmul_rn(6.0f, sg)));
      if (active) {
        const float eff = __fmul_rn(e4m3_to_float(sbyte), sg);
        uint64_t x2[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x2[i] = pack2(v[2 * i], v[2 * i + 1]);
        uint32_t c0, c1;
        encode_codes(x2, eff, __frcp_rn(eff), c0, c1);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(o.out) + r * (cols / 2) + u * 8) = make_uint2(c0, c1);
      }
    } else {
      amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      const int e = mx_exponent(amax, FMT == NVFP4_OUT_MXFP8 ? 8 : 2);
      sbyte = amax != amax ? 255u : static_cast<uint32_t>(e + 127);
      const float inv = exp2_int(-e);
      if (active) {
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(v[i], inv);
        if constexpr (FMT == NVFP4_OUT_MXFP8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_e4m3(y[4 * i], y[4 * i + 1]) | (pack_e4m3(y[4 * i + 2], y[4 * i + 3]) << 16);
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(o.out) + r * cols + u * 16) =
              make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          const uint32_t c0 = cvt_e2m1x8(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
          const uint32_t c1 = cvt_e2m1x8(y[8], y[9], y[10], y[11], y[12], y[13], y[14], y[15]);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(o.out) + r * (cols / 2) + u * 8) = make_uint2(c0, c1);
        }
      }
    }
    const int64_t b = u / kLanes;
    if (o.swizzled || (nblk & 3) == 0) {
      // four consecutive blocks' bytes in one 32-bit store; a block past the row's end
      // is the tile's padding and contributes 0
      if (!active) sbyte = 0;
      const uint32_t s1 = __shfl_down_sync(0xFFFFFFFFu, sbyte, kLanes);
      const uint32_t s2 = __shfl_down_sync(0xFFFFFFFFu, sbyte, 2 * kLanes);
      const uint32_t s3 = __shfl_down_sync(0xFFFFFFFFu, sbyte, 3 * kLanes);
      if (active && (lane % (4 * kLanes)) == 0) {
        const int64_t atoms = (nblk + 3) / 4;
        const int64_t at = o.swizzled ? ((r >> 7) * atoms + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4
                                      : r * nblk + b;
        *reinterpret_cast<uint32_t*>(o.scales + at) = sbyte | (s1 << 8) | (s2 << 16) | (s3 << 24);
      }
    } else if (active && (lane % kLanes) == 0) {
      o.scales[r * nblk + b] = static_cast<uint8_t>(sbyte);
    }
  }
}

// Zeroes the row padding of a swizzled scale buffer: the 16-byte lines of its last row
// group (rows q * 32 + line of the group in word q), by threads `tid` of `threads`.
__device__ __forceinline__ void zero_row_padding(uint8_t* scales, int64_t rows, int64_t nblk, int64_t tid,
                                                 int64_t threads) {
  const int64_t tail = rows & 127;
  if (tail == 0) return;
  const int64_t atoms = (nblk + 3) / 4;
  uint8_t* base = scales + (rows >> 7) * atoms * 512;
  for (int64_t i = tid; i < atoms * 32; i += threads) {
    uint32_t* line = reinterpret_cast<uint32_t*>(base + i * 16);
    const int64_t l = i & 31;
    if (l >= tail) {
      *reinterpret_cast<uint4*>(line) = make_uint4(0u, 0u, 0u, 0u);
    } else {
#pragma unroll
      for (int q = 1; q < 4; ++q)
        if (l + 32 * q >= tail) line[q] = 0u;
    }
  }
}

// 16-byte lines that a padding CTA of `threads` threads zeroes per thread, and the CTAs needed.
int64_t padding_lines(int64_t rows, int64_t cols, const RowOutput& o) {
  if (o.format == NVFP4_OUT_BF16 || !o.swizzled || (rows & 127) == 0) return 0;
  const int64_t nblk = cols / (o.format == NVFP4_OUT_NVFP4 ? 16 : 32);
  return (nblk + 3) / 4 * 32;
}

__device__ __forceinline__ unsigned long long ld_shared_cluster_u64(uint32_t cluster_addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr) : "memory");
  return v;
}

__device__ __forceinline__ double cluster_max(double mine, unsigned long long* slot) {
  if (threadIdx.x == 0) *slot = amax_bits(mine);
  cluster_sync();
  unsigned long long g = 0;
#pragma unroll
  for (uint32_t i = 0; i < static_cast<uint32_t>(kCluster); ++i)
    g = max(g, ld_shared_cluster_u64(mapa_shared(smem_u32(slot), i)));
  cluster_sync();  // no CTA leaves while another still reads its word
  return __longlong_as_double(static_cast<long long>(g));
}

// Sum over the CTA (every thread gets it), in a fixed order.  One __syncthreads; `part`
// must not be reused before another one.
template <typename T>
__device__ __forceinline__ T block_sum(T s, T* part) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  s = lane < nw ? part[lane] : T{0};
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s;
}

// Maximum over the CTA of a magnitude (>= 0 or NaN) as its bit pattern; valid in every thread.
__device__ __forceinline__ float block_max(float m, uint32_t* part) {
  uint32_t b = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m) & 0x7FFFFFFFu);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) part[threadIdx.x >> 5] = b;
  __syncthreads();
  b = __reduce_max_sync(0xFFFFFFFFu, lane < nw ? part[lane] : 0u);
  return __uint_as_float(b);
}

// 1 / sqrt(mean square + eps) = up (r + r_lo), up a power of two and r in [1, 2] (above that where
// up would leave binary32), r_lo what its float leaves.  h * up is exact and near 1, whatever the
// row's magnitude; its product with a BF16 weight is exact too, so that v is rounded once, by r.
struct InvRms {
  float up, r, r_lo;
};

// From m = (mean square + eps) 4^f.  With m = 4^k t, t in [1, 4): r = 2 / sqrt(t) by the function
// and one Newton step, r + r (1 - t (r / 2)^2) / 2, whose residual takes the square in two floats.
__device__ __forceinline__ InvRms inv_rms(float m, int f) {
  if (!(m >= 0x1p-126f && m < __int_as_float(0x7F800000)))  // zero, infinity, NaN
    return {1.0f, m > 0.0f ? 0.0f : m == 0.0f ? __int_as_float(0x7F800000) : m, 0.0f};
  const int e = (__float_as_int(m) >> 23) - 127, k = e >> 1;
  const float t = __int_as_float(__float_as_int(m) - (k << 24));
  const float r = rsqrtf(t), q = __fmul_rn(r, r);
  const float d = __fmaf_rn(-t, __fmaf_rn(r, r, -q), __fmaf_rn(-t, q, 1.0f));
  const int up = max(-149, min(127, f - k - 1));
  const float rest = 2.0f * exp2_float(f - k - 1 - up), hi = __fmaf_rn(0.5f * r, d, r);
  return {exp2_float(up), hi * rest, __fmaf_rn(0.5f * r, d, r - hi) * rest};
}

// Sum over the CTA of (h x)^2, h the row's values from memory.  Out of line, for the few rows that
// need it: inlined, the branch cost 8192 x 5375 86 us instead of 75.
__device__ __noinline__ float scaled_squares(const uint16_t* h, int64_t cols, float x, float* part) {
  float s = 0.0f;
#pragma unroll 1
  for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) {
    const float v = bf16_bits_to_float(h[c]) * x;
    s = __fmaf_rn(v, v, s);
  }
  return block_sum(s, part);
}

// The same of a row, from this thread's part of the sum of squares.  BF16 squares reach from
// 2^-266 to 2^256: a sum that left binary32's range, or came near its lower end with nothing in
// eps to cover that, is taken once more of scaled values.  h: the row's cols values in memory (0:
// no row), the CTA's own stores of them visible since the first sum's barrier.
__device__ __forceinline__ InvRms row_inv_rms(const NormArgs& a, float mine, float (*part)[32], const uint16_t* h,
                                              int64_t cols) {
  const float s = block_sum(mine, part[0]);
  const float m = __fmaf_rn(s, a.inv_cols, __fmaf_rn(s, a.inv_cols_lo, a.eps));
  if (s < 1e38f && m >= 0x1p-100f) return inv_rms(m, 0);
  const int f = s < 1e38f ? 80 : -80;
  const float x = scaled_squares(h, cols, exp2_float(f), part[1]), eps = a.eps * exp2_float(f) * exp2_float(f);
  return inv_rms(__fmaf_rn(x, a.inv_cols, eps), f);
}

// Sum of squares of the values of N words of BF16 pairs, in four parts.
template <int N>
__device__ __forceinline__ float unit_squares(const uint32_t (&h)[N]) {
  uint64_t s[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t x = pack2(bf16_lo(h[i]), bf16_hi(h[i]));
    s[i & 1] = fma2(x, x, s[i & 1]);
  }
  float a, b, c, d;
  unpack2(s[0], a, b);
  unpack2(s[1], c, d);
  return (a + b) + (c + d);
}

// One CTA per row; thread t owns units t, t + T, ... (U of them), kept in registers
// between the sum of squares and the output, so each input is read once.
template <int FMT, int U, int PHASE>
__global__ void __launch_bounds__(norm_threads(U)) norm_kernel(const NormArgs a, const RowOutput o) {
  __shared__ float sums[2][32];
  __shared__ uint32_t maxima[32];
  __shared__ unsigned long long cta_max;
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t units = a.cols / kUnit;
  const int T = blockDim.x;
  if (PHASE != kCluster1 && blockIdx.x >= a.rows) {  // a padding CTA
    zero_row_padding(o.scales, a.rows, a.cols / (FMT == NVFP4_OUT_NVFP4 ? 16 : 32),
                     (static_cast<int64_t>(blockIdx.x) - a.rows) * T + threadIdx.x,
                     (static_cast<int64_t>(gridDim.x) - a.rows) * T);
    return;
  }
  // the second launch walks the rows backwards: the last rows of the first are in L2
  const int64_t r = PHASE == kFormat ? a.rows - 1 - blockIdx.x : blockIdx.x;
  const bool row = PHASE != kCluster1 || r < a.rows;
  uint32_t h[U][8];
  const bool add = PHASE != kFormat && a.residual != nullptr;
  const uint16_t* src = PHASE == kFormat && a.residual ? a.residual_out + r * a.ld_res_out : a.x + r * a.ld_x;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int64_t u = threadIdx.x + static_cast<int64_t>(k) * T;
    if (row && u < units) {
      load_unit(src + u * kUnit, a.wide, h[k]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = 0u;
    }
  }
  if (add && U > 4) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t u = threadIdx.x + static_cast<int64_t>(k) * T;
      if (row && u < units) {
        uint32_t q[8];
        load_unit(a.residual + r * a.ld_res + u * kUnit, a.wide, q);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          h[k][i] = pack_bf16(bf16_lo(h[k][i]) + bf16_lo(q[i]), bf16_hi(h[k][i]) + bf16_hi(q[i]));
        store_unit(a.residual_out + r * a.ld_res_out + u * kUnit, a.wide, h[k]);
      }
    }
  } else if (add) {  // all loads of the residual in flight together
    uint32_t q[U][8];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t u = threadIdx.x + static_cast<int64_t>(k) * T;
      if (row && u < units) load_unit(a.residual + r * a.ld_res + u * kUnit, a.wide, q[k]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t u = threadIdx.x + static_cast<int64_t>(k) * T;
      if (row && u < units) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          h[k][i] = pack_bf16(bf16_lo(h[k][i]) + bf16_lo(q[k][i]), bf16_hi(h[k][i]) + bf16_hi(q[k][i]));
        store_unit(a.residual_out + r * a.ld_res_out + u * kUnit, a.wide, h[k]);
      }
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < U; ++k) s += unit_squares(h[k]);
  const InvRms inv = row_inv_rms(a, s, sums, add ? a.residual_out + r * a.ld_res_out : src, row ? a.cols : 0);
#pragma unroll
  for (int k = 0; k < U; ++k) as_words(h[k]);
  const uint64_t up = pack2(inv.up, inv.up), rstd = pack2(inv.r, inv.r), rstd_lo = pack2(inv.r_lo, inv.r_lo);
  const uint64_t one = pack2(1.0f, 1.0f), offset = pack2(a.weight_offset, a.weight_offset);

  // (h up)(weight + offset) of unit k
  auto weighted = [&](int k, uint64_t (&x)[8]) {
    const int64_t u = threadIdx.x + static_cast<int64_t>(k) * T;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = mul2(pack2(bf16_lo(h[k][i]), bf16_hi(h[k][i])), up);
    if (a.weight != nullptr && u < units) {
      uint32_t w[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(a.weight + u * kUnit) + half);
        w[4 * half] = q.x, w[4 * half + 1] = q.y, w[4 * half + 2] = q.z, w[4 * half + 3] = q.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], fma2(pack2(bf16_lo(w[i]), bf16_hi(w[i])), one, offset));
    }
  };

  float sg = 1.0f;
  if constexpr (PHASE == kCluster1 || PHASE == kAmax) {
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      uint64_t x[8];
      float v[16];
      weighted(k, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) unpack2(x[i], v[2 * i], v[2 * i + 1]);
      if (row && threadIdx.x + static_cast<int64_t>(k) * T < units) m = max_nan(m, amax16(v));
    }
    // the row's largest |v| in binary64: the tensor scale moves every rounding border of the output
    const double amax = row ? block_max(m, maxima) * (static_cast<double>(inv.r) + inv.r_lo) : 0.0;
    if constexpr (PHASE == kAmax) {
      if (threadIdx.x == 0) publish_amax(amax, o.amax_word);
      return;
    }
    sg = tensor_scale(cluster_max(amax, &cta_max));
  } else if constexpr (FMT == NVFP4_OUT_NVFP4) {
    sg = PHASE == kFormat ? tensor_scale(__longlong_as_double(*o.amax_word)) : *o.gs_in;
  }
  if (FMT == NVFP4_OUT_NVFP4 && o.gs_out && blockIdx.x == 0 && threadIdx.x == 0) *o.gs_out = sg;
  if (row) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t u = threadIdx.x + static_cast<int64_t>(k) * T;
      if (U > 1 && u - threadIdx.x >= units) break;
      uint64_t x[8];
      float v[16];
      weighted(k, x);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        unpack2(FMT == NVFP4_OUT_BF16 ? mul2(x[i], rstd) : fma2(x[i], rstd, mul2(x[i], rstd_lo)), v[2 * i],
                v[2 * i + 1]);
      emit<FMT>(v, r, u, u < units, a.cols, sg, o);
    }
  }
  if (PHASE == kCluster1 && o.swizzled)
    zero_row_padding(o.scales, a.rows, a.cols / 16, static_cast<int64_t>(blockIdx.x) * T + threadIdx.x,
                     static_cast<int64_t>(gridDim.x) * T);
}

// BF16 rows that the 16-value units do not fit (odd sizes, strides or addresses, or rows
// longer than a CTA's registers hold): one value per thread and step.  CACHED: a thread's
// kAny values stay in registers; else the second pass re-reads h (each thread its own
// values, so x may be the output).
constexpr int kAny = 8;
template <bool CACHED>
__global__ void __launch_bounds__(512) norm_any_kernel(const NormArgs a, uint16_t* out, int64_t ld_out) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t r = blockIdx.x;
  const uint16_t* x = a.x + r * a.ld_x;
  const uint16_t* q = a.residual ? a.residual + r * a.ld_res : nullptr;
  uint16_t* ho = a.residual_out + r * a.ld_res_out;
  auto value = [&](int64_t c) {  // h of column c, stored on the way
    const float f = bf16_bits_to_float(x[c]);
    if (q == nullptr) return f;
    const uint32_t h = pack_bf16(f + bf16_bits_to_float(q[c]), 0.0f) & 0xFFFFu;
    ho[c] = static_cast<uint16_t>(h);
    return bf16_bits_to_float(h);
  };
  auto finish = [&](int64_t c, float f, InvRms inv) {
    float v = __fmul_rn(f, inv.up);
    if (a.weight) v = __fmul_rn(v, __fadd_rn(bf16_bits_to_float(a.weight[c]), a.weight_offset));
    out[r * ld_out + c] = static_cast<uint16_t>(pack_bf16(__fmul_rn(v, inv.r), 0.0f));
  };
  if constexpr (CACHED) {
    __shared__ float sums[2][32];
    float f[kAny];
#pragma unroll
    for (int i = 0; i < kAny; ++i) {
      const int64_t c = threadIdx.x + i * static_cast<int64_t>(blockDim.x);
      f[i] = c < a.cols ? value(c) : 0.0f;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kAny; ++i) s = __fmaf_rn(f[i], f[i], s);
    const InvRms inv = row_inv_rms(a, s, sums, q ? ho : x, a.cols);
#pragma unroll
    for (int i = 0; i < kAny; ++i) {
      const int64_t c = threadIdx.x + i * static_cast<int64_t>(blockDim.x);
      if (c < a.cols) finish(c, f[i], inv);
    }
  } else {
    __shared__ double sums[32];
    double s = 0.0;  // (the row may have 2^31 values, and they are read once: no second sum)
    for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const double f = value(c);
      s = __fma_rn(f, f, s);
    }
    const double m = block_sum(s, sums) / static_cast<double>(a.cols) + static_cast<double>(a.eps);
    // (down to 2^-266 over 2^31 columns)
    const int f = m > 0x1p100 && m < 0x1p300 ? -100 : m < 0x1p-100 ? 100 : 0;
    const InvRms inv = inv_rms(static_cast<float>(m * (f < 0 ? 0x1p-200 : f > 0 ? 0x1p200 : 1.0)), f);
    const uint16_t* h = q ? ho : x;
    for (int64_t c = threadIdx.x; c < a.cols; c += blockDim.x) finish(c, bf16_bits_to_float(h[c]), inv);
  }
}

// BF16 rows of any width in dense matrices: row r begins s = r cols mod 8 values behind a
// 16-byte boundary, the same in every matrix, so that the row is read and written in the
// 16-byte vectors that cover it; the two at its ends go value by value.  The weight, which
// does not share that shift, is read in words and shifted by half a word for odd s.
// (8192 x 5375 with a residual: 74 us; value by value 162.)
template <int V>
__global__ void __launch_bounds__(512) norm_dense_kernel(const NormArgs a, uint16_t* out) {
  __shared__ float sums[2][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int cols = static_cast<int>(a.cols), T = blockDim.x;
  const int64_t start = static_cast<int64_t>(blockIdx.x) * cols;
  const int s = static_cast<int>(start & 7);
  const int64_t base = start - s;
  const int nvec = (s + cols + 7) >> 3;
  const bool add = a.residual != nullptr;
  auto whole = [&](int j) { return 8 * j >= s && 8 * j - s + 8 <= cols; };
  // the vector's values inside the row; others are 0
  auto load = [&](const uint16_t* p, int j, uint32_t (&w)[4]) {
    if (whole(j)) {
      const uint4 v = ld_v4(p + base + 8 * j);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 8 * j - s + 2 * i;
        const uint32_t lo = c >= 0 && c < cols ? p[start + c] : 0u, hi = c + 1 >= 0 && c + 1 < cols ? p[start + c + 1] : 0u;
        w[i] = lo | (hi << 16);
      }
    }
  };
  auto store = [&](uint16_t* p, int j, const uint32_t (&w)[4]) {
    if (whole(j)) {
      *reinterpret_cast<uint4*>(p + base + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = 8 * j - s + i;
        if (c >= 0 && c < cols) p[start + c] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
      }
    }
  };
  uint32_t h[V][4], q[V][4];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int j = threadIdx.x + k * T;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[k][i] = q[k][i] = 0u;
    if (j < nvec) {
      load(a.x, j, h[k]);
      if (add) load(a.residual, j, q[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int j = threadIdx.x + k * T;
    if (add && j < nvec) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[k][i] = pack_bf16(bf16_lo(h[k][i]) + bf16_lo(q[k][i]), bf16_hi(h[k][i]) + bf16_hi(q[k][i]));
      store(a.residual_out, j, h[k]);
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < V; ++k) sum += unit_squares(h[k]);
  const InvRms inv = row_inv_rms(a, sum, sums, (add ? a.residual_out : a.x) + start, a.cols);
#pragma unroll
  for (int k = 0; k < V; ++k) as_words(h[k]);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int j = threadIdx.x + k * T;
    if (j >= nvec) break;
    uint32_t w[5] = {};
    const int c0 = 8 * j - s;  // column of the vector's first value
    if (a.weight != nullptr) {
      // five words from column c0 - (c0 & 1) on, those that hold a column of the row; the
      // last word of an odd row would reach past it
      const uint32_t* words = reinterpret_cast<const uint32_t*>(a.weight);
      const int w0 = c0 >> 1;
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        const int at = w0 + i;
        if (at >= 0 && 2 * at + 1 < cols)
          w[i] = __ldg(words + at);
        else if (at >= 0 && 2 * at < cols)
          w[i] = __ldg(a.weight + 2 * at);
      }
    }
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo = __fmul_rn(bf16_lo(h[k][i]), inv.up), hi = __fmul_rn(bf16_hi(h[k][i]), inv.up);
      if (a.weight != nullptr) {
        const uint32_t ww = c0 & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
        lo = __fmul_rn(lo, __fadd_rn(bf16_lo(ww), a.weight_offset));
        hi = __fmul_rn(hi, __fadd_rn(bf16_hi(ww), a.weight_offset));
      }
      y[i] = pack_bf16(__fmul_rn(lo, inv.r), __fmul_rn(hi, inv.r));
    }
    store(out, j, y);
  }
}

// silu_times of the sixteen values of a unit, two to a packed instruction, for |g| < 80.
//   e^-g = 2^h (1 + l ln 2), h = RN(-g log2 e), l what h leaves of -g log2 e, with the second
//   word of log2 e; d = 1 + e^-g; 1 / d by the approximate reciprocal and one Newton step.
// The error stays near one unit in the last place, so the block formats' rounding borders see
// no more of it than a plain binary32 evaluation has.  Written out because the issue rate
// bounds this kernel: 12 instructions a value instead of 21 took 8192 x 21504 to MXFP8 from
// 172 us to 157 (135 now, 6.5 TB/s).
__device__ __forceinline__ void silu_unit(const uint32_t (&g)[8], const uint32_t (&u)[8], float (&v)[16]) {
  float big = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) big = max3_abs(big, bf16_lo(g[i]), bf16_hi(g[i]));
  if (!(big < 80.0f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = silu_times(bf16_lo(g[i]), bf16_lo(u[i]));
      v[2 * i + 1] = silu_times(bf16_hi(g[i]), bf16_hi(u[i]));
    }
    return;
  }
  const uint64_t m_l2e = pack2(-1.44269502f, -1.44269502f);
  const uint64_t l2e = pack2(1.44269502f, 1.44269502f);             // RN(log2 e)
  const uint64_t l2e_lo = pack2(1.92596299e-8f, 1.92596299e-8f);    // log2 e - RN(log2 e)
  const uint64_t ln2 = pack2(0.693147182f, 0.693147182f), m_one = pack2(-1.0f, -1.0f), one = pack2(1.0f, 1.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t x = pack2(bf16_lo(g[i]), bf16_hi(g[i]));
    const uint64_t h = mul2(x, m_l2e);
    const uint64_t ml = fma2(x, l2e_lo, fma2(x, l2e, h));  // -l: the inner one exact
    float h0, h1, e0, e1;
    unpack2(h, h0, h1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(h0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(h1));
    // -d = -1 - e (1 + l ln 2), and 1 + l ln 2 = 1 - ln 2 (-l)
    const uint64_t nd = fma2(pack2(e0, e1), fma2(ml, ln2, m_one), m_one);
    float d0, d1, r0, r1;
    unpack2(nd, d0, d1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(-d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(-d1));
    const uint64_t r = pack2(r0, r1);
    const uint64_t q = mul2(mul2(x, fma2(fma2(nd, r, one), r, r)), pack2(bf16_lo(u[i]), bf16_hi(u[i])));
    unpack2(q, v[2 * i], v[2 * i + 1]);
  }
}

constexpr int kGateThreads = 256;
// CTAs of gate_kernel that an SM is to hold (64 or 80 registers a thread; NVFP4's encoding at
// 64 is 4 % slower).
constexpr int gate_ctas(int fmt, int phase) { return fmt == NVFP4_OUT_NVFP4 && phase != kAmax ? 3 : 4; }

// One warp per 32 consecutive units of a row.
template <int FMT, int PHASE>
__global__ void __launch_bounds__(kGateThreads, gate_ctas(FMT, PHASE)) gate_kernel(const GateArgs a, const RowOutput o) {
  __shared__ uint32_t maxima[32];
  __shared__ unsigned long long cta_max;
  grid_dependency_wait();
  grid_dependents_launch();
  const int rows = static_cast<int>(a.rows), units = static_cast<int>(a.cols / kUnit), chunks = (units + 31) / 32;
  const int lane = threadIdx.x & 31;
  // The warp's tasks: chunk c0 of row r0, then step_r rows and step_c chunks further,
  // with a carry (no division per task).
  const int warp = blockIdx.x * (kGateThreads / 32) + (threadIdx.x >> 5), warps = gridDim.x * (kGateThreads / 32);
  const int r0 = warp / chunks, c0 = warp - r0 * chunks;
  const int step_r = warps / chunks, step_c = warps - step_r * chunks;

  // The tasks' values in turn: f(r, u, active, v) for each, the next task's loads requested
  // before f.  `back`: from the last task to the first.  The amax pass takes two sets of
  // registers in turn (46 us instead of 51 for 4096 x 14336); where the encoding needs the
  // registers, moving a set is faster (60 us instead of 66).
  constexpr int kSets = PHASE == kAmax ? 2 : 1;
  auto each = [&](bool back, auto f) {
    struct Pair {
      uint32_t g[8], u[8];
    } p[kSets];
    int r = r0, c = c0;
    auto row = [&]() { return back ? rows - 1 - r : r; };
    auto unit = [&]() { return (back ? chunks - 1 - c : c) * 32 + lane; };
    auto request = [&](Pair& t) {
      const int u = unit();
      if (r < rows && u < units) {
        const int64_t at = row(), off = static_cast<int64_t>(u) * kUnit;
        load_unit(a.gate + at * a.ld_gate + off, a.wide, t.g);
        load_unit(a.up + at * a.ld_up + off, a.wide, t.u);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) t.g[i] = t.u[i] = 0u;
      }
    };
    request(p[0]);
    while (r < rows) {
#pragma unroll
      for (int k = 0; k < kSets; ++k) {
        if (k == 1 && r >= rows) break;
        const int at = row(), u = unit();
        r += step_r;
        c += step_c;
        if (c >= chunks) {
          c -= chunks;
          ++r;
        }
        const Pair t = p[k];
        request(p[kSets - 1 - k]);
        float v[16];
        silu_unit(t.g, t.u, v);
        f(at, u, u < units, v);
      }
    }
  };

  float sg = 1.0f;
  if constexpr (PHASE == kCluster1 || PHASE == kAmax) {
    float m = 0.0f;
    // (an inactive lane's values are 0)
    each(false, [&](int, int, bool, const float(&v)[16]) { m = max_nan(m, amax16(v)); });
    m = block_max(m, maxima);
    if constexpr (PHASE == kAmax) {
      if (threadIdx.x == 0) publish_amax(m, o.amax_word);
      return;
    }
    sg = tensor_scale(cluster_max(m, &cta_max));
  } else if constexpr (FMT == NVFP4_OUT_NVFP4) {
    sg = PHASE == kFormat ? tensor_scale(__longlong_as_double(*o.amax_word)) : *o.gs_in;
  }
  if (FMT == NVFP4_OUT_NVFP4 && o.gs_out && blockIdx.x == 0 && threadIdx.x == 0) *o.gs_out = sg;
  // the second launch walks backwards: the end of the first's reads is in L2
  each(PHASE == kFormat, [&](int r, int u, bool active, const float(&v)[16]) {
    emit<FMT>(v, r, u, active, a.cols, sg, o);
  });
  if (FMT == NVFP4_OUT_BF16 && blockIdx.x == 0 && static_cast<int>(threadIdx.x) < a.tail) {
    const int64_t c = a.cols + threadIdx.x;
    static_cast<uint16_t*>(o.out)[c] = static_cast<uint16_t>(
        pack_bf16(silu_times(bf16_bits_to_float(a.gate[c]), bf16_bits_to_float(a.up[c])), 0.0f));
  }
  if (FMT != NVFP4_OUT_BF16 && o.swizzled)
    zero_row_padding(o.scales, a.rows, a.cols / (FMT == NVFP4_OUT_NVFP4 ? 16 : 32),
                     static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                     static_cast<int64_t>(gridDim.x) * blockDim.x);
}

// BF16 values that the 16-value units do not fit: 1024 of a row per CTA and step.
__global__ void __launch_bounds__(256) gate_any_kernel(const GateArgs a, uint16_t* out, int64_t ld_out) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t parts = (a.cols + 1023) / 1024, tasks = a.rows * parts;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int64_t r = task / parts, c0 = (task - r * parts) * 1024 + threadIdx.x;
    const uint16_t *g = a.gate + r * a.ld_gate, *u = a.up + r * a.ld_up;
    uint16_t* y = out + r * ld_out;
    float gv[4], uv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = c0 + 256 * i;
      gv[i] = c < a.cols ? bf16_bits_to_float(g[c]) : 0.0f;
      uv[i] = c < a.cols ? bf16_bits_to_float(u[c]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = c0 + 256 * i;
      if (c < a.cols) y[c] = static_cast<uint16_t>(pack_bf16(silu_times(gv[i], uv[i]), 0.0f));
    }
  }
}

int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), int64_t grid, int threads, int cluster, cudaStream_t stream, int* launches,
                   Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaGetLastError();
}

bool fits_units(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; }
bool fits_wide(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && ld % 16 == 0; }

// Whether every matrix of a BF16 norm lies dense from a 16-byte boundary on.
bool dense(const NormArgs& a, const RowOutput& o) {
  auto one = [&](const void* p, int64_t ld) { return fits_units(p, 0) && (ld == a.cols || a.rows == 1); };
  return one(a.x, a.ld_x) && one(o.out, o.ld_out) && (reinterpret_cast<uintptr_t>(a.weight) & 3u) == 0 &&
         (!a.residual || (one(a.residual, a.ld_res) && one(a.residual_out, a.ld_res_out)));
}

template <int FMT, int PHASE>
cudaError_t norm_launch_u(const NormArgs& a, const RowOutput& o, int* launches, cudaStream_t stream) {
  const int64_t units = a.cols / kUnit;
  // Few rows: as many threads as a row has units, for the shortest chain of loads per
  // thread; more rows than the SMs hold CTAs: two units per thread.
  int U = a.rows <= 2 * 148 ? 1 : 2;
  while (U < 8 && (units + U - 1) / U > norm_threads(U)) U *= 2;
  int T = static_cast<int>(((units + U - 1) / U + 31) / 32 * 32);
  if (T < 64) T = 64;
  const int64_t pad = PHASE == kCluster1 || PHASE == kAmax ? 0 : padding_lines(a.rows, a.cols, o);
  const int64_t grid = PHASE == kCluster1 ? kCluster : a.rows + (pad + T - 1) / T;
  const int cluster = PHASE == kCluster1 ? kCluster : 1;
  if (U == 1) return launch(norm_kernel<FMT, 1, PHASE>, grid, T, cluster, stream, launches, a, o);
  if (U == 2) return launch(norm_kernel<FMT, 2, PHASE>, grid, T, cluster, stream, launches, a, o);
  if (U == 4) return launch(norm_kernel<FMT, 4, PHASE>, grid, T, cluster, stream, launches, a, o);
  return launch(norm_kernel<FMT, 8, PHASE>, grid, T, cluster, stream, launches, a, o);
}

template <int FMT, int PHASE>
cudaError_t gate_launch(const GateArgs& a, const RowOutput& o, int* launches, cudaStream_t stream) {
  constexpr int T = kGateThreads;
  if (PHASE == kCluster1)
    return launch(gate_kernel<FMT, PHASE>, kCluster, T, kCluster, stream, launches, a, o);
  const int64_t warps = a.rows * ((a.cols / kUnit + 31) / 32);
  int64_t grid = (warps + T / 32 - 1) / (T / 32);
  // (a grid of resident CTAs only, each with the same work, is 2 to 4 % slower)
  const int64_t cap = static_cast<int64_t>(sm_count()) * 16;
  if (grid > cap) grid = cap;
  if (PHASE != kAmax) {
    const int64_t pad = (padding_lines(a.rows, a.cols, o) + T - 1) / T;
    if (grid < pad) grid = pad < cap ? pad : cap;
  }
  return launch(gate_kernel<FMT, PHASE>, grid, T, 1, stream, launches, a, o);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& args, const RowOutput& output, int* launches, cudaStream_t stream) {
  NormArgs a = args;
  RowOutput o = output;
  const double inv_cols = 1.0 / static_cast<double>(a.cols);
  a.inv_cols = static_cast<float>(inv_cols);
  a.inv_cols_lo = static_cast<float>(inv_cols - a.inv_cols);
  a.wide = fits_wide(a.x, a.ld_x) &&
           (!a.residual || (fits_wide(a.residual, a.ld_res) && fits_wide(a.residual_out, a.ld_res_out)));
  o.wide = fits_wide(o.out, o.ld_out);
  const bool units = a.cols % kUnit == 0 && a.cols <= kNormMaxCols &&
                     fits_units(a.x, a.ld_x) && fits_units(a.weight, 0) &&
                     (!a.residual || (fits_units(a.residual, a.ld_res) && fits_units(a.residual_out, a.ld_res_out)));
  switch (o.format) {
    case NVFP4_OUT_BF16:
      if (units && fits_units(o.out, o.ld_out)) return norm_launch_u<NVFP4_OUT_BF16, kOnePass>(a, o, launches, stream);
      if (dense(a, o) && a.cols <= 8 * 512 * 4 - 16) {
        const int64_t nvec = (a.cols + 14) / 8;  // at most, whatever the shift
        const int V = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4;
        const int T = static_cast<int>(((nvec + V - 1) / V + 31) / 32 * 32);
        uint16_t* y = static_cast<uint16_t*>(o.out);
        return V == 1   ? launch(norm_dense_kernel<1>, a.rows, T, 1, stream, launches, a, y)
               : V == 2 ? launch(norm_dense_kernel<2>, a.rows, T, 1, stream, launches, a, y)
                        : launch(norm_dense_kernel<4>, a.rows, T, 1, stream, launches, a, y);
      }
      if (a.cols <= 512 * kAny) {
        const int T = static_cast<int>(((a.cols + kAny - 1) / kAny + 31) / 32 * 32);
        return launch(norm_any_kernel<true>, a.rows, T, 1, stream, launches, a, static_cast<uint16_t*>(o.out), o.ld_out);
      }
      return launch(norm_any_kernel<false>, a.rows, 512, 1, stream, launches, a, static_cast<uint16_t*>(o.out),
                    o.ld_out);
    case NVFP4_OUT_MXFP8: return norm_launch_u<NVFP4_OUT_MXFP8, kOnePass>(a, o, launches, stream);
    case NVFP4_OUT_MXFP4: return norm_launch_u<NVFP4_OUT_MXFP4, kOnePass>(a, o, launches, stream);
    default: break;
  }
  if (o.gs_in) return norm_launch_u<NVFP4_OUT_NVFP4, kOnePass>(a, o, launches, stream);
  if (a.rows <= kCluster) return norm_launch_u<NVFP4_OUT_NVFP4, kCluster1>(a, o, launches, stream);
  cudaError_t e = cudaMemsetAsync(o.amax_word, 0, sizeof(*o.amax_word), stream);
  if (e == cudaSuccess) e = norm_launch_u<NVFP4_OUT_NVFP4, kAmax>(a, o, launches, stream);
  if (e == cudaSuccess) e = norm_launch_u<NVFP4_OUT_NVFP4, kFormat>(a, o, launches, stream);
  return e;
}

cudaError_t launch_silu_mul(const GateArgs& args, const RowOutput& output, int* launches, cudaStream_t stream) {
  GateArgs a = args;
  RowOutput o = output;
  a.wide = fits_wide(a.gate, a.ld_gate) && fits_wide(a.up, a.ld_up);
  o.wide = fits_wide(o.out, o.ld_out);
  switch (o.format) {
    case NVFP4_OUT_BF16: {
      const int64_t n = a.rows * a.cols;
      if (a.cols % kUnit != 0 && n >= kUnit && n <= kMaxFlat &&
          (a.rows == 1 || (a.ld_gate == a.cols && a.ld_up == a.cols && o.ld_out == a.cols)) && fits_units(a.gate, 0) && fits_units(a.up, 0) && fits_units(o.out, 0)) {
        // dense matrices of any width: one row of all values, whose last few are a tail
        a.rows = 1;
        a.tail = static_cast<int>(n % kUnit);
        a.cols = a.ld_gate = a.ld_up = o.ld_out = n - a.tail;
        a.wide = fits_wide(a.gate, 0) && fits_wide(a.up, 0);
        o.wide = fits_wide(o.out, 0);
        return gate_launch<NVFP4_OUT_BF16, kOnePass>(a, o, launches, stream);
      }
      if (a.cols % kUnit == 0 && fits_units(a.gate, a.ld_gate) && fits_units(a.up, a.ld_up) &&
          fits_units(o.out, o.ld_out))
        return gate_launch<NVFP4_OUT_BF16, kOnePass>(a, o, launches, stream);
      int64_t grid = a.rows * ((a.cols + 1023) / 1024);
      const int64_t cap = static_cast<int64_t>(sm_count()) * 16;
      if (grid > cap) grid = cap;
      return launch(gate_any_kernel, grid, 256, 1, stream, launches, a, static_cast<uint16_t*>(o.out), o.ld_out);
    }
    case NVFP4_OUT_MXFP8: return gate_launch<NVFP4_OUT_MXFP8, kOnePass>(a, o, launches, stream);
    case NVFP4_OUT_MXFP4: return gate_launch<NVFP4_OUT_MXFP4, kOnePass>(a, o, launches, stream);
    default: break;
  }
  if (o.gs_in) return gate_launch<NVFP4_OUT_NVFP4, kOnePass>(a, o, launches, stream);
  // a small output: one cluster computes the amax and formats
  if (a.rows * a.cols <= kClusterMax) return gate_launch<NVFP4_OUT_NVFP4, kCluster1>(a, o, launches, stream);
  cudaError_t e = cudaMemsetAsync(o.amax_word, 0, sizeof(*o.amax_word), stream);
  if (e == cudaSuccess) e = gate_launch<NVFP4_OUT_NVFP4, kAmax>(a, o, launches, stream);
  if (e == cudaSuccess) e = gate_launch<NVFP4_OUT_NVFP4, kFormat>(a, o, launches, stream);
  return e;
}

}  // namespace nvfp4
