// matvec.cu -- y = x W^T for 1 to 16 tokens, W in 4 bits (NVFP4 or MXFP4), x in BF16 or
// MXFP8, y in BF16; with a second weight, y = silu(x G^T) * (x W^T) in the same pass.
//   y[m, n] = s_g sum_k x[m, k] q[n, k] s[n, k / G],  G = 16 (E4M3 s) or 32 (E8M0 s).
//
// Bound: the weight stream, N K (1/2 + 1/G) bytes from HBM; the products ride along on
// mma.sync m16n8k16 (f16 x f16 -> f32): 16 weight rows x 8 tokens, so up to 8 tokens need
// the mma of one (14336 x 4096 NVFP4: 9.0 us for 1 token, 12.1 for 8, 15.3 for 16).
//
// Exactness: an E2M1 code times an E4M3 scale has at most 6 significant bits and lies in
// [2^-10, 2688], so NVFP4 weights are exact in binary16.  E8M0 scales do not fit binary16; there
// the mma runs on the bare codes of one block and the binary32 partial product is multiplied by the
// block's power of two.  x becomes binary16 under a power of two per token (over the part of K that
// a CTA handles), its largest finite magnitude just below 2^15 (MXFP4 weights: 2^14); there it is
// exact down to 2^-31 (2^-30) of that largest one.  Smaller values -- one may be the only one that
// meets a weight other than zero -- are left out, and a CTA that has some goes over its weights
// again for them, under their own power of two, until none is left.  So x is exact too, and sums
// are binary32 throughout.
//
// Layout.  K is cut into chunks of 256 values (128 where K is no multiple of 64), N into
// tiles of 16 rows: 4 neighbours in each of the 4 row quarters of a 128-row group, whose
// scales lie side by side in the 128 x 4 scale tiles (row order is free).  A CTA owns a
// run of tiles -- all of K, or, where rows are few and long, one part of it in a cluster
// that shares the tiles -- and puts its part of x into shared memory once, cut into mma
// fragments.  Its (tile, chunk) items, chunks fastest, are dealt to the warps in equal
// runs; a warp keeps a tile's sums in registers along the chunks.  Weights come through
// a ring of asynchronous copies in shared memory, private to the warp, 128 (64)
// contiguous bytes per row.  The mma's k order is free as long as both operands agree:
// for NVFP4 a lane takes the codes whose scales are its own, for MXFP4 ldmatrix deals
// each 16-byte block to a quad, so that an mma stays inside one scale block.  A tile that
// ends in another warp's run leaves its sums in a slot per warp; the slots meet in a fixed
// order (a cluster's through distributed shared memory): no atomics on sums, no
// workspace, the same bits on every call.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "layer_ops.h"
#include "ptx.cuh"
#include "silu.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kDepth = 2;        // weight items in flight per warp (3 and 4: no faster, less room for x)
constexpr int kPad = 16;         // floats per token of a 16-row partial
constexpr int kTokenWords = 8 * kMatvecMaxTokens + 4;
constexpr int kMaxPasses = 12;   // binary32 has 277 binades, a pass takes 30 at least
constexpr int kUnit = 256;       // K is divided in units of this between a cluster's CTAs
constexpr int kSmem = 226 * 1024;

struct Params {
  MatvecArgs a;
  int tiles;          // of 16 rows (gated: 8 of each weight)
  int units;          // of 256 K values
  int atoms;          // scale atoms (4 blocks) per 128-row group
  int batch;          // tiles between two reductions
  int split;          // CTAs of a cluster that share tiles, each a part of K
  int x_units;        // units of a part, at most
  int sums_at;        // a cluster's sums, bytes into shared memory
  bool sums_over_x;   // they take the place of x (one batch)
  uint32_t m_inv;     // ceil(2^32 / M): x / M = mulhi(x, m_inv) for the small x it is used on
  int tiles_q, tiles_r, units_q, units_r;  // tiles per CTA (cluster) and units per part, and remainders
};

// First of `items` that warp w handles (w = kWarps: the end): equal runs, none empty before
// a warp that has one.
__device__ __forceinline__ int run_start(int items, int w) {
  return items < kWarps ? min(w, items) : items * w / kWarps;
}

__device__ __forceinline__ int div_m(const Params& p, int x) {
  return p.a.M == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), p.m_inv));
}

// Asynchronous 16-byte copies, global to shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// the eight E2M1 codes of a word as four binary16 pairs, element 2i in the low half
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 2^k as a BF16 pair
__device__ __forceinline__ uint32_t exp2_bf16x2(int k) { return static_cast<uint32_t>(k + 127) * 0x00800080u; }

__device__ __forceinline__ int exponent(float s) { return max(-126, min(127, (__float_as_int(s) >> 23 & 0xFF) - 127)); }

// s 2^k as the product of two factors, each with half the power of two: what they multiply in turn
// does not leave binary32 on the way unless the result does (a tensor scale is often 2^-15, a
// token's scaling up to 2^120).
__device__ __forceinline__ float2 two_factors(float s, int k) {
  const int e = exponent(s), half = (e + k) / 2;
  return make_float2(s * exp2_float(-e) * exp2_float(half), exp2_float(e + k - half));
}

__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  return d;
}

// two E8M0 bytes times `by` (a BF16 pair) as floats (exact down to 2^-133; 255 is NaN)
__device__ __forceinline__ void e8m0x2_to_float(uint32_t two, uint32_t by, float& lo, float& hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  if (by != exp2_bf16x2(0)) d = mul_bf16x2(d, by);
  lo = __uint_as_float(d << 16);
  hi = __uint_as_float(d & 0xFFFF0000u);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// d += a b, a 16 x 16 (rows of W), b 16 x 8 (tokens)
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two E4M3 codes as floats
__device__ __forceinline__ void e4m3x2_to_float(uint32_t two, float& lo, float& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}\n"
      : "=f"(lo), "=f"(hi)
      : "r"(e4m3x2_to_half2(two)));
}

// eight E4M3 codes times their scale
__device__ __forceinline__ void fp8_values(uint32_t lo4, uint32_t hi4, float s, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    e4m3x2_to_float(((i < 2 ? lo4 : hi4) >> (16 * (i & 1))) & 0xFFFFu, lo, hi);
    v[2 * i] = lo * s;
    v[2 * i + 1] = hi * s;
  }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_shared_cluster(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared4(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared4(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Four 8 x 16-byte matrices of shared memory (lane l: the address of row l & 7 of matrix
// l >> 3): register i holds word t of row g of matrix i.
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}

// Power of two 2^e, e a binary32 exponent
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The exponent E by which a token's values are scaled down, from the bits of its largest finite
// magnitude: 2^-E brings it into [2^(T-1), 2^T), tiny ones as near as binary32 allows.  MXFP4's block
// scales are taken times 2^-6, so that sums of weights up to 2^110 have room beside so large an x.
template <bool MX>
constexpr int kTop = MX ? 14 : 15;
template <bool MX>
constexpr int kScaleShift = MX ? 6 : 0;
template <bool MX>
__device__ __forceinline__ int down_exponent(uint32_t top) {
  return top == 0u ? 0 : max(-126, static_cast<int>(top >> 23) - 126 - kTop<MX>);
}

// The bits of 2^(E + L), the lowest magnitude that is certain to be exact in binary16 after scaling, whose
// last bit is 2^-24: BF16 has 8 bits, E4M3 4.  (No lower than 2^-126; below, both have fewer bits.)
template <bool MX8>
__device__ __forceinline__ uint32_t lowest(int E) {
  return static_cast<uint32_t>(max(E + (MX8 ? -21 : -17) + 127, 1)) << 23;
}

// The same without that lower end.
__device__ __forceinline__ uint32_t lowest_exactly(bool mx8, int E) {
  const int k = E + (mx8 ? -21 : -17);  // -147 at least
  return k >= -126 ? static_cast<uint32_t>(k + 127) << 23 : 1u << (k + 149);
}

// x in shared memory.  The part from unit u0 on (n units) of every token becomes mma fragments
// of scaled binary16: 512 bytes per (unit, token), in which place (j, t) of 16 bytes holds the 8
// values that lane t of a quad multiplies with its word j of the unit's codes.
// Odd tokens have the places of each pair j, j + 1 exchanged, so that two tokens' quads
// read 8 different bank groups.  One warp per (unit, token), a lane per piece of 8 values.
// fetch() copies the pieces as they come (E4M3: 8 bytes, then the word that holds their
// scale), ahead of the weight stream; stage() puts their values in place.  (Copying
// straight to the places, whose stride is 64 bytes or more, took 600 cycles a copy.)
// Rolled loops: the code runs once per launch, from a cold instruction cache.
template <bool MX, int WORDS>
struct Stager {
  const Params& p;
  const int u0, pairs;
  uint4* const xs;

  // Calls f(pair, unit, token) for the warp's pairs.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int M = p.a.M, step_u = div_m(p, kWarps), step_m = kWarps - step_u * M;
    int pair = threadIdx.x >> 5, u = div_m(p, pair), m = pair - u * M;
#pragma unroll 1
    for (; pair < pairs; pair += kWarps) {
      f(pair, u, m);
      u += step_u;
      m += step_m;
      if (m >= M) {
        m -= M;
        ++u;
      }
    }
  }
  __device__ __forceinline__ uint4* raw(int pair) const { return xs + pair * 32 + (threadIdx.x & 31); }
  __device__ __forceinline__ int k_of(int u) const { return (u0 + u) * kUnit + (threadIdx.x & 31) * 8; }
  __device__ __forceinline__ int scale_of(int m, int k) const {
    const int b = k >> 5, row = p.a.x_row0 + m;
    return p.a.x_swizzled ? (b >> 2) * 512 + row * 16 + (b & 3) : row * static_cast<int>(p.a.K >> 5) + b;
  }

  __device__ __forceinline__ void fetch() const {
    const MatvecArgs& a = p.a;
    each([&](int pair, int u, int m) {
      const int k = k_of(u);
      const uint32_t dst = smem_u32(raw(pair));
      if (k >= a.K) {
        st_shared16(dst, make_uint4(0u, 0u, a.x_scales ? 0x7F7F7F7Fu : 0u, 0u));
      } else if (a.x_scales == nullptr) {
        copy16(dst, static_cast<const uint8_t*>(a.x) + (m * a.ld_x + k) * 2);
      } else {
        copy8(dst, static_cast<const uint8_t*>(a.x) + m * a.ld_x + k);
        const int at = scale_of(m, k), word = at & ~3;
        if (a.x_swizzled || word + 4 <= a.x_rows * static_cast<int>(a.K >> 5))
          copy4(dst + 8, a.x_scales + word);
        else  // the last bytes of a linear buffer that ends inside a word
          st_shared4(dst + 8, static_cast<uint32_t>(__ldg(a.x_scales + at)) * 0x01010101u);
      }
    });
    copies_commit();
  }

  // the values of an MXFP8 piece; returns their scale
  __device__ __forceinline__ float fp8(uint4 v, int u, int m, float (&f)[8]) const {
    float s, unused;
    e8m0x2_to_float((v.z >> (8 * (scale_of(m, k_of(u)) & 3))) & 0xFFu, exp2_bf16x2(0), s, unused);
    fp8_values(v.x, v.y, s, f);
    return s;
  }

  // The values of a piece; returns an MXFP8 piece's scale.
  template <bool MX8>
  __device__ __forceinline__ float values(uint4 v, int u, int m, float (&f)[8]) const {
    if constexpr (MX8) {
      return fp8(v, u, m, f);
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
      return 0.0f;
    }
  }

  // This lane's place in a pair's 512 bytes.
  __device__ __forceinline__ uint32_t place() const {
    const int lane = threadIdx.x & 31;
    const int j = MX ? lane >> 2 : WORDS == 8 ? lane & 7 : (lane >> 4) * 4 + (lane & 3);
    const int t = MX ? lane & 3 : WORDS == 8 ? lane >> 3 : (lane >> 2) & 3;
    return smem_u32(xs + j * 4 + t);
  }
  __device__ __forceinline__ void put(uint32_t place, int pair, int m, const float (&f)[8], float down) const {
    st_shared16((place + pair * 512) ^ ((m & 1) << 6),
                make_uint4(pack_half(f[0] * down, f[1] * down), pack_half(f[2] * down, f[3] * down),
                           pack_half(f[4] * down, f[5] * down), pack_half(f[6] * down, f[7] * down)));
  }

  // top: a zeroed word per token, receives the bits of its largest finite magnitude.
  template <bool MX8>
  __device__ __forceinline__ void find_top(uint32_t* top) const {
    each([&](int pair, int u, int m) {
      const uint4 v = *raw(pair);
      uint32_t big = 0;
      if constexpr (MX8) {
        float f[8];
        fp8(v, u, m, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b = __float_as_uint(f[e]) & 0x7FFFFFFFu;
          big = max(big, b < 0x7F800000u ? b : 0u);  // infinities and NaN do not set the scale
        }
      } else {
        const uint32_t k = 0x7FFF7FFFu;
        const uint32_t two = __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
        big = max(two & 0xFFFFu, two >> 16);
        if (big >= 0x7F80u) {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          big = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t b = (w[e >> 1] >> (16 * (e & 1))) & 0x7FFFu;
            big = max(big, b < 0x7F80u ? b : 0u);
          }
        }
        big <<= 16;
      }
      big = __reduce_max_sync(0xFFFFFFFFu, big);
      if ((threadIdx.x & 31) == 0) atomicMax(top + m, big);
    });
  }

  // Every lane takes the pieces it copied and scales them by `top`.  Returns whether a value of the
  // thread's is too small for that.
  template <bool MX8>
  __device__ __forceinline__ bool stage(const uint32_t* top) const {
    bool far = false;
    const uint32_t to = place();
    each([&](int pair, int u, int m) {
      const uint4 v = *raw(pair);
      __syncwarp();  // the pair's pieces have been read: its 512 bytes may be written
      float f[8];
      const float s = values<MX8>(v, u, m, f);
      const int E = down_exponent<MX>(top[m]);
      const uint32_t from = lowest<MX8>(E);
      if (!MX8 || s * 0x1p-9f < __uint_as_float(from)) {  // (2^-9: the smallest E4M3 value but 0)
        uint32_t least = 2u * from - 1u;                  // magnitudes as doubled bits less 1: a zero is the largest
#pragma unroll
        for (int e = 0; e < 8; ++e) least = min(least, __float_as_uint(f[e]) * 2u - 1u);
        far |= least < 2u * from - 1u;
      }
      put(to, pair, m, f, exp2_int(-E));
    });
    return far;
  }

  // The same of pieces fetched again and of the values below the token's limit[m] alone: those from
  // there on and too small ones are left out (zeros), and next[m] (zeroed) receives the largest of
  // the latter.
  __device__ __forceinline__ void stage_below(bool mx8, const uint32_t* top, const uint32_t* limit,
                                              uint32_t* next) const {
    const uint32_t to = place();
    each([&](int pair, int u, int m) {
      const uint4 v = *raw(pair);
      __syncwarp();
      float f[8];
      if (mx8)
        values<true>(v, u, m, f);
      else
        values<false>(v, u, m, f);
      const int E = down_exponent<MX>(top[m]);
      const uint32_t from = lowest_exactly(mx8, E), end = limit[m];
      uint32_t big = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(f[e]) & 0x7FFFFFFFu;
        if (b < min(from, end)) big = max(big, b);
        f[e] = b < from || b >= end ? 0.0f : f[e];
      }
      big = __reduce_max_sync(0xFFFFFFFFu, big);
      if (big != 0u && (threadIdx.x & 31) == 0) atomicMax(next + m, big);
      put(to, pair, m, f, exp2_int(-E));
    });
  }
};

// One item in a warp's ring: 16 R rows of codes (the 16-byte pieces of a row permuted so that
// every access below is free of bank conflicts), then its scale lines, 4 R per atom.
template <bool MX, int WORDS, int R>
struct ItemBytes {
  static constexpr int kRow = WORDS * 16;                   // bytes of codes per row
  static constexpr int kAtoms = WORDS / (MX ? 4 : 2);       // scale atoms
  static constexpr int kScales = 16 * R * kRow;             // where the scales begin
  static constexpr int kBytes = kScales + 64 * R * kAtoms;
  __device__ static int place(int m, int piece) {
    return m * kRow + ((piece ^ (WORDS == 8 ? m & 7 : (m >> 1) & 3)) << 4);
  }
};

// WORDS: 32-bit words of codes per lane and row of an item: 8 (chunks of 256) or 4 (128).
// R: 16-row groups of a tile (2 only with WORDS 4: each word of x then serves two of them).
template <bool MX, int NT, bool GATED, int WORDS, int R>
__global__ void __launch_bounds__(kThreads, 1) matvec_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  using Ring = ItemBytes<MX, WORDS, R>;
  constexpr int kPerUnit = 8 / WORDS;              // chunks per unit
  constexpr int kLines = (GATED ? 2 : 4) * R;      // neighbour lines of a tile
  constexpr int kCopies = WORDS / 2 * R;           // copies per lane for the codes
  static_assert(WORDS == 4 || R == 1, "a 256-value chunk of one 16-row group, or 128 of one or two");
  constexpr int W = kWarps;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int M = p.a.M, slot = M * kPad * R;
  const uint32_t ring = smem_u32(smem) + warp * kDepth * Ring::kBytes;
  uint4* xs = reinterpret_cast<uint4*>(smem + W * kDepth * Ring::kBytes);
  // per token: largest magnitude; of one pass of many: the same of its values, the limit below which they
  // lie, and the largest that it leaves out; what sums are multiplied by; and a word: x too wide for one pass
  uint32_t* top = reinterpret_cast<uint32_t*>(xs + p.x_units * M * 32);
  uint32_t *const cur = top + kMatvecMaxTokens, *const limit = cur + kMatvecMaxTokens;
  uint32_t* const next = limit + kMatvecMaxTokens;
  float2* factors = reinterpret_cast<float2*>(next + kMatvecMaxTokens);
  uint32_t* wide = top + kTokenWords - 4;
  uint8_t* first = reinterpret_cast<uint8_t*>(top + kTokenWords);  // per tile: first and last warp
  uint8_t* last = first + p.batch;
  float* part = reinterpret_cast<float*>(first + (2 * p.batch + 15) / 16 * 16);  // slot of (tile, warp): tile + warp
  const int rank = p.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int group = p.split > 1 ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int T0 = group * p.tiles_q + min(group, p.tiles_r), T1 = T0 + p.tiles_q + (group < p.tiles_r);
  const int u0 = rank * p.units_q + min(rank, p.units_r), un = p.units_q + (rank < p.units_r);
  const int row_bytes = static_cast<int>(p.a.K / 2);
  const int chunk0 = u0 * kPerUnit;
  // chunks of this part (the last unit may end inside its first chunk of 128), those whole
  const int chunks = min(un * kPerUnit, (row_bytes + Ring::kRow - 1) / Ring::kRow - chunk0);
  const int whole = min(chunks, row_bytes / Ring::kRow - chunk0);
  const int64_t group_bytes = static_cast<int64_t>(p.atoms) * 512;
  const int N = static_cast<int>(p.a.N);
  if (threadIdx.x < kMatvecMaxTokens) top[threadIdx.x] = *wide = 0u;

  // Load side: walks the items of this warp, batch after batch, kDepth ahead of the other.
  // A lane copies 16-byte pieces of row quarter lq, with WORDS 8 of one row per copy, with
  // WORDS 4 of two.
  const int lq = WORDS == 8 ? lane >> 3 : (lane >> 2) & 3;
  const int lpiece = WORDS == 8 ? lane & 7 : lane & 3;
  const int lline = WORDS == 8 ? 0 : lane >> 4;  // line of the first copy
  const uint32_t ldst = ring + (WORDS == 8 ? Ring::place(lq, lpiece) : Ring::place(lane >> 2, lpiece));
  const uint32_t sdst = ring + Ring::kScales + lane * 16;
  const int64_t lane_off = (32 * lq + lline) * static_cast<int64_t>(row_bytes) + lpiece * 16;
  const uint8_t* const codes0 = (GATED ? p.a.gate.codes : p.a.w.codes) + lane_off;
  const int64_t gate_to_w = GATED ? static_cast<int64_t>(reinterpret_cast<uintptr_t>(p.a.w.codes) -
                                                         reinterpret_cast<uintptr_t>(p.a.gate.codes))
                                  : 0;
  // a lane per 16-byte scale line, 4 R lines of each atom: rows 4 line .. of the tile
  const bool scale_lane = lane < 4 * R * Ring::kAtoms;
  const int satom = lane / (4 * R), sline = lane % (4 * R);
  const uint8_t* const scales0 = (GATED && (sline & 2) == 0 ? p.a.gate.scales : p.a.w.scales) + satom * 512 +
                                 (GATED ? (sline >> 2) * 2 + (sline & 1) : sline) * 16;
  // Segments: consecutive chunks of one tile.
  int ltile = T0, lt = 0, lc = 0, left = 0;  // batch: first tile; next tile and chunk; items left
  int run = 0;                               // items left of the segment
  bool full = false;                         // every row and byte of its items is inside the weight
  int rows = 0, lchunk = 0;                  // otherwise: rows of this lane's quarter, the chunk
  const uint8_t *pc = codes0, *ps = scales0;
  auto segment = [&]() {
    while (left == 0 && ltile < T1) {
      const int nt = min(p.batch, T1 - ltile), items = nt * chunks, i0 = run_start(items, warp);
      left = run_start(items, warp + 1) - i0;
      lt = i0 / chunks;
      lc = i0 - lt * chunks;
      if (left == 0) ltile += nt;  // (fewer items than warps)
    }
    if (left == 0) return;
    const int line = (ltile + lt) * kLines;
    const int row0 = (line >> 5) * 128 + (line & 31);
    lchunk = chunk0 + lc;
    pc = codes0 + static_cast<int64_t>(row0) * row_bytes + lchunk * Ring::kRow;
    ps = scales0 + (line >> 5) * group_bytes + (line & 31) * 16 + lchunk * static_cast<int64_t>(Ring::kAtoms * 512);
    full = (line >> 5) * 128 + 128 <= N && lc < whole;
    rows = N - row0 - 32 * lq - lline;
    run = full ? min(left, whole - lc) : 1;
    left -= run;
    lc += run;
    if (lc == chunks) {
      lc = 0;
      ++lt;
    }
    if (left == 0) ltile += min(p.batch, T1 - ltile);
  };
  auto load = [&](int at) {  // at: the slot's offset in the ring
    if (run == 0) segment();
    if (run > 0) {
      const uint8_t* pw = pc + gate_to_w;
      const uint32_t d0 = ldst + at, d1 = (ldst ^ 64u) + at;
      if (full) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          // line of the copy (less lline): rows 4 line .. of the tile, the gate's before w's in each 16
          const int l = WORDS == 8 ? (GATED ? i & 1 : i) : (GATED ? i & ~1 : 2 * i);
          const bool of_w = GATED && (WORDS == 8 ? i >= 2 : i & 1);
          copy16((WORDS == 8 && (i & 1) ? d1 : d0) + i * 512,
                 (of_w ? pw : pc) + static_cast<uint64_t>(static_cast<uint32_t>(row_bytes)) * l);
        }
        if (scale_lane) copy16(sdst + at, ps);
      } else {
        // a row or piece outside the weight keeps what the ring held: the row's sums are never
        // written, the piece meets zeros of x
        const bool in = lchunk * Ring::kRow + lpiece * 16 < row_bytes;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int l = WORDS == 8 ? (GATED ? i & 1 : i) : (GATED ? i & ~1 : 2 * i);
          const bool of_w = GATED && (WORDS == 8 ? i >= 2 : i & 1);
          if (in && l < rows)
            copy16((WORDS == 8 && (i & 1) ? d1 : d0) + i * 512,
                   (of_w ? pw : pc) + static_cast<int64_t>(row_bytes) * l);
        }
        // scales past the row's end are cleared, whatever the padding holds: zero by zero
        const int blocks = row_bytes / (MX ? 16 : 8) - 4 * (lchunk * Ring::kAtoms + satom);
        if (scale_lane) {
          if (blocks >= 4) {
            copy16(sdst + at, ps);
          } else {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (blocks > 0) {
              const uint32_t mask = (1u << (8 * blocks)) - 1u;
              v = __ldg(reinterpret_cast<const uint4*>(ps));
              v = make_uint4(v.x & mask, v.y & mask, v.z & mask, v.w & mask);
            }
            st_shared16(sdst + at, v);
          }
        }
      }
      pc += Ring::kRow;
      ps += Ring::kAtoms * 512;
      --run;
    }
    copies_commit();  // (empty past the end: the wait counts groups)
  };
  if (p.split > 1 && !p.sums_over_x) cluster_arrive();  // waited for before the first store into another CTA
  __syncthreads();  // `top` is zeroed
  segment();
  grid_dependency_wait();
  grid_dependents_launch();
  const Stager<MX, WORDS> stager{p, u0, un * M, xs};
  stager.fetch();
#pragma unroll 1
  for (int d = 0; d < kDepth; ++d) load(d * Ring::kBytes);
  copies_wait<kDepth>();  // x, not yet the weights
  // (a loop for each kind of x: 8 tokens of MXFP8, 4096 x 14336 MXFP4, 13.5 us instead of 14.1)
  const bool mx8 = p.a.x_scales != nullptr;
  bool far;
  if (mx8) {
    stager.template find_top<true>(top);
    __syncthreads();
    far = stager.template stage<true>(top);
  } else {
    stager.template find_top<false>(top);
    __syncthreads();
    far = stager.template stage<false>(top);
  }
  if (far) *wide = 1u;
  __syncthreads();  // (with a reduction of the flag: 16 tokens, 5376 x 21504, 0.4 us slower)
  const bool many = *wide != 0u;  // passes over the weights

  // Compute side: a lane's places in a slot of the ring and in x (a token that is not there
  // repeats the last one: its sums are not kept).
  const uint32_t codes_at = ring + (MX ? Ring::place((lane & 7) + (lane & 8), lane >> 4) : Ring::place(g, t * (WORDS / 4)));
  const uint32_t scales_at = ring + Ring::kScales + g * 4 + (MX ? 0 : (WORDS == 8 ? t : t >> 1) * 64 * R);
  uint32_t x_at[NT], x_flip[NT];  // of word 0 of the part; 64 for odd tokens
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int m = min(g + 8 * n, M - 1);
    x_at[n] = smem_u32(xs + m * 32 + t);
    x_flip[n] = (m & 1) * 64;
  }
  // What the sums of each token are multiplied by: the tensor scale (gated: also the gate's) and the power of
  // two that x was scaled down by; by the first threads, from their token's largest magnitude.
  auto set_factors = [&](const uint32_t* of) {
    if (threadIdx.x < (GATED ? 2 : 1) * kMatvecMaxTokens) {
      const float* gs = GATED && threadIdx.x >= kMatvecMaxTokens ? p.a.gate.gs : p.a.w.gs;
      factors[threadIdx.x] = two_factors(
          gs ? *gs : 1.0f, down_exponent<MX>(of[threadIdx.x % kMatvecMaxTokens]) + kScaleShift<MX>);
    }
  };
  if (!many) set_factors(top);
  int at = 0;  // the slot's offset in the ring
  for (int tile0 = T0; tile0 < T1; tile0 += p.batch) {
    const int nt = min(p.batch, T1 - tile0);
    const int items = nt * chunks;
    const int i0 = run_start(items, warp);
    bool more = false;
    int pass = 0;
    do {
      if (many) {  // (out of the way of the usual call: as part of its start, 1 token, 14336 x 4096, 10.0 us, not 9.0)
        copies_wait<0>();
        ltile = tile0, left = run = at = 0;  // the loads start again with this batch
        if (threadIdx.x < kMatvecMaxTokens) {
          uint32_t &c = cur[threadIdx.x], &l = limit[threadIdx.x], &n = next[threadIdx.x];
          l = pass == 0 ? 0xFFFFFFFFu : n == 0u ? 0u : lowest_exactly(mx8, down_exponent<MX>(c));
          c = pass == 0 ? top[threadIdx.x] : n;
          n = 0u;
        }
        __syncthreads();
        set_factors(cur);
        stager.fetch();
#pragma unroll 1
        for (int d = 0; d < kDepth; ++d) load(d * Ring::kBytes);
        copies_wait<kDepth>();
        stager.stage_below(mx8, cur, limit, next);
        __syncthreads();
        more = false;
        for (int m = 0; m < M; ++m) more = more || next[m] != 0u;
      }
      int todo = run_start(items, warp + 1) - i0;
      int ti = i0 / chunks, c = i0 - ti * chunks;
      while (todo > 0) {
        const int stop = min(chunks, c + todo);
        todo -= stop - c;
        if (lane == 0) {
          if (c == 0) first[ti] = static_cast<uint8_t>(warp);
          if (stop == chunks) last[ti] = static_cast<uint8_t>(warp);
        }
        float acc[R][NT][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[r][n][0] = acc[r][n][1] = acc[r][n][2] = acc[r][n][3] = 0.0f;
#pragma unroll 1
        for (; c < stop; ++c) {
          copies_wait<kDepth - 1>();
          __syncwarp();  // every lane's copies of this item have landed
          uint32_t wa[R][WORDS], wb[R][WORDS];
          uint32_t ha[R][WORDS / 2], hb[R][WORDS / 2];  // NVFP4: block scales, twice each
          float fa[R][WORDS], fb[R][WORDS];             // MXFP4: block scales
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint32_t src = codes_at + at + r * 16 * Ring::kRow, ssrc = scales_at + at + r * 64;
            if constexpr (MX) {
              // word j: lane t's word of the chunk's block j
#pragma unroll
              for (int j = 0; j < WORDS; j += 2)
                ldmatrix4(src ^ (j << 4), wa[r][j], wb[r][j], wa[r][j + 1], wb[r][j + 1]);
#pragma unroll
              for (int h = 0; h < WORDS / 4; ++h) {
                const uint32_t sca = ld_shared4(ssrc + 64 * R * h), scb = ld_shared4(ssrc + 64 * R * h + 32);
                const uint32_t by = exp2_bf16x2(-kScaleShift<MX>);
                e8m0x2_to_float(sca & 0xFFFFu, by, fa[r][4 * h], fa[r][4 * h + 1]);
                e8m0x2_to_float(sca >> 16, by, fa[r][4 * h + 2], fa[r][4 * h + 3]);
                e8m0x2_to_float(scb & 0xFFFFu, by, fb[r][4 * h], fb[r][4 * h + 1]);
                e8m0x2_to_float(scb >> 16, by, fb[r][4 * h + 2], fb[r][4 * h + 3]);
              }
            } else {
              // word j: codes 8 j .. of the lane's own 32 (16) bytes of the row
#pragma unroll
              for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 a = ld_shared16(src ^ (i << 4));
                const uint4 b = ld_shared16((src ^ (i << 4)) + 8 * Ring::kRow);
                wa[r][4 * i] = a.x, wa[r][4 * i + 1] = a.y, wa[r][4 * i + 2] = a.z, wa[r][4 * i + 3] = a.w;
                wb[r][4 * i] = b.x, wb[r][4 * i + 1] = b.y, wb[r][4 * i + 2] = b.z, wb[r][4 * i + 3] = b.w;
              }
              uint32_t sca = ld_shared4(ssrc), scb = ld_shared4(ssrc + 32);
              if constexpr (WORDS == 4) {
                sca >>= 16 * (t & 1);
                scb >>= 16 * (t & 1);
              }
#pragma unroll
              for (int h = 0; h < WORDS / 4; ++h) {
                const uint32_t a2 = e4m3x2_to_half2((sca >> (16 * h)) & 0xFFFFu);
                const uint32_t b2 = e4m3x2_to_half2((scb >> (16 * h)) & 0xFFFFu);
                ha[r][2 * h] = __byte_perm(a2, 0u, 0x1010), ha[r][2 * h + 1] = __byte_perm(a2, 0u, 0x3232);
                hb[r][2 * h] = __byte_perm(b2, 0u, 0x1010), hb[r][2 * h + 1] = __byte_perm(b2, 0u, 0x3232);
              }
            }
          }
          __syncwarp();  // the slot has been read by every lane
          load(at);
          at = at == (kDepth - 1) * Ring::kBytes ? 0 : at + Ring::kBytes;
          const uint32_t xc = (c / kPerUnit) * M * 512 + (c % kPerUnit) * (WORDS * 64);
#pragma unroll
          for (int j = 0; j < WORDS; ++j) {
            uint4 x[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
              x[n] = ld_shared16(x_at[n] + xc + (j & 1 ? 0u - x_flip[n] : x_flip[n]) + j * 64);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              uint32_t a[4], b[4];
              codes_to_half(wa[r][j], a);
              codes_to_half(wb[r][j], b);
#pragma unroll
              for (int i = 0; i < 4 && !MX; ++i) {
                a[i] = mul_half2(a[i], ha[r][j >> 1]);
                b[i] = mul_half2(b[i], hb[r][j >> 1]);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float(&d)[4] = acc[r][n];
                if constexpr (MX) {
                  float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma(q, a[0], b[0], a[1], b[1], x[n].x, x[n].y);
                  mma(q, a[2], b[2], a[3], b[3], x[n].z, x[n].w);
                  d[0] = __fmaf_rn(q[0], fa[r][j], d[0]);
                  d[1] = __fmaf_rn(q[1], fa[r][j], d[1]);
                  d[2] = __fmaf_rn(q[2], fb[r][j], d[2]);
                  d[3] = __fmaf_rn(q[3], fb[r][j], d[3]);
                } else {
                  mma(d, a[0], b[0], a[1], b[1], x[n].x, x[n].y);
                  mma(d, a[2], b[2], a[3], b[3], x[n].z, x[n].w);
                }
              }
            }
          }
        }
        float* out = part + (ti + warp) * slot + g;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int m = 8 * n + 2 * t + (i & 1);
              if (m < M) {
                float& o = out[(r * M + m) * kPad + 8 * (i >> 1)];
                float v = acc[r][n][i];
                if (many) {  // the passes meet under their factors
                  const float2 f = factors[GATED && i < 2 ? kMatvecMaxTokens + m : m];
                  v = v * f.x * f.y + (pass == 0 ? 0.0f : o);
                }
                o = v;
              }
            }
        c = 0;
        ++ti;
      }
      if (many) {
        __syncthreads();  // x, `next` and the factors have been read
        ++pass;
        more = more && pass < kMaxPasses;
        if (!more && threadIdx.x < 2 * kMatvecMaxTokens) factors[threadIdx.x] = make_float2(1.0f, 1.0f);
      }
    } while (more);
    __syncthreads();
    // Outputs, four to a thread: i = (group of 16 rows, token, line), the line's rows of the
    // four quarters.
    constexpr int kOut = GATED ? 2 : 4;  // lines of a 16-row group
    const int outputs = nt * R * kOut * M;
    const int out_line = lane % kOut;
    // sums of output i over the warps that had a part of its tile (gated: both products), under the
    // tensor scale and with the token's scaling undone
    auto sum = [&](int i, float4& s, float4& v) {
      const int tr = div_m(p, i / kOut), m = i / kOut - tr * M, ti = tr / R;
      const int w0 = first[ti], w1 = last[ti];
      const float* q = part + ((ti + w0) * R + tr % R) * (M * kPad) + m * kPad + 4 * out_line;
      s = *reinterpret_cast<const float4*>(q);
      if (GATED) v = *reinterpret_cast<const float4*>(q + 8);
      for (int w = w0; w < w1; ++w) {
        q += slot;
        s = add4(s, *reinterpret_cast<const float4*>(q));
        if (GATED) v = add4(v, *reinterpret_cast<const float4*>(q + 8));
      }
      const float2 f = factors[GATED ? kMatvecMaxTokens + m : m];
      s = make_float4(s.x * f.x * f.y, s.y * f.x * f.y, s.z * f.x * f.y, s.w * f.x * f.y);
      if (GATED) {
        const float2 h = factors[m];
        v = make_float4(v.x * h.x * h.y, v.y * h.x * h.y, v.z * h.x * h.y, v.w * h.x * h.y);
      }
    };
    auto write = [&](int i, float4 s, float4 v) {
      const int tr = div_m(p, i / kOut), m = i / kOut - tr * M;
      const int line = tile0 * kLines + tr * (kLines / R) + out_line;
      const int row = (line >> 5) * 128 + (line & 31);
      uint16_t* const y = p.a.out + m * p.a.ld_out + row;
      const float ss[4] = {s.x, s.y, s.z, s.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = GATED ? silu_times_short(ss[k], vv[k]) : ss[k];
        if (row + 32 * k < N) y[32 * k] = static_cast<uint16_t>(pack_bf16(f, 0.0f));
      }
    };
    if (p.split == 1) {
      for (int i = threadIdx.x; i < outputs; i += kThreads) {
        float4 s, v = {};
        sum(i, s, v);
        write(i, s, v);
      }
    } else {
      // 32 threads' outputs at a time belong to one CTA of the cluster in turn: every CTA puts
      // its sums into the owner's memory (that of x when it is no longer needed), 16 bytes a
      // store, and the owner adds them in rank order
      if (p.sums_over_x) {
        cluster_sync();  // every CTA is through with its items
      } else if (tile0 == T0) {
        cluster_wait();  // every CTA has started
      }
      float4* sums = reinterpret_cast<float4*>(smem + p.sums_at);
      const int shift = __ffs(p.split) - 1;                                 // split is a power of two
      const int mine = ((outputs + 32 * p.split - 1) >> (5 + shift)) << 5;  // outputs per CTA, at most
      const uint32_t my_sums = smem_u32(sums + rank * mine + lane);
      for (int b = warp; b * 32 < outputs; b += W) {
        if (b * 32 + lane < outputs) {
          float4 s, v;
          sum(b * 32 + lane, s, v);
          const uint32_t dst = mapa_shared(my_sums + (b >> shift) * 512, b & (p.split - 1));
          st_shared_cluster(dst, s);
          if (GATED) st_shared_cluster(dst + 16 * p.split * mine, v);
        }
      }
      cluster_sync();
      for (int b = warp; b * 32 < mine; b += W) {
        const int i = ((b << shift) + rank) * 32 + lane;
        if (i >= outputs) break;
        float4 s = {}, v = {};
        for (int k = 0; k < p.split; ++k) {
          s = add4(s, sums[k * mine + b * 32 + lane]);
          if (GATED) v = add4(v, sums[(p.split + k) * mine + b * 32 + lane]);
        }
        write(i, s, v);
      }
      if (tile0 + p.batch < T1) cluster_sync();  // the sums may be overwritten
    }
    __syncthreads();  // the slots may be overwritten
  }
}

template <bool MX, int NT, bool GATED, int WORDS, int R>
cudaError_t launch_one(const Params& p, int grid, int threads, size_t smem, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool raised[64];  // per device: the kernel may use more than 48 KB (idempotent)
  if (dev >= 64 || !raised[dev]) {
    e = cudaFuncSetAttribute(matvec_kernel<MX, NT, GATED, WORDS, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) raised[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, matvec_kernel<MX, NT, GATED, WORDS, R>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The kernel's shapes.  kNarrow: K no multiple of 64.  kPaired: more than 8 tokens, whose x
// costs shared memory twice the reads: two 16-row groups share them (16 tokens: 5376 x 21504
// 26.3 us against 26.9 with kWide's tiles, 21504 x 5376 22.9 / 23.3, 1024 x 4096 5.0 / 4.7;
// 8 tokens, 14336 x 4096: 12.8 / 12.1).
enum Shape { kWide, kNarrow, kPaired };

template <bool MX>
size_t ring_bytes(Shape s) {
  return static_cast<size_t>(kWarps) * kDepth *
         (s == kWide ? ItemBytes<MX, 8, 1>::kBytes : s == kNarrow ? ItemBytes<MX, 4, 1>::kBytes
                                                                  : ItemBytes<MX, 4, 2>::kBytes);
}

template <bool MX, bool GATED>
cudaError_t launch_format(const Params& p, Shape s, int grid, size_t smem, cudaStream_t stream) {
  if (s == kWide) return launch_one<MX, 1, GATED, 8, 1>(p, grid, kThreads, smem, stream);
  if (s == kNarrow) return launch_one<MX, 1, GATED, 4, 1>(p, grid, kThreads, smem, stream);
  return launch_one<MX, 2, GATED, 4, 2>(p, grid, kThreads, smem, stream);
}

// Shared memory of a launch: rings, x, then slots for as many tiles as fit, at most `tiles`
// of them (0: not even one), and a cluster's sums -- in x's place when that, and only that,
// lets one batch be all.
struct Plan {
  int tiles;
  size_t smem, sums_at;
  bool over_x;
};

Plan plan(int M, int x_units, int tiles, int split, size_t ring, int R) {
  const size_t x = static_cast<size_t>(x_units) * M * 512, slot = static_cast<size_t>(M) * kPad * R * 4;
  const size_t fixed = ring + x + kTokenWords * 4 + 16 + kWarps * slot;
  if (fixed + slot + 2 > kSmem) return {0, 0, 0, false};
  const int slots = static_cast<int>(std::min<size_t>(tiles, (kSmem - fixed) / (slot + 2)));
  if (split == 1) return {slots, fixed + slots * (slot + 2), 0, false};
  // sums: 16 R per tile and token, in whole rounds of 32 threads' and the cluster's CTAs
  const size_t round = static_cast<size_t>(split) * 32 * 16 * 2 + 16, sum = static_cast<size_t>(M) * 64 * R;
  size_t n = fixed + round > kSmem ? 0 : (kSmem - fixed - round) / (slot + 2 + sum);
  if (n < static_cast<size_t>(tiles) && slots == tiles && tiles * sum + round <= x)
    return {tiles, fixed + tiles * (slot + 2), ring, true};
  n = std::min<size_t>(n, tiles);
  const size_t at = (fixed + n * (slot + 2) + 15) / 16 * 16;
  return {static_cast<int>(n), at + round + n * sum, at, false};
}

}  // namespace

namespace {

// The launch of so many tokens: whether x of them fits any split, then its shape and parameters.
struct Launch {
  Params p;
  Shape shape;
  int groups;
  size_t smem;
};

bool prepare(const MatvecArgs& a, Launch& l) {
  l = {};
  Params& p = l.p;
  p.a = a;
  const bool gated = a.gate.codes != nullptr;
  l.shape = a.M > 8 ? kPaired : a.K % 64 == 0 ? kWide : kNarrow;
  const int R = l.shape == kPaired ? 2 : 1;
  const int64_t tail = a.N % 128;
  const int lines_per_tile = (gated ? 2 : 4) * R;
  const int64_t lines = a.N / 128 * 32 + (tail < 32 ? tail : 32);  // neighbour lines, 4 rows each
  p.tiles = static_cast<int>((lines + lines_per_tile - 1) / lines_per_tile);
  p.units = static_cast<int>((a.K + kUnit - 1) / kUnit);
  p.atoms = static_cast<int>((a.K / (a.mx ? 32 : 16) + 3) / 4);
  const size_t ring = a.mx ? ring_bytes<true>(l.shape) : ring_bytes<false>(l.shape);
  // CTAs per cluster: the fewest items for the busiest CTA among the splits whose part of x
  // fits.  Clusters that the GPU holds at a time, of CTAs that fill an SM: 148, 74, 33, 15.
  static const int kSplits[4] = {1, 2, 4, 8}, kGroups[4] = {148, 74, 33, 15};
  int64_t best = -1;
  for (int i = 0; i < 4; ++i) {
    const int s = kSplits[i], n = p.tiles < kGroups[i] ? p.tiles : kGroups[i];
    const int x_units = (p.units + s - 1) / s, tiles = (p.tiles + n - 1) / n;
    const Plan q = plan(a.M, x_units, tiles, s, ring, R);
    // (in quarters of the time of an item of 16 x 256 weights: a unit of a token to stage 1, a
    // cluster's barriers, and its wait for the slowest CTA, 8)
    const int64_t items = static_cast<int64_t>(tiles) * x_units * R, pieces = static_cast<int64_t>(x_units) * a.M;
    const int64_t cost = (items * 4 + kWarps - 1) / kWarps + (pieces + kWarps - 1) / kWarps + (s > 1 ? 8 : 0);
    if (q.tiles == 0 || s > p.units || (best >= 0 && cost >= best)) continue;
    best = cost;
    p.split = s;
    p.batch = q.tiles;
    p.x_units = x_units;
    l.groups = n;
    l.smem = q.smem;
    p.sums_at = static_cast<int>(q.sums_at);
    p.sums_over_x = q.over_x;
  }
  if (best < 0) return false;
  p.m_inv = static_cast<uint32_t>(((uint64_t{1} << 32) + a.M - 1) / a.M);
  p.tiles_q = p.tiles / l.groups, p.tiles_r = p.tiles % l.groups;
  p.units_q = p.units / p.split, p.units_r = p.units % p.split;
  return true;
}

}  // namespace

bool plan_matvec(const MatvecArgs& a, MatvecPlan* plan) {
  Launch l;
  if (!prepare(a, l)) {
    if (a.M == 1) return false;
    MatvecArgs first = a, second = a;
    first.M = a.M / 2;
    second.M = a.M - first.M;
    MatvecPlan rest;
    if (!plan_matvec(second, &rest) || !plan_matvec(first, plan)) return false;
    plan->launches += rest.launches;
    return true;
  }
  const int tiles = l.p.tiles_q + (l.p.tiles_r > 0);
  *plan = {l.p.split, (tiles + l.p.batch - 1) / l.p.batch, l.p.sums_over_x, 1};
  return true;
}

cudaError_t launch_matvec(const MatvecArgs& a, int* launches, cudaStream_t stream) {
  Launch l;
  if (!prepare(a, l)) {  // x of this many tokens fits no split: half of them at a time
    if (a.M == 1) return cudaErrorInvalidValue;
    MatvecArgs first = a, second = a;
    first.M = a.M / 2;
    second.M = a.M - first.M;
    const int64_t bytes = a.x_scales ? 1 : 2;
    second.x = static_cast<const uint8_t*>(a.x) + first.M * a.ld_x * bytes;
    second.x_row0 += first.M;
    second.out = a.out + first.M * a.ld_out;
    const cudaError_t e = launch_matvec(first, launches, stream);
    return e != cudaSuccess ? e : launch_matvec(second, launches, stream);
  }
  const int grid = l.groups * l.p.split;
  ++*launches;
  const bool gated = a.gate.codes != nullptr;
  if (a.mx) return gated ? launch_format<true, true>(l.p, l.shape, grid, l.smem, stream)
                         : launch_format<true, false>(l.p, l.shape, grid, l.smem, stream);
  return gated ? launch_format<false, true>(l.p, l.shape, grid, l.smem, stream)
               : launch_format<false, false>(l.p, l.shape, grid, l.smem, stream);
}

}  // namespace nvfp4
