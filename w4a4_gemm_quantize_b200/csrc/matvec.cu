// matvec.cu -- y = x W^T for 1 to 16 tokens, W in 4 bits (NVFP4 or MXFP4), x in BF16 or
// MXFP8, y in BF16; with a second weight, y = silu(x G^T) * (x W^T) in the same pass.
//   y[m, n] = s_g sum_k x[m, k] q[n, k] s[n, k / G],  G = 16 (E4M3 s) or 32 (E8M0 s).
//
// Bound: the weight stream, N K (1/2 + 1/G) bytes from HBM; the products ride along on
// mma.sync m16n8k16 (f16 x f16 -> f32): 16 weight rows x 8 tokens, so up to 8 tokens cost
// what one does.
//
// Exactness: an E2M1 code times an E4M3 scale has at most 6 significant bits and lies in
// [2^-10, 2688], so NVFP4 weights are exact in binary16.  E8M0 scales do not fit
// binary16; there the mma runs on the bare codes of one block and the binary32 partial
// product is multiplied by the block's power of two.  x becomes binary16 scaled by a
// power of two per token and K slice, its largest finite magnitude in [2^7, 2^8): values
// down to 2^-21 of that largest one keep all their bits, smaller ones are rounded at
// 2^-32 of it, below the binary32 sum's own rounding.  Sums are binary32 throughout.
//
// Layout: the K axis is cut into chunks of 128 values, dealt round-robin to the CTA's
// warps; a warp keeps its chunks of x in shared memory as mma fragments and walks down
// the CTA's weight rows, 16 at a time, each lane loading 16 bytes (32 codes) of two
// rows.  The mma's k order is free as long as both operands agree, so the fragments are
// cut to what a lane has loaded: no shuffles for NVFP4, and a 4 x 4 word transpose
// within the quad for MXFP4 (each mma then stays inside one scale block).  Row order is
// free too: a tile's 16 rows are 4 neighbours in each of the 4 row quarters of a
// 128-row group, whose scales lie in 64 contiguous bytes per 4 blocks.  A CTA owns a
// run of such neighbour lines, so that rows divide over the SMs to within 4.  At the end
// the warps' partial sums meet in shared memory in a fixed order: no atomics, no
// workspace, the same bits on every call.
#include <cuda_runtime.h>

#include "layer_ops.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kChunk = 128;      // K values of one warp step
constexpr int kMaxWarps = 16;
constexpr int kDepth = 4;        // weight steps in flight per warp
constexpr int kPad = 20;         // floats per token of a 16-row partial (padded: conflict-free)
constexpr int kMaxSlice = 12;    // chunks of x a warp holds at a time, at most
constexpr int kXBytes = 10240;   // shared memory for them, per warp
constexpr int kSmem = 220 * 1024;

struct Params {
  MatvecArgs a;
  int64_t lines;      // 4-row neighbour lines of the weight
  int chunks;         // ceil(K / 128)
  int slice;          // chunks of x per warp and slice
  int batch;          // row tiles between two reductions
  int64_t atoms;      // scale atoms (4 blocks) per 128-row group
  uint32_t last_mask; // MXFP4: the scale bytes of the last chunk that are blocks of the row
};

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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

__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  return d;
}

// two E8M0 bytes as floats (exact; 255 is NaN)
__device__ __forceinline__ void e8m0x2_to_float(uint32_t two, float& lo, float& hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
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

// w[b] of lane t <- w[t] of lane b, within each quad of lanes
__device__ __forceinline__ void transpose_quad(uint32_t (&w)[4], int t) {
  const bool odd = t & 1, high = t & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t r = __shfl_xor_sync(0xFFFFFFFFu, odd ? w[i] : w[i + 1], 1);
    (odd ? w[i] : w[i + 1]) = r;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t r = __shfl_xor_sync(0xFFFFFFFFu, high ? w[i] : w[i + 2], 2);
    (high ? w[i] : w[i + 2]) = r;
  }
}

// Eight consecutive values of x: BF16 (16 bytes) or E4M3 with their scale byte.
struct Piece {
  uint4 v;
  uint32_t scale;
};

__device__ __forceinline__ Piece load_piece(const MatvecArgs& a, int m, int64_t k) {
  Piece p{make_uint4(0u, 0u, 0u, 0u), 127u};
  if (k >= a.K) return p;
  if (a.x_scales == nullptr) {
    p.v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + m * a.ld_x + k));
  } else {
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + m * a.ld_x + k));
    p.v.x = c.x;
    p.v.y = c.y;
    const int64_t b = k >> 5;
    p.scale = __ldg(a.x_scales + (a.x_swizzled ? (b >> 2) * 512 + m * 16 + (b & 3) : m * (a.K >> 5) + b));
  }
  return p;
}

__device__ __forceinline__ void piece_values(const Piece& p, bool fp8, float (&v)[8]) {
  if (!fp8) {
    const uint32_t w[4] = {p.v.x, p.v.y, p.v.z, p.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    float s, unused;
    e8m0x2_to_float(p.scale, s, unused);
    const uint32_t w[2] = {p.v.x, p.v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = e4m3x2_to_half2((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
      float lo, hi;
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}\n"
          : "=f"(lo), "=f"(hi)
          : "r"(h));
      v[2 * i] = lo * s;
      v[2 * i + 1] = hi * s;
    }
  }
}

// Puts x's chunks first, first + W, ... (n of them) of every token into the warp's shared
// memory as scaled binary16 mma fragments: 16 bytes for (chunk, word j, token, lane t)
// hold the 8 values from k = 32 t + 8 j (NVFP4) or 32 j + 8 t (MXFP4) of the chunk.
// mult[m] = the power of two that undoes token m's scaling.
template <bool MX>
__device__ __noinline__ void stage_x(const Params& p, int first, int W, int n, uint4* xs, float* mult) {
  const int lane = threadIdx.x & 31;
  const bool fp8 = p.a.x_scales != nullptr;
  const int M = p.a.M, pieces = n * 16;
  for (int m = 0; m < M; ++m) {
    Piece q[kMaxSlice / 2];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kMaxSlice / 2; ++i) {
      const int id = lane + 32 * i;
      if (id >= pieces) break;
      const int64_t k = static_cast<int64_t>(first + (id >> 4) * W) * kChunk + (id & 15) * 8;
      q[i] = load_piece(p.a, m, k);
    }
#pragma unroll
    for (int i = 0; i < kMaxSlice / 2; ++i) {
      if (lane + 32 * i >= pieces) break;
      float v[8];
      piece_values(q[i], fp8, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
        top = max(top, b < 0x7F800000u ? b : 0u);  // infinities and NaN keep to themselves
      }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    // the largest magnitude 2^e.. goes to [2^7, 2^8); E stays a binary32 exponent
    const int E = top == 0u ? 0 : max(-126, static_cast<int>(top >> 23) - 127 - 7);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - E) << 23);
    if (lane == 0) mult[m] = __uint_as_float(static_cast<uint32_t>(127 + E) << 23);
#pragma unroll
    for (int i = 0; i < kMaxSlice / 2; ++i) {
      const int id = lane + 32 * i;
      if (id >= pieces) break;
      float v[8];
      piece_values(q[i], fp8, v);
      uint4 h;
      h.x = pack_half(v[0] * down, v[1] * down);
      h.y = pack_half(v[2] * down, v[3] * down);
      h.z = pack_half(v[4] * down, v[5] * down);
      h.w = pack_half(v[6] * down, v[7] * down);
      const int c = id >> 4, o = id & 15;
      const int j = MX ? o >> 2 : o & 3, t = MX ? o & 3 : o >> 2;
      xs[((c * 4 + j) * M + m) * 4 + t] = h;
    }
  }
}

// 128 K values of a lane's two weight rows: 32 codes each, and their scales (NVFP4: the
// two bytes of the lane's blocks; MXFP4: the four bytes of the chunk's blocks).
struct Step {
  uint4 a, b;
  uint32_t sa, sb;
};

template <bool MX, int NT, bool GATED>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) matvec_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float mults[kMaxWarps][kMatvecMaxTokens];
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int kLines = GATED ? 2 : 4;  // neighbour lines of a 16-row tile
  const int W = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int M = p.a.M;
  uint4* xs = reinterpret_cast<uint4*>(smem) + static_cast<size_t>(warp) * p.slice * M * 16;
  float* part = reinterpret_cast<float*>(smem + static_cast<size_t>(W) * p.slice * M * 256);
  float* mult = mults[warp];
  const int64_t l0 = p.lines * blockIdx.x / gridDim.x, l1 = p.lines * (blockIdx.x + 1) / gridDim.x;
  const int tiles = static_cast<int>((l1 - l0 + kLines - 1) / kLines);
  const int mine = p.chunks > warp ? (p.chunks - warp + W - 1) / W : 0;  // chunks of this warp
  const int64_t row_bytes = p.a.K / 2;

  for (int tile0 = 0; tile0 < tiles; tile0 += p.batch) {
    const int nt = min(p.batch, tiles - tile0);
    if (mine > 0) {
      // the load side of the pipeline runs kDepth steps ahead of the compute side, both
      // through slices (outermost), tiles, chunks
      int ls = 0, lt = 0, lj = 0;  // first chunk of the slice, tile, chunk
      const uint8_t *pa = nullptr, *pb = nullptr, *sa = nullptr, *sb = nullptr;
      bool va = false, vb = false, more = true;
      auto rows_of_tile = [&]() {
        const int64_t line = l0 + static_cast<int64_t>(tile0 + lt) * kLines + (g >> 2);
        const int64_t lb = GATED ? line : line + 2;
        const int64_t ra = (line >> 5) * 128 + (line & 31) + 32 * (g & 3);
        const int64_t rb = (lb >> 5) * 128 + (lb & 31) + 32 * (g & 3);
        va = line < l1 && ra < p.a.N;
        vb = lb < l1 && rb < p.a.N;
        const Weight4& wa = GATED ? p.a.gate : p.a.w;
        pa = wa.codes + ra * row_bytes + t * 16;
        pb = p.a.w.codes + rb * row_bytes + t * 16;
        const int lane_off = (MX ? 0 : (t >> 1) * 512 + (t & 1) * 2) + (g & 3) * 4;
        sa = wa.scales + (line >> 5) * p.atoms * 512 + (line & 31) * 16 + lane_off;
        sb = p.a.w.scales + (lb >> 5) * p.atoms * 512 + (lb & 31) * 16 + lane_off;
      };
      rows_of_tile();
      auto load = [&](Step& s) {
        s.a = s.b = make_uint4(0u, 0u, 0u, 0u);
        s.sa = s.sb = 0u;
        if (!more) return;
        const int c = warp + (ls + lj) * W;
        const bool in = c * static_cast<int64_t>(kChunk) + 32 * t < p.a.K;
        const int64_t co = static_cast<int64_t>(c) * (kChunk / 2);
        const int64_t so = static_cast<int64_t>(c) * (MX ? 512 : 1024);
        if (va && in) s.a = ld_stream(pa + co);
        if (vb && in) s.b = ld_stream(pb + co);
        if constexpr (MX) {
          if (va) s.sa = __ldg(reinterpret_cast<const uint32_t*>(sa + so));
          if (vb) s.sb = __ldg(reinterpret_cast<const uint32_t*>(sb + so));
          if (c == p.chunks - 1) {  // the padding's bytes, whatever they hold, scale zero codes
            s.sa &= p.last_mask;
            s.sb &= p.last_mask;
          }
        } else {
          if (va && in) s.sa = __ldg(reinterpret_cast<const uint16_t*>(sa + so));
          if (vb && in) s.sb = __ldg(reinterpret_cast<const uint16_t*>(sb + so));
        }
        if (++lj == min(p.slice, mine - ls)) {
          lj = 0;
          if (++lt == nt) {
            lt = 0;
            ls += p.slice;
            more = ls < mine;
          }
          if (more) rows_of_tile();
        }
      };
      Step ring[kDepth];
#pragma unroll
      for (int d = 0; d < kDepth; ++d) load(ring[d]);

      int cs = 0, ct = 0, cj = 0;
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
      bool done = false;
      while (!done) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          if (done) break;
          if (cj == 0 && ct == 0) {  // a new slice of x
            __syncwarp();            // every lane is through with the last one
            stage_x<MX>(p, warp + cs * W, W, min(p.slice, mine - cs), xs, mult);
            __syncwarp();
          }
          Step& s = ring[d];
          uint32_t wa[4] = {s.a.x, s.a.y, s.a.z, s.a.w}, wb[4] = {s.b.x, s.b.y, s.b.z, s.b.w};
          uint32_t ha2[2], hb2[2];
          float fa[4], fb[4];
          if constexpr (MX) {
            transpose_quad(wa, t);
            transpose_quad(wb, t);
            e8m0x2_to_float(s.sa & 0xFFFFu, fa[0], fa[1]);
            e8m0x2_to_float(s.sa >> 16, fa[2], fa[3]);
            e8m0x2_to_float(s.sb & 0xFFFFu, fb[0], fb[1]);
            e8m0x2_to_float(s.sb >> 16, fb[2], fb[3]);
          } else {
            const uint32_t a2 = e4m3x2_to_half2(s.sa), b2 = e4m3x2_to_half2(s.sb);
            ha2[0] = __byte_perm(a2, 0u, 0x1010), ha2[1] = __byte_perm(a2, 0u, 0x3232);
            hb2[0] = __byte_perm(b2, 0u, 0x1010), hb2[1] = __byte_perm(b2, 0u, 0x3232);
          }
          load(s);  // the slot is free
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a[4], b[4];
            codes_to_half(wa[j], a);
            codes_to_half(wb[j], b);
            if constexpr (!MX) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                a[i] = mul_half2(a[i], ha2[j >> 1]);
                b[i] = mul_half2(b[i], hb2[j >> 1]);
              }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int m = g + 8 * n;
              uint4 x = make_uint4(0u, 0u, 0u, 0u);
              if (m < M) x = xs[((cj * 4 + j) * M + m) * 4 + t];
              if constexpr (MX) {
                float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma(q, a[0], b[0], a[1], b[1], x.x, x.y);
                mma(q, a[2], b[2], a[3], b[3], x.z, x.w);
                acc[n][0] = __fmaf_rn(q[0], fa[j], acc[n][0]);
                acc[n][1] = __fmaf_rn(q[1], fa[j], acc[n][1]);
                acc[n][2] = __fmaf_rn(q[2], fb[j], acc[n][2]);
                acc[n][3] = __fmaf_rn(q[3], fb[j], acc[n][3]);
              } else {
                mma(acc[n], a[0], b[0], a[1], b[1], x.x, x.y);
                mma(acc[n], a[2], b[2], a[3], b[3], x.z, x.w);
              }
            }
          }
          if (++cj == min(p.slice, mine - cs)) {  // the tile's share of this slice
            cj = 0;
            float* out = part + static_cast<size_t>(ct * W + warp) * M * kPad;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int m = 8 * n + 2 * t + (i & 1);
                if (m < M) {
                  float* q = out + m * kPad + g + 8 * (i >> 1);
                  const float v = acc[n][i] * mult[m];
                  *q = cs == 0 ? v : *q + v;
                }
                acc[n][i] = 0.0f;
              }
            }
            if (++ct == nt) {
              ct = 0;
              cs += p.slice;
              done = cs >= mine;
            }
          }
        }
      }
    }
    __syncthreads();
    constexpr int kRows = GATED ? 8 : 16;  // outputs of a tile per token
    const float sw = p.a.w.gs ? *p.a.w.gs : 1.0f, sgate = GATED && p.a.gate.gs ? *p.a.gate.gs : 1.0f;
    for (int i = threadIdx.x; i < nt * kRows * M; i += blockDim.x) {
      const int r = i % kRows, m = (i / kRows) % M, ti = i / (kRows * M);
      const float* q = part + static_cast<size_t>(ti) * W * M * kPad + m * kPad + r;
      float s = 0.0f, u = 0.0f;
      for (int w = 0; w < W; ++w) {
        s += q[w * M * kPad];
        if (GATED) u += q[w * M * kPad + 8];
      }
      const int64_t line = l0 + static_cast<int64_t>(tile0 + ti) * kLines + (r >> 2);
      const int64_t row = (line >> 5) * 128 + (line & 31) + 32 * (r & 3);
      if (line >= l1 || row >= p.a.N) continue;
      float y;
      if (GATED) {
        const float gt = s * sgate;
        y = gt / (1.0f + expf(-gt)) * (u * sw);
      } else {
        y = s * sw;
      }
      p.a.out[m * p.a.ld_out + row] = static_cast<uint16_t>(pack_bf16(y, 0.0f));
    }
    __syncthreads();  // the partial sums may be overwritten
  }
}

template <bool MX, int NT, bool GATED>
cudaError_t launch_one(const Params& p, int grid, int threads, size_t smem, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool raised[64];  // per device: the kernel may use more than 48 KB (idempotent)
  if (dev >= 64 || !raised[dev]) {
    e = cudaFuncSetAttribute(matvec_kernel<MX, NT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) raised[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, matvec_kernel<MX, NT, GATED>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool MX>
cudaError_t launch_format(const Params& p, int grid, int threads, size_t smem, cudaStream_t stream) {
  const bool gated = p.a.gate.codes != nullptr;
  if (p.a.M <= 8)
    return gated ? launch_one<MX, 1, true>(p, grid, threads, smem, stream)
                 : launch_one<MX, 1, false>(p, grid, threads, smem, stream);
  return gated ? launch_one<MX, 2, true>(p, grid, threads, smem, stream)
               : launch_one<MX, 2, false>(p, grid, threads, smem, stream);
}

}  // namespace

cudaError_t launch_matvec(const MatvecArgs& a, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.chunks = static_cast<int>((a.K + kChunk - 1) / kChunk);
  const int W = p.chunks < kMaxWarps ? p.chunks : kMaxWarps;
  const int per_sm = kMaxWarps / W;  // CTAs of short rows share an SM
  const int64_t tail = a.N % 128;
  p.lines = a.N / 128 * 32 + (tail < 32 ? tail : 32);
  p.atoms = ((a.K / (a.mx ? 32 : 16)) + 3) / 4;
  const int last_blocks = static_cast<int>(a.K / 32 - (p.chunks - 1) * int64_t{4});
  p.last_mask = last_blocks == 4 ? 0xFFFFFFFFu : (1u << (8 * last_blocks)) - 1u;
  int dev = 0, sms = 148;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t slots = static_cast<int64_t>(sms) * per_sm;
  const int grid = static_cast<int>(p.lines < slots ? p.lines : slots);
  // x: as many of a warp's chunks as its share of shared memory holds, in equal slices
  const int per_warp = (p.chunks + W - 1) / W;
  int most = kXBytes / (a.M * 256);
  if (most > kMaxSlice) most = kMaxSlice;
  const int slices = (per_warp + most - 1) / most;
  p.slice = (per_warp + slices - 1) / slices;
  // partial sums: as many tiles as the rest holds
  const size_t x_bytes = static_cast<size_t>(W) * p.slice * a.M * 256;
  const size_t tile_bytes = static_cast<size_t>(W) * a.M * kPad * sizeof(float);
  const int lines_per_tile = a.gate.codes ? 2 : 4;
  const int64_t tiles = ((p.lines + grid - 1) / grid + lines_per_tile - 1) / lines_per_tile;
  const int64_t room = static_cast<int64_t>((kSmem / per_sm - x_bytes) / tile_bytes);
  p.batch = static_cast<int>(tiles < room ? tiles : room);
  const size_t smem = x_bytes + p.batch * tile_bytes;
  return a.mx ? launch_format<true>(p, grid, W * 32, smem, stream) : launch_format<false>(p, grid, W * 32, smem, stream);
}

}  // namespace nvfp4
