// layer_ops.h -- host-side declarations of the decoder-layer operators' launchers
// (row_ops.cu, matvec.cu), called by the entry points in layer_api.cu with arguments
// that are already validated.  All pointers are device pointers.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace nvfp4 {

// Where a row operator's output goes.  format: nvfp4_out_format.  BF16: out with row
// stride ld_out elements; the block formats: dense codes in out, one scale byte per
// block in scales (128 x 4 tiles when swizzled, else row-major).
struct RowOutput {
  void* out;
  int64_t ld_out;
  uint8_t* scales;
  bool swizzled;
  int format;
  const float* gs_in;  // NVFP4: the given tensor scale, or null: computed from the output's amax
  float* gs_out;       // NVFP4: receives the tensor scale (may be null)
  unsigned long long* amax_word;  // NVFP4 without gs_in: scratch for the output's amax (binary64)
  bool wide;           // (launchers) BF16 rows of out at multiples of 32 bytes
};

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;  // null: none
  const uint16_t* weight;    // null: ones
  uint16_t* residual_out;    // null exactly when residual is
  int64_t ld_x, ld_res, ld_res_out;
  int64_t rows, cols;
  float eps, weight_offset;
  float inv_cols, inv_cols_lo;  // (launcher) 1 / cols, in two floats
  bool wide;  // (launcher) rows of every matrix but the output at multiples of 32 bytes
};

struct GateArgs {
  const uint16_t* gate;
  const uint16_t* up;
  int64_t ld_gate, ld_up;
  int64_t rows, cols;
  bool wide;  // (launcher) rows of both at multiples of 32 bytes
  int tail;   // (launcher) values behind the last unit of row 0
};

// Each adds the number of kernels it enqueued to *launches.  rows, cols >= 1.
cudaError_t launch_rms_norm(const NormArgs& a, const RowOutput& o, int* launches, cudaStream_t stream);
cudaError_t launch_silu_mul(const GateArgs& a, const RowOutput& o, int* launches, cudaStream_t stream);

// One 4-bit weight (N x K): packed codes, swizzled scales, tensor scale (NVFP4; null for MXFP4).
struct Weight4 {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* gs;
};

struct MatvecArgs {
  const void* x;            // BF16, or E4M3 codes when x_scales is not null
  const uint8_t* x_scales;  // null, or one E8M0 byte per 32 values
  bool x_swizzled;
  int x_row0, x_rows;       // x_scales: the row of token 0, and the rows of the whole buffer
  int64_t ld_x;             // elements between rows of x (BF16: 2 bytes each, E4M3: 1)
  Weight4 w, gate;          // gate.codes null: no gate
  bool mx;                  // MXFP4 weights, else NVFP4
  int M;
  int64_t N, K;
  uint16_t* out;
  int64_t ld_out;
};

constexpr int kMatvecMaxTokens = 16;

// How a call is cut (host side only; pointers tell BF16, gate and format, and are not read): CTAs of a
// cluster that share K, batches of tiles per CTA at most, whether a cluster's sums take x's place
// in shared memory -- of the first launch -- and the launches.  False: it fits no launch.
struct MatvecPlan {
  int split, batches;
  bool sums_over_x;
  int launches;
};
bool plan_matvec(const MatvecArgs& a, MatvecPlan* plan);

// One launch, or several when x of so many tokens does not fit shared memory.
cudaError_t launch_matvec(const MatvecArgs& a, int* launches, cudaStream_t stream);

}  // namespace nvfp4
