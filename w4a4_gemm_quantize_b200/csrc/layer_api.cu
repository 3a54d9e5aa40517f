// layer_api.cu -- the extern "C" entry points of the decoder-layer operators declared in
// include/nvfp4.h: host-side validation and launches.  No allocation, no synchronisation.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/nvfp4.h"
#include "internal.h"
#include "layer_ops.h"

namespace {

constexpr size_t kRowWorkspace = 256;  // the first 8 bytes: the output's amax
constexpr int64_t kMaxRows = int64_t{1} << 30;
constexpr int64_t kMaxBlockCols = 65536;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A rows x cols region of elements of `size` bytes with row stride ld.
struct Region {
  const void* p;
  int64_t rows, cols, ld, size;
};

bool same_place(const Region& a, const Region& b) {
  return a.p == b.p && a.size == b.size && (a.ld == b.ld || a.rows <= 1);
}

// Whether two regions may share a byte.  Exact for regions of the same row stride (column
// slices of one buffer), else by their address ranges.
bool overlap(const Region& a, const Region& b) {
  if (!a.p || !b.p || a.rows <= 0 || a.cols <= 0 || b.rows <= 0 || b.cols <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + static_cast<uintptr_t>(((a.rows - 1) * a.ld + a.cols) * a.size);
  const uintptr_t b1 = b0 + static_cast<uintptr_t>(((b.rows - 1) * b.ld + b.cols) * b.size);
  if (a1 <= b0 || b1 <= a0) return false;
  const uintptr_t pitch = static_cast<uintptr_t>(a.ld * a.size);
  if (pitch != static_cast<uintptr_t>(b.ld * b.size) || pitch == 0) return true;
  // columns of b relative to a's, modulo the pitch
  const uintptr_t off = b0 >= a0 ? (b0 - a0) % pitch : (pitch - (a0 - b0) % pitch) % pitch;
  return off < static_cast<uintptr_t>(a.cols * a.size) || off + static_cast<uintptr_t>(b.cols * b.size) > pitch;
}

struct RowCall {
  int64_t rows, cols, ld_out;
  int format, layout;
  const float* gs_in;
  void* out;
  uint8_t* scales;
  float* gs_out;
  void* workspace;
  size_t workspace_bytes;
};

size_t scale_bytes(const RowCall& c) {
  return c.format == NVFP4_OUT_NVFP4 ? nvfp4_scales_bytes(c.rows, c.cols, static_cast<nvfp4_sf_layout>(c.layout))
                                     : mxfp4_scales_bytes(c.rows, c.cols, static_cast<nvfp4_sf_layout>(c.layout));
}

Region out_region(const RowCall& c) {
  if (c.format == NVFP4_OUT_BF16) return {c.out, c.rows, c.cols, c.ld_out, 2};
  const int64_t bytes = c.rows * (c.format == NVFP4_OUT_MXFP8 ? c.cols : c.cols / 2);
  return {c.out, 1, bytes, bytes, 1};
}

// Whether `bytes` bytes at p lie in a region (not in the gaps between its rows).
bool inside(const void* p, int64_t bytes, const Region& r) {
  return overlap(r, {p, p ? 1 : 0, bytes / r.size, r.ld, r.size});
}

// Whether a tensor scale or the workspace shares a byte with another argument: none may, but
// for the given scale written over itself.  rin: inputs, rout: outputs.
template <size_t I, size_t O>
bool words_overlap(const RowCall& c, const Region (&rin)[I], const Region (&rout)[O]) {
  const void* ws = c.format == NVFP4_OUT_NVFP4 && !c.gs_in ? c.workspace : nullptr;
  constexpr int64_t kWs = kRowWorkspace;
  for (const Region& r : rin)
    if (inside(c.gs_out, 4, r) || inside(ws, kWs, r)) return true;
  for (const Region& r : rout)
    if (inside(c.gs_in, 4, r) || inside(c.gs_out, 4, r) || inside(ws, kWs, r)) return true;
  return inside(c.gs_out, 4, {ws, ws ? 1 : 0, kWs, kWs, 1});
}

// The checks of the output's side that need no look at the inputs.
nvfp4_status validate_output(const RowCall& c) {
  if (c.rows < 0 || c.cols < 1) return NVFP4_ERR_INVALID_ARG;
  if (c.format < NVFP4_OUT_BF16 || c.format > NVFP4_OUT_NVFP4) return NVFP4_ERR_INVALID_ARG;
  if (c.layout != NVFP4_SF_SWIZZLED && c.layout != NVFP4_SF_LINEAR) return NVFP4_ERR_INVALID_ARG;
  if (c.rows > kMaxRows || c.cols > INT32_MAX) return NVFP4_ERR_SHAPE;
  const bool nv = c.format == NVFP4_OUT_NVFP4, block = c.format != NVFP4_OUT_BF16;
  if (!nv && (c.gs_in || c.gs_out)) return NVFP4_ERR_INVALID_ARG;
  if (!block && (c.scales || c.ld_out < c.cols)) return NVFP4_ERR_INVALID_ARG;
  if (block && c.cols % (nv ? 16 : 32) != 0) return NVFP4_ERR_SHAPE;
  if (c.rows > 0 && (!c.out || (block && !c.scales))) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(c.out, block ? 16 : 2) || !aligned(c.scales, 16) || !aligned(c.gs_in, 4) || !aligned(c.gs_out, 4) ||
      !aligned(c.workspace, 16))
    return NVFP4_ERR_ALIGNMENT;
  if (nv && !c.gs_in && (!c.workspace || c.workspace_bytes < kRowWorkspace)) return NVFP4_ERR_WORKSPACE;
  return NVFP4_OK;
}

// An input matrix: present, wide enough, aligned as the format asks.
nvfp4_status validate_input(const void* p, int64_t ld, const RowCall& c) {
  if (c.rows > 0 && !p) return NVFP4_ERR_INVALID_ARG;
  if (ld < c.cols) return NVFP4_ERR_INVALID_ARG;
  const bool block = c.format != NVFP4_OUT_BF16;
  if (!aligned(p, block ? 16 : 2) || (block && ld % 8 != 0)) return NVFP4_ERR_ALIGNMENT;
  return NVFP4_OK;
}

// NVFP4's tensor scale of an empty result: the given one, or 1.
nvfp4_status publish_empty(const RowCall& c, cudaStream_t s) {
  if (c.format != NVFP4_OUT_NVFP4 || !c.gs_out) return NVFP4_OK;
  static const float one = 1.0f;
  const cudaError_t e = c.gs_in ? cudaMemcpyAsync(c.gs_out, c.gs_in, sizeof(float), cudaMemcpyDeviceToDevice, s)
                                : cudaMemcpyAsync(c.gs_out, &one, sizeof(float), cudaMemcpyHostToDevice, s);
  return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

nvfp4::RowOutput row_output(const RowCall& c) {
  return {c.out,   c.ld_out, c.scales, c.layout == NVFP4_SF_SWIZZLED, c.format, c.gs_in, c.gs_out,
          static_cast<unsigned long long*>(c.workspace), false};
}

nvfp4_status matvec(const void* x, const uint8_t* x_scales, int x_layout, int64_t M, int64_t K, int64_t ld_x,
                    const nvfp4::Weight4& w, const nvfp4::Weight4& gate, bool mx, int64_t N, void* out, int64_t ld_out,
                    void* stream) {
  nvfp4::g_last_launches = 0;
  if (M < 0 || N < 1 || K < 1 || ld_x < K || ld_out < N) return NVFP4_ERR_INVALID_ARG;
  if (x_scales && x_layout != NVFP4_SF_SWIZZLED && x_layout != NVFP4_SF_LINEAR) return NVFP4_ERR_INVALID_ARG;
  if (K % 32 != 0 || M > nvfp4::kMatvecMaxTokens || N > kMaxRows || K > (int64_t{1} << 19)) return NVFP4_ERR_SHAPE;
  if (!w.codes || !w.scales || (!mx && !w.gs) || (M > 0 && (!x || !out))) return NVFP4_ERR_INVALID_ARG;
  if ((gate.codes != nullptr) != (gate.scales != nullptr) || (!mx && (gate.codes != nullptr) != (gate.gs != nullptr)))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(x_scales, 16) || ld_x % (x_scales ? 16 : 8) != 0 || !aligned(w.codes, 16) ||
      !aligned(w.scales, 16) || !aligned(gate.codes, 16) || !aligned(gate.scales, 16) || !aligned(w.gs, 4) ||
      !aligned(gate.gs, 4) || !aligned(out, 2))
    return NVFP4_ERR_ALIGNMENT;
  const Region o{out, M, N, ld_out, 2};
  const int64_t codes = N * (K / 2), scales = (N + 127) / 128 * 128 * ((K / (mx ? 32 : 16) + 3) / 4 * 4);
  const int64_t xs =  // swizzled: whole 128 x 4 tiles
      x_scales ? static_cast<int64_t>(mxfp4_scales_bytes(M, K, static_cast<nvfp4_sf_layout>(x_layout))) : 0;
  if (overlap(o, {x, M, K, ld_x, x_scales ? 1 : 2}) || overlap(o, {x_scales, 1, xs, xs, 1}))
    return NVFP4_ERR_INVALID_ARG;
  for (const nvfp4::Weight4& t : {w, gate})
    if (overlap(o, {t.codes, 1, codes, codes, 1}) || overlap(o, {t.scales, 1, scales, scales, 1}) ||
        inside(t.gs, 4, o))
      return NVFP4_ERR_INVALID_ARG;
  const nvfp4_status st = nvfp4_check_device();
  if (st != NVFP4_OK || M == 0) return st;
  const nvfp4::MatvecArgs a{x,    x_scales, x_layout == NVFP4_SF_SWIZZLED, 0, static_cast<int>(M), ld_x, w, gate, mx,
                            static_cast<int>(M), N, K, static_cast<uint16_t*>(out), ld_out};
  return nvfp4::launch_matvec(a, &nvfp4::g_last_launches, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? NVFP4_OK
             : NVFP4_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t nvfp4_row_workspace_bytes(void) { return kRowWorkspace; }

nvfp4_status nvfp4_rms_norm(const void* x, int64_t rows, int64_t cols, int64_t ld_x, const void* residual,
                            int64_t ld_residual, void* residual_out, int64_t ld_residual_out, const void* weight,
                            float weight_offset, float eps, nvfp4_out_format out_format, nvfp4_sf_layout layout,
                            const float* global_scale_in, void* out, int64_t ld_out, uint8_t* scales,
                            float* global_scale_out, void* workspace, size_t workspace_bytes, void* stream) {
  nvfp4::g_last_launches = 0;
  const RowCall c{rows, cols, ld_out, out_format, layout, global_scale_in, out, scales, global_scale_out, workspace,
                  workspace_bytes};
  nvfp4_status st = validate_output(c);
  if (st != NVFP4_OK) return st;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(weight_offset)) return NVFP4_ERR_INVALID_ARG;
  st = validate_input(x, ld_x, c);
  if (st != NVFP4_OK) return st;
  if ((residual != nullptr) != (residual_out != nullptr)) return NVFP4_ERR_INVALID_ARG;
  if (residual) {
    st = validate_input(residual, ld_residual, c);
    if (st == NVFP4_OK) st = validate_input(residual_out, ld_residual_out, c);
    if (st != NVFP4_OK) return st;
  }
  const bool block = out_format != NVFP4_OUT_BF16;
  if (!aligned(weight, block ? 16 : 2)) return NVFP4_ERR_ALIGNMENT;
  if (block && cols > kMaxBlockCols) return NVFP4_ERR_SHAPE;
  const Region rx{x, rows, cols, ld_x, 2}, rr{residual, rows, cols, ld_residual, 2},
      ro{residual_out, rows, cols, ld_residual_out, 2}, rw{weight, weight ? 1 : 0, cols, cols, 2}, y = out_region(c),
      sc{scales, scales ? 1 : 0, static_cast<int64_t>(block ? scale_bytes(c) : 0), 1, 1};
  if (overlap(y, ro) || overlap(y, rw) || overlap(ro, rw) || (overlap(ro, rr) && !same_place(ro, rr)) ||
      (overlap(ro, rx) && !same_place(ro, rx)))
    return NVFP4_ERR_INVALID_ARG;
  for (const Region& in : {rx, rr})
    if (overlap(y, in) && (block || !same_place(y, in))) return NVFP4_ERR_INVALID_ARG;
  for (const Region& other : {rx, rr, ro, rw, y})
    if (overlap(sc, other)) return NVFP4_ERR_INVALID_ARG;
  if (words_overlap(c, {rx, rr, rw}, {y, ro, sc})) return NVFP4_ERR_INVALID_ARG;
  st = nvfp4_check_device();
  if (st != NVFP4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return publish_empty(c, s);
  const nvfp4::NormArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(residual),
                          static_cast<const uint16_t*>(weight), static_cast<uint16_t*>(residual_out), ld_x,
                          ld_residual, ld_residual_out, rows, cols, eps, weight_offset, 0.0f, 0.0f, false};
  return nvfp4::launch_rms_norm(a, row_output(c), &nvfp4::g_last_launches, s) == cudaSuccess ? NVFP4_OK
                                                                                            : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_silu_mul(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int64_t rows,
                            int64_t cols, nvfp4_out_format out_format, nvfp4_sf_layout layout,
                            const float* global_scale_in, void* out, int64_t ld_out, uint8_t* scales,
                            float* global_scale_out, void* workspace, size_t workspace_bytes, void* stream) {
  nvfp4::g_last_launches = 0;
  const RowCall c{rows, cols, ld_out, out_format, layout, global_scale_in, out, scales, global_scale_out, workspace,
                  workspace_bytes};
  nvfp4_status st = validate_output(c);
  if (st == NVFP4_OK) st = validate_input(gate, ld_gate, c);
  if (st == NVFP4_OK) st = validate_input(up, ld_up, c);
  if (st != NVFP4_OK) return st;
  const bool block = out_format != NVFP4_OUT_BF16;
  const Region rg{gate, rows, cols, ld_gate, 2}, ru{up, rows, cols, ld_up, 2}, y = out_region(c),
      sc{scales, scales ? 1 : 0, static_cast<int64_t>(block ? scale_bytes(c) : 0), 1, 1};
  for (const Region& in : {rg, ru})
    if (overlap(y, in) && (block || !same_place(y, in))) return NVFP4_ERR_INVALID_ARG;
  for (const Region& other : {rg, ru, y})
    if (overlap(sc, other)) return NVFP4_ERR_INVALID_ARG;
  if (words_overlap(c, {rg, ru}, {y, sc})) return NVFP4_ERR_INVALID_ARG;
  st = nvfp4_check_device();
  if (st != NVFP4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return publish_empty(c, s);
  const nvfp4::GateArgs a{static_cast<const uint16_t*>(gate), static_cast<const uint16_t*>(up), ld_gate, ld_up, rows,
                          cols, false, 0};
  return nvfp4::launch_silu_mul(a, row_output(c), &nvfp4::g_last_launches, s) == cudaSuccess ? NVFP4_OK
                                                                                            : NVFP4_ERR_CUDA;
}

nvfp4_status nvfp4_matvec(const void* x, const uint8_t* x_scales, nvfp4_sf_layout x_layout, int64_t M, int64_t K,
                          int64_t ld_x, const uint8_t* w_codes, const uint8_t* w_scales,
                          const float* w_global_scale, const uint8_t* gate_codes, const uint8_t* gate_scales,
                          const float* gate_global_scale, int64_t N, void* out, int64_t ld_out, void* stream) {
  return matvec(x, x_scales, x_layout, M, K, ld_x, {w_codes, w_scales, w_global_scale},
                {gate_codes, gate_scales, gate_global_scale}, false, N, out, ld_out, stream);
}

nvfp4_status mxfp4_matvec(const void* x, const uint8_t* x_scales, nvfp4_sf_layout x_layout, int64_t M, int64_t K,
                          int64_t ld_x, const uint8_t* w_codes, const uint8_t* w_scales, const uint8_t* gate_codes,
                          const uint8_t* gate_scales, int64_t N, void* out, int64_t ld_out, void* stream) {
  return matvec(x, x_scales, x_layout, M, K, ld_x, {w_codes, w_scales, nullptr}, {gate_codes, gate_scales, nullptr},
                true, N, out, ld_out, stream);
}

nvfp4_status nvfp4_matvec_plan(int64_t M, int64_t N, int64_t K, int mxfp4_weights, int gated, int32_t plan[4]) {
  if (!plan || M < 1 || N < 1 || K < 1) return NVFP4_ERR_INVALID_ARG;
  if (K % 32 != 0 || M > nvfp4::kMatvecMaxTokens || N > kMaxRows || K > (int64_t{1} << 19)) return NVFP4_ERR_SHAPE;
  nvfp4::MatvecArgs a{};
  static const uint8_t some = 0;  // (only told from null)
  a.mx = mxfp4_weights != 0;
  if (gated) a.gate.codes = &some;
  a.M = static_cast<int>(M), a.N = N, a.K = K;
  nvfp4::MatvecPlan p;
  if (!nvfp4::plan_matvec(a, &p)) return NVFP4_ERR_SHAPE;
  plan[0] = p.split, plan[1] = p.batches, plan[2] = p.sums_over_x, plan[3] = p.launches;
  return NVFP4_OK;
}

}  // extern "C"
