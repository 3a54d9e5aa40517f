"""NVFP4 quantization and the W4A4 block-scaled GEMM on B200 (sm_100a).

A thin ctypes binding over ``libnvfp4_b200.so`` (declared in ``include/nvfp4.h``).
It only marshals arguments: torch provides device memory and the current CUDA
stream; every step of the computation runs in the library's CUDA kernels.  There
is no CPU fallback: if the library is missing or the device is not sm_100, the
calls raise.

Format and method: web page "Tu pipeline NVFP4: meter 62 GB de modelo en 24 GB
de laptop", section 2 "Qué es realmente NVFP4" (E2M1 codes in blocks of 16
along K, one E4M3 scale per block, one FP32 scale per tensor; absmax or MSE
block scales) and "NVFP4 en difusión: la misma cuantización, un motor
completamente distinto", section 2 (packed (out, in/2) codes, (out, in/16)
scales, out = (A s_a)(B s_b)^T in BF16, activations quantized on every call).

Every call serves inference: nothing here has a gradient, and results are detached
from tensors that require one.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4_b200.so")

SCALE_ABSMAX = 0
SCALE_MSE = 1
SCALE_FOUR_OVER_SIX = 2
SF_SWIZZLED = 0
SF_LINEAR = 1
OUT_BF16 = 0
OUT_MXFP8 = 1
OUT_MXFP4 = 2
OUT_NVFP4 = 3
MATVEC_MAX_TOKENS = 16

_MODES = {"absmax": SCALE_ABSMAX, "mse": SCALE_MSE, "four_over_six": SCALE_FOUR_OVER_SIX,
          SCALE_ABSMAX: SCALE_ABSMAX, SCALE_MSE: SCALE_MSE, SCALE_FOUR_OVER_SIX: SCALE_FOUR_OVER_SIX}
_LAYOUTS = {"swizzled": SF_SWIZZLED, "linear": SF_LINEAR, SF_SWIZZLED: SF_SWIZZLED, SF_LINEAR: SF_LINEAR}
_FORMATS = {"bf16": OUT_BF16, "mxfp8": OUT_MXFP8, "mxfp4": OUT_MXFP4, "nvfp4": OUT_NVFP4}

STATUS = {0: "NVFP4_OK", 1: "NVFP4_ERR_INVALID_ARG", 2: "NVFP4_ERR_SHAPE", 3: "NVFP4_ERR_ALIGNMENT",
          4: "NVFP4_ERR_UNSUPPORTED_DEVICE", 5: "NVFP4_ERR_CUDA", 6: "NVFP4_ERR_TIMEOUT",
          7: "NVFP4_ERR_WORKSPACE"}

# Every symbol include/nvfp4.h declares, with its ctypes signature.
_P, _I64, _SZ, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "nvfp4_status_string": ([_I], ctypes.c_char_p),
    "nvfp4_check_device": ([], _I),
    "nvfp4_codes_bytes": ([_I64, _I64], _SZ),
    "nvfp4_scales_bytes": ([_I64, _I64, _I], _SZ),
    "nvfp4_quantize_workspace_bytes": ([_I64, _I64], _SZ),
    "nvfp4_quantize": ([_P, _I64, _I64, _I64, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "nvfp4_dequantize": ([_P, _P, _I, _P, _I64, _I64, _P, _I64, _P], _I),
    "nvfp4_gemm_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "nvfp4_gemm": ([_P, _P, _P, _I64, _P, _P, _P, _I64, _I64, _P, _I64, _P, _SZ, _P], _I),
    "nvfp4_linear_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "nvfp4_linear": ([_P, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _P, _I64, _P, _SZ, _P], _I),
    "nvfp4_linear_fused": ([_P, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _P, _I64, _P, _SZ, _P], _I),
    "nvfp4_linear_lora_workspace_bytes": ([_I64, _I64, _I64, _I64], _SZ),
    "nvfp4_linear_lora": ([_P, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _P, _P, _I64, _P, _I64, _P, _P, _SZ, _P], _I),
    "mxfp4_scales_bytes": ([_I64, _I64, _I], _SZ),
    "mxfp4_quantize": ([_P, _I64, _I64, _I64, _I, _P, _P, _P], _I),
    "mxfp4_dequantize": ([_P, _P, _I, _I64, _I64, _P, _I64, _P], _I),
    "mxfp4_gemm": ([_P, _P, _I64, _P, _P, _I64, _I64, _P, _I64, _P, _SZ, _P], _I),
    "nvfp4_row_workspace_bytes": ([], _SZ),
    "nvfp4_rms_norm": ([_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _F, _F, _I, _I, _P, _P, _I64, _P, _P, _P, _SZ,
                        _P], _I),
    "nvfp4_silu_mul": ([_P, _I64, _P, _I64, _I64, _I64, _I, _I, _P, _P, _I64, _P, _P, _P, _SZ, _P], _I),
    "nvfp4_matvec": ([_P, _P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _I64, _P, _I64, _P], _I),
    "mxfp4_matvec": ([_P, _P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _I64, _P, _I64, _P], _I),
    "nvfp4_matvec_plan": ([_I64, _I64, _I64, _I, _I, ctypes.POINTER(ctypes.c_int32)], _I),
    "nvfp4_read_device_error": ([_P, _P, ctypes.POINTER(ctypes.c_uint32)], _I),
    "nvfp4_last_launch_count": ([], _I),
    "nvfp4_quantize_noalloc": ([_P, _I64, _I64, _I64, _I, _I, _P, _P, _P, _P, _P, _P], _I),
    "nvfp4_selftest_wait_timeout": ([_P, ctypes.c_uint32, _P], _I),
}


class Nvfp4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status})")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the CUDA library (raises if it was not built: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} not found: build it with `python -m w4a4_gemm_quantize_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != 0:
        raise Nvfp4Error(status, where)


# What torch.cuda.current_device and current_stream ask, without their host time (a few microseconds a call); a
# torch that lacks these names has the public calls.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                   or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _stream(stream) -> int:
    if stream is None:
        return _current_stream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


@dataclass
class NVFP4Tensor:
    """A quantized rows x cols tensor: packed codes, E4M3 scales, FP32 global scale."""
    codes: torch.Tensor          # uint8 (rows, cols/2)
    scales: torch.Tensor         # uint8, flat swizzled buffer or (rows, cols/16) linear
    global_scale: torch.Tensor   # float32 (1,)
    rows: int
    cols: int
    layout: int = SF_SWIZZLED
    block_err: Optional[torch.Tensor] = None  # float32 (rows, cols/16)

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel() + 4


def codes_bytes(rows: int, cols: int) -> int:
    return load_library().nvfp4_codes_bytes(rows, cols)


def scales_bytes(rows: int, cols: int, layout=SF_SWIZZLED) -> int:
    return load_library().nvfp4_scales_bytes(rows, cols, _LAYOUTS[layout])


def nvfp4_quantize(x: torch.Tensor, mode="absmax", layout="swizzled", global_scale: Optional[torch.Tensor] = None,
                   block_err: bool = False, out: Optional[NVFP4Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> NVFP4Tensor:
    """Quantize a 2-D BF16 CUDA tensor (row stride multiple of 8, cols % 16 == 0)."""
    lib = load_library()
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a 2-D row-major bfloat16 CUDA tensor")
    rows, cols = x.shape
    m, lay = _MODES[mode], _LAYOUTS[layout]
    dev = x.device
    if out is None:
        codes = torch.empty(lib.nvfp4_codes_bytes(rows, cols), dtype=torch.uint8, device=dev).view(rows, cols // 2)
        nsf = lib.nvfp4_scales_bytes(rows, cols, lay)
        scales = torch.empty(nsf, dtype=torch.uint8, device=dev)
        if lay == SF_LINEAR:
            scales = scales.view(rows, cols // 16)
        gs = torch.empty(1, dtype=torch.float32, device=dev)
        err = torch.empty((rows, cols // 16), dtype=torch.float32, device=dev) if block_err else None
        out = NVFP4Tensor(codes, scales, gs, rows, cols, lay, err)
    if workspace is None and global_scale is None:
        workspace = torch.empty(lib.nvfp4_quantize_workspace_bytes(rows, cols), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.nvfp4_quantize(_ptr(x), rows, cols, x.stride(0), m, lay, _ptr(global_scale), _ptr(out.codes),
                            _ptr(out.scales), _ptr(out.global_scale), _ptr(out.block_err), _ptr(workspace),
                            ws_bytes, _stream(stream))
    _check(st, "nvfp4_quantize")
    return out


def nvfp4_quantize_noalloc(x: torch.Tensor, mode="absmax", layout="swizzled",
                           global_scale: Optional[torch.Tensor] = None, block_err: bool = False,
                           out: Optional[NVFP4Tensor] = None, stream=None) -> NVFP4Tensor:
    """nvfp4_quantize without a workspace, for callers that cannot allocate device
    memory: the library's own 256-byte scratch block per GPU is used instead.
    Calls that overlap on the GPU share that block and race; serialize them."""
    lib = load_library()
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a 2-D row-major bfloat16 CUDA tensor")
    rows, cols = x.shape
    lay = _LAYOUTS[layout]
    if out is None:
        dev = x.device
        codes = torch.empty(lib.nvfp4_codes_bytes(rows, cols), dtype=torch.uint8, device=dev).view(rows, cols // 2)
        scales = torch.empty(lib.nvfp4_scales_bytes(rows, cols, lay), dtype=torch.uint8, device=dev)
        if lay == SF_LINEAR:
            scales = scales.view(rows, cols // 16)
        gs = torch.empty(1, dtype=torch.float32, device=dev)
        err = torch.empty((rows, cols // 16), dtype=torch.float32, device=dev) if block_err else None
        out = NVFP4Tensor(codes, scales, gs, rows, cols, lay, err)
    st = lib.nvfp4_quantize_noalloc(_ptr(x), rows, cols, x.stride(0), _MODES[mode], lay, _ptr(global_scale),
                                    _ptr(out.codes), _ptr(out.scales), _ptr(out.global_scale),
                                    _ptr(out.block_err), _stream(stream))
    _check(st, "nvfp4_quantize_noalloc")
    return out


def nvfp4_dequantize(q: NVFP4Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """BF16 reconstruction q * s_b * s_g of a quantized tensor."""
    lib = load_library()
    if out is None:
        out = torch.empty(q.rows, q.cols, dtype=torch.bfloat16, device=q.codes.device)
    st = lib.nvfp4_dequantize(_ptr(q.codes), _ptr(q.scales), q.layout, _ptr(q.global_scale), q.rows, q.cols,
                              _ptr(out), out.stride(0), _stream(stream))
    _check(st, "nvfp4_dequantize")
    return out


def nvfp4_gemm(a: NVFP4Tensor, b: NVFP4Tensor, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """C = (A s_a)(B s_b)^T s_gA s_gB in BF16; A is M x K, B is N x K, scales swizzled."""
    lib = load_library()
    if a.cols != b.cols:
        raise ValueError("A and B must share K")
    if a.layout != SF_SWIZZLED or b.layout != SF_SWIZZLED:
        raise ValueError("nvfp4_gemm needs swizzled scales")
    M, N, K = a.rows, b.rows, a.cols
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.codes.device)
    if workspace is None:
        workspace = torch.empty(lib.nvfp4_gemm_workspace_bytes(M, N, K), dtype=torch.uint8, device=a.codes.device)
    st = lib.nvfp4_gemm(_ptr(a.codes), _ptr(a.scales), _ptr(a.global_scale), M, _ptr(b.codes), _ptr(b.scales),
                        _ptr(b.global_scale), N, K, _ptr(out), out.stride(0), _ptr(workspace),
                        workspace.numel(), _stream(stream))
    _check(st, "nvfp4_gemm")
    return out


def read_device_error(workspace: torch.Tensor, stream=None) -> int:
    """Synchronize and return the raw device status word of a GEMM workspace (0 = ok)."""
    word = ctypes.c_uint32(0)
    st = load_library().nvfp4_read_device_error(_ptr(workspace), _stream(stream), ctypes.byref(word))
    if st not in (0, 6):
        _check(st, "nvfp4_read_device_error")
    return word.value


def selftest_wait_timeout(workspace: torch.Tensor, timeout_us: int = 20000, stream=None) -> None:
    """Launch the bounded-wait diagnostic (see include/nvfp4.h); read the result with read_device_error."""
    _check(load_library().nvfp4_selftest_wait_timeout(_ptr(workspace), timeout_us, _stream(stream)),
           "nvfp4_selftest_wait_timeout")


def last_launch_count() -> int:
    return load_library().nvfp4_last_launch_count()


def linear(x: torch.Tensor, w: NVFP4Tensor, x_global_scale: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
           fused: bool = False) -> torch.Tensor:
    """W4A4 linear layer C = Q(x) w^T in BF16: the activation x (M x K BF16) is
    quantized on this call with absmax block scales -- under `x_global_scale` (a
    device float, e.g. a calibrated activation scale) or, if None, amax(|x|)/2688
    computed on the device -- and multiplied by the pre-quantized weight w (N x K).
    fused=True (M <= 32) quantizes the activation inside the GEMM kernel
    (nvfp4_linear_fused); the result is the same bit for bit."""
    lib = load_library()
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a 2-D row-major bfloat16 CUDA tensor")
    if w.layout != SF_SWIZZLED or w.cols != x.shape[1]:
        raise ValueError("w must share K with x and have swizzled scales")
    M, K = x.shape
    N = w.rows
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(lib.nvfp4_linear_workspace_bytes(M, N, K), dtype=torch.uint8, device=x.device)
    fn = lib.nvfp4_linear_fused if fused else lib.nvfp4_linear
    st = fn(_ptr(x), M, K, x.stride(0), _ptr(x_global_scale), _ptr(w.codes), _ptr(w.scales),
            _ptr(w.global_scale), N, _ptr(out), out.stride(0), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "nvfp4_linear_fused" if fused else "nvfp4_linear")
    return out


def linear_lora(x: torch.Tensor, w: NVFP4Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
                x_global_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                t_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """W4A4 linear layer with a low-rank branch, y = Q(x) w^T + (x A^T) B^T in BF16:
    lora_a (R x K) and lora_b (N x R) BF16 CUDA tensors, rank R in {16, 32, 48, 64};
    t = x A^T is rounded to BF16 (returned in t_out if given) and t B^T is added to the
    W4A4 GEMM's FP32 accumulator before the single BF16 rounding."""
    lib = load_library()
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a 2-D row-major bfloat16 CUDA tensor")
    M, K = x.shape
    N, R = w.rows, lora_a.shape[0]
    if w.layout != SF_SWIZZLED or w.cols != K:
        raise ValueError("w must share K with x and have swizzled scales")
    for t, shape in ((lora_a, (R, K)), (lora_b, (N, R))):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"low-rank factors must be contiguous bfloat16 of shapes {(R, K)} and {(N, R)}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(lib.nvfp4_linear_lora_workspace_bytes(M, N, K, R), dtype=torch.uint8,
                                device=x.device)
    st = lib.nvfp4_linear_lora(_ptr(x), M, K, x.stride(0), _ptr(x_global_scale), _ptr(w.codes), _ptr(w.scales),
                               _ptr(w.global_scale), N, _ptr(lora_a), _ptr(lora_b), R, _ptr(out), out.stride(0),
                               _ptr(t_out), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "nvfp4_linear_lora")
    return out


@dataclass
class MXFP4Tensor:
    """A rows x cols tensor in MXFP4: packed E2M1 codes and one E8M0 scale per 32 values."""
    codes: torch.Tensor   # uint8 (rows, cols/2)
    scales: torch.Tensor  # uint8, flat swizzled buffer or (rows, cols/32) linear
    rows: int
    cols: int
    layout: int = SF_SWIZZLED


def mxfp4_quantize(x: torch.Tensor, layout="swizzled", out: Optional[MXFP4Tensor] = None, stream=None) -> MXFP4Tensor:
    """Quantize a 2-D BF16 CUDA tensor (cols % 32 == 0) to MXFP4."""
    lib = load_library()
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("x must be a 2-D row-major bfloat16 CUDA tensor")
    rows, cols = x.shape
    lay = _LAYOUTS[layout]
    if out is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty(lib.mxfp4_scales_bytes(rows, cols, lay), dtype=torch.uint8, device=x.device)
        if lay == SF_LINEAR:
            scales = scales.view(rows, cols // 32)
        out = MXFP4Tensor(codes, scales, rows, cols, lay)
    _check(lib.mxfp4_quantize(_ptr(x), rows, cols, x.stride(0), lay, _ptr(out.codes), _ptr(out.scales),
                              _stream(stream)), "mxfp4_quantize")
    return out


def mxfp4_dequantize(q: MXFP4Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    lib = load_library()
    if out is None:
        out = torch.empty(q.rows, q.cols, dtype=torch.bfloat16, device=q.codes.device)
    _check(lib.mxfp4_dequantize(_ptr(q.codes), _ptr(q.scales), q.layout, q.rows, q.cols, _ptr(out), out.stride(0),
                                _stream(stream)), "mxfp4_dequantize")
    return out


def mxfp4_gemm(a: MXFP4Tensor, b: MXFP4Tensor, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """C = A B^T in BF16 for MXFP4 operands (A M x K, B N x K, swizzled scales)."""
    lib = load_library()
    if a.cols != b.cols or a.layout != SF_SWIZZLED or b.layout != SF_SWIZZLED:
        raise ValueError("A and B must share K and have swizzled scales")
    M, N, K = a.rows, b.rows, a.cols
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.codes.device)
    if workspace is None:
        workspace = torch.empty(lib.nvfp4_gemm_workspace_bytes(M, N, K), dtype=torch.uint8, device=a.codes.device)
    _check(lib.mxfp4_gemm(_ptr(a.codes), _ptr(a.scales), M, _ptr(b.codes), _ptr(b.scales), N, K, _ptr(out),
                          out.stride(0), _ptr(workspace), workspace.numel(), _stream(stream)), "mxfp4_gemm")
    return out


# ---------------------------------------------------------------------------------------------
# The operators around a layer's products: norm, gate, and the weight-only product of a few tokens
# ---------------------------------------------------------------------------------------------

@dataclass
class MXFP8Tensor:
    """A rows x cols tensor in MXFP8: E4M3 codes and one E8M0 scale per 32 values."""
    codes: torch.Tensor   # float8_e4m3fn (rows, cols)
    scales: torch.Tensor  # uint8, flat swizzled buffer or (rows, cols/32) linear
    rows: int
    cols: int
    layout: int = SF_SWIZZLED


class _On:
    """The device and stream of one call: makes the tensors' device current, and where the caller names a stream,
    allocates on it (a temporary is not reused before that stream is through with it)."""

    def __init__(self, device: torch.device, stream):
        self.contexts = [torch.cuda.device(device)]
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            self.contexts.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _ld(t: torch.Tensor, name: str, shape=None, dev: int = -1) -> int:
    """Checks a BF16 matrix argument (of `shape`, on device `dev`) and returns its row stride (a single row's is its
    length, rounded up)."""
    own = t.shape
    if t.dtype is not torch.bfloat16 or len(own) != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D bfloat16 CUDA tensor")
    if shape is not None:
        if own != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(own)}")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    rows, cols = own
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must be row-major (stride 1 along its rows)")
    return ld if rows > 1 else -(-cols // 16) * 16


def _like(t: torch.Tensor, name: str, dtype, numel: int, like: torch.Tensor) -> None:
    if t.dtype is not dtype or t.numel() != numel or t.get_device() != like.get_device() or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {numel} elements on {like.device}")


def _weight(t, dev: int) -> None:
    """Checks that a 4-bit weight's tensors are those of its stated size, one byte to a code pair and to a block scale,
    and on device `dev`."""
    nvfp4, c, s = isinstance(t, NVFP4Tensor), t.codes, t.scales
    if c.get_device() != dev or s.get_device() != dev or (nvfp4 and t.global_scale.get_device() != dev):
        raise ValueError(f"the weights must be on x's device, cuda:{dev}")
    if (c.numel() != t.rows * (t.cols // 2) or s.numel() != _swizzled_bytes(t.rows, t.cols // (16 if nvfp4 else 32))
            or c.element_size() != 1 or s.element_size() != 1 or not c.is_contiguous() or not s.is_contiguous()):
        raise ValueError(f"a weight's codes or scales are not those of a {t.rows} x {t.cols} tensor")
    if nvfp4 and (t.global_scale.dtype is not torch.float32 or t.global_scale.numel() != 1):
        raise ValueError("a weight's global_scale must be one float32")


def _swizzled_bytes(rows: int, blocks: int) -> int:
    """nvfp4_scales_bytes / mxfp4_scales_bytes of the SWIZZLED layout."""
    return (rows + 127) // 128 * 128 * ((blocks + 3) // 4 * 4)


def _block_output(fmt: int, layout: int, x: torch.Tensor, out, global_scale):
    """The block-format output of a row operator on x's shape: (tensor object, codes, scales, tensor scale)."""
    rows, cols = x.shape
    block = 16 if fmt == OUT_NVFP4 else 32
    blocks = cols // block
    if blocks * block != cols:
        raise ValueError(f"{cols} columns are no whole number of {block}-value blocks")
    if fmt == OUT_MXFP8:
        kind, width, dtype = MXFP8Tensor, cols, torch.float8_e4m3fn
    else:
        kind, width, dtype = NVFP4Tensor if block == 16 else MXFP4Tensor, cols // 2, torch.uint8
    if out is None:
        dev = x.device
        codes = torch.empty(rows, width, dtype=dtype, device=dev)
        if layout == SF_LINEAR:
            scales = torch.empty(rows, blocks, dtype=torch.uint8, device=dev)
        else:
            scales = torch.empty(_swizzled_bytes(rows, blocks), dtype=torch.uint8, device=dev)
        if fmt != OUT_NVFP4:
            return kind(codes, scales, rows, cols, layout), codes, scales, None
        gs = torch.empty(1, dtype=torch.float32, device=dev)
        return NVFP4Tensor(codes, scales, gs, rows, cols, layout), codes, scales, gs
    if not isinstance(out, kind) or (out.rows, out.cols, out.layout) != (rows, cols, layout):
        raise ValueError(f"out must be a {kind.__name__} of {rows} x {cols} with the asked scale layout")
    _like(out.codes, "out.codes", dtype, rows * width, x)
    _like(out.scales, "out.scales", torch.uint8,
          rows * blocks if layout == SF_LINEAR else _swizzled_bytes(rows, blocks), x)
    if fmt != OUT_NVFP4:
        return out, out.codes, out.scales, None
    _like(out.global_scale, "out.global_scale", torch.float32, 1, x)
    return out, out.codes, out.scales, out.global_scale


def _output(fmt: int, layout: int, x: torch.Tensor, dev: int, out, global_scale, workspace):
    """Output and workspace of a row operator on x: (what the caller gets; the addresses and sizes that the C call
    takes: data, row stride, scales, tensor scale in and out; the workspace, to be held until the call is made)."""
    rows, cols = x.shape
    if fmt == OUT_BF16:
        if global_scale is not None:
            raise ValueError("global_scale is NVFP4's tensor scale; this format has none")
        if out is None:
            out = torch.empty(rows, cols, dtype=torch.bfloat16, device=x.device)
            return out, out.data_ptr(), cols if rows > 1 else -(-cols // 16) * 16, None, None, None, None
        return out, out.data_ptr(), _ld(out, "out", x.shape, dev), None, None, None, None
    result, codes, scales, gs = _block_output(fmt, layout, x, out, global_scale)
    if fmt != OUT_NVFP4:
        if global_scale is not None:
            raise ValueError("global_scale is NVFP4's tensor scale; this format has none")
        return result, codes.data_ptr(), cols, scales.data_ptr(), None, None, None
    if global_scale is not None:
        _like(global_scale, "global_scale", torch.float32, 1, x)
        return result, codes.data_ptr(), cols, scales.data_ptr(), global_scale.data_ptr(), gs.data_ptr(), None
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=x.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {x.device}")
    return result, codes.data_ptr(), cols, scales.data_ptr(), None, gs.data_ptr(), workspace


def _choices(out_format, layout):
    try:
        return _FORMATS[out_format], _LAYOUTS[layout]
    except (KeyError, TypeError):
        raise ValueError(f"out_format must be one of {list(_FORMATS)}, layout 'swizzled' or 'linear'; got "
                         f"{out_format!r}, {layout!r}") from None


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6, weight_offset: float = 0.0, out_format: str = "bf16", layout="swizzled",
             global_scale: Optional[torch.Tensor] = None, out=None, residual_out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None):
    """Root-mean-square norm of the rows of a 2-D BF16 tensor, the residual's addition before it and the
    quantizer behind it (see nvfp4_rms_norm in include/nvfp4.h):

        h = BF16(x + residual);  v = h / sqrt(mean(h^2) + eps) * (weight + weight_offset)

    out_format: "bf16" -> a tensor, "mxfp8" -> MXFP8Tensor, "mxfp4" -> MXFP4Tensor, "nvfp4" -> NVFP4Tensor, whose
    tensor scale is `global_scale` (a device float) or computed from v.  Returns the output, or with a residual
    (output, h); residual_out may be `residual` itself to update the stream in place.  No gradient: the results are
    detached."""
    fmt, lay = _choices(out_format, layout)
    ld_x = _ld(x, "x")
    dev = x.get_device()
    if stream is not None or dev != _current_device():
        with _On(x.device, stream):
            return rms_norm(x, weight, residual, eps, weight_offset, out_format, layout, global_scale, out,
                            residual_out, workspace)
    shape = rows, cols = x.shape
    result, data, ld_out, scales, gs_in, gs_out, ws = _output(fmt, lay, x, dev, out, global_scale, workspace)
    w = None
    if weight is not None:
        _like(weight, "weight", torch.bfloat16, cols, x)
        w = weight.data_ptr()
    r = ro = None
    ld_r = ld_ro = 0
    if residual is not None:
        ld_r, r = _ld(residual, "residual", shape, dev), residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty(rows, cols, dtype=torch.bfloat16, device=x.device)
            ld_ro = cols if rows > 1 else ld_x
        else:
            ld_ro = _ld(residual_out, "residual_out", shape, dev)
        ro = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    st = (_lib or load_library()).nvfp4_rms_norm(x.data_ptr(), rows, cols, ld_x, r, ld_r, ro, ld_ro, w, weight_offset,
                                                 eps, fmt, lay, gs_in, data, ld_out, scales, gs_out, _ptr(ws),
                                                 0 if ws is None else ws.nbytes, _current_stream(dev))
    if st:
        _check(st, "nvfp4_rms_norm")
    return result if residual is None else (result, residual_out)


def silu_mul(gate: torch.Tensor, up: torch.Tensor, out_format: str = "bf16", layout="swizzled",
             global_scale: Optional[torch.Tensor] = None, out=None, workspace: Optional[torch.Tensor] = None,
             stream=None):
    """silu(gate) * up of two 2-D BF16 tensors (strided views, such as the halves of one product, are fine), written
    as `out_format` like rms_norm's output (see nvfp4_silu_mul in include/nvfp4.h).  No gradient: the result is
    detached."""
    fmt, lay = _choices(out_format, layout)
    ld_g = _ld(gate, "gate")
    dev = gate.get_device()
    if stream is not None or dev != _current_device():
        with _On(gate.device, stream):
            return silu_mul(gate, up, out_format, layout, global_scale, out, workspace)
    rows, cols = gate.shape
    ld_u = _ld(up, "up", gate.shape, dev)
    result, data, ld_out, scales, gs_in, gs_out, ws = _output(fmt, lay, gate, dev, out, global_scale, workspace)
    st = (_lib or load_library()).nvfp4_silu_mul(gate.data_ptr(), ld_g, up.data_ptr(), ld_u, rows, cols, fmt, lay,
                                                 gs_in, data, ld_out, scales, gs_out, _ptr(ws),
                                                 0 if ws is None else ws.nbytes, _current_stream(dev))
    if st:
        _check(st, "nvfp4_silu_mul")
    return result


def matvec(x, w, w_gate=None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = x w^T in BF16 for up to MATVEC_MAX_TOKENS rows of x (2-D BF16 tensor, or MXFP8Tensor) and a 4-bit weight w
    (NVFP4Tensor or MXFP4Tensor, N x K, swizzled scales); the activation is not rounded to 4 bits.  With w_gate, a
    second weight of the same kind and shape: silu(x w_gate^T) * (x w^T) in one pass.  More rows: use linear,
    nvfp4_gemm or mxfp4_gemm.  No gradient: the result is detached."""
    if isinstance(x, torch.Tensor):
        data, scales, x_lay, ld_x = x, None, SF_SWIZZLED, _ld(x, "x")
        M, K = x.shape
    else:
        if not isinstance(x, MXFP8Tensor) or not x.codes.is_cuda:
            raise ValueError("x must be a 2-D bfloat16 CUDA tensor or an MXFP8Tensor on a CUDA device")
        data, scales, M, K = x.codes, x.scales, x.rows, x.cols
        if x.layout not in (SF_SWIZZLED, SF_LINEAR):
            raise ValueError(f"unknown scale layout {x.layout!r}")
        ld_x, x_lay = K, x.layout
        _like(data, "x.codes", torch.float8_e4m3fn, M * K, data)
        _like(scales, "x.scales", torch.uint8,
              M * (K // 32) if x_lay == SF_LINEAR else _swizzled_bytes(M, K // 32), data)
    nvfp4 = isinstance(w, NVFP4Tensor)
    if not nvfp4 and not isinstance(w, MXFP4Tensor):
        raise ValueError("w must be an NVFP4Tensor or an MXFP4Tensor")
    N, dev = w.rows, data.get_device()
    for t in (w,) if w_gate is None else (w, w_gate):
        if type(t) is not type(w) or t.rows != N or t.cols != K or t.layout != SF_SWIZZLED:
            raise ValueError("the weights must share K with x, one kind and shape, and have swizzled scales")
        _weight(t, dev)
    if stream is not None or dev != _current_device():
        with _On(data.device, stream):
            return matvec(x, w, w_gate, out)
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=data.device)
        ld_out = N
    else:
        ld_out = max(_ld(out, "out", (M, N), dev), N)
    gc, gsc = (None, None) if w_gate is None else (w_gate.codes.data_ptr(), w_gate.scales.data_ptr())
    if nvfp4:
        st = (_lib or load_library()).nvfp4_matvec(data.data_ptr(), _ptr(scales), x_lay, M, K, ld_x,
                                                   w.codes.data_ptr(), w.scales.data_ptr(), w.global_scale.data_ptr(),
                                                   gc, gsc, None if w_gate is None else w_gate.global_scale.data_ptr(),
                                                   N, out.data_ptr(), ld_out, _current_stream(dev))
    else:
        st = (_lib or load_library()).mxfp4_matvec(data.data_ptr(), _ptr(scales), x_lay, M, K, ld_x,
                                                   w.codes.data_ptr(), w.scales.data_ptr(), gc, gsc, N,
                                                   out.data_ptr(), ld_out, _current_stream(dev))
    if st:
        _check(st, "nvfp4_matvec" if nvfp4 else "mxfp4_matvec")
    return out


def matvec_plan(M: int, N: int, K: int, mxfp4_weights: bool = False, gated: bool = False):
    """How matvec cuts a call of these sizes: (CTAs that share K, batches of tiles per CTA, whether a cluster's sums
    take x's place in shared memory, launches); see nvfp4_matvec_plan in include/nvfp4.h."""
    plan = (ctypes.c_int32 * 4)()
    _check(load_library().nvfp4_matvec_plan(M, N, K, int(mxfp4_weights), int(gated), plan), "nvfp4_matvec_plan")
    return plan[0], plan[1], bool(plan[2]), plan[3]


def mxfp8_scales_bytes(rows: int, cols: int, layout=SF_SWIZZLED) -> int:
    """Bytes of an MXFP8 tensor's E8M0 scales (the layouts are MXFP4's: one byte per 32 values)."""
    return load_library().mxfp4_scales_bytes(rows, cols, _LAYOUTS[layout])
