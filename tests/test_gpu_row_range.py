"""rms_norm and silu_mul at the ends of their arguments' range, against the 64-bit definitions
(tests/layer_reference.py)."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import w4a4_gemm_quantize_b200 as nv

pytestmark = pytest.mark.gpu


def bf16(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


# powers of two of the rows: subnormal values, squares that leave binary32 below and above, their sum alone above
POWERS = [-130, -120, -100, -76, -70, -64, -40, 0, 40, 58, 62, 64, 100, 124]


# 512: 16-value units; 16384: several per thread; 251 dense rows of another width; 4097 and 70001: one value at a time
@pytest.mark.parametrize("cols", [32, 512, 16384, 251, 4097, 70001])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_rows_of_any_magnitude(cuda_device, cols, eps):
    """The squares of BF16 values reach from 2^-266 to 2^256: no row may turn to zeros or infinities over that."""
    rows = len(POWERS)
    x = torch.ldexp(bf16((rows, cols), 1).float(), torch.tensor(POWERS, device="cuda")[:, None]).to(torch.bfloat16)
    w = bf16((1, cols), 2).view(-1)
    v, _ = ref.norm64(x, None, w, eps)
    assert np.isfinite(v).all()
    ref.check_bf16(nv.rms_norm(x, w, eps=eps), v, ref.NORM_DELTA)
    wide = torch.zeros((rows, cols + 1), dtype=torch.bfloat16, device="cuda")   # the path of single values
    wide[:, 1:] = x
    ref.check_bf16(nv.rms_norm(wide[:, 1:], w, eps=eps), v, ref.NORM_DELTA)
    if cols % 32 == 0:
        for fmt in ("mxfp8", "mxfp4", "nvfp4"):
            q = nv.rms_norm(x, w, eps=eps, out_format=fmt, layout="linear")
            ref.check_blocks(q, v, fmt, "linear", ref.NORM_DELTA)


def test_norm_of_a_row_whose_sum_of_squares_passes_binary32(cuda_device):
    """4096 values of 4e17: their mean square is 1.6e35, their sum 6.6e38."""
    x = torch.full((3, 4096), 4e17, dtype=torch.bfloat16, device="cuda")
    assert (nv.rms_norm(x) == 1.0).all()
