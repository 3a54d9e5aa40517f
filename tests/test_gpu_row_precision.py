"""How few roundings lie between the inputs of rms_norm and silu_mul and a block format's borders.  A block's scale and
codes follow from v and from the tensor scale, and one step of a 4-bit code is up to half the value, so a rounding too
many shows there first."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import w4a4_gemm_quantize_b200 as nv

pytestmark = pytest.mark.gpu


# rows: one cluster computes scale and output (1, 8), two launches (9, 300); cols: 1 to 8 units per thread
@pytest.mark.parametrize("rows,cols", [(1, 4096), (8, 1024), (9, 2048), (300, 4096), (2, 16384), (2, 65536)])
@pytest.mark.parametrize("weighted", [True, False])
def test_norm_tensor_scale_and_codes_have_one_rounding(cuda_device, rows, cols, weighted):
    """h of small whole numbers and rows of 2^k values: the mean square is exact (its sum of at most cols * 16 is a
    whole number below 2^24), h * weight has 16 bits, so v is off by the rounding of its product with the root, 2^-24,
    and the root's own error (two floats: 2^-44), and the tensor scale, taken from the product in 64 bits, by its own
    rounding alone."""
    g = torch.Generator(device="cuda").manual_seed(rows * cols)
    one_rounding = 2.0 ** -24 * (1 + 2.0 ** -10)
    for i in range(24):
        x = torch.randint(-4, 5, (rows, cols), generator=g, device="cuda").to(torch.bfloat16)
        w = torch.randn(cols, generator=g, device="cuda").to(torch.bfloat16) if weighted else None
        q = nv.rms_norm(x, w, eps=0.0, out_format="nvfp4", layout="linear")
        v, _ = ref.norm64(x, None, w, 0.0)
        want = np.abs(v).max() / 2688.0
        assert abs(q.global_scale.item() - want) <= one_rounding * want, i
        ref.check_blocks(q, v, "nvfp4", "linear", one_rounding)


def test_norm_tensor_scale_with_residual_and_offset(cuda_device):
    """The sum of the residual is small whole numbers, weight + 1 is exact in binary32 and its product with h has at
    most 3 + 17 bits."""
    g = torch.Generator(device="cuda").manual_seed(5)
    for i in range(24):
        x, r = (torch.randint(-2, 3, (40, 2048), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        w = (torch.randint(-512, 513, (2048,), generator=g, device="cuda") / 1024.0).to(torch.bfloat16)
        q, h = nv.rms_norm(x, w, r, eps=0.0, weight_offset=1.0, out_format="nvfp4")
        v, _ = ref.norm64(x, r, w, 0.0, 1.0)
        want = np.abs(v).max() / 2688.0
        assert abs(q.global_scale.item() - want) <= 2.0 ** -24 * (1 + 2.0 ** -10) * want, i
