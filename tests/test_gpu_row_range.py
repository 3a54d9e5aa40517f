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


@pytest.mark.parametrize("cols", [512, 333])                 # 16-value units, one value at a time
def test_gate_of_far_negative_values(cuda_device, cols):
    """e^-g passes binary32 from g = -88.7 on, where a large up value still brings the product back into range."""
    g = torch.linspace(-78.0, -185.0, 64, device="cuda")[:, None].expand(64, cols)
    u = torch.ldexp(bf16((64, cols), 1).float().clamp(-3.9, 3.9), torch.arange(cols, device="cuda") % 126).to(torch.bfloat16)
    g = g.to(torch.bfloat16).contiguous()
    v = ref.gate64(g, u)
    assert (np.abs(v) < 3e38).all() and (np.abs(v) > 1e-20).mean() > 0.1
    ref.check_bf16(nv.silu_mul(g, u), v, ref.GATE_DELTA)
    if cols % 32 == 0:
        ref.check_blocks(nv.silu_mul(g, u, out_format="mxfp8", layout="linear"), v, "mxfp8", "linear", ref.GATE_DELTA)


def test_gated_product_of_far_negative_gates(cuda_device):
    """The same behind the products: a gate of -99 (the quantized -1 times 96) and an up product of 2^126."""
    K = 32
    def weight(value):                                       # N = 16 rows of one value, exact in NVFP4
        w = torch.zeros((16, K), dtype=torch.bfloat16, device="cuda")
        w[:, 0] = value
        return nv.nvfp4_quantize(w, global_scale=torch.ones(1, device="cuda"))
    x = torch.zeros((2, K), dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0] = 96.0, 2.0 ** 5
    gate, up = weight(-1.0), weight(6.0)
    up.global_scale.fill_(2.0 ** 117)
    y, _ = ref.matvec64(x, up, gate)
    assert np.abs(y[0]).min() > 1e-4 and np.isfinite(y).all()
    # one product per sum: the gate is off by 3 roundings, so e^gate by 99 * 3 * 2^-24, and BF16 by half a step
    got = nv.matvec(x, up, gate).double().cpu().numpy()
    assert (np.abs(got - y) <= np.abs(y) * (2.0 ** -8 + 2.0 ** -14)).all()


@pytest.mark.parametrize("power", [-133, -126, 0, 127])
def test_norm_of_one_value_in_a_row_of_millions(cuda_device, power):
    """One value among 2^22 zeros, down to BF16's smallest: the mean square goes to 2^-288."""
    cols = 2 ** 22 + 3
    x = torch.zeros((1, cols), dtype=torch.bfloat16, device="cuda")
    x[0, 12345] = 2.0 ** power
    y = nv.rms_norm(x, eps=0.0).double().cpu().numpy()
    v = np.zeros((1, cols))
    v[0, 12345] = np.sqrt(cols)
    assert np.count_nonzero(y) == 1 and abs(y[0, 12345] - v[0, 12345]) <= v[0, 12345] * 2.0 ** -8
