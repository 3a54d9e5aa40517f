"""matvec over the whole range of its activations, against the 64-bit product of the dequantized weight
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


@pytest.mark.parametrize("N,K", [(96, 4096), (40, 21504)])              # one CTA per tile, clusters
@pytest.mark.parametrize("gated", [False, True])
def test_large_tokens_under_a_small_tensor_scale(cuda_device, N, K, gated):
    """Tokens whose product with the codes and block scales passes binary32 while the tensor scale, about 2^-15, brings
    the result back: plain outputs stay finite, a far negative gate gives a zero and no NaN."""
    powers = torch.tensor([100, 108, 112, 114, 116, 118, 0, 120], device="cuda")
    x = torch.ldexp(bf16((8, K), 1).float().clamp(-3.9, 3.9), powers[:, None]).to(torch.bfloat16)
    w = nv.nvfp4_quantize(bf16((N, K), 2, 0.02))
    if not gated:
        y, bound = ref.matvec64(x, w)
        assert np.abs(y).max() < 3e38
        ref.check_product(nv.matvec(x, w), y, bound)
        return
    gate = nv.nvfp4_quantize(-w.codes.new_ones((N, K)).to(torch.bfloat16) * 0.02)   # the gate: -0.02 times the token's sum
    x = x.abs()
    g, _ = ref.matvec64(x, gate)
    want = nv.matvec(x[6:7], w, gate)                                   # the token of ordinary size
    got = nv.matvec(x, w, gate)
    assert torch.equal(got[6:7], want)
    far = (g < -1e30) & (g > -3.4e38)                                   # e^-2^100 and less; beyond, the FP32 sum is -inf
    assert far.sum() >= 6 * N
    assert (got.double().cpu().numpy()[far] == 0).all()
