"""matvec refuses weights whose tensors are not what the kernel reads."""
import pytest
import torch

import w4a4_gemm_quantize_b200 as nv

pytestmark = pytest.mark.gpu


def test_weights_of_other_types_are_refused(cuda_device):
    w = nv.nvfp4_quantize(torch.randn(64, 96, device="cuda").to(torch.bfloat16))
    x = torch.randn(2, 96, device="cuda").to(torch.bfloat16)
    for gs in (w.global_scale.bfloat16(), w.global_scale.double(), w.global_scale.expand(2), w.global_scale[:0]):
        bad = nv.NVFP4Tensor(w.codes, w.scales, gs, 64, 96)
        for call in (lambda: nv.matvec(x, bad), lambda: nv.matvec(x, w, bad)):
            with pytest.raises(ValueError):
                call()
    for bad in (nv.NVFP4Tensor(w.codes.int(), w.scales, w.global_scale, 64, 96),
                nv.NVFP4Tensor(w.codes, w.scales.half(), w.global_scale, 64, 96)):
        with pytest.raises(ValueError):
            nv.matvec(x, bad)
    assert torch.equal(nv.matvec(x, nv.NVFP4Tensor(w.codes.view(torch.int8), w.scales, w.global_scale.view(()), 64, 96)),
                       nv.matvec(x, w))
