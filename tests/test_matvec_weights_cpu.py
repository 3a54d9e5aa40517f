"""The check of matvec's weights, on host tensors (device -1): sizes, types and devices of what the kernel reads."""
import pytest
import torch

import w4a4_gemm_quantize_b200 as nv


def weight(kind="nvfp4", **other):
    parts = dict(codes=torch.zeros((64, 48), dtype=torch.uint8),
                 scales=torch.zeros(128 * (8 if kind == "nvfp4" else 4), dtype=torch.uint8))
    if kind == "nvfp4":
        parts["global_scale"] = torch.ones(1)
    parts.update(other)
    return (nv.NVFP4Tensor if kind == "nvfp4" else nv.MXFP4Tensor)(**parts, rows=64, cols=96)


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_a_weight_as_the_quantizer_makes_it(kind):
    nv._weight(weight(kind), -1)
    nv._weight(weight(kind, codes=torch.zeros((64, 48), dtype=torch.int8)), -1)          # the same bytes


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("other", [
    dict(codes=torch.zeros((64, 48), dtype=torch.int32)), dict(codes=torch.zeros((64, 47), dtype=torch.uint8)),
    dict(codes=torch.zeros((48, 64), dtype=torch.uint8).t()), dict(scales=torch.zeros(1, dtype=torch.uint8)),
    dict(scales=torch.zeros(1024, dtype=torch.float32)), dict(scales=torch.zeros(512, dtype=torch.float16))])
def test_codes_and_scales_of_another_size_or_type(kind, other):
    with pytest.raises(ValueError):
        nv._weight(weight(kind, **other), -1)


@pytest.mark.parametrize("gs", [torch.ones(1, dtype=torch.bfloat16), torch.ones(1, dtype=torch.float16),
                                torch.ones(1, dtype=torch.float64), torch.ones(2), torch.ones(0)])
def test_a_tensor_scale_that_is_not_one_float32(gs):
    with pytest.raises(ValueError):
        nv._weight(weight(global_scale=gs), -1)


def test_another_device():
    with pytest.raises(ValueError):
        nv._weight(weight(), 0)
