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


def mxfp8(x, layout):
    """x as MXFP8 through plain torch operations."""
    v = x.float().view(x.shape[0], -1, 32)
    amax = v.abs().amax(2, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 9, -127).clamp(-127, 127)
    # 2^-e in two factors: with e down to -127 it may pass binary32
    codes = (v * torch.ldexp(torch.ones_like(amax), -e // 2) * torch.ldexp(torch.ones_like(amax), -e - (-e // 2)))
    codes = codes.clamp(-448, 448).to(torch.float8_e4m3fn).view(x.shape)
    s = (e + 127).to(torch.uint8).view(x.shape[0], -1)
    if layout == "linear":
        return nv.MXFP8Tensor(codes, s.contiguous(), *x.shape, nv.SF_LINEAR)
    import oracle
    return nv.MXFP8Tensor(codes, torch.from_numpy(oracle.swizzle_scales(s.cpu().numpy())).cuda(), *x.shape)


def values(x):
    return x if isinstance(x, torch.Tensor) else torch.from_numpy(ref.dequantize64(x))


def banded(M, N, K, kind, group, powers, seed):
    """x whose values lie at 2^powers, a random one for each `group` of columns, and a weight whose row n is zero but
    where x is near a power of its own: what a token holds at other powers must not cost that row a bit."""
    r = np.random.default_rng(seed)
    p = r.choice(powers, K // group).repeat(group)
    x = torch.ldexp(bf16((M, K), seed).float(), torch.from_numpy(p).cuda()).to(torch.bfloat16)
    centre = torch.from_numpy(r.choice(p, N)).cuda()[:, None]
    w = torch.where((torch.from_numpy(p).cuda()[None] - centre).abs() <= 4, bf16((N, K), seed + 1, 0.02).float(), 0.0)
    w = w.to(torch.bfloat16)
    return x, nv.nvfp4_quantize(w) if kind == "nvfp4" else nv.mxfp4_quantize(w)


# several chunks of K and one, part of a chunk, odd blocks; one CTA for all of K and clusters; 1 to 16 tokens
BANDED = [(1, 5, 64), (3, 130, 1056), (1, 300, 4096), (8, 1000, 544), (9, 77, 4096), (16, 300, 2080), (16, 40, 21504),
          (5, 200, 14336), (12, 3000, 96)]


@pytest.mark.parametrize("M,N,K", BANDED)
@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_values_of_any_magnitude_in_one_token(cuda_device, M, N, K, kind):
    """Single values (BF16) and blocks (MXFP8) from 2^-120 to 2^100 next to one another."""
    x, w = banded(M, N, K, kind, 1, np.arange(-120, 101), M + N)
    y, bound = ref.matvec64(x, w)
    ref.check_product(nv.matvec(x, w), y, bound, f"{kind} {M}x{N}x{K}")
    for layout in ("linear", "swizzled"):
        x, w = banded(M, N, K, kind, 32, np.arange(-100, 101), M + N)
        x8 = mxfp8(x, layout)
        y, bound = ref.matvec64(values(x8), w)
        got = nv.matvec(x8, w)
        ref.check_product(got, y, bound, f"{kind} mxfp8 {M}x{N}x{K}")
        assert torch.equal(got, nv.matvec(x8, w))                       # the same bits on every call


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 40, 544), (4, 300, 4096), (16, 100, 21504)])
def test_values_of_any_magnitude_in_a_gated_product(cuda_device, kind, M, N, K):
    x, w = banded(M, N, K, kind, 1, np.arange(-70, 3), 3)
    _, g = banded(M, N, K, kind, 1, np.arange(-70, 3), 3)               # the same rows' powers
    if kind == "nvfp4":
        g.global_scale.mul_(2.0)
    y, bound = ref.matvec64(x, w, g)
    ref.check_product(nv.matvec(x, w, g), y, bound, f"gated {kind}", min_exact=0.85)


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_a_large_value_over_zero_codes(cuda_device, kind):
    """2^p next to values near 1, for p up to where nothing of them was left: the large value's weight is zero."""
    K = 96
    w = torch.full((16, K), 3.0, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 0
    w = nv.nvfp4_quantize(w) if kind == "nvfp4" else nv.mxfp4_quantize(w)
    for p in (20, 24, 25, 28, 30, 33, 40, 64, 100, 127):
        x = torch.full((2, K), 1.3125, dtype=torch.bfloat16, device="cuda")
        x[:, 0] = 2.0 ** p
        y, bound = ref.matvec64(x, w)
        ref.check_product(nv.matvec(x, w), y, bound, f"2^{p}")


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_values_of_any_magnitude_handled_token_by_token(cuda_device, kind):
    """Rows so long that the tokens are handled apart, their scale rows at odd offsets."""
    x, w = banded(3, 40, 2 ** 19 - 32, kind, 32, np.arange(-60, 61), 1)
    for t in (x, mxfp8(x, "linear"), mxfp8(x, "swizzled")):
        y, bound = ref.matvec64(values(t), w)
        ref.check_product(nv.matvec(t, w), y, bound, kind)
        assert nv.last_launch_count() == 3


@pytest.mark.parametrize("power", [-120, -60, 60, 109])
@pytest.mark.parametrize("spread", [False, True])
def test_mxfp4_weights_of_any_magnitude(cuda_device, power, spread):
    """Weights up to 2^110, values of x near one another and 40 binades apart (one pass and two)."""
    M, N, K = 8, 130, 1056
    x = bf16((M, K), 1).float()
    x = torch.ldexp(x, torch.full((), 100 if power == -120 else -3, device="cuda"))
    if spread:
        x[:, ::3] *= 2.0 ** -40
    x = x.to(torch.bfloat16)
    w = nv.mxfp4_quantize(torch.ldexp(bf16((N, K), 2).float().clamp(-1.9, 1.9), torch.full((), power, device="cuda")).bfloat16())
    y, bound = ref.matvec64(x, w)
    ref.check_product(nv.matvec(x, w), y, bound)


@pytest.mark.parametrize("scale", [-30, -15, -9, 0, 20])
def test_nvfp4_tensor_scales_of_any_magnitude(cuda_device, scale):
    """Passes meet under their own factors, of which the tensor scale is a part."""
    x, w = banded(3, 77, 544, "nvfp4", 1, np.arange(-60, 41), 9)
    w.global_scale.fill_(1.37 * 2.0 ** scale)
    y, bound = ref.matvec64(x, w)
    ref.check_product(nv.matvec(x, w), y, bound)


@pytest.mark.parametrize("scale,power", [(100, -90), (118, -8), (-126, 100), (-100, 105), (60, 40), (-60, -60)])
def test_tensor_scales_against_tokens(cuda_device, scale, power):
    """A tensor scale and a token at the ends of their ranges whose product is an ordinary number."""
    M, N, K = 3, 40, 96
    w = nv.nvfp4_quantize(bf16((N, K), 2, 1.0), global_scale=torch.tensor([1.0 / 64], device="cuda"))
    w.global_scale.fill_(1.37 * 2.0 ** scale)
    for spread in (False, True):
        x = bf16((M, K), 1).float()
        if spread:
            x[:, ::2] *= 2.0 ** -34
        x = torch.ldexp(x, torch.full((), power, device="cuda")).to(torch.bfloat16)
        y, bound = ref.matvec64(x, w)
        assert np.abs(y).max() < 3e38
        ref.check_product(nv.matvec(x, w), y, bound)


def test_mxfp8_values_down_to_the_smallest(cuda_device):
    """E4M3's smallest values under E8M0's smallest scales, 2^-136, beside large ones: exact like all others."""
    N, K = 40, 96
    w = nv.mxfp4_quantize(torch.ldexp(bf16((N, K), 1).float(), torch.full((), 90, device="cuda")).to(torch.bfloat16))
    codes = torch.randint(1, 8, (2, K), device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)     # 2^-9 to 7 2^-9
    for big in (0, 60, 134):
        scales = torch.tensor([[big, 0, 1], [0, 2, big]], dtype=torch.uint8, device="cuda")
        x = nv.MXFP8Tensor(codes, scales, 2, K, nv.SF_LINEAR)
        y, bound = ref.matvec64(values(x), w)
        ref.check_product(nv.matvec(x, w), y, bound)
    zero_first = w.codes.clone()
    zero_first[:, :16] = 0                                              # nothing but the smallest values is left
    w0 = nv.MXFP4Tensor(zero_first, w.scales, N, K)
    y, bound = ref.matvec64(values(x), w0)
    ref.check_product(nv.matvec(x, w0), y, bound)


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(4, 40, 2304), (12, 130, 4096)])
def test_non_finite_values_beside_small_ones(cuda_device, kind, M, N, K):
    """Infinities and NaN in calls that take several passes: they stay in their token and their formula."""
    x, w = banded(M, N, K, kind, 1, np.arange(-90, 60), 5)
    clean = nv.matvec(x, w)
    z = x.clone()
    z[1, 77] = float("inf")
    z[2, 2200] = float("nan")
    got = nv.matvec(z, w)
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(got[keep], clean[keep])
    assert got[2].isnan().all()
    col = ref.dequantize64(w)[:, 77]
    want = np.where(col == 0, np.nan, np.copysign(np.inf, col))
    assert np.array_equal(got[1].double().cpu().numpy(), want, equal_nan=True)


def test_tokens_of_zeros_and_of_one_value_beside_wide_ones(cuda_device):
    """Tokens that are through after no pass, one and several, in one call."""
    x, w = banded(9, 77, 1088, "nvfp4", 1, np.arange(-100, 60), 8)
    x[0] = 0
    x[3] = 0
    x[3, 1000] = 2.0 ** -70
    x[5] = 1.5
    y, bound = ref.matvec64(x, w)
    got = nv.matvec(x, w)
    ref.check_product(got, y, bound)
    assert (got[0] == 0).all()
