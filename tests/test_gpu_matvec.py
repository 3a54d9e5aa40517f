"""matvec on the GPU against the 64-bit product of the dequantized weight (tests/layer_reference.py), and the layer
operators run together as a decoder's MLP uses them."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import w4a4_gemm_quantize_b200 as nv

pytestmark = pytest.mark.gpu


def bf16(shape, seed, std=1.0, outliers=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda") * std
    if outliers:
        x[:, torch.randperm(shape[1], generator=g, device="cuda")[:outliers]] *= 50
    return x.to(torch.bfloat16)


def weight(N, K, kind, seed):
    w = bf16((N, K), seed, 0.02)
    return nv.nvfp4_quantize(w) if kind == "nvfp4" else nv.mxfp4_quantize(w)


def mxfp8(x, layout="linear"):
    """x as MXFP8 through plain torch operations."""
    v = x.float().view(x.shape[0], -1, 32)
    amax = v.abs().amax(2, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 9, -127).clamp(-127, 127)
    codes = torch.ldexp(v, -e).clamp(-448, 448).to(torch.float8_e4m3fn).view(x.shape)
    s = (e + 127).to(torch.uint8).view(x.shape[0], -1)
    if layout == "linear":
        return nv.MXFP8Tensor(codes, s.contiguous(), *x.shape, nv.SF_LINEAR)
    import oracle
    return nv.MXFP8Tensor(codes, torch.from_numpy(oracle.swizzle_scales(s.cpu().numpy())).cuda(), *x.shape)


def values(x):
    return x if isinstance(x, torch.Tensor) else torch.from_numpy(ref.dequantize64(x))


# N: one row, fewer than a 128-row group's lines, partial groups, more tiles than one round of partial sums;
# K: one block pair, partial chunks, fewer chunks than warps, several slices of x
SHAPES = [(1, 1, 32), (1, 5, 64), (3, 33, 96), (2, 130, 1056), (5, 1001, 160), (8, 256, 2048), (9, 200, 4096),
          (16, 300, 4128), (16, 77, 21504), (1, 14336, 4096), (7, 520, 14336), (11, 96, 28672), (1, 64, 65536),
          (16, 8192, 512), (13, 20000, 128), (16, 40, 65536), (1, 33, 524288), (12, 30000, 2048), (2, 65536, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_matvec(cuda_device, M, N, K, kind):
    x = bf16((M, K), M, outliers=min(4, K // 32))
    w = weight(N, K, kind, N + K)
    y, bound = ref.matvec64(x, w)
    got = nv.matvec(x, w)
    ref.check_product(got, y, bound, f"{kind} {M}x{N}x{K}")
    assert torch.equal(got, nv.matvec(x, w))                        # the same bits on every call
    for layout in ("linear", "swizzled"):
        x8 = mxfp8(x, layout)
        y, bound = ref.matvec64(values(x8), w)
        ref.check_product(nv.matvec(x8, w), y, bound, f"{kind} mxfp8 {M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 1000, 5376), (4, 130, 1056), (16, 515, 4096), (16, 4000, 8192),
                                   (9, 40, 21504), (2, 30000, 256)])
@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_matvec_gated(cuda_device, M, N, K, kind):
    x = bf16((M, K), M)
    w, g = weight(N, K, kind, 1), weight(N, K, kind, 2)
    if kind == "nvfp4":
        g.global_scale.mul_(4.0)                                    # each product under its own tensor scale
    y, bound = ref.matvec64(x, w, g)
    ref.check_product(nv.matvec(x, w, g), y, bound, f"gated {kind} {M}x{N}x{K}", min_exact=0.85)
    x8 = mxfp8(x)
    y, bound = ref.matvec64(values(x8), w, g)
    ref.check_product(nv.matvec(x8, w, g), y, bound, f"gated {kind} mxfp8 {M}x{N}x{K}", min_exact=0.85)


def test_matvec_on_many_shapes(cuda_device):
    """Sizes drawn over the whole range: every split of K over a cluster, tiles and chunks that end anywhere."""
    r = np.random.default_rng(7)
    for i in range(60):
        M, K = int(r.integers(1, 17)), 32 * int(np.exp(r.uniform(0, np.log(700))))
        N = int(np.exp(r.uniform(0, np.log(min(6000, 4e7 / K)))))
        kind, gated, fp8 = ("nvfp4", "mxfp4")[i % 2], r.random() < 0.3, r.random() < 0.4
        x = bf16((M, K), i)
        x = mxfp8(x, ("linear", "swizzled")[i // 2 % 2]) if fp8 else x
        w, g = weight(N, K, kind, i), weight(N, K, kind, i + 100) if gated else None
        y, bound = ref.matvec64(values(x), w, g)
        ref.check_product(nv.matvec(x, w, g), y, bound, f"{kind} {M}x{N}x{K} gated={gated} fp8={fp8}", 0.85)


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_matvec_long_rows_token_by_token(cuda_device, kind):
    """Rows so long that x is handled a few tokens at a time, its scale rows at odd offsets."""
    M, N, K = 3, 40, 2 ** 19 - 32
    w = weight(N, K, kind, 1)
    for x in (bf16((M, K), 2), mxfp8(bf16((M, K), 2)), mxfp8(bf16((M, K), 2), "swizzled")):
        y, bound = ref.matvec64(values(x), w)
        ref.check_product(nv.matvec(x, w), y, bound, f"{kind} {M}x{N}x{K}")
        assert nv.last_launch_count() == 3


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_matvec_past_two_to_the_31_bytes_of_codes(cuda_device, kind):
    """A weight whose last rows lie more than 2^31 bytes behind its first: random codes, sampled rows checked."""
    N, K, M = 140_000, 32768, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    block = 16 if kind == "nvfp4" else 32
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    n = (N + 127) // 128 * 128 * (K // block)
    low, high = (0x30, 0x48) if kind == "nvfp4" else (118, 126)
    scales = torch.randint(low, high, (n,), generator=g, device="cuda", dtype=torch.uint8)
    if kind == "nvfp4":
        w = nv.NVFP4Tensor(codes, scales, torch.tensor([0.01], device="cuda"), N, K)
    else:
        w = nv.MXFP4Tensor(codes, scales, N, K)
    x = bf16((M, K), 1)
    got = nv.matvec(x, w)
    group = slice((N // 128) * 128, N)                       # the last rows, and rows of two groups on the way
    for rows in (slice(0, 128), slice(65536, 65536 + 128), group):
        a, b = rows.start, rows.stop
        per_group = 128 * (K // block)
        part = scales[a // 128 * per_group: (b + 127) // 128 * per_group]
        sub = (nv.NVFP4Tensor(codes[a:b], part, w.global_scale, b - a, K) if kind == "nvfp4"
               else nv.MXFP4Tensor(codes[a:b], part, b - a, K))
        m = torch.from_numpy(dequantize_any(sub)).cuda()
        y = x.double() @ m.t()
        S = (x.double().abs() @ m.abs().t()) * 2.0 ** -14
        ref.check_product(got[:, a:b], y.cpu().numpy(), S.cpu().numpy(), f"rows {a}..{b}")


def dequantize_any(w):
    """ref.dequantize64 without its look at the scales' padding (which is random here)."""
    import oracle
    block = 16 if isinstance(w, nv.NVFP4Tensor) else 32
    s = oracle.unswizzle_scales(w.scales.cpu().numpy(), w.rows, w.cols // block)
    eff = ref.e4m3_values(s) * float(w.global_scale.item()) if block == 16 else 2.0 ** (s.astype(np.float64) - 127)
    v = ref.code_values(w, "fp4").reshape(w.rows, -1, block)
    return (v * eff[..., None]).reshape(w.rows, w.cols)


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_matvec_strides_and_margins(cuda_device, kind):
    """x a column slice, y a column slice of odd stride: nothing beside them is read into it or written."""
    M, N, K = 5, 333, 544
    buf = bf16((M, K + 64), 1)
    buf[:, :32] = float("nan")
    buf[:, 32 + K:] = float("nan")
    x = buf[:, 32:32 + K]
    w = weight(N, K, kind, 3)
    out = torch.full((M + 1, N + 6), 7.0, dtype=torch.bfloat16, device="cuda")
    got = nv.matvec(x, w, out=out[:M, 3:3 + N])
    assert torch.equal(got, nv.matvec(x.contiguous(), w))
    out[:M, 3:3 + N] = 7.0
    assert (out == 7.0).all()


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_matvec_reads_no_row_or_block_past_the_weight(cuda_device, kind):
    """Scale padding of any content (NaN scales) does not reach the result."""
    M, N, K = 3, 45, 96
    w = weight(N, K, kind, 3)
    x = bf16((M, K), 1)
    want = nv.matvec(x, w)
    import oracle
    nblk = K // (16 if kind == "nvfp4" else 32)
    lin = oracle.unswizzle_scales(w.scales.cpu().numpy(), N, nblk)
    full = np.full((128, -(-nblk // 4) * 4), 0x7F if kind == "nvfp4" else 0xFF, np.uint8)
    full[:N, :nblk] = lin
    w.scales.copy_(torch.from_numpy(oracle.swizzle_scales(full)))
    assert torch.equal(nv.matvec(x, w), want)


def test_matvec_mxfp4_scales_of_every_power(cuda_device):
    """E8M0 scales from 2^-127 to 2^100 in one weight: no binary16 holds them, the products must be exact."""
    N, K = 256, 128
    r = np.random.default_rng(0)
    w = weight(N, K, "mxfp4", 5)
    byte = np.tile(np.minimum(np.arange(N), 227)[:, None], (1, K // 32)).astype(np.uint8)
    byte[:, 1] = np.maximum(byte[:, 0].astype(int) - 20, 0)            # blocks of one row far apart
    byte[:, 2] = r.integers(0, 228, N)
    import oracle
    w.scales.copy_(torch.from_numpy(oracle.swizzle_scales(byte)))
    x = bf16((2, K), 6)
    y, bound = ref.matvec64(x, w)
    ref.check_product(nv.matvec(x, w), y, bound)


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_matvec_scale_of_the_activation(cuda_device, kind):
    """Tokens from 2^-120 to 2^110, zero tokens, and values far apart within a token."""
    M, N, K = 16, 96, 4096
    x = bf16((M, K), 1).float()
    p = torch.tensor([-120, -100, -60, -20, -1, 0, 1, 20, 60, 100, 108, 0, 0, 0, 0, 0], device="cuda")
    x = torch.ldexp(x, p[:, None])
    x[11] = 0
    x[12, :] = 0
    x[12, 4095] = 3.0
    x[13, ::2] *= 2.0 ** -19                      # within the 21 binades that stay exact
    x[14, ::2] *= 2.0 ** -30                      # below: rounded at 2^-32 of the largest
    x[15, 64:] *= 2.0 ** -40
    x = x.to(torch.bfloat16)
    w = weight(N, K, kind, 3)
    y, bound = ref.matvec64(x, w)
    ref.check_product(nv.matvec(x, w), y, bound)


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_matvec_with_non_finite_activations(cuda_device, kind):
    """Infinities and NaN stay in their token; its finite values keep their scaling."""
    M, N, K = 4, 40, 2304
    x = bf16((M, K), 1)
    w = weight(N, K, kind, 3)
    clean = nv.matvec(x, w)
    z = x.clone()
    z[1, 77] = float("inf")
    z[2, 2200] = float("nan")
    got = nv.matvec(z, w)
    assert torch.equal(got[[0, 3]], clean[[0, 3]])
    assert got[2].isnan().all()
    col = ref.dequantize64(w)[:, 77]
    want = np.where(col == 0, np.nan, np.copysign(np.inf, col))
    assert np.array_equal(got[1].double().cpu().numpy(), want, equal_nan=True)


def test_matvec_empty_batch_and_refusals(cuda_device):
    w, m = weight(64, 96, "nvfp4", 1), weight(64, 96, "mxfp4", 1)
    x = bf16((2, 96), 1)
    assert nv.matvec(x[:0], w).shape == (0, 64)
    lin = nv.nvfp4_quantize(bf16((64, 96), 1), layout="linear")
    for call in (lambda: nv.matvec(x, lin), lambda: nv.matvec(x[:, :64], w), lambda: nv.matvec(x.float(), w),
                 lambda: nv.matvec(x, w, m), lambda: nv.matvec(x, w, weight(32, 96, "nvfp4", 1)),
                 lambda: nv.matvec(x, x), lambda: nv.matvec(x, w, out=torch.empty((2, 63), dtype=torch.bfloat16,
                                                                                  device="cuda")),
                 lambda: nv.matvec(nv.MXFP8Tensor(x, x, 2, 96), w),
                 lambda: nv.matvec(x, nv.NVFP4Tensor(w.codes[:32], w.scales, w.global_scale, 64, 96)),
                 lambda: nv.matvec(x, nv.NVFP4Tensor(w.codes, w.scales[:-4], w.global_scale, 64, 96)),
                 lambda: nv.matvec(x, nv.NVFP4Tensor(w.codes, w.scales.cpu(), w.global_scale, 64, 96)),
                 lambda: nv.matvec(x, nv.NVFP4Tensor(w.codes, w.scales, w.global_scale.cpu(), 64, 96))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: nv.matvec(bf16((17, 96), 1), w), lambda: nv.matvec(bf16((2, 100), 1)[:, :96], w),
                 lambda: nv.matvec(x, nv.nvfp4_quantize(bf16((96, 96), 1)), out=x)):
        with pytest.raises(nv.Nvfp4Error):
            call()


def test_matvec_two_streams_and_graph(cuda_device):
    """Two calls at once on two streams, and a captured call replayed on new tokens: no shared state."""
    w1, w2 = weight(2000, 4096, "nvfp4", 1), weight(2000, 4096, "mxfp4", 2)
    x = bf16((8, 4096), 1)
    want1, want2 = nv.matvec(x, w1), nv.matvec(x, w2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(nv.matvec(x, w1, stream=s1), nv.matvec(x, w2, stream=s2)) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want1) and torch.equal(b, want2) for a, b in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nv.matvec(x, w1)
        z = nv.matvec(x, w2, w2)
    for seed in (5, 6):
        x.copy_(bf16((8, 4096), seed))
        graph.replay()
        assert torch.equal(y, nv.matvec(x, w1)) and torch.equal(z, nv.matvec(x, w2, w2))


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
@pytest.mark.parametrize("tokens", [1, 16])
def test_decode_mlp(cuda_device, kind, fmt, tokens):
    """One MLP of a decoder layer at decode: norm (residual added) -> gated matvec -> matvec, 4-bit weights.  Each
    step is checked on the inputs the step before it produced."""
    H, F = 1056, 2208
    x, r = bf16((tokens, H), 1), bf16((tokens, H), 2, outliers=4)
    nw = (1 + bf16((1, H), 3, 0.1).float()).to(torch.bfloat16).view(-1)
    gate, up, down = weight(F, H, kind, 4), weight(F, H, kind, 5), weight(H, F, kind, 6)
    a, h = nv.rms_norm(x, nw, r, out_format=fmt)
    y = nv.matvec(a, up, gate)
    z = nv.matvec(y, down)
    v, h64 = ref.norm64(x, r, nw, 1e-6)
    assert np.array_equal(h.double().cpu().numpy(), h64)
    if fmt == "bf16":
        ref.check_bf16(a, v, ref.NORM_DELTA)
    else:
        ref.check_blocks(a, v, fmt, "swizzled", ref.NORM_DELTA)
    ref.check_product(y, *ref.matvec64(values(a), up, gate), "gated", 0.85)
    ref.check_product(z, *ref.matvec64(y, down), "down")


@pytest.mark.parametrize("kind", ["nvfp4", "mxfp4"])
def test_prompt_mlp(cuda_device, kind):
    """The same layer on a prompt: norm and gate write what the library's block-scaled GEMMs read."""
    T, H, F = 200, 1024, 1536
    x, r = bf16((T, H), 1), bf16((T, H), 2, outliers=4)
    up, down = weight(2 * F, H, kind, 5), weight(H, F, kind, 6)
    gemm = nv.nvfp4_gemm if kind == "nvfp4" else nv.mxfp4_gemm
    a, h = nv.rms_norm(x, None, r, out_format=kind)
    both = gemm(a, up)
    b = nv.silu_mul(both[:, :F], both[:, F:], out_format=kind)
    z = gemm(b, down)
    v, _ = ref.norm64(x, r, None, 1e-6)
    ref.check_blocks(a, v, kind, "swizzled", ref.NORM_DELTA)
    ref.check_blocks(b, ref.gate64(both[:, :F], both[:, F:]), kind, "swizzled", ref.GATE_DELTA)
    for out, p, q in ((both, a, up), (z, b, down)):
        A, B = (torch.from_numpy(ref.dequantize64(t)).cuda() for t in (p, q))
        y, S = (A @ B.t()).cpu().numpy(), (A.abs() @ B.abs().t()).cpu().numpy()
        ref.check_product(out, y, 1e-3 * S + 1e-6, "gemm")           # the GEMM's stated bound
