"""rms_norm and silu_mul on the GPU against their 64-bit definitions (tests/layer_reference.py): every format, both
scale layouts, sizes from one value to long rows, strides, in-place calls, special values, streams and graphs."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import oracle
import workloads
import w4a4_gemm_quantize_b200 as nv

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "mxfp8", "mxfp4", "nvfp4"]


def bf16(shape, seed, std=1.0, outliers=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda") * std
    if outliers:
        x[:, torch.randperm(shape[1], generator=g, device="cuda")[:outliers]] *= 50
    return x.to(torch.bfloat16)


def check(q, v, fmt, layout, delta, sg=None, where=""):
    if fmt == "bf16":
        ref.check_bf16(q, v, delta, where)
    else:
        ref.check_blocks(q, v, fmt, layout, delta, sg)


# (1, 32) one block; 4096, 5376 the layers' rows; 16 * 1024 + 32: more than a unit per thread; 65536 the longest
NORM_SHAPES = [(1, 32), (1, 4096), (3, 96), (8, 5376), (9, 1056), (130, 2080), (300, 5376), (2, 16416), (301, 16416),
               (2, 40000), (1, 65536)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_norm(cuda_device, rows, cols, fmt):
    x, r = bf16((rows, cols), 1), bf16((rows, cols), 2, outliers=min(4, cols // 32))
    w = (1 + bf16((1, cols), 3, 0.2).float()).to(torch.bfloat16).view(-1)
    for layout, residual, weight, offset in (("swizzled", r, w, 0.0), ("linear", None, w, 1.0), ("linear", r, None, 0.0)):
        res = nv.rms_norm(x, weight, residual, eps=1e-5, weight_offset=offset, out_format=fmt, layout=layout)
        v, h = ref.norm64(x, residual, weight, 1e-5, offset)
        q = res
        if residual is not None:
            q, stream = res
            assert np.array_equal(stream.double().cpu().numpy(), h)
        check(q, v, fmt, layout, ref.NORM_DELTA, where=f"{fmt} {rows}x{cols}")


@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 7), (5, 33), (9, 3), (19, 8), (17, 1001), (777, 2201), (1, 130001),
                                       (3, 65552), (4, 2200), (20, 4099), (9, 16365), (9, 16369), (8, 12346)])
def test_norm_bf16_of_any_size(cuda_device, rows, cols):
    x, r, w = bf16((rows, cols), 1), bf16((rows, cols), 2), bf16((1, cols), 3).view(-1)
    for residual, weight in ((r, w), (None, w), (r, None)):
        res = nv.rms_norm(x, weight, residual, weight_offset=0.5)
        out, h = res if residual is not None else (res, x)
        v, h64 = ref.norm64(x, residual, weight, 1e-6, 0.5)
        assert np.array_equal(h.double().cpu().numpy(), h64)
        ref.check_bf16(out, v, ref.NORM_DELTA)
    want, h = nv.rms_norm(x, w, r)
    # from addresses and strides that take the path of single values
    wide = torch.zeros((rows + 2, cols + 3), dtype=torch.bfloat16, device="cuda")
    wide[1:-1, 1:-2] = x
    assert torch.equal(nv.rms_norm(wide[1:-1, 1:-2], w, r)[1], h)
    # nothing beside the outputs is written
    for shift in (16, 15):                               # at a 32-byte address, and at one of single values
        flat = [torch.full((rows * cols + 32,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        y, ho = (f[shift:shift + rows * cols].view(rows, cols) for f in flat)
        nv.rms_norm(x, w, r, out=y, residual_out=ho)
        ref.check_bf16(y, ref.norm64(x, r, w, 1e-6)[0], ref.NORM_DELTA)
        assert torch.equal(ho, h) and (shift != 16 or torch.equal(y, want))  # (the other path adds in another order)
        for f in flat:
            assert (f[:shift] == 7.0).all() and (f[shift + rows * cols:] == 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_norm_on_column_slices(cuda_device, fmt):
    """Row strides wider than the row, outputs between other columns, rows behind the last one: all left as they were."""
    buf = bf16((40, 1024), 5)
    keep = buf.clone()
    x, r = buf[:37, 64:576], bf16((37, 4096), 6)[:, 512:1024]
    out = torch.full((40, 1024), 7.0, dtype=torch.bfloat16, device="cuda") if fmt == "bf16" else None
    res = nv.rms_norm(x, None, r, out_format=fmt, out=out[:37, 256:768] if out is not None else None)
    v, h = ref.norm64(x, r, None, 1e-6)
    assert np.array_equal(res[1].double().cpu().numpy(), h)
    check(res[0], v, fmt, "swizzled", ref.NORM_DELTA)
    assert torch.equal(buf, keep)
    if out is not None:
        out[:37, 256:768] = 7.0
        assert (out == 7.0).all()


@pytest.mark.parametrize("rows,cols", [(5, 512), (400, 2048), (3, 100), (2, 40000)])
def test_norm_in_place(cuda_device, rows, cols):
    """The residual updated in place, the BF16 output over x; and the residual stream written over x."""
    x, r = bf16((rows, cols), 1), bf16((rows, cols), 2)
    want, h = nv.rms_norm(x, None, r)
    x1, r1 = x.clone(), r.clone()
    out, ro = nv.rms_norm(x1, None, r1, out=x1, residual_out=r1)
    assert out is x1 and ro is r1
    assert torch.equal(out, want) and torch.equal(ro, h)
    x2 = x.clone()
    out, ro = nv.rms_norm(x2, None, r, residual_out=x2)
    assert torch.equal(out, want) and torch.equal(x2, h)
    if cols % 32 == 0:
        for fmt in ("nvfp4", "mxfp8"):
            a, _ = nv.rms_norm(x, None, r, out_format=fmt)
            r3 = r.clone()
            b, _ = nv.rms_norm(x, None, r3, out_format=fmt, residual_out=r3)
            assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scales, b.scales)
            assert torch.equal(r3, h)


@pytest.mark.parametrize("rows", [1, 8, 200])
def test_norm_exact_values_encode_like_the_quantizer(cuda_device, rows):
    """Rows whose root mean square is a power of two normalise without any rounding, so the codes and scales must be
    the quantizer's of those values, bit for bit: ties included (the values sit on rounding borders)."""
    r = np.random.default_rng(rows)
    patterns = [[5, 2, 1, 1, 1, 0, 0, 0] * 2,                                # mean square 4
                [15, 5, 2, 1, 1] + [0] * 11,                                # 16
                [7, 3, 2, 1, 1] + [0] * 11]                                 # 4
    cols = 512
    x = np.zeros((rows, cols))
    for i in range(rows):
        row = np.concatenate([r.permutation(patterns[i % 3]) for _ in range(cols // 16)])
        x[i] = row * r.choice([-1.0, 1.0], cols) * 2.0 ** r.integers(-3, 4)
    xt = workloads.to_bf16(x.astype(np.float32))
    v = (x / np.sqrt((x ** 2).mean(1, keepdims=True))).astype(np.float32)
    vt = workloads.to_bf16(v)
    assert np.array_equal(vt.double().numpy(), v.astype(np.float64))          # the values are BF16
    codes, sc = oracle.quantize_mx(vt)
    q = nv.rms_norm(xt.cuda(), eps=0.0, out_format="mxfp4", layout="linear")
    assert np.array_equal(q.codes.cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy(), sc)
    for sg in (None, np.float32(0.0123)):
        codes, sc, want_sg, _ = oracle.quantize(vt, oracle.SCALE_ABSMAX, sg)
        given = None if sg is None else torch.tensor([sg], device="cuda")
        q = nv.rms_norm(xt.cuda(), eps=0.0, out_format="nvfp4", global_scale=given)
        assert q.global_scale.item() == want_sg
        assert np.array_equal(q.codes.cpu().numpy(), codes)
        assert np.array_equal(q.scales.cpu().numpy(), oracle.swizzle_scales(sc))
    out = nv.rms_norm(xt.cuda(), eps=0.0)
    assert np.array_equal(out.cpu().double().numpy(), v.astype(np.float64))


@pytest.mark.parametrize("fmt", FORMATS)
def test_norm_of_zero_rows_and_extreme_rows(cuda_device, fmt):
    x = torch.zeros((6, 128), dtype=torch.bfloat16, device="cuda")
    q = nv.rms_norm(x, out_format=fmt, layout="linear")                   # all zero: eps alone under the root
    check(q, np.zeros((6, 128)), fmt, "linear", ref.NORM_DELTA)
    x[1] = bf16((1, 128), 3)[0]
    x[2] = bf16((1, 128), 4)[0] * 1e-20                                   # eps outweighs it
    x[3] = bf16((1, 128), 5)[0] * 1e15
    x[4, 5] = -3.0
    v, _ = ref.norm64(x, None, None, 1e-6)
    check(nv.rms_norm(x, out_format=fmt, layout="linear"), v, fmt, "linear", ref.NORM_DELTA)


def test_norm_with_non_finite_values(cuda_device):
    """A row with a NaN or an infinity is its formula's NaNs and zeros; the other rows are as without it."""
    x = bf16((5, 256), 1)
    clean = nv.rms_norm(x)
    y = x.clone()
    y[1, 7] = float("nan")
    y[3, 9] = float("inf")
    out = nv.rms_norm(y)
    assert torch.equal(out[[0, 2, 4]], clean[[0, 2, 4]])
    assert out[1].isnan().all() and out[3, 9].isnan() and (out[3, :9] == 0).all()
    q = nv.rms_norm(y, out_format="mxfp8", layout="linear")
    assert (q.scales[1] == 255).all() and (q.scales[3, 0] == 255)
    c = nv.rms_norm(x, out_format="mxfp8", layout="linear")
    assert torch.equal(q.scales[[0, 2, 4]], c.scales[[0, 2, 4]])
    assert torch.equal(q.codes.view(torch.uint8)[[0, 2, 4]], c.codes.view(torch.uint8)[[0, 2, 4]])
    gs = torch.tensor([0.002], device="cuda")
    q = nv.rms_norm(y, out_format="nvfp4", layout="linear", global_scale=gs)
    assert (q.scales[1] == 0x7F).all()


GATE_SHAPES = [(1, 32), (1, 14336), (37, 1440), (7, 96), (129, 544), (1000, 1056), (64, 14336)]


@pytest.mark.parametrize("rows,cols", GATE_SHAPES)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", ["swizzled", "linear"])
def test_gate(cuda_device, rows, cols, fmt, layout):
    g, u = bf16((rows, cols), 1, 3.0), bf16((rows, cols), 2)
    q = nv.silu_mul(g, u, out_format=fmt, layout=layout)
    check(q, ref.gate64(g, u), fmt, layout, ref.GATE_DELTA)


@pytest.mark.parametrize("op", ["norm", "gate"])
@pytest.mark.parametrize("rows,cols", [(3, 80), (200, 4112)])
def test_nvfp4_sixteen_wide_tail_and_given_scale(cuda_device, op, rows, cols):
    """cols a multiple of 16 but not of 32, the tensor scale given (small enough that scales saturate in places)."""
    x, u = bf16((rows, cols), 1, 2.0), bf16((rows, cols), 2)
    for sg in (0.0031, 1e-5):
        gs = torch.tensor([sg], device="cuda")
        if op == "norm":
            q = nv.rms_norm(x, None, out_format="nvfp4", global_scale=gs)
            v, delta = ref.norm64(x, None, None, 1e-6)[0], ref.NORM_DELTA
        else:
            q = nv.silu_mul(x, u, out_format="nvfp4", global_scale=gs)
            v, delta = ref.gate64(x, u), ref.GATE_DELTA
        ref.check_blocks(q, v, "nvfp4", "swizzled", delta, float(np.float32(sg)))
    q = nv.rms_norm(x, out_format="nvfp4") if op == "norm" else nv.silu_mul(x, u, out_format="nvfp4")
    ref.check_blocks(q, ref.norm64(x, None, None, 1e-6)[0] if op == "norm" else v, "nvfp4", "swizzled", delta)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (1, 15), (1, 16), (1, 5001), (100, 333), (64, 1000), (3, 1025)])
def test_gate_bf16_of_any_size(cuda_device, rows, cols):
    g, u = bf16((rows, cols), 1, 3.0), bf16((rows, cols), 2)
    want = ref.gate64(g, u)
    ref.check_bf16(nv.silu_mul(g, u), want, ref.GATE_DELTA)
    wide = torch.zeros((rows, cols + 3), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:-2] = g
    ref.check_bf16(nv.silu_mul(wide[:, 1:-2], u), want, ref.GATE_DELTA)
    flat = torch.full((rows * cols + 32,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = flat[16:16 + rows * cols].view(rows, cols)
    ref.check_bf16(nv.silu_mul(g, u, out=y), want, ref.GATE_DELTA)
    assert (flat[:16] == 7.0).all() and (flat[-16:] == 7.0).all()
    if rows * cols >= 16:
        ref.check_bf16(nv.silu_mul(g, u, out=g), want, ref.GATE_DELTA)      # in place


@pytest.mark.parametrize("cols", [512, 100])
def test_gate_on_the_halves_of_a_product_and_in_place(cuda_device, cols):
    both = bf16((70, 2 * cols), 1, 2.0)
    g, u = both[:, :cols], both[:, cols:]
    want = nv.silu_mul(g.contiguous(), u.contiguous())
    assert torch.equal(nv.silu_mul(g, u), want)
    half = u.clone()
    out = nv.silu_mul(g, u, out=g)
    assert torch.equal(out, want) and torch.equal(both[:, :cols], want) and torch.equal(both[:, cols:], half)


def test_gate_every_bf16_argument(cuda_device):
    """silu of every BF16 value: tails, subnormals, infinities, NaN."""
    bits = np.arange(65536, dtype=np.uint16).reshape(256, 256)
    g = workloads.from_bits(bits).cuda()
    out = nv.silu_mul(g, torch.ones_like(g))
    g64 = g.double().cpu().numpy()
    with np.errstate(all="ignore"):
        v = g64 / (1.0 + np.exp(-g64))
    v[np.isneginf(g64)] = np.nan                         # -inf / inf, as the formula has it
    got = out.double().cpu().numpy()
    deep = np.isfinite(g64) & (g64 < -87.0)              # e^-g leaves binary32's range: 0, off by at most 1e-36
    assert (np.abs(got[deep]) <= 2e-36).all()
    v[deep] = got[deep]
    ref.check_bf16(out, v, ref.GATE_DELTA)


@pytest.mark.parametrize("op", ["norm", "gate"])
def test_empty_rows(cuda_device, op):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    for fmt in FORMATS:
        q = nv.rms_norm(x, out_format=fmt) if op == "norm" else nv.silu_mul(x, x, out_format=fmt)
        if fmt == "nvfp4":
            assert q.global_scale.item() == 1.0 and q.codes.shape == (0, 32)


@pytest.mark.parametrize("op", ["norm", "gate"])
@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("rows", [1, 5, 161])
def test_outputs_stay_inside_their_buffers(cuda_device, op, fmt, rows):
    """Codes and scales between 4 KiB margins that nothing may touch; a workspace of any content."""
    cols, block = 2080, 16 if fmt == "nvfp4" else 32
    x, u = bf16((rows, cols), 1), bf16((rows, cols), 2)
    width = cols if fmt == "mxfp8" else cols // 2
    size = nv.mxfp8_scales_bytes if fmt == "mxfp8" else nv.scales_bytes

    def margin(n):
        t = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        return t, t[4096:4096 + n]

    tc, codes = margin(rows * width)
    ts, scales = margin(size(rows, cols, "swizzled"))
    if fmt == "mxfp8":
        out = nv.MXFP8Tensor(codes.view(torch.float8_e4m3fn).view(rows, width), scales, rows, cols)
    else:
        out = nv.NVFP4Tensor(codes.view(rows, width), scales, torch.zeros(1, device="cuda"), rows, cols)
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    call = (lambda **k: nv.rms_norm(x, out_format=fmt, **k)) if op == "norm" else \
        (lambda **k: nv.silu_mul(x, u, out_format=fmt, **k))
    q = call(out=out, workspace=ws)
    fresh = call()
    assert q is out
    assert torch.equal(q.codes.view(torch.uint8), fresh.codes.view(torch.uint8)) and torch.equal(q.scales, fresh.scales)
    for t in (tc, ts):
        assert (t[:4096] == 0xA5).all() and (t[-4096:] == 0xA5).all()


def test_refusals(cuda_device):
    x = bf16((4, 64), 1)
    for call in (lambda: nv.rms_norm(x.float()), lambda: nv.rms_norm(x[0]), lambda: nv.rms_norm(x.t()),
                 lambda: nv.rms_norm(x, x[0, :32]), lambda: nv.rms_norm(x, None, x[:2]),
                 lambda: nv.rms_norm(x, residual_out=x), lambda: nv.rms_norm(x, out=x[:, :32]),
                 lambda: nv.rms_norm(x, global_scale=torch.ones(1, device="cuda")),
                 lambda: nv.rms_norm(x, out_format="nvfp4", global_scale=torch.ones(1)),
                 lambda: nv.rms_norm(bf16((4, 48), 1), out_format="mxfp8"),
                 lambda: nv.rms_norm(x, out_format="mxfp8", out=nv.rms_norm(x, out_format="mxfp4")),
                 lambda: nv.rms_norm(x, out_format="mxfp8", out=nv.rms_norm(x, out_format="mxfp8", layout="linear")),
                 lambda: nv.silu_mul(x, x[:2]), lambda: nv.silu_mul(x, x.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: nv.rms_norm(x, eps=-1.0), lambda: nv.rms_norm(x[:1].expand(4, 64)),
                 lambda: nv.rms_norm(bf16((4, 72), 1)[:, 4:68], out_format="mxfp8"),
                 lambda: nv.rms_norm(x, None, x, residual_out=x, out=x),
                 lambda: nv.silu_mul(x, x, out_format="nvfp4", workspace=torch.empty(64, dtype=torch.uint8,
                                                                                     device="cuda"))):
        with pytest.raises(nv.Nvfp4Error):
            call()


@pytest.mark.parametrize("op", ["norm", "gate"])
@pytest.mark.parametrize("rows", [4, 300])
def test_graph_replay_on_new_inputs(cuda_device, op, rows):
    """Captured once and replayed on other data: the computed tensor scale is of the data at replay."""
    x, u = bf16((rows, 2048), 1), bf16((rows, 2048), 2)

    def call():
        return nv.rms_norm(x, None, u, out_format="nvfp4")[0] if op == "norm" else nv.silu_mul(x, u, out_format="nvfp4")
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = call()
    for seed, std in ((7, 40.0), (8, 0.01)):
        x.copy_(bf16((rows, 2048), seed, std))
        u.copy_(bf16((rows, 2048), seed + 100, std))
        graph.replay()
        want = call()
        assert q.global_scale.item() == want.global_scale.item()
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)


def test_on_another_stream(cuda_device):
    """The work goes to the named stream, behind what is queued there; temporaries live until it is done."""
    side = torch.cuda.Stream()
    x = bf16((300, 4096), 1)
    want = nv.rms_norm(x, out_format="nvfp4")
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        y = torch.zeros_like(x)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            y.copy_(x)
        q = nv.rms_norm(y, out_format="nvfp4", stream=s)
        junk = [torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(8)]  # not over the workspace
        side.synchronize()
        assert len(junk) == 8 and torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    with torch.cuda.stream(side):
        q = nv.rms_norm(x, out_format="nvfp4")
    side.synchronize()
    assert torch.equal(q.codes, want.codes)


@pytest.mark.parametrize("op", ["norm", "gate"])
def test_past_two_to_the_31_elements(cuda_device, op):
    """Rows whose element offsets pass 32 bits, in BF16 and in NVFP4 under a computed tensor scale: the first and last
    rows equal the same rows computed alone."""
    rows, cols = 66_000, 32768
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.view(-1).view(torch.int16).random_(0x3C00, 0x4000)              # BF16 magnitudes of 2^-7 to 2
    if op == "norm":
        def call(t, **k):
            return nv.rms_norm(t, **k)
    else:
        def call(t, **k):
            return nv.silu_mul(t, t, **k)
    parts = (slice(0, 3), slice(65536, 65539), slice(rows - 3, rows))
    out = call(x)
    for p in parts:
        assert torch.equal(out[p], call(x[p].clone()))
    del out
    q = call(x, out_format="nvfp4", layout="linear")
    for p in parts:
        alone = call(x[p].clone(), out_format="nvfp4", layout="linear", global_scale=q.global_scale)
        assert torch.equal(q.codes[p], alone.codes) and torch.equal(q.scales[p], alone.scales)


def test_rows_and_formats_drawn_at_random(cuda_device):
    """Sizes drawn over the whole range, odd ones among them, each format and operator."""
    r = np.random.default_rng(11)
    for i in range(80):
        fmt = FORMATS[i % 4]
        step = {"bf16": 1, "nvfp4": 16}.get(fmt, 32)
        cols = step * int(np.exp(r.uniform(0, np.log(12000 / step))))
        rows = int(np.exp(r.uniform(0, np.log(2e6 / cols))))
        layout = ("swizzled", "linear")[i // 4 % 2]
        x, y = bf16((rows, cols), i, 2.0), bf16((rows, cols), i + 1000)
        if r.random() < 0.5:
            w = bf16((1, cols), 5).view(-1)
            q, h = nv.rms_norm(x, w, y, out_format=fmt, layout=layout)
            v, h64 = ref.norm64(x, y, w, 1e-6)
            assert np.array_equal(h.double().cpu().numpy(), h64)
            delta = ref.NORM_DELTA
        else:
            q, v, delta = nv.silu_mul(x, y, out_format=fmt, layout=layout), ref.gate64(x, y), ref.GATE_DELTA
        check(q, v, fmt, layout, delta, where=f"{fmt} {rows}x{cols}")
