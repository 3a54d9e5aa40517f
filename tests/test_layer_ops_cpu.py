"""The decoder-layer operators on a machine without a GPU: the C entry points' checks answer before any CUDA
call, and the Python calls refuse what they cannot run.  No compute call is made here."""
import ctypes

import numpy as np
import pytest
import torch

import layer_reference as ref
import w4a4_gemm_quantize_b200 as nv
from w4a4_gemm_quantize_b200 import build as nvbuild

NO_DEVICE = (4, 5)   # everything valid: the device check runs and fails without a GPU


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return nv.load_library()


def P(v):
    return ctypes.c_void_p(v) if v else None


def norm(lib, x=1 << 20, rows=4, cols=64, ld=64, res=0, ld_res=64, res_out=0, ld_res_out=64, weight=0, offset=0.0,
         eps=1e-6, fmt=0, layout=0, gs=0, out=2 << 20, ld_out=64, scales=0, gs_out=0, ws=0, ws_bytes=256):
    return lib.nvfp4_rms_norm(P(x), rows, cols, ld, P(res), ld_res, P(res_out), ld_res_out, P(weight), offset, eps, fmt,
                              layout, P(gs), P(out), ld_out, P(scales), P(gs_out), P(ws), ws_bytes, None)


def test_rms_norm_validation(lib):
    block = dict(scales=3 << 20)
    assert norm(lib) in NO_DEVICE
    assert norm(lib, cols=33, ld=33, ld_out=33) in NO_DEVICE           # BF16: any size and stride
    assert norm(lib, x=(1 << 20) + 2) in NO_DEVICE
    assert norm(lib, x=(1 << 20) + 1) == 3
    assert norm(lib, rows=-1) == 1 and norm(lib, cols=0) == 1
    assert norm(lib, rows=0) in NO_DEVICE
    assert norm(lib, x=0) == 1 and norm(lib, out=0) == 1
    assert norm(lib, ld=63) == 1 and norm(lib, ld_out=63) == 1
    assert norm(lib, fmt=4) == 1 and norm(lib, fmt=-1) == 1 and norm(lib, layout=2) == 1
    assert norm(lib, eps=-1.0) == 1 and norm(lib, eps=float("nan")) == 1 and norm(lib, eps=float("inf")) == 1
    assert norm(lib, eps=0.0) in NO_DEVICE and norm(lib, offset=float("inf")) == 1
    assert norm(lib, scales=3 << 20) == 1                              # BF16 has no scales
    assert norm(lib, gs=3 << 20) == 1 and norm(lib, gs_out=3 << 20) == 1
    for fmt in (1, 2):
        assert norm(lib, fmt=fmt, **block) in NO_DEVICE
        assert norm(lib, fmt=fmt) == 1                                 # no scales
        assert norm(lib, fmt=fmt, cols=48, **block) == 2
        assert norm(lib, fmt=fmt, gs=4 << 20, **block) == 1
        assert norm(lib, fmt=fmt, x=(1 << 20) + 8, **block) == 3
        assert norm(lib, fmt=fmt, ld=68, **block) == 3
        assert norm(lib, fmt=fmt, weight=(4 << 20) + 2, **block) == 3
        assert norm(lib, fmt=fmt, cols=65536 + 32, ld=65536 + 32, scales=8 << 20, out=16 << 20) == 2
    assert norm(lib, fmt=3, **block) == 7                              # computed scale, no workspace
    assert norm(lib, fmt=3, ws=4 << 20, ws_bytes=255, **block) == 7
    assert norm(lib, fmt=3, ws=(4 << 20) + 8, **block) == 3
    assert norm(lib, fmt=3, ws=4 << 20, **block) in NO_DEVICE
    assert norm(lib, fmt=3, gs=4 << 20, **block) in NO_DEVICE
    assert norm(lib, fmt=3, gs=(4 << 20) + 2, **block) == 3
    assert norm(lib, fmt=3, cols=24, gs=4 << 20, **block) == 2
    assert norm(lib, rows=(1 << 30) + 1) == 2


def test_rms_norm_residual_and_overlap(lib):
    A, B, C, D = 1 << 20, 2 << 20, 3 << 20, 4 << 20
    assert norm(lib, res=C) == 1 and norm(lib, res_out=C) == 1
    assert norm(lib, res=C, res_out=D) in NO_DEVICE
    assert norm(lib, res=C, res_out=C) in NO_DEVICE                    # in place
    assert norm(lib, res=C, res_out=A) in NO_DEVICE                    # over x
    assert norm(lib, res=C, res_out=C + 128) == 1                      # shifted by a row
    assert norm(lib, res=C, res_out=B) == 1                            # over the output
    assert norm(lib, out=A) in NO_DEVICE                               # BF16 over x
    assert norm(lib, out=A, ld_out=128) == 1                           # same place, other stride
    assert norm(lib, out=A + 128) == 1
    assert norm(lib, weight=B) == 1                                    # the weight under the output
    assert norm(lib, fmt=1, scales=C, out=A) == 1                      # codes over x
    assert norm(lib, fmt=1, scales=B) == 1 and norm(lib, fmt=1, scales=A) == 1
    # column slices of one buffer share an address range but no byte
    assert norm(lib, x=A, ld=128, out=A + 128, ld_out=128) in NO_DEVICE
    assert norm(lib, x=A, ld=128, out=A + 126, ld_out=128) == 1
    assert norm(lib, x=A + 128, ld=128, out=A, ld_out=128) in NO_DEVICE
    assert norm(lib, x=A + 126, ld=128, out=A, ld_out=128) == 1


def gate(lib, g=1 << 20, ld_g=64, u=2 << 20, ld_u=64, rows=4, cols=64, fmt=0, layout=0, gs=0, out=3 << 20, ld_out=64,
         scales=0, gs_out=0, ws=0, ws_bytes=256):
    return lib.nvfp4_silu_mul(P(g), ld_g, P(u), ld_u, rows, cols, fmt, layout, P(gs), P(out), ld_out, P(scales),
                              P(gs_out), P(ws), ws_bytes, None)


def test_silu_mul_validation(lib):
    assert gate(lib) in NO_DEVICE
    assert gate(lib, g=0) == 1 and gate(lib, u=0) == 1 and gate(lib, out=0) == 1
    assert gate(lib, ld_g=63) == 1 and gate(lib, ld_u=63) == 1
    assert gate(lib, u=(2 << 20) + 1) == 3
    assert gate(lib, cols=1) in NO_DEVICE
    assert gate(lib, fmt=2, scales=4 << 20, u=(2 << 20) + 8) == 3
    assert gate(lib, fmt=2, scales=4 << 20, ld_u=68) == 3
    assert gate(lib, fmt=2, scales=4 << 20, cols=48) == 2
    assert gate(lib, fmt=3, scales=4 << 20) == 7
    assert gate(lib, fmt=3, scales=4 << 20, ws=5 << 20) in NO_DEVICE
    assert gate(lib, out=1 << 20) in NO_DEVICE and gate(lib, out=2 << 20) in NO_DEVICE   # in place
    assert gate(lib, out=(1 << 20) + 2) == 1
    assert gate(lib, fmt=1, scales=4 << 20, out=2 << 20) == 1
    # gate and up are the halves of one product, the output over the first half
    A = 1 << 20
    assert gate(lib, g=A, ld_g=128, u=A + 128, ld_u=128, out=A, ld_out=128) in NO_DEVICE
    assert gate(lib, g=A, ld_g=128, u=A + 128, ld_u=128, out=A, ld_out=64) == 1


@pytest.mark.parametrize("mx", [False, True])
def test_matvec_validation(lib, mx):
    def mv(x=1 << 20, xs=0, xl=0, M=4, K=64, ld=64, wc=2 << 20, wsc=3 << 20, gs=4 << 20, gc=0, gsc=0, ggs=0, N=96,
           out=5 << 20, ld_out=96):
        if mx:
            return lib.mxfp4_matvec(P(x), P(xs), xl, M, K, ld, P(wc), P(wsc), P(gc), P(gsc), N, P(out), ld_out, None)
        return lib.nvfp4_matvec(P(x), P(xs), xl, M, K, ld, P(wc), P(wsc), P(gs), P(gc), P(gsc), P(ggs), N, P(out),
                                ld_out, None)

    assert mv() in NO_DEVICE and mv(M=0) in NO_DEVICE and mv(M=16) in NO_DEVICE
    assert mv(M=17) == 2 and mv(K=48, ld=48) == 2 and mv(K=(1 << 19) + 32, ld=1 << 20) == 2
    assert mv(M=-1) == 1 and mv(N=0) == 1 and mv(K=0) == 1
    assert mv(ld=32) == 1 and mv(ld_out=95) == 1
    assert mv(x=0) == 1 and mv(out=0) == 1 and mv(wc=0) == 1 and mv(wsc=0) == 1
    assert mv(x=(1 << 20) + 8) == 3 and mv(ld=68) == 3 and mv(out=(5 << 20) + 1) == 3
    assert mv(out=(5 << 20) + 2, N=95, ld_out=97) in NO_DEVICE
    assert mv(xs=6 << 20) in NO_DEVICE and mv(xs=6 << 20, ld=72) == 3 and mv(xs=6 << 20, xl=3) == 1
    assert mv(wc=(2 << 20) + 8) == 3 and mv(wsc=(3 << 20) + 8) == 3
    assert mv(gc=6 << 20) == 1 and mv(gsc=6 << 20) == 1
    assert mv(gc=6 << 20, gsc=7 << 20, ggs=8 << 20) in NO_DEVICE
    assert mv(out=1 << 20) == 1                                        # over x
    assert mv(out=2 << 20) == 1 and mv(out=(3 << 20) + 2) == 1         # over the weight's codes, its scales
    assert mv(gc=6 << 20, gsc=7 << 20, ggs=8 << 20, out=7 << 20) == 1  # over the gate's scales
    if not mx:
        assert mv(gs=0) == 1 and mv(gs=(4 << 20) + 2) == 3
        assert mv(gc=6 << 20, gsc=7 << 20) == 1                        # the gate's tensor scale is missing


def test_row_workspace(lib):
    assert lib.nvfp4_row_workspace_bytes() == 256
    assert nv.mxfp8_scales_bytes(130, 96, "linear") == 390
    assert nv.mxfp8_scales_bytes(130, 96) == 256 * 4


def test_python_calls_refuse_host_tensors_and_wrong_arguments():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.rms_norm(x)
    with pytest.raises(ValueError):
        nv.silu_mul(x, x)
    with pytest.raises(ValueError):
        nv.matvec(x, nv.MXFP4Tensor(x, x, 4, 64))
    with pytest.raises(ValueError):
        nv.matvec(nv.MXFP8Tensor(x, x, 4, 64), nv.MXFP4Tensor(x, x, 4, 64))
    for bad in ("fp8", None, 1):
        with pytest.raises(ValueError):
            nv.rms_norm(x, out_format=bad)
    with pytest.raises(ValueError):
        nv.silu_mul(x, x, out_format="mxfp8", layout="rows")


def test_reference_roundings_agree_with_torch_and_the_oracle_grid():
    """The tests' own roundings: E4M3 against torch's conversion, E2M1 against its grid's nearest value."""
    y = np.concatenate([np.linspace(0, 500, 20011), 2.0 ** np.linspace(-14, 9, 20011)])
    want = torch.from_numpy(np.minimum(y, 448.0).astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.round_e4m3(y.astype(np.float32).astype(np.float64)), want)
    y = np.linspace(0, 8, 10007)
    near = np.min(np.abs(y[:, None] - ref.E2M1[None]), axis=1)
    assert np.allclose(np.abs(ref.round_e2m1(y) - y), near)


@pytest.mark.parametrize("mx", [False, True])
def test_matvec_refuses_an_output_over_swizzled_activation_scales(lib, mx):
    """Swizzled scales take whole 128 x 4 tiles: 4 x 256 values' scales lie in 1024 bytes, not in the 32 they are."""
    S, W = 6 << 20, 2 << 20

    def mv(out, layout):
        tail = [] if mx else [P(0)]
        gs = [] if mx else [P(4 << 20)]
        call = lib.mxfp4_matvec if mx else lib.nvfp4_matvec
        return call(P(1 << 20), P(S), layout, 4, 256, 256, P(W), P(3 << 20), *gs, P(0), P(0), *tail, 96, P(out), 96, None)

    for out in (S, S + 32, S + 560, S + 1022, S - 700):
        assert mv(out, 0) == 1, out
    assert mv(S + 1024, 0) in NO_DEVICE and mv(S - 768, 0) in NO_DEVICE   # the output has 4 x 96 x 2 = 768 bytes
    assert mv(S + 30, 1) == 1 and mv(S + 32, 1) in NO_DEVICE              # linear: 32 bytes


def test_tensor_scales_and_workspace_share_no_byte_with_other_arguments(lib):
    """The 4-byte tensor scales are inputs and outputs like the matrices, and the workspace is written."""
    X, OUT, SC, GI, GO, WS = (i << 20 for i in range(1, 7))
    for call in (lambda **k: norm(lib, x=X, out=OUT, fmt=3, scales=SC, ws_bytes=256, **k),
                 lambda **k: gate(lib, g=X, u=9 << 20, out=OUT, fmt=3, scales=SC, ws_bytes=256, **k)):
        assert call(gs=GI, gs_out=GO) in NO_DEVICE and call(ws=WS, gs_out=GO) in NO_DEVICE
        assert call(gs=GI, gs_out=GI) in NO_DEVICE                     # the given scale, in place
        for taken in (X, OUT, SC):
            assert call(gs=GI, gs_out=taken + 8) == 1
            assert call(ws=taken + 16, gs_out=GO) == 1
        for output in (OUT, SC):
            assert call(gs=output + 8, gs_out=GO) == 1
        assert call(ws=WS, gs_out=WS + 252) == 1 and call(ws=WS, gs_out=WS + 256) in NO_DEVICE
    assert norm(lib, x=X, res=7 << 20, res_out=8 << 20, out=OUT, fmt=3, scales=SC, gs=(8 << 20) + 4, gs_out=GO) == 1
    assert norm(lib, x=X, weight=10 << 20, out=OUT, fmt=3, scales=SC, gs=GI, gs_out=10 << 20) == 1

    def mv(gs, ggs, out):
        return lib.nvfp4_matvec(P(X), P(0), 0, 4, 64, 64, P(OUT), P(SC), P(gs), P(7 << 20), P(8 << 20), P(ggs), 96,
                                P(out), 96, None)
    assert mv(GI, GO, WS) in NO_DEVICE
    assert mv(WS + 4, GO, WS) == 1 and mv(GI, WS + 4, WS) == 1
