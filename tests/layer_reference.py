"""The decoder-layer operators in 64 bits, and the comparisons their tests use (test infrastructure).

A rounding to a format is monotone, so where a kernel's binary32 value may differ from the 64-bit one by a
relative delta, its code must lie between the roundings of v (1 - delta) and v (1 + delta): ``check_blocks``
asks exactly that of every scale and every code, with no slack beyond it.

Where the deltas come from:
* norm: a thread sums at most 16 * 8 squares one after the other, 10 levels of a tree follow; every step is off
  by at most 2^-24 of the sum, so the sum by (128 + 10) 2^-24, its root by half of that, and the quotient,
  the root itself and the two products by 2^-24 each: under 2^-17.  (Rows the vector kernel does not take:
  at most cols / 512 squares per thread; ``NORM_DELTA`` holds up to 131072 columns.)
* gate: e^-g to 2 units in the last place (2^-22), 1 + e, the quotient and the product 2^-23 each: under 2^-20.
* encoding: the scale's reciprocal and one product, 2^-23.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle

NORM_DELTA = 2.0 ** -16
GATE_DELTA = 2.0 ** -20
ENCODE_DELTA = 2.0 ** -22
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def norm64(x, residual, weight, eps, offset=0.0):
    """(v, h): h the BF16 residual stream (as doubles), v the normalised row."""
    h = x.double()
    if residual is not None:
        h = (x.float() + residual.float()).to(torch.bfloat16).double()
    v = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    if weight is not None:
        v = v * (weight.double() + offset)
    return v.cpu().numpy(), h.cpu().numpy()


def gate64(gate, up):
    g = gate.double()
    return (g / (1.0 + torch.exp(-g)) * up.double()).cpu().numpy()


def check_bf16(got, v, delta, where=""):
    """BF16 output: half a step (2^-8 relative, 2^-134 below the normal range) of a value within delta of v."""
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(v)), f"{where}: NaNs differ"
    inf = np.isinf(v)
    assert np.array_equal(got[inf], v[inf]), f"{where}: infinities differ"
    ok = ~np.isnan(v) & ~inf
    err = np.abs(got - np.where(ok, v, 0.0))[ok]
    bound = np.abs(v[ok]) * (2.0 ** -8 + 2 * delta) + 2.0 ** -133
    assert (err <= bound).all(), f"{where}: worst {np.max(err / bound):.3f} of the bound"


def round_e2m1(y):
    """|y| to the nearest E2M1 magnitude, saturating (ties: either neighbour serves a monotone bound)."""
    return E2M1[np.searchsorted((E2M1[1:] + E2M1[:-1]) / 2, y)]


def round_e4m3(y):
    """Non-negative y to the nearest E4M3 value, saturating at 448."""
    e = np.maximum(np.floor(np.log2(np.maximum(y, 2.0 ** -300))), -6.0)
    step = 2.0 ** (e - 3)
    return np.minimum(np.round(y / step) * step, 448.0)


def e4m3_values(byte):
    t = torch.from_numpy(np.ascontiguousarray(byte))
    return t.view(torch.float8_e4m3fn).double().numpy()


def scales_of(q, rows, nblk, layout):
    s = q.scales.cpu().numpy()
    if layout == "linear":
        return s.reshape(rows, nblk)
    lin = oracle.unswizzle_scales(s, rows, nblk)
    assert np.array_equal(oracle.swizzle_scales(lin), s), "padding of the swizzled scales is not zero"
    return lin


def code_values(q, fmt):
    if fmt == "mxfp8":
        return q.codes.double().cpu().numpy()
    c = q.codes.cpu().numpy()
    n = np.stack([c & 15, c >> 4], 2).reshape(c.shape[0], -1)
    return np.where(n >= 8, -1.0, 1.0) * E2M1[n & 7]


def check_blocks(q, v, fmt, layout, delta, sg=None):
    """Every scale and code of a block-format output against v; sg: NVFP4's given tensor scale.
    Returns the values the output stands for (64 bits)."""
    rows, cols = v.shape
    block = 16 if fmt == "nvfp4" else 32
    nblk = cols // block
    byte = scales_of(q, rows, nblk, layout)
    b = np.abs(v).reshape(rows, nblk, block)
    amax = b.max(2)
    if fmt == "nvfp4":
        got_sg = float(q.global_scale.item())
        if sg is None:
            want = amax.max() / 2688.0 if amax.max() > 0 else 1.0
            assert abs(got_sg - want) <= want * (delta + 2.0 ** -23), (got_sg, want)
        else:
            assert got_sg == sg
        lo, hi = (round_e4m3(amax * (1 + s * (delta + ENCODE_DELTA)) / (6.0 * got_sg)) for s in (-1, 1))
        dec = e4m3_values(byte)
        assert ((lo <= dec) & (dec <= hi)).all(), "block scales"
        eff = dec * got_sg
        rnd = round_e2m1
    else:
        emax = 8 if fmt == "mxfp8" else 2

        def exponent(a):
            e = np.floor(np.log2(np.maximum(a, 2.0 ** -300))) - emax
            return np.where(a > 0, np.clip(e, -127, 127), -127)

        lo, hi = exponent(amax * (1 - delta)), exponent(amax * (1 + delta))
        e = byte.astype(np.int64) - 127
        assert ((lo <= e) & (e <= hi)).all(), "block scales"
        eff = 2.0 ** e.astype(np.float64)
        rnd = round_e4m3 if fmt == "mxfp8" else round_e2m1
    codes = code_values(q, fmt)
    mag = np.abs(codes).reshape(rows, nblk, block)
    d = delta + ENCODE_DELTA
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(eff[..., None] > 0, b / eff[..., None], 0.0)
    assert ((rnd(y * (1 - d)) <= mag) & (mag <= rnd(y * (1 + d)))).all(), "codes"
    nonzero = codes != 0
    assert (np.sign(codes)[nonzero] == np.sign(v)[nonzero]).all(), "signs"
    return (codes.reshape(rows, nblk, block) * eff[..., None]).reshape(rows, cols)


def dequantize64(w):
    """The values of an NVFP4Tensor / MXFP4Tensor / MXFP8Tensor (64 bits, numpy)."""
    import w4a4_gemm_quantize_b200 as nv
    fmt = {nv.NVFP4Tensor: "nvfp4", nv.MXFP4Tensor: "mxfp4", nv.MXFP8Tensor: "mxfp8"}[type(w)]
    nblk = w.cols // (16 if fmt == "nvfp4" else 32)
    s = scales_of(w, w.rows, nblk, "linear" if w.layout == nv.SF_LINEAR else "swizzled")
    if fmt == "nvfp4":
        eff = e4m3_values(s) * float(w.global_scale.item())
    else:
        eff = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127.0))
    return (code_values(w, fmt).reshape(w.rows, nblk, -1) * eff[..., None]).reshape(w.rows, w.cols)


def matvec64(x, w, gate=None):
    """(y, bound): y = x w^T (gated: silu(x gate^T) * it) in 64 bits on the GPU, and the error allowed before the
    BF16 rounding: binary32 accumulation, 2^-14 of the sum of magnitudes S.  By operation count: a warp keeps a tile's
    sums over its part of K, a chain of at most K / 16 mma, each off by at most 2^-22 of S (operand alignment inside
    the mma included); 16 warps' and 8 CTAs' sums follow: (K / 16 + 24) 2^-22 S, which is 2^-14 S up to K = 3700.
    Longer rows are held to the same 2^-14, tighter than their count: the partial sums stay far below S and their
    roundings have both signs (the largest excess over half a BF16 step, K up to 524288, was 2^-26 S)."""
    x = x.double().cuda()

    def product(q):
        m = torch.from_numpy(dequantize64(q)).cuda()
        return x @ m.t(), (x.abs() @ m.abs().t()) * 2.0 ** -14
    y, b = product(w)
    if gate is not None:
        g, bg = product(gate)
        s = g / (1.0 + torch.exp(-g))
        b = s.abs() * b + 1.1 * bg * (y.abs() + b) + (s * y).abs() * GATE_DELTA
        y = s * y
    return y.cpu().numpy(), b.cpu().numpy()


def check_product(got, y, bound, where="", min_exact=0.9):
    got = got.double().cpu().numpy()
    finite = np.isfinite(y)
    assert np.array_equal(np.isnan(got), np.isnan(y)), f"{where}: NaNs differ"
    inf = np.isinf(y)
    assert np.array_equal(got[inf], y[inf]), f"{where}: infinities differ"
    err, allow = np.abs(got[finite] - y[finite]), (bound + np.abs(y) * 2.0 ** -8 + 2.0 ** -133)[finite]
    assert (err <= allow).all(), f"{where}: worst {np.max(err / allow):.3f} of the bound"
    rne = torch.from_numpy(y[finite].astype(np.float32)).to(torch.bfloat16).double().numpy()
    if rne.size >= 64:
        assert np.mean(got[finite] == rne) >= min_exact, f"{where}: {np.mean(got[finite] == rne):.3f} equal BF16(ref)"
