"""The decoder-layer operators of the library, as cases to measure: rms_norm, silu_mul, matvec.

``run`` computes a case with elementary torch operations in 32 bits, or, where ``own`` is true, with the
library's calls.  Outputs held in 8 bits are returned as float8 codes and power-of-two scales; outputs held
in 4 bits as the BF16 values they stand for (the library's dequantize call).  ``exact`` is the definition in
64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one token's hidden state before an 8-bit-activation product: pure latency
        {"name": "norm token mxfp8", "op": "norm", "rows": 1, "cols": 4096, "residual": True, "format": "mxfp8"},
        # a long prompt of the 31B-class layer before its W4A4 product, activation scale computed on the call
        {"name": "norm prompt nvfp4", "op": "norm", "rows": 8192, "cols": 5376, "residual": True, "format": "nvfp4"},
        # a ragged batch, a hidden size that is no multiple of a block, 16-bit output, no residual
        {"name": "norm ragged bf16", "op": "norm", "rows": 777, "cols": 2201, "residual": False, "format": "bf16"},
        # one token's MLP gate
        {"name": "gate token mxfp8", "op": "gate", "rows": 1, "cols": 14336, "residual": False, "format": "mxfp8"},
        # a small batch of odd size between two MXFP4 products
        {"name": "gate batch mxfp4", "op": "gate", "rows": 37, "cols": 14336, "residual": False, "format": "mxfp4"},
        # the 8B-class prompt's gate before the down product, activation scale computed on the call
        {"name": "gate prompt nvfp4", "op": "gate", "rows": 4096, "cols": 14336, "residual": False, "format": "nvfp4"},
        # the largest gate: the 31B-class layer at 8192 tokens, 8-bit output
        {"name": "gate large mxfp8", "op": "gate", "rows": 8192, "cols": 21504, "residual": False, "format": "mxfp8"},
        # decode: one token through the 8B-class up product, weight-only NVFP4
        {"name": "matvec token", "op": "matvec", "M": 1, "N": 14336, "K": 4096, "w": "nvfp4", "x": "bf16",
         "gated": False},
        # decode: one token through the 31B-class gate and up products together
        {"name": "matvec gated", "op": "matvec", "M": 1, "N": 21504, "K": 5376, "w": "nvfp4", "x": "bf16",
         "gated": True},
        # eight sequences, MXFP4 weights and 8-bit activations, long rows (the down product)
        {"name": "matvec batch mx", "op": "matvec", "M": 8, "N": 4096, "K": 14336, "w": "mxfp4", "x": "mxfp8",
         "gated": False},
        # sixteen sequences, the 31B-class down product
        {"name": "matvec batch 16", "op": "matvec", "M": 16, "N": 5376, "K": 21504, "w": "nvfp4", "x": "bf16",
         "gated": False},
        # a small projection of odd sizes: latency
        {"name": "matvec small", "op": "matvec", "M": 3, "N": 1001, "K": 1056, "w": "mxfp4", "x": "bf16",
         "gated": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gate", "matvec"])
    if op == "matvec":
        K, gated = 32 * _log(rng, 2, 672), rng.random() < 0.3
        most = 2 * 21504 * 5376 // K // (2 if gated else 1)  # no more weights than the largest listed layer
        return {"op": op, "M": rng.randint(1, 16), "N": _log(rng, 16, min(32768, most)), "K": K,
                "w": rng.choice(["nvfp4", "mxfp4"]), "x": rng.choice(["bf16", "mxfp8"]), "gated": gated}
    fmt = rng.choice(["bf16", "mxfp8", "mxfp4", "nvfp4"])
    step = {"bf16": 1, "nvfp4": 16}.get(fmt, 32)
    cols = step * _log(rng, max(1, 64 // step), (8192 if op == "norm" else 21504) // step)
    return {"op": op, "rows": _log(rng, 1, 8192), "cols": cols, "residual": op == "norm" and rng.random() < 0.7,
            "format": fmt}


def work(case):
    if case["op"] == "matvec":
        M, N, K = case["M"], case["N"], case["K"]
        weights = (2 if case["gated"] else 1) * N * (K // 2 + K // (16 if case["w"] == "nvfp4" else 32))
        x = M * K * 2 if case["x"] == "bf16" else M * (K + K // 32)
        return {"bytes": weights + x + 2 * M * N, "flops": (4 if case["gated"] else 2) * M * N * K}
    n = case["rows"] * case["cols"]
    reads = 4 if case["op"] == "gate" or case["residual"] else 2
    writes = {"mxfp8": 1 + 1 / 32}.get(case["format"], 2) + (2 if case["residual"] else 0)
    return {"bytes": n * (reads + writes) + (2 * case["cols"] if case["op"] == "norm" else 0), "flops": 6 * n}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


def _activation(rows, cols, g):
    """N(0, 1) with four channels fifty times as large, as decoder activations have them."""
    x = _normal((rows, cols), g)
    x[:, torch.randperm(cols, generator=g, device="cuda")[:4]] *= 50.0
    return x.to(torch.bfloat16)


def _e2m1_index(a):
    """Index of the E2M1 magnitude nearest to a >= 0, ties to the even index."""
    i = (a > 0.25).to(torch.uint8)
    for mid, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        i += (a >= mid) if up else (a > mid)
    return i


def _swizzle(s):
    """(rows, blocks) scale bytes -> the flat 128 x 4 tile layout, padding zero."""
    rows, blocks = s.shape
    rp, cp = -(-rows // 128) * 128, -(-blocks // 4) * 4
    p = torch.zeros((rp, cp), dtype=torch.uint8, device=s.device)
    p[:rows, :blocks] = s
    return p.view(rp // 128, 4, 32, cp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _weight(N, K, kind, g):
    """A N(0, 0.02) weight in 4 bits: packed codes, swizzled scales, and the NVFP4 tensor scale."""
    block = 16 if kind == "nvfp4" else 32
    sg = 0.02 * 5.5 / 2688.0
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N, K // block), dtype=torch.uint8, device="cuda")
    for r in range(0, N, 8192):
        w = _normal((min(8192, N - r), K // block, block), g, 0.02)
        amax = w.abs().amax(2, keepdim=True)
        if kind == "nvfp4":
            s = (amax / (6.0 * sg)).clamp_(max=448.0).to(torch.float8_e4m3fn)
            byte, eff = s.view(torch.uint8), s.float() * sg
        else:
            e = torch.frexp(amax)[1] - 3
            byte, eff = (e + 127).to(torch.uint8), torch.ldexp(torch.ones_like(amax), e)
        y = w / eff.clamp(min=1e-30)
        q = (_e2m1_index(y.abs()) | ((y < 0).to(torch.uint8) << 3)).view(-1, K)
        codes[r:r + 8192] = q[:, 0::2] | (q[:, 1::2] << 4)
        scales[r:r + 8192] = byte.view(-1, K // block)
    return {"codes": codes, "scales": _swizzle(scales), "N": N, "K": K, "kind": kind,
            "global_scale": torch.tensor([sg], dtype=torch.float32, device="cuda")}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "matvec":
        x = _activation(case["M"], case["K"], g)
        s = {"case": case, "w": _weight(case["N"], case["K"], case["w"], g), "gate": None}
        if case["gated"]:
            s["gate"] = _weight(case["N"], case["K"], case["w"], g)
        if case["x"] == "mxfp8":
            v = x.float().view(case["M"], -1, 32)
            e = (torch.frexp(v.abs().amax(2, keepdim=True))[1] - 9).clamp(-127, 127)
            s["x_codes"] = (v * torch.ldexp(torch.ones_like(v), -e)).clamp(-448, 448).to(torch.float8_e4m3fn).view(
                case["M"], case["K"])
            s["x_scales"] = (e + 127).to(torch.uint8).view(case["M"], -1)
        else:
            s["x"] = x
        return s
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "norm":
        return {"case": case, "x": _normal((rows, cols), g).to(torch.bfloat16),
                "residual": _activation(rows, cols, g) if case["residual"] else None,
                "weight": (1.0 + _normal((cols,), g, 0.2)).to(torch.bfloat16)}
    return {"case": case, "gate": _normal((rows, cols), g, 2.0).to(torch.bfloat16),
            "up": _normal((rows, cols), g).to(torch.bfloat16)}


# ---------------------------------------------------------------------------------------------
# one pass: the library's calls, or elementary operations
# ---------------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "matvec":
        x = state["x"].float() if case["x"] == "bf16" else _mx_values(state["x_codes"], state["x_scales"])
        y = x @ _weight_values(state["w"]).t()
        if case["gated"]:
            g = x @ _weight_values(state["gate"]).t()
            y = g / (1.0 + torch.exp(-g)) * y
        return {"out": y.to(torch.bfloat16)}
    out = {}
    if case["op"] == "norm":
        h = state["x"]
        if case["residual"]:
            h = (h.float() + state["residual"].float()).to(torch.bfloat16)
            out["residual"] = h
        h = h.float()
        v = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * state["weight"].float()
    else:
        g = state["gate"].float()
        v = g / (1.0 + torch.exp(-g)) * state["up"].float()
    out.update(_output(v, case["format"]))
    return out


def _own(state, case):
    import w4a4_gemm_quantize_b200 as nv
    if case["op"] == "matvec":
        if case["x"] == "bf16":
            x = state["x"]
        else:
            x = nv.MXFP8Tensor(state["x_codes"], state["x_scales"], case["M"], case["K"], nv.SF_LINEAR)
        gate = _tensor(nv, state["gate"]) if case["gated"] else None
        return {"out": nv.matvec(x, _tensor(nv, state["w"]), gate)}
    out, fmt = {}, case["format"]
    layout = "linear" if fmt == "mxfp8" else "swizzled"
    if case["op"] == "norm":
        q = nv.rms_norm(state["x"], state["weight"], state["residual"], eps=EPS, out_format=fmt, layout=layout)
        if case["residual"]:
            q, out["residual"] = q
    else:
        q = nv.silu_mul(state["gate"], state["up"], out_format=fmt, layout=layout)
    if fmt == "bf16":
        out["out"] = q
    elif fmt == "mxfp8":
        out["codes"], out["scales"] = q.codes, q.scales.view(torch.float8_e8m0fnu)
    else:
        out["values"] = nv.nvfp4_dequantize(q) if fmt == "nvfp4" else nv.mxfp4_dequantize(q)
    return out


def _tensor(nv, w):
    if w["kind"] == "nvfp4":
        return nv.NVFP4Tensor(w["codes"], w["scales"], w["global_scale"], w["N"], w["K"])
    return nv.MXFP4Tensor(w["codes"], w["scales"], w["N"], w["K"])


def _unswizzle(s, rows, blocks):
    rp, cp = -(-rows // 128) * 128, -(-blocks // 4) * 4
    return s.view(rp // 128, cp // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rp, cp)[:rows, :blocks]


def _weight_values(w):
    """The weight in 32 bits: code value x block scale x tensor scale."""
    N, K = w["N"], w["K"]
    block = 16 if w["kind"] == "nvfp4" else 32
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], 1)   # byte -> its two values
    v = pairs.index_select(0, w["codes"].view(-1).int()).view(N, K // block, block)
    s = _unswizzle(w["scales"], N, K // block)
    if block == 16:
        s = s.contiguous().view(torch.float8_e4m3fn).float() * w["global_scale"]
    else:
        s = torch.ldexp(torch.ones((), device="cuda"), s.int() - 127)
    return (v * s.unsqueeze(2)).view(N, K)


def _mx_values(codes, scales):
    rows, cols = codes.shape
    s = torch.ldexp(torch.ones((), device="cuda"), scales.int() - 127)
    return (codes.float().view(rows, -1, 32) * s.unsqueeze(2)).view(rows, cols)


def _output(v, fmt):
    rows, cols = v.shape
    if fmt == "bf16":
        return {"out": v.to(torch.bfloat16)}
    b = v.view(rows, -1, 16 if fmt == "nvfp4" else 32)
    amax = b.abs().amax(2, keepdim=True)
    if fmt == "mxfp8":
        e = torch.where(amax > 0, torch.frexp(amax)[1] - 9, -127).clamp(-127, 127)
        codes = torch.ldexp(b, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(rows, cols)
        return {"codes": codes, "scales": (e + 127).to(torch.uint8).view(rows, -1).view(torch.float8_e8m0fnu)}
    if fmt == "mxfp4":
        e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
        eff = torch.ldexp(torch.ones_like(amax), e)
        y = b * torch.ldexp(torch.ones_like(amax), -e)
    else:
        top = amax.amax()
        sg = torch.where(top > 0, top / 2688.0, 1.0)
        eff = (amax / (6.0 * sg)).clamp(max=448.0).to(torch.float8_e4m3fn).float() * sg
        y = b * torch.where(eff > 0, 1.0 / eff, 0.0)
    a = y.abs()
    mag = (0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + (a > 2.5) * 1.0
           + (a >= 3.5) * 1.0 + (a > 5.0) * 2.0)
    return {"values": (torch.copysign(mag, y) * eff).to(torch.bfloat16).view(rows, cols)}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def _grid_round(y, mantissa_bits, lowest_exponent, largest):
    """y rounded to a small float format: nearest, ties to even, saturating."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -300))).clamp(min=lowest_exponent)
                      - mantissa_bits)
    return (torch.round(y / step) * step).clamp(-largest, largest)


def _exact_weight(w):
    c = w["codes"].to(torch.int16)
    n = torch.stack([c & 15, c >> 4], 2).view(w["N"], w["K"])
    exponent, mantissa = ((n >> 1) & 3).double(), (n & 1).double()
    v = torch.where(exponent > 0, (1.0 + mantissa / 2.0) * torch.exp2(exponent - 1.0), mantissa / 2.0)
    v = torch.where(n >= 8, -v, v)
    block = 16 if w["kind"] == "nvfp4" else 32
    r = torch.arange(w["N"], device="cuda").view(-1, 1)
    b = torch.arange(w["K"] // block, device="cuda").view(1, -1)
    atoms = -(-(w["K"] // block) // 4)
    at = ((r // 128) * atoms + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    byte = w["scales"][at].double()
    if block == 16:
        e, m = torch.floor(byte / 8.0), byte % 8.0
        s = torch.where(e > 0, (1.0 + m / 8.0) * torch.exp2(e - 7.0), m / 8.0 * 2.0 ** -6) * w["global_scale"].double()
    else:
        s = torch.exp2(byte - 127.0)
    return (v.view(w["N"], -1, block) * s.unsqueeze(2)).view(w["N"], w["K"])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        if case["x"] == "bf16":
            x = s["x"].double()
        else:
            x = s["x_codes"].double() * torch.exp2(s["x_scales"].double() - 127.0).repeat_interleave(32, 1)
        y = x @ _exact_weight(s["w"]).t()
        if case["gated"]:
            y = y * torch.nn.functional.silu(x @ _exact_weight(s["gate"]).t())
        return {"out": y}
    out = {}
    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(torch.bfloat16).double()
            out["residual"] = h
        v = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].double()
    else:
        v = torch.nn.functional.silu(s["gate"].double()) * s["up"].double()
    fmt, (rows, cols) = case["format"], v.shape
    if fmt == "bf16":
        return {**out, "out": v}
    b = v.view(rows, -1, 16 if fmt == "nvfp4" else 32)
    amax = b.abs().amax(2, keepdim=True)
    if fmt == "nvfp4":
        sg = amax.max() / 2688.0
        scale = _grid_round(amax / (6.0 * sg), 3, -6, 448.0) * sg
    else:
        scale = torch.exp2((torch.floor(torch.log2(amax.clamp(min=2.0 ** -200))) - (8 if fmt == "mxfp8" else 2))
                           .clamp(-127, 127))
    y = torch.where(scale > 0, b / scale, torch.zeros_like(b))
    if fmt == "mxfp8":
        return {**out, "codes": _grid_round(y, 3, -6, 448.0).view(rows, cols), "scales": scale.view(rows, -1)}
    return {**out, "values": (_grid_round(y, 1, 0, 6.0) * scale).view(rows, cols)}
