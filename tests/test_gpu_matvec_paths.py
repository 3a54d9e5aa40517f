"""matvec on sizes that take every way it cuts a call (tests/matvec_paths.py), against the 64-bit product."""
import numpy as np
import pytest
import torch

import layer_reference as ref
import w4a4_gemm_quantize_b200 as nv
from matvec_paths import PATHS

pytestmark = pytest.mark.gpu

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def weight(N, K, kind, g):
    """Any codes, block scales over a few binades; their values (64 bits) row by row in `rows`."""
    block = 16 if kind == "nvfp4" else 32
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    codes[:, :8] = 0                                                   # 16 columns of zeros, for x's large values
    nblk = K // block
    low, high = (0x30, 0x48) if kind == "nvfp4" else (118, 126)
    lin = torch.randint(low, high, (N, nblk), generator=g, device="cuda", dtype=torch.uint8)
    rp, cp = -(-N // 128) * 128, -(-nblk // 4) * 4
    full = torch.zeros((rp, cp), dtype=torch.uint8, device="cuda")
    full[:N, :nblk] = lin
    scales = full.view(rp // 128, 4, 32, cp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()
    gs = torch.tensor([0.0123], device="cuda")
    q = nv.NVFP4Tensor(codes, scales, gs, N, K) if kind == "nvfp4" else nv.MXFP4Tensor(codes, scales, N, K)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")

    def rows(a, b):
        c = codes[a:b].int()
        v = torch.stack([table[c & 15], table[c >> 4]], 2).view(b - a, nblk, block)
        s = lin[a:b].contiguous()
        s = s.view(torch.float8_e4m3fn).double() * gs.double() if kind == "nvfp4" else torch.exp2(s.double() - 127.0)
        return (v * s.unsqueeze(2)).view(b - a, K)
    return q, rows


def product(x, rows, N):
    """x w^T and sum |x w| in 64 bits, a slice of the rows at a time."""
    x, step = x.double(), max(1, 4_000_000 // x.shape[1])
    y, s = [], []
    for a in range(0, N, step):
        w = rows(a, min(N, a + step))
        y.append(x @ w.t())
        s.append(x.abs() @ w.abs().t())
    return torch.cat(y, 1), torch.cat(s, 1)


@pytest.mark.parametrize("M,N,K,kind,gated", PATHS)
def test_every_way_of_cutting_a_call(cuda_device, M, N, K, kind, gated):
    g = torch.Generator(device="cuda").manual_seed(N + K)
    w, rows = weight(N, K, kind, g)
    gate, gate_rows = weight(N, K, kind, g) if gated else (None, None)
    near = torch.randn((M, K), generator=g, device="cuda") * (0.02 if gated else 1.0)
    far, last = near.clone(), near.clone()                             # more passes than one over the weights:
    far[:, 16::2] *= 2.0 ** -40                                        # its first holds the result,
    last[:, 3], last[1::2, 5] = 2.0 ** 90, 2.0 ** 45                   # its second, in odd tokens its third does
    for x in (near.to(torch.bfloat16), far.to(torch.bfloat16), last.to(torch.bfloat16)):
        got = nv.matvec(x, w, gate)
        y, s = product(x, rows, N)
        bound = s * 2.0 ** -14                                         # as layer_reference.matvec64 has it
        if gated:
            z, sz = product(x, gate_rows, N)
            e = z / (1.0 + torch.exp(-z))
            bound = e.abs() * bound + 1.1 * sz * 2.0 ** -14 * (y.abs() + bound) + (e * y).abs() * ref.GATE_DELTA
            y = e * y
        ref.check_product(got, y.cpu().numpy(), bound.cpu().numpy(), f"{kind} {M}x{N}x{K}", 0.85)
        assert torch.equal(got, nv.matvec(x, w, gate))                 # the same bits on every call


@pytest.mark.parametrize("M,N,K,kind,gated", [s for s in PATHS if s[1] * s[2] < 2e7])
def test_every_way_beside_others(cuda_device, M, N, K, kind, gated):
    """Two streams at once and a captured call: nothing is shared between calls."""
    g = torch.Generator(device="cuda").manual_seed(N)
    w, _ = weight(N, K, kind, g)
    gate = weight(N, K, kind, g)[0] if gated else None
    x = (torch.randn((M, K), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    far = x.clone()
    far[0, 5] = 2.0 ** -50
    want, want_far = nv.matvec(x, w, gate), nv.matvec(far, w, gate)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(nv.matvec(x, w, gate, stream=s1), nv.matvec(far, w, gate, stream=s2)) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want_far) for a, b in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nv.matvec(x, w, gate)
    x.copy_(far)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want_far)
