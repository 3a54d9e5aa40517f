"""Sizes that together take every way matvec cuts a call, shared by the CPU test that they do and the GPU test that the
results are right."""
import w4a4_gemm_quantize_b200 as nv

# (M, N, K, kind, gated)
PATHS = [
    # more than 8 tokens: tiles of 32 rows
    (16, 5376, 21504, "nvfp4", False), (15, 70, 32000, "mxfp4", False), (16, 11584, 4096, "nvfp4", False),
    (16, 6208, 14336, "nvfp4", False), (16, 40960, 8192, "mxfp4", False), (16, 266665, 64, "nvfp4", False),
    (16, 1472, 21504, "nvfp4", True), (16, 4032, 14336, "nvfp4", True), (14, 69, 36416, "mxfp4", True),
    (16, 5815, 5952, "mxfp4", True), (16, 139540, 64, "mxfp4", True),
    # up to 8 tokens, K a multiple of 64
    (6, 6555, 12544, "nvfp4", False), (8, 82, 73536, "nvfp4", False), (8, 71, 74688, "mxfp4", False),
    (8, 4319, 35392, "nvfp4", True), (8, 348588, 64, "mxfp4", True), (7, 87, 80512, "nvfp4", True),
    # up to 8 tokens, K no multiple of 64
    (8, 25866, 11296, "mxfp4", False), (6, 64, 119648, "nvfp4", False), (8, 6974, 22496, "nvfp4", True),
    (8, 107, 88416, "mxfp4", True),
]


def shape(M, K):
    return "paired" if M > 8 else "wide" if K % 64 == 0 else "narrow"


def way(M, N, K, kind, gated):
    """(tiles, K shared by a cluster, several batches of tiles per CTA, a cluster's sums over x)"""
    split, batches, over_x, launches = nv.matvec_plan(M, N, K, kind == "mxfp4", gated)
    assert launches == 1
    return shape(M, K), split > 1, batches > 1, over_x
