"""How matvec cuts its calls, on a machine without a GPU: the sizes of the GPU test take every way."""
import pytest

import w4a4_gemm_quantize_b200 as nv
from matvec_paths import PATHS, way
from w4a4_gemm_quantize_b200 import build as nvbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    nvbuild.build()
    return nv.load_library()


def test_the_gpu_tests_sizes_take_every_way():
    """Each kind of tile, K whole or shared by a cluster, one batch of tiles per CTA or several, the sums over x; and
    each of these ways in both formats and with a gate for some kind of tile."""
    ways = [way(*s) for s in PATHS]
    for tiles in ("paired", "wide", "narrow"):
        assert (tiles, False, True, False) in ways, tiles
        assert (tiles, True, True, False) in ways, tiles
        assert (tiles, True, False, True) in ways, tiles
    for kind in ("nvfp4", "mxfp4"):
        for gated in (False, True):
            some = {way(*s)[1:] for s in PATHS if s[3] == kind and s[4] == gated}
            assert some & {(False, True, False), (True, True, False)} and (True, False, True) in some, (kind, gated)


def test_plan_of_calls():
    assert nv.matvec_plan(1, 14336, 4096) == (1, 1, False, 1)
    assert nv.matvec_plan(3, 40, 2 ** 19 - 32)[3] == 3               # x of one token at a time
    assert nv.matvec_plan(16, 64, 65536)[0] > 1                      # few long rows: a cluster shares them
    for M, N, K in ((0, 64, 64), (1, 0, 64), (1, 64, 0), (17, 64, 64), (1, 64, 48), (1, 64, 2 ** 19 + 32)):
        with pytest.raises(nv.Nvfp4Error):
            nv.matvec_plan(M, N, K)
