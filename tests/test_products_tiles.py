"""The choice of tiles of the grouped and fp8 products (host only): each case of the GPU tests takes the tile that it
is listed for."""
import os

import pytest

from grouped_cases import BF16, CASES, E4M3, GROUPED, LONG, SMS, case_id, plan
from input_adaptive_reduced_colnorm_b200 import build as rmm_build
import input_adaptive_reduced_colnorm_b200 as rmm

OK, INVALID, UNSUPPORTED = range(3)


@pytest.fixture(scope="module", autouse=True)
def built():
    rmm_build.build()


@pytest.mark.parametrize("case", CASES + LONG, ids=case_id)
def test_cases_take_their_tiles(case):
    dtype, sizes, d, m, tile = case
    outside = 5 if len(sizes) > 1 else 0
    assert plan(dtype, sum(sizes) + outside, d, m, len(sizes)) == tile


def test_every_tile_has_a_case():
    """Over a grid of sizes nothing is chosen that the cases leave out."""
    sizes = (1, 7, 16, 17, 33, 64, 65, 200, 513, 1030, 4096, 8192)
    widths = (1, 130, 300, 1000, 1522, 2048, 2600, 4096, 6000, 9000, 14336, 20000, 40000)
    seen = {(t, plan(t, n, d, m, g)) for t in (BF16, E4M3) for n in sizes for d in (1, 130, 300, 1000, 2200, 4200, 14336)
            for m in widths for g in (1, 2, 3, 8, 20, 64, 128)}
    assert seen == {(c[0], c[4]) for c in CASES} == {(c[0], c[4]) for c in LONG}
    assert {(c[0], c[4][:2]) for c in CASES} == {(c[0], c[4][:2]) for c in GROUPED}


def test_expiring_hook_refusals():
    """It checks its arguments as the calls do, and enqueues nothing for no rows."""
    P = 0x10000
    L = rmm.lib()

    def f(e4m3, n=0, X=P, off=P, sw=P):
        return L.rmm_debug_grouped_expire_producer(e4m3, X, n, 256, 256, P, 8, P, 2, 256 * 512, 512, 512, sw, off, P * 2,
                                                   512, None)
    assert f(0) == OK and f(1) == OK
    assert f(2) == INVALID
    assert f(0, off=None) == INVALID and f(1, off=None) == INVALID
    assert f(0, n=8, X=None) == INVALID and f(1, n=8, X=None) == INVALID
    assert f(0, n=8, X=2 * P) == INVALID and f(1, n=8, X=2 * P) == INVALID  # in place
    assert f(1, sw=None) == INVALID and f(0, sw=None) == OK


def test_plan_refusals():
    import ctypes
    L, out = rmm.lib(), ctypes.cast((ctypes.c_int32 * 3)(), ctypes.c_void_p)
    good = (1, 8, 256, 512, 2, SMS, out)
    assert L.rmm_debug_grouped_plan(*good) == OK
    for i, bad in ((0, 2), (1, 0), (2, 0), (3, 0), (4, 0), (5, 0), (6, None)):
        assert L.rmm_debug_grouped_plan(*good[:i], bad, *good[i + 1:]) == INVALID
    for i, most in ((1, (1 << 31) - 257), (2, 1 << 24), (3, (1 << 31) - 513), (4, 1024), (5, 1 << 20)):
        assert L.rmm_debug_grouped_plan(*good[:i], most, *good[i + 1:]) == OK
        assert L.rmm_debug_grouped_plan(*good[:i], most + 1, *good[i + 1:]) == UNSUPPORTED


def test_no_code_for_e4m3_pairs():
    """e4m3 tiles are single CTAs': their sources hold no pair form of the e4m3 product."""
    assert plan(E4M3, 8192, 4096, 14336, 8)[:2] == (128, 256)
    for f in os.listdir(rmm_build.CSRC):
        with open(os.path.join(rmm_build.CSRC, f)) as h:
            assert "cta_group::2.kind::f8f6f4" not in h.read(), f
