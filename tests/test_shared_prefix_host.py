"""How shared-prefix decode is launched, by its sizes, and what its tests' bounds let through (no GPU)."""
import numpy as np
import pytest
import torch

import rows_cases


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_193_gb300 import build, _lib
    build.build()
    return _lib.load()


@pytest.mark.parametrize("S,G,Hq,Hkv,D,B,width", [(4, 1, 32, 8, 128, 16, 8), (64, 1, 64, 8, 128, 16, 2176), (256, 1, 32, 8, 128, 16, 160),
                                                  (90, 7, 16, 16, 64, 32, 330), (7, 1, 32, 8, 128, 16, 435), (7, 1, 32, 8, 128, 16, 436)])
@pytest.mark.parametrize("dt", [0, 1])
def test_a_bound_past_the_tables_width_is_that(lib, S, G, Hq, Hkv, D, B, width, dt):
    """No prefix is longer than the tables: whether it is taken once goes by their width, whatever the bound.  (A bound that
    is larger may mean fewer parts, by which a join may move; not whether anything is shared.)"""
    def launches(bound):
        return lib.pa_shared_prefix_launches(S, G, Hq, Hkv, D, B, width, bound, dt)

    for bound in (width + 1, 2 * width, 1 << 20):
        assert (launches(bound) > 1) == (launches(width) > 1)


@pytest.mark.parametrize("width,bound", [(40, 40), (40, 33), (40, 30), (40, 4), (700, 300), (9000, 33), (9000, 9000)])
@pytest.mark.parametrize("S,G", [(1, 1), (9, 1), (64, 1), (130, 3), (300, 1), (2000, 1), (2000, 70)])
@pytest.mark.parametrize("dt", [0, 1])
def test_the_join_is_apart_where_a_test_asks_for_it(lib, S, G, width, bound, dt):
    """And with it in the rest's kernel: of every launch that there is, a warp to a head for short lists among them."""
    try:
        for Hq, Hkv, D, B in ((8, 2, 128, 16), (32, 8, 128, 16), (16, 16, 64, 32), (64, 4, 128, 32)):
            for apart in (0, 1):
                assert lib.pa_test_set_share(0, apart) == 0
                assert lib.pa_shared_prefix_launches(S, G, Hq, Hkv, D, B, width, bound, dt) == 2 + apart
    finally:
        assert lib.pa_test_set_share(-1, -1) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [0, 3, 5])
def test_a_prefix_of_one_page_less_is_past_the_bound(page, fp8):
    """A page of the prefix that is left out, as a kernel would that counts one too few: every sequence that holds the prefix
    is outside its bound, one that does not is untouched."""
    case = rows_cases.Shared("cpu", [(6, [40, 3, -90])], 4, 2, D=64, fp8=fp8)
    good = case.expected()
    rows_cases.within(torch.from_numpy(good[0]), good)
    full, lens = case.tables.clone(), list(case.lens)
    for s in range(2):
        row = torch.cat([full[s, :page], full[s, page + 1:], torch.tensor([-1], dtype=torch.int32)])
        case.tables[s] = row
        case.lens[s] = lens[s] - 16
    wrong = case.expected()[0]
    assert np.array_equal(wrong[2], good[0][2])
    for s in range(2):
        with pytest.raises(AssertionError):
            rows_cases.within(torch.from_numpy(wrong[s]), tuple(x[s] for x in good))
