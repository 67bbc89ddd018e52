"""How shared-prefix decode is launched, by its sizes (no GPU)."""
import pytest


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
