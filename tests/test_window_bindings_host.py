"""The Python side of the rotary append's and the windowed attention's bindings, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def native():
    from paged_kv_cache_207_gb300 import build, _native
    build.build()
    return _native


def test_bounds_past_int32_stay_on_their_side(native):
    for x, want in ((-2**32 + 5, -2**31), (-2**63, -2**31), (-2**31, -2**31), (-7, -7), (0, 0), (2**31 - 1, 2**31 - 1),
                    (2**31, 2**31 - 1), (2**32 + 5, 2**31 - 1), (2**100, 2**31 - 1)):
        assert native._bound(x) == want, x
