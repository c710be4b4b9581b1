"""The cache operators without a GPU: what is refused at the ends of sizes and factors."""

import pytest

from test_kv_cpu import INVALID, UNSUPPORTED, _append, _attend


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** 101, -2.0 ** 101, 3e38, -3e38, float("-inf")])
def test_scales_beyond_their_limit(lib, fp8, scale):
    so = lib.load_library()
    assert _attend(so, fp8, scale=scale) == INVALID
    assert b"scale" in so.rope_last_error()


@pytest.mark.parametrize("sizes", [
    dict(B=2 ** 31 - 1, S=1, Nq=1, Nkv=1), dict(B=2 ** 31 - 200, S=1, Nq=1, Nkv=1),    # rows of Q, and blocks
    dict(B=1, S=2 ** 31 - 100, Nq=1, Nkv=1), dict(B=3, S=715827882, Nq=1, Nkv=1),      # rows of Q
    dict(B=2 ** 28 - 1, S=1, Nq=8, Nkv=8), dict(B=2 ** 27 - 1, S=2, Nq=8, Nkv=8),      # blocks
])
def test_appends_just_below_2_31_rows(lib, sizes):
    """Rows and blocks are counted in 32 bits by CTAs that may reach beyond the last one."""
    so = lib.load_library()
    assert _append(so, H=2, L=1, **sizes) == UNSUPPORTED
    assert b"2^31" in so.rope_last_error()
