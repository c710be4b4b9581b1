"""The cache operators without a GPU: what is refused at the ends of sizes and factors."""

import pytest

from test_kv_cpu import INVALID, _attend


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** 101, -2.0 ** 101, 3e38, -3e38, float("-inf")])
def test_scales_beyond_their_limit(lib, fp8, scale):
    so = lib.load_library()
    assert _attend(so, fp8, scale=scale) == INVALID
    assert b"scale" in so.rope_last_error()
