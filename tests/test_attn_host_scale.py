"""A scale whose product with log2(e) is no FP32 number would make NaN of every score that is zero: refused."""
import pytest

from test_attn_host import INVALID, call, dg      # noqa: F401  (fixtures)


@pytest.mark.parametrize("name", ["det_attn_decode", "det_attn", "det_attn_bwd"])
def test_scales_at_the_end_of_the_range(call, name):      # noqa: F811
    for scale in (3.4028234e38, 2.5e38, float("inf"), 0.0, -1e-30):
        assert call(name, scale=scale) == INVALID
    for scale in (2.0 ** 127, 1e-45, 1e38):
        assert call(name, scale=scale, D=12) == INVALID and call(name, scale=scale) != INVALID
