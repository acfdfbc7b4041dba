"""The scale of paged attention is used times log2 e: both have to be finite numbers."""
import pytest

from tests.test_paged_abi import INVALID, OK, attention, mnb  # noqa: F401  (mnb: a fixture)


@pytest.mark.parametrize("scale,rc", [(3.0e38, INVALID), (-3.0e38, INVALID), (2.5e38, INVALID), (1.9e38, OK),
                                      (-1.9e38, OK), (0.0, OK)])
def test_scale_whose_product_overflows(mnb, scale, rc):  # noqa: F811
    assert attention(mnb, B=0, scale=scale) == rc
