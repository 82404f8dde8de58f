"""The choice of products is checked on the host, without a GPU."""
import inspect

import pytest

from test_linear_abi import _call, m, rs  # noqa: F401


@pytest.mark.parametrize("products,code", [(-1, -1), (2, -1), (0, 0), (1, 0)])
def test_products(m, products, code):  # noqa: F811
    for mx in (False, True):
        assert _call(m, {"rows": 0, "products": products}, mx=mx) == code
    if code:
        assert b"products" in m._lib().replayssm_last_error()


def test_exact_products_unless_asked(rs, m):  # noqa: F811
    assert inspect.signature(rs.linear).parameters["fast_products"].default is False
    assert m.RssmLinearDesc().products == 0
