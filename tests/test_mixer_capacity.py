"""Calls of more threads than one launch holds are refused on the host."""
import ctypes
import math

import pytest

from test_mixer_abi import m, rs  # noqa: F401


@pytest.fixture
def conv(m):  # noqa: F811
    L = m._lib()
    heads = 16000                                      # 1024256 channels: 501 workgroups a row
    cc = 64 * heads + 256

    def call(batch, total=None):
        d = m.RssmConvDesc(batch, 0, heads, 64, 128, 1, 4, 1, 1, 1, 0.0, math.inf)
        st, io = m.RssmConvState(*([16] * 6), None), m.RssmConvIO(16, cc, 16, heads, 16, 16, 16, 16)
        if total is None:
            return L.replayssm_conv_step(ctypes.byref(d), ctypes.byref(st), ctypes.byref(io), None)
        return L.replayssm_conv_prefill(ctypes.byref(d), ctypes.byref(st), total, 16, 0, None, ctypes.byref(io), None)
    return call


def test_conv(m, conv):  # noqa: F811
    """2^24 workgroups of 256 threads or more: tokens from 33488 rows on, packed ones from 33488 tiles of 32."""
    for call in (dict(batch=1 << 20), dict(batch=33488), dict(batch=1, total=1 << 30), dict(batch=1, total=33488 * 32)):
        assert conv(**call) == -3 and b"launch" in m._lib().replayssm_last_error(), call
