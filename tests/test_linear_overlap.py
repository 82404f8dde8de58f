"""Outputs of the projections and of rows in 8 bits that overlap what the call reads (or each other) are refused on the
host, without a GPU: other workgroups may still read there.  Addresses are placeholders, nothing may be launched."""
import ctypes

import pytest

from test_linear_abi import _call, m, rs  # noqa: F401

FAR = 1 << 32
# 4 rows of 64 inputs, 96 outputs, bf16: where every buffer of the product lies when it is by itself
AT = dict(x=FAR, weight=2 * FAR, bias=3 * FAR, residual=4 * FAR, out=5 * FAR, x_scales=6 * FAR, weight_scales=7 * FAR,
          out_scales=8 * FAR)


def _linear(m, desc=None, **io):  # noqa: F811
    d = {"res_dtype": 1, **(desc or {})}
    b = {**AT, **io}
    if d["res_dtype"] == 4:
        b["residual"] = None
    return _call(m, d, b, mx=d.get("in_dtype") == 2)


BYTES = {"x": 4 * 64 * 2, "weight": 96 * 64 * 2, "bias": 96 * 4, "residual": 4 * 96 * 2}


@pytest.mark.parametrize("name", list(BYTES))
@pytest.mark.parametrize("end", ["first", "last"])
def test_product_over_an_operand(m, name, end):  # noqa: F811
    out = AT[name] + (BYTES[name] - 2 if end == "last" else 2 - 4 * 96 * 2)
    assert _linear(m, out=out) == -1
    assert b"overlap" in m._lib().replayssm_last_error()


@pytest.mark.parametrize("desc,io", [
    ({}, dict(out=AT["x"])),                                                     # 96 outputs over 64 inputs
    ({"out_dtype": 0}, dict(out=AT["residual"])),                                # the residual's place, another type
    ({"n_out": 64}, dict(out=AT["weight"])),
    ({"out_dtype": 2, "res_dtype": 4}, dict(out=AT["out"], out_scales=AT["out"] + 4 * 96 - 1)),   # scales over codes
    ({"out_dtype": 2, "res_dtype": 4}, dict(out_scales=AT["x"] + 64)),
    ({"out_dtype": 2}, dict(out=AT["residual"])),
    ({"in_dtype": 2}, dict(out=AT["x_scales"] - 4 * 96 * 2 + 1)),
    ({"in_dtype": 2}, dict(out=AT["weight_scales"] + 96 * 2 - 1)),
    ({"in_dtype": 2, "out_dtype": 2, "n_out": 64, "res_dtype": 4}, dict(out=AT["x"])),             # 8-bit rows in place
    ({}, dict(x_pitch=512, out=AT["x"] + 2 * 3 * 512)),                          # the last of strided rows
    ({}, dict(x_pitch=512, out=AT["x"] + 2 * 64 + 896 - 768 + 2)),               # from between two rows into the next
])
def test_products_that_overlap(m, desc, io):  # noqa: F811
    assert _linear(m, desc, **io) == -1
    assert b"overlap" in m._lib().replayssm_last_error()


def _refused(m, rc):  # noqa: F811
    assert rc == -1 and b"overlap" in m._lib().replayssm_last_error()


def test_rows_in_8_bits_that_overlap(m):  # noqa: F811
    L = m._lib()
    X, C, S, Y, Z, W, R, O, P = (FAR * i for i in range(1, 10))
    q = lambda c=C, s=S, pitch=64: L.replayssm_quantize_mx(4, 64, X, 1, pitch, c, s, None)  # noqa: E731
    for kw in (dict(c=X), dict(c=X + 496), dict(s=X - 7), dict(s=X + 511), dict(s=C), dict(s=C + 255), dict(c=S),
               dict(pitch=640, c=X + 3 * 1280 + 112)):
        _refused(m, q(**kw))
    gn = lambda c=C, s=S: L.replayssm_gated_norm_mx(4, 64, 2, Y, 0, Z, 1, 300, W, 1e-5, 0, c, s, None)  # noqa: E731
    for kw in (dict(c=Y), dict(c=Y + 1008), dict(s=Y + 1023), dict(c=Z), dict(c=Z + 608), dict(s=Z + 127), dict(c=W),
               dict(s=W + 255), dict(s=C + 8)):
        _refused(m, gn(**kw))
    an = lambda x=X, r=R, o=O, xt=1, c=C, s=S, p=P: L.replayssm_add_norm_mx(  # noqa: E731
        4, 64, x, xt, r, o, 0, W, p, 1.0, 1e-5, c, s, None)
    for kw in (dict(c=X), dict(c=R), dict(c=O), dict(s=X + 511), dict(s=R + 1023), dict(s=O + 1023), dict(c=W), dict(s=P),
               dict(s=C + 255), dict(o=X), dict(o=X + 4, xt=0), dict(o=R + 4), dict(o=R - 4), dict(o=W), dict(o=P - 1020),
               dict(x=None, o=None, p=None, c=R), dict(x=None, o=None, p=None, s=R + 1023)):
        _refused(m, an(**kw))


def test_calls_without_rows_overlap_nothing(m):  # noqa: F811
    assert _linear(m, {"rows": 0}, out=AT["x"]) == 0
    L = m._lib()
    assert L.replayssm_quantize_mx(0, 64, FAR, 1, 64, FAR, FAR, None) == 0
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_pitches_that_64_bits_hold_only_as_elements(m):  # noqa: F811
    """Their bytes between rows are more than 2^63."""
    L = m._lib()
    for pitch in (1 << 62, (1 << 62) + 16, (1 << 63) - 1):
        _refused(m, L.replayssm_quantize_mx(4, 64, FAR, 0, pitch, FAR, 2 * FAR, None))
        _refused(m, L.replayssm_gated_norm_mx(4, 64, 1, FAR, 0, 2 * FAR, 0, pitch, 3 * FAR, 1e-5, 0, 2 * FAR, 4 * FAR, None))
