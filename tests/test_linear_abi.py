"""Refusals of the products and of rows in 8 bits, without a GPU: bad arguments
are turned away on the host before any launch, by the C ABI and by the binding."""
import ctypes
import math
import os

import pytest
import torch

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def rs():
    import state_space_recurrence_amd as rs
    if not os.path.exists(rs.LIB_PATH):
        from state_space_recurrence_amd import build
        build.build()
    return rs


@pytest.fixture(scope="module")
def m(rs):
    from state_space_recurrence_amd import projection
    projection._lib()
    return projection


def _call(m, desc=None, io=None, mx=False):
    """replayssm_linear's status with these fields changed; placeholders as pointers: nothing may be launched."""
    d = dict(rows=4, n_in=64, n_out=96, in_dtype=2 if mx else 1, out_dtype=1, res_dtype=4, activation=0, scale=1.0)
    d.update(desc or {})
    b = dict(x=16, x_pitch=d["n_in"], x_scales=16 if mx else None, weight=16, weight_scales=16 if mx else None, bias=None,
             residual=None, out=16, out_scales=16)
    b.update(io or {})
    D, I = m.RssmLinearDesc(**d), m.RssmLinearIO(**b)
    return m._lib().replayssm_linear(ctypes.addressof(D), ctypes.addressof(I), None)


@pytest.mark.parametrize("desc,code", [
    ({"rows": -1}, -1), ({"rows": (1 << 26) + 1}, -1), ({"n_in": 0}, -1), ({"n_out": 0}, -1), ({"n_in": (1 << 20) + 1}, -1),
    ({"n_out": (1 << 20) + 1}, -1), ({"in_dtype": 0}, -2), ({"in_dtype": 3}, -2), ({"out_dtype": 3}, -2),
    ({"out_dtype": 4}, -2), ({"res_dtype": 2}, -2), ({"res_dtype": 5}, -2), ({"activation": -1}, -1), ({"activation": 4}, -1),
    ({"out_dtype": 2, "n_out": 48}, -1), ({"rows": 1 << 26, "n_out": 1 << 20}, -3), ({"rows": 1 << 26, "n_out": 1024}, -3),
    ({"rows": 0}, 0), ({"rows": 0, "out_dtype": 2}, 0),
])
def test_descriptor(m, desc, code):
    assert _call(m, desc) == code
    if code:
        assert m._lib().replayssm_last_error().decode()


def test_descriptor_mx(m):
    assert _call(m, {"n_in": 48}, mx=True) == -1 and b"32" in m._lib().replayssm_last_error()
    assert _call(m, {"rows": 0}, mx=True) == 0


@pytest.mark.parametrize("mx,desc,io,text", [
    (False, {}, {"x": None}, "NULL"), (False, {}, {"weight": None}, "NULL"), (False, {}, {"out": None}, "NULL"),
    (True, {}, {"x_scales": None}, "NULL"), (True, {}, {"weight_scales": None}, "NULL"),
    (True, {}, {"x": 24}, "16 bytes"), (True, {}, {"weight": 8}, "16 bytes"),
    (False, {"out_dtype": 2}, {"out_scales": None}, "NULL"), (False, {"out_dtype": 2}, {"out": 20}, "16 bytes"),
    (False, {}, {"residual": 16}, "res_dtype"), (False, {"res_dtype": 0}, {}, "res_dtype"),
    (False, {}, {"x_pitch": 63}, "x_pitch"), (True, {}, {"x_pitch": 65}, "x_pitch"),
    (False, {}, {"x_pitch": (1 << 22) + 1}, "x_pitch"),
])
def test_buffers(m, mx, desc, io, text):
    assert _call(m, desc, io, mx) in (-1, -3)
    assert text in m._lib().replayssm_last_error().decode()


def test_null_structs(m):
    L = m._lib()
    assert L.replayssm_linear(None, None, None) == -1
    d = m.RssmLinearDesc(4, 64, 96, 1, 1, 4, 0, 1.0)
    assert L.replayssm_linear(ctypes.addressof(d), None, None) == -1
    d.rows = 0
    assert L.replayssm_linear(ctypes.addressof(d), None, None) == 0


def test_rows_in_8_bits_refuse(m):
    L = m._lib()
    q = lambda rows=4, dim=64, x=16, xt=1, pitch=64, c=16, s=16: L.replayssm_quantize_mx(  # noqa: E731
        rows, dim, x, xt, pitch, c, s, None)
    assert q(rows=-1) == -1 and q(rows=(1 << 26) + 1) == -1 and q(dim=0) == -1 and q(dim=33, pitch=33) == -1
    assert q(dim=(1 << 20) + 32, pitch=1 << 21) == -3 and q(xt=2) == -2 and q(x=None) == -1 and q(c=None) == -1
    assert q(s=None) == -1 and q(c=8) == -1 and q(pitch=63) == -1 and q(rows=0, x=None) == 0
    gn = lambda rows=4, dim=64, groups=1, y=16, yt=0, zt=1, pitch=64, eps=1e-5, before=0, c=16, s=16: \
        L.replayssm_gated_norm_mx(rows, dim, groups, y, yt, 16, zt, pitch, 16, eps, before, c, s, None)  # noqa: E731
    assert gn(rows=-1) == -1 and gn(dim=0) == -1 and gn(groups=0) == -1 and gn(dim=96, groups=2, pitch=96) == -1
    assert gn(dim=16416, pitch=16416) == -3 and gn(yt=2) == -2 and gn(zt=4) == -2 and gn(pitch=63) == -1
    assert gn(eps=-1.0) == -1 and gn(eps=math.nan) == -1 and gn(eps=math.inf) == -1 and gn(before=2) == -1
    assert gn(y=None) == -1 and gn(c=None) == -1 and gn(s=None) == -1 and gn(c=4) == -1 and gn(rows=0, y=None) == 0
    an = lambda rows=4, dim=64, x=16, xt=1, ro=16, rt=0, post=None, eps=1e-5, c=16, s=16: L.replayssm_add_norm_mx(  # noqa: E731
        rows, dim, x, xt, 16, ro, rt, 16, post, 1.0, eps, c, s, None)
    assert an(rows=-1) == -1 and an(dim=40) == -1 and an(dim=16416) == -3 and an(xt=2) == -2 and an(rt=4) == -2
    assert an(ro=None) == -1 and an(x=None) == -1 and an(x=None, ro=None, post=16) == -1 and an(eps=-0.5) == -1
    assert an(c=None) == -1 and an(s=None) == -1 and an(c=1) == -1 and an(rows=0) == 0


def _device_tensors(monkeypatch):
    """Tensors that say they are on device 0, the current one (nothing is launched)."""
    class Dev(torch.Tensor):
        is_cuda = True
        at = 0

        def get_device(self):
            return self.at
    from state_space_recurrence_amd import projection
    monkeypatch.setattr(projection, "_current_device", lambda: 0)
    return lambda t: t.as_subclass(Dev)


def test_binding_refuses(rs):
    """Shapes, types, devices and pairs are checked before the library is called."""
    E = rs.ReplaySSMError
    x, w = torch.zeros(2, 64, dtype=BF16), torch.zeros(96, 64, dtype=BF16)
    pair = lambda n, k: (torch.zeros(n, k, dtype=torch.float8_e4m3fn),  # noqa: E731
                         torch.zeros(n, k // 32, dtype=torch.float8_e8m0fnu))
    for match, args, kw in (
            ("activation", (x, w), dict(activation="tanh")), ("x: expected a device", (x, w), {}),
            ("pairs", (x, pair(96, 64)), {}), ("pairs", (pair(2, 64), w), {}), ("x: expected", ((), ()), {}),
            ("x: expected", (None, None), {}), ("x: expected a device", (pair(2, 64), pair(96, 64)), {})):
        with pytest.raises(E, match=match):
            rs.linear(*args, **kw)
    for bad in (torch.zeros(64), torch.zeros(2, 48), torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.float16)):
        with pytest.raises(E):
            rs.quantize_mx(bad)
        with pytest.raises(E):
            rs.gated_norm_mx(bad, bad, torch.ones(64))
        with pytest.raises(E):
            rs.add_norm_mx(bad, bad, torch.ones(64))


def test_binding_refuses_device_tensors(rs, monkeypatch):
    """What is refused once the operands themselves are device tensors."""
    mk = _device_tensors(monkeypatch)
    E = rs.ReplaySSMError
    x, w = mk(torch.zeros(2, 64, dtype=BF16)), mk(torch.zeros(96, 64, dtype=BF16))
    f = lambda *s: mk(torch.zeros(*s))  # noqa: E731
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    pair = lambda n, k: (f(n, k).to(e4), f(n, k // 32).to(e8))  # noqa: E731
    for match, kw in (("bias", dict(bias=f(95))), ("bias", dict(bias=f(96).to(BF16))), ("bias", dict(bias=torch.zeros(96))),
                      ("residual", dict(residual=f(2, 95))), ("residual", dict(residual=f(2, 96).to(torch.float16))),
                      ("out", dict(out=f(2, 95))), ("out", dict(out_dtype=torch.float16)),
                      ("out", dict(out=f(2, 96).to(e4))), ("pair", dict(out=(f(2, 96),))),
                      ("out codes", dict(out=(f(2, 96), f(2, 3)))), ("out scales", dict(out=(f(2, 96).to(e4), f(2, 3))))):
        with pytest.raises(E, match=match):
            rs.linear(x, w, **kw)
    for match, args in (("n_in", (f(64).to(BF16), w)), ("n_in", (x, f(64).to(BF16))), ("n_in", (x, None)),
                        ("x:", (f(2, 64), w)), ("weight", (x, f(96, 64))), ("weight", (x, f(96, 32).to(BF16))),
                        ("multiple of 32", (pair(2, 48), pair(96, 48))), ("pair", (pair(2, 64) + (x,), pair(96, 64))),
                        ("x codes", ((x, f(2, 2).to(e8)), pair(96, 64))), ("x scales", ((pair(2, 64)[0], f(2, 2)), pair(96, 64))),
                        ("weight scales", (pair(2, 64), (pair(96, 64)[0], f(95, 2).to(e8))))):
        with pytest.raises(E, match=match):
            rs.linear(*args)
    with pytest.raises(E, match="multiple of 32"):
        rs.linear(x, mk(torch.zeros(95, 64, dtype=BF16)), out_dtype=e4)
    with pytest.raises(E, match="weight"):
        rs.linear(x, mk(torch.zeros(96, 128, dtype=BF16))[:, ::2])
    with pytest.raises(E, match="strides"):
        rs.linear(mk(torch.zeros(2, 128, dtype=BF16))[:, ::2], w)
    with pytest.raises(E, match="residual_out"):
        rs.add_norm_mx(None, f(2, 64), f(64), residual_out=f(2, 64))
    with pytest.raises(E, match="residual_out"):
        rs.add_norm_mx(None, f(2, 64), f(64), post_weight=f(64))
    for bad in (dict(y=f(2, 32)), dict(y=f(2, 64).to(torch.float16)), dict(y=torch.zeros(2, 64)), dict(y=f(1, 128)),
                dict(weight=f(63)), dict(z=f(2, 128)[:, ::2])):
        with pytest.raises(E):
            rs.gated_norm_mx(**{**dict(y=f(2, 64), z=f(2, 64), weight=f(64)), **bad})
    for bad in (dict(x=f(2, 32)), dict(x=f(2, 64).to(torch.float16)), dict(residual_out=f(2, 64).to(BF16)),
                dict(post_weight=f(32)), dict(residual=f(2, 128)[:, ::2])):
        with pytest.raises(E):
            rs.add_norm_mx(**{**dict(x=f(2, 64), residual=f(2, 64), weight=f(64)), **bad})


def test_tensors_of_other_devices_are_refused(rs, monkeypatch):
    mk = _device_tensors(monkeypatch)
    x, w, b = mk(torch.zeros(2, 64, dtype=BF16)), mk(torch.zeros(96, 64, dtype=BF16)), mk(torch.zeros(96))
    b.at = 1
    with pytest.raises(rs.ReplaySSMError, match="bias: is on device 1"):
        rs.linear(x, w, b)
    x.at = 1
    with pytest.raises(rs.ReplaySSMError, match="not the current"):
        rs.linear(x, w)
    r = mk(torch.zeros(2, 64))
    with pytest.raises(rs.ReplaySSMError, match="x: is on device 1"):
        rs.add_norm_mx(x, r, mk(torch.zeros(64)))
    with pytest.raises(rs.ReplaySSMError, match="y: expected"):
        rs.gated_norm_mx(x, r, mk(torch.zeros(64)))
