"""The mixer operators' refusals, without a GPU: bad arguments are turned away
on the host before any launch, by the C ABI and by the binding."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rs():
    import state_space_recurrence_amd as rs
    if not os.path.exists(rs.LIB_PATH):
        from state_space_recurrence_amd import build
        build.build()
    return rs


@pytest.fixture(scope="module")
def m(rs):
    from state_space_recurrence_amd import mixer
    mixer._lib()
    return mixer


def _desc(m, **kw):
    d = dict(batch=4, n_slots=0, n_heads=8, head_dim=64, d_state=128, n_groups=2, width=4, max_draft=5, in_dtype=1,
             activation=1, dt_min=0.0, dt_max=math.inf)
    d.update(kw)
    return m.RssmConvDesc(**d)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), ({"width": 2}, 0), ({"in_dtype": 0}, 0), ({"batch": 0}, 0),
    ({"batch": -1}, -1), ({"n_slots": -1}, -1), ({"n_heads": 7}, -1), ({"n_groups": 0}, -1), ({"n_heads": 0}, -1),
    ({"head_dim": 32}, -2), ({"d_state": 64}, -2), ({"width": 1}, -2), ({"width": 5}, -2),
    ({"max_draft": 0}, -3), ({"max_draft": 9}, -3), ({"in_dtype": 2}, -2), ({"activation": 2}, -1),
    ({"dt_min": 1.0, "dt_max": 0.5}, -1), ({"dt_min": math.nan}, -1), ({"n_heads": 1 << 15}, -1),
    ({"batch": 1 << 21}, -1),
])
def test_conv_descriptor(m, kw, code):
    L = m._lib()
    d = _desc(m, **kw)
    assert L.replayssm_conv_check_desc(ctypes.byref(d)) == code
    if code:
        assert L.replayssm_last_error().decode()


def test_ring_rows(m):
    rows = lambda **kw: m._lib().replayssm_conv_ring_rows(ctypes.byref(_desc(m, **kw)))  # noqa: E731
    assert rows(width=4, max_draft=5) == 8 and rows(width=4, max_draft=1) == 6
    assert rows(width=2, max_draft=1) == 2 and rows(width=2, max_draft=8) == 9
    assert rows(width=9) == 0


def test_conv_calls_refuse(m):
    L = m._lib()
    R = ctypes.byref
    d, st, io = _desc(m), m.RssmConvState(), m.RssmConvIO()
    assert L.replayssm_conv_step(None, R(st), R(io), None) == -1
    assert L.replayssm_conv_step(R(d), None, R(io), None) == -1
    assert L.replayssm_conv_step(R(d), R(st), R(io), None) == -1 and b"ring" in L.replayssm_last_error()
    full = m.RssmConvState(*([16] * 6), None)             # placeholders: nothing is launched
    assert L.replayssm_conv_step(R(d), R(full), None, None) == -1
    assert L.replayssm_conv_step(R(d), R(full), R(io), None) == -1
    cc = 8 * 64 + 2 * 2 * 128
    short = m.RssmConvIO(16, cc - 1, 16, 8, 16, 16, 16, 16)
    assert L.replayssm_conv_step(R(d), R(full), R(short), None) == -1 and b"pitch" in L.replayssm_last_error()
    ok = m.RssmConvIO(16, cc, 16, 8, 16, 16, 16, 16)
    for T in (0, 6, -1):
        assert L.replayssm_conv_verify(R(d), R(full), T, R(ok), None) == -3
        assert L.replayssm_conv_accept(R(d), R(full), 16, T, None) == -3
    assert L.replayssm_conv_accept(R(d), R(full), None, 2, None) == -1
    few = _desc(m, n_slots=2)
    assert L.replayssm_conv_step(R(few), R(full), R(ok), None) == -1 and b"n_slots" in L.replayssm_last_error()
    pre = lambda total, cu, fz, st=full, io=ok: L.replayssm_conv_prefill(  # noqa: E731
        R(d), R(st), total, cu, fz, None, R(io), None)
    assert pre(-1, 16, 0) == -1 and pre((1 << 30) + 1, 16, 0) == -1 and pre(8, 16, 2) == -1 and pre(8, None, 0) == -1
    assert pre(0, None, 0) == 0                            # no tokens: nothing to do
    empty = _desc(m, batch=0)
    assert L.replayssm_conv_step(R(empty), R(st), R(io), None) == 0


def test_packed_prefill_refuses(rs, m):
    L = m._lib()
    d = rs._make_desc(4, 8, 64, 128, 1, 16, 1, rs.BF16)
    st = rs.RssmState(*([16] * 11))
    A = ctypes.addressof
    call = lambda total=8, cu=16, fz=0, x=16, C=16, y=16, yt=0: L.replayssm_prefill_packed(  # noqa: E731
        A(d), A(st), total, cu, fz, None, x, 16, C, 16, y, yt, None, 0, None)
    assert call(total=-1) == -1 and call(total=1 << 29) == -1 and call(fz=3) == -1 and call(yt=2) == -2
    assert call(cu=None) == -1 and call(x=None) == -1 and call(C=None) == -1
    assert L.replayssm_prefill_packed(None, A(st), 8, 16, 0, None, 16, 16, 16, 16, 16, 0, None, 0, None) == -1
    assert L.replayssm_prefill_packed(A(d), None, 8, 16, 0, None, 16, 16, 16, 16, 16, 0, None, 0, None) == -1
    assert call(total=0, cu=None) == 0
    ws = lambda n: L.replayssm_prefill_packed_workspace(A(d), n)  # noqa: E731
    assert ws(-1) == 0 and ws(0) == 0 and ws(1 << 31) == 0 and ws(100000) > 0
    assert L.replayssm_prefill_packed(A(d), A(st), 100000, 16, 0, None, 16, 16, 16, 16, 16, 0, 16, ws(100000) - 1,
                                      None) == -1 and b"workspace" in L.replayssm_last_error()
    low = rs._make_desc(4, 8, 64, 128, 1, 16, 1, rs.BF16, ckpt_dtype=rs.BF16, out_dtype=rs.FP4_E2M1)
    assert L.replayssm_prefill_packed_workspace(A(low), 100000) == 0
    wide = rs._make_desc(4, (1 << 15) + 1, 64, 128, 1, 16, 1, rs.BF16)
    assert L.replayssm_prefill_packed(A(wide), A(st), 8, 16, 0, None, 16, 16, 16, 16, 16, 0, None, 0, None) == -3


def test_norms_refuse(m):
    L = m._lib()
    gn = lambda rows=4, dim=64, groups=1, y=16, yt=0, zt=1, pitch=64, eps=1e-5, before=0, out=16, ot=1: \
        L.replayssm_gated_norm(rows, dim, groups, y, yt, 16, zt, pitch, 16, eps, before, out, ot, None)  # noqa: E731
    assert gn(rows=-1) == -1 and gn(dim=0) == -1 and gn(dim=65, groups=2, pitch=65) == -1 and gn(groups=0) == -1
    assert gn(dim=16385, pitch=16385) == -3 and gn(yt=2) == -2 and gn(zt=4) == -2 and gn(ot=3) == -2
    assert gn(pitch=63) == -1 and gn(eps=-1.0) == -1 and gn(eps=math.nan) == -1 and gn(eps=math.inf) == -1
    assert gn(before=2) == -1 and gn(y=None) == -1 and gn(out=None) == -1
    assert gn(rows=0, y=None) == 0
    an = lambda rows=4, dim=64, x=16, xt=1, ro=16, rt=0, eps=1e-5, ot=1: L.replayssm_add_norm(  # noqa: E731
        rows, dim, x, xt, 16, ro, rt, 16, None, 1.0, eps, 16, ot, None)
    assert an(rows=-1) == -1 and an(dim=0) == -1 and an(dim=20000) == -3 and an(xt=2) == -2 and an(rt=4) == -2
    assert an(ot=5) == -2 and an(x=None) == -1 and an(ro=None) == -1 and an(eps=-0.5) == -1 and an(rows=0) == 0


def test_binding_refuses_bad_tensors(rs):
    """Shapes, types, devices and strides are checked before the library is called."""
    E = rs.ReplaySSMError
    Cc = 8 * 64 + 2 * 128
    cs = rs.ConvState(2, 8, 1, torch.zeros(Cc, 4), device="cpu")
    with pytest.raises(E, match="u:"):
        rs.conv_step(cs, torch.zeros(2, Cc, dtype=torch.bfloat16), torch.zeros(2, 8, dtype=torch.bfloat16))
    with pytest.raises(E, match="slots"):
        rs.conv_step(cs, torch.zeros(3, Cc), torch.zeros(3, 8))
    for kw in (dict(weight=torch.zeros(Cc, 5)), dict(weight=torch.zeros(Cc - 1, 4)), dict(bias=torch.zeros(3)),
               dict(dt_bias=torch.zeros(7)), dict(activation="gelu"), dict(in_dtype=torch.float16),
               dict(max_draft=9), dict(dt_limit=(2.0, 1.0))):
        args = dict(weight=torch.zeros(Cc, 4), device="cpu")
        args.update(kw)
        with pytest.raises(E):
            rs.ConvState(2, 8, 1, **args)
    w = torch.ones(64)
    with pytest.raises(E, match="y:"):
        rs.gated_norm(torch.zeros(2, 64), torch.zeros(2, 64), w)
    with pytest.raises(E, match="rows, dim"):
        rs.add_norm(torch.zeros(64), torch.zeros(64), w)
    with pytest.raises(E, match="x:"):
        rs.add_norm(torch.zeros(2, 64), torch.zeros(2, 64), w)
    with pytest.raises(E, match="cu_seqlens"):
        rs.conv_prefill(cs, torch.zeros(2, Cc), torch.zeros(2, 8), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(E, match="offset"):
        rs.conv_prefill(cs, torch.zeros(2, Cc), torch.zeros(2, 8), torch.zeros(0, dtype=torch.int32))


def test_view_pitch(rs, m, monkeypatch):
    """Which strided views of projection rows are taken, and their pitch (device check aside)."""
    class Dev(torch.Tensor):
        is_cuda = True
    mk = lambda t: t.as_subclass(Dev)  # noqa: E731
    f = torch.float32
    base = torch.zeros(6, 100)
    assert m._pitch(mk(base[:, 10:40]), (6,), 30, f, "u") == 100
    assert m._pitch(mk(base[:, 10:40].unflatten(0, (2, 3))), (2, 3), 30, f, "u") == 100
    assert m._pitch(mk(base[:1, :30]), (1,), 30, f, "u") == 100
    assert m._pitch(mk(base[:0, :30]), (0,), 30, f, "u") >= 30
    assert m._pitch(mk(torch.zeros(1, 3, 100)[:, :, :30]), (1, 3), 30, f, "u") == 100
    assert m._pitch(mk(torch.zeros(4, 1, 100)[:, :, :30]), (4, 1), 30, f, "u") == 100
    assert m._pitch(mk(torch.zeros(5, 1)), (5,), 1, f, "dt") == 1
    for bad, lead, width in ((base.t()[:6, :3], (6,), 3), (torch.zeros(2, 4, 100)[:, :3, :30], (2, 3), 30),
                             (base[:, ::2], (6,), 50), (torch.zeros(1, 30).expand(6, 30), (6,), 30)):
        with pytest.raises(rs.ReplaySSMError, match="strides"):
            m._pitch(mk(bad), lead, width, f, "u")


SAN = ["-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer"]


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="needs g++ and the ROCm headers")
def test_mixer_host_checks_under_sanitizers(tmp_path):
    """mixer_api.cpp with launchers that abort, under AddressSanitizer and UndefinedBehaviorSanitizer (host code)."""
    exe = str(tmp_path / "mixer_checks")
    src = os.path.join(ROOT, "state_space_recurrence_amd", "csrc")
    cmd = ["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
           "-I" + src, os.path.join(src, "mixer_api.cpp"), os.path.join(ROOT, "tests", "sanitize", "mixer_api_checks.cpp"),
           "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0:abort_on_error=1"})
    assert r.returncode == 0 and "0 failed" in r.stdout, r.stdout + r.stderr
