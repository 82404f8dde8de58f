"""GPU parity of the mixer operators (convolution, packed prefill, norms)
against plain 64-bit forms, at the sizes and values where they can go wrong."""
import math

import pytest
import torch

import mixer_ref as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def rs():
    need_gpu()
    import state_space_recurrence_amd as rs
    rs.lib()
    return rs


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _conv(rs, slots, H, G, W, dtype, seed=0, *, bias=True, act="silu", max_draft=1, dt_limit=(0.0, math.inf)):
    g = _gen(seed)
    Cc = 64 * H + 256 * G
    w = (torch.rand(Cc, W, generator=g) * 2 - 1) / math.sqrt(W)
    b = 0.1 * torch.randn(Cc, generator=g) if bias else None
    db = torch.randn(H, generator=g) - 2 if bias else None
    cs = rs.ConvState(slots, H, G, w, b, db, max_draft=max_draft, in_dtype=dtype, activation=act, dt_limit=dt_limit)
    return cs, w, b, db


def _rows(g, lead, H, G, dtype, extra=0):
    """Projection rows [z | x B C | dt] and the views of x B C and dt."""
    Cc = 64 * H + 256 * G
    r = torch.randn(*lead, 64 * H + Cc + H + extra, generator=g).to(dtype)
    d = r.cuda()
    return r[..., 64 * H:64 * H + Cc], r[..., 64 * H + Cc:64 * H + Cc + H], \
        d[..., 64 * H:64 * H + Cc], d[..., 64 * H + Cc:64 * H + Cc + H]


def _history(cs, slot):
    h, W, R = int(cs.head[slot]), cs.width, cs.ring_rows
    return torch.stack([cs.ring[slot, (h - k) % R] for k in range(W - 1, 0, -1)]).cpu()


def _check_conv(got, out, err, dtv, dterr, dtype, H, G, what):
    u = ref.half_step(dtype) if dtype != F32 else 0.0
    flat = torch.cat([got[0].flatten(-2), got[1].flatten(-2), got[2].flatten(-2)], -1)
    # +1e-37: results below the smallest normal number may be flushed
    ref.assert_within(flat, out, err * (1 + u) + u * out.abs() + 1e-37, what)
    ref.assert_within(got[3], dtv, dterr * (1 + u) + u * dtv + 1e-37, what + " dt")


@pytest.mark.parametrize("W,H,G,dtype,bias,act", [
    (4, 8, 1, BF16, True, "silu"), (3, 3, 3, F32, True, "silu"), (2, 6, 2, BF16, False, None),
    (4, 5, 1, F32, False, "silu"), (4, 42, 2, BF16, True, "silu"),
])
def test_conv_step_tokens(rs, W, H, G, dtype, bias, act):
    """Tokens one by one on a mapped pool with a padding row, over more tokens than the ring has rows."""
    S, n = 6, 4
    cs, w, b, db = _conv(rs, S, H, G, W, dtype, seed=W, bias=bias, act=act, dt_limit=(0.01, 1.5))
    g = _gen(5)
    slots = [4, -1, 0, 5]
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    hist = {s: torch.zeros(W - 1, cs.channels, dtype=dtype) for s in slots if s >= 0}
    for t in range(9):
        u, d, ug, dg = _rows(g, (n,), H, G, dtype, extra=t % 3)   # odd pitches and offsets too
        before = cs.snapshot()
        got = rs.conv_step(cs, ug, dg, slots=sl)
        for r, s in enumerate(slots):
            if s < 0:
                continue
            out, err, hist[s] = ref.conv(hist[s], u[r:r + 1], w, b, act is not None)
            dv, de = ref.dt(d[r:r + 1], db, 0.01, 1.5)
            _check_conv([x[r:r + 1] for x in got], out, err, dv, de, dtype, H, G, f"token {t} slot {s}")
            assert torch.equal(_history(cs, s), hist[s])
        for s in (1, 2, 3):   # slots of no row
            assert torch.equal(cs.ring[s], before["ring"][s]) and int(cs.head[s]) == int(before["head"][s])
    cs.check_device_errors()
    assert int(cs.work.abs().sum()) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_rounds_of_drafts(rs, dtype):
    """Verify sees each draft's predecessors; accept keeps a prefix; rejected drafts (NaN) leave no trace."""
    H, G, W, T, n = 6, 2, 4, 8, 5
    cs, w, b, db = _conv(rs, n, H, G, W, dtype, seed=3, max_draft=T)
    g = _gen(7)
    hist = [torch.zeros(W - 1, cs.channels, dtype=dtype) for _ in range(n)]
    for rnd in range(6):
        t = [1, 5, 8, 3, 8, 2][rnd]
        u, d, ug, dg = _rows(g, (n, t), H, G, dtype)
        keep = torch.randint(0, t + 1, (n,), generator=g, dtype=torch.int32)
        ug = ug.clone()
        for r in range(n):
            ug[r, int(keep[r]):] = float("nan")
        got = rs.conv_verify(cs, ug, dg)
        for r in range(n):
            k = int(keep[r])
            out, err, _ = ref.conv(hist[r], u[r], w, b)
            dv, de = ref.dt(d[r], db)
            _check_conv([x[r, :k] for x in got], out[:k], err[:k], dv[:k], de[:k], dtype, H, G, f"round {rnd} row {r}")
            assert torch.equal(_history(cs, r), hist[r])          # verify moves nothing
            assert all(torch.isnan(x[r, k:].float()).all() for x in got[:3])
        rs.conv_accept(cs, keep.cuda(), t)
        for r in range(n):
            hist[r] = torch.cat([hist[r], u[r, :int(keep[r])]])[-(W - 1):]
            assert torch.equal(_history(cs, r), hist[r])
    cs.check_device_errors()
    rs.conv_accept(cs, torch.tensor([9, -1, 0, 1, 2], dtype=torch.int32, device="cuda"), 8)
    with pytest.raises(rs.ReplaySSMError, match="n_keep"):
        cs.check_device_errors()


LENGTHS = [
    [0, 1, 2, 3, 0, 64, 33, 5, 32, 31, 1, 1, 0],   # none, single tokens, tile borders
    [300],
    [1],
    [0, 0, 7],
    [95, 1, 2, 1],
]


def _lens_case(lens, seed, extra_slots=2):
    g = _gen(seed)
    n = len(lens)
    slots = torch.randperm(n + extra_slots, generator=g)[:n].to(torch.int32)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    fresh = (torch.rand(n, generator=g) < 0.4).to(torch.int32)
    return g, n, slots, cu, fresh


@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("W,H,G,dtype", [(4, 6, 1, BF16), (3, 8, 2, F32), (2, 33, 1, BF16)])
def test_conv_packed_prompts(rs, lens, W, H, G, dtype):
    """Two packed calls in a row, some rows fresh, then single tokens on the same slots."""
    g, n, slots, cu, fresh = _lens_case(lens, 11)
    cs, w, b, db = _conv(rs, n + 2, H, G, W, dtype, seed=1)
    hist = [torch.zeros(W - 1, cs.channels, dtype=dtype) for _ in range(n)]
    sl = slots.cuda()
    for call in range(2):
        u, d, ug, dg = _rows(g, (sum(lens),), H, G, dtype, extra=call)
        fr = fresh if call else None
        got = rs.conv_prefill(cs, ug, dg, cu.cuda(), fresh=None if fr is None else fr.cuda(), slots=sl)
        for r in range(n):
            a, e = int(cu[r]), int(cu[r + 1])
            h0 = torch.zeros_like(hist[r]) if fr is not None and fr[r] and e > a else hist[r]
            out, err, hist[r] = ref.conv(h0, u[a:e], w, b)
            dv, de = ref.dt(d[a:e], db)
            _check_conv([x[a:e] for x in got], out, err, dv, de, dtype, H, G, f"call {call} row {r}")
            assert torch.equal(_history(cs, int(slots[r])), hist[r]), (call, r)
    u, d, ug, dg = _rows(g, (n,), H, G, dtype)
    got = rs.conv_step(cs, ug, dg, slots=sl)
    for r in range(n):
        out, err, hist[r] = ref.conv(hist[r], u[r:r + 1], w, b)
        dv, de = ref.dt(d[r:r + 1], db)
        _check_conv([x[r:r + 1] for x in got], out, err, dv, de, dtype, H, G, f"after, row {r}")
    cs.check_device_errors()
    assert int(cs.work.abs().sum()) == 0


def test_conv_pieces_equal_whole(rs):
    """A prompt in pieces (1, 2, 40, 3, ...) gives the whole prompt's outputs and history bit for bit."""
    H, G, W = 4, 1, 4
    a, *_ = _conv(rs, 1, H, G, W, BF16, seed=2)
    c, *_ = _conv(rs, 1, H, G, W, BF16, seed=2)
    _, _, u, d = _rows(_gen(3), (113,), H, G, BF16)
    cu = lambda k: torch.tensor([0, k], dtype=torch.int32, device="cuda")  # noqa: E731
    whole = rs.conv_prefill(a, u, d, cu(113))
    at, parts = 0, []
    for k in (1, 2, 40, 3, 1, 66):
        parts.append(rs.conv_prefill(c, u[at:at + k], d[at:at + k], cu(k)))
        at += k
    for i in range(4):
        assert torch.equal(whole[i], torch.cat([p[i] for p in parts]))
    assert torch.equal(_history(a, 0), _history(c, 0))


def test_conv_neighbours_do_not_leak(rs):
    """Infinities and NaN of one packed sequence or slot stay out of the others; tokens of no sequence are skipped."""
    H, G = 2, 1
    cs, w, b, db = _conv(rs, 3, H, G, 4, F32, seed=4)
    cs.ring[1] = float("nan")
    u, d, ug, dg = _rows(_gen(9), (24,), H, G, F32)
    ug, dg = ug.clone(), dg.clone()
    ug[8:16] = float("inf")
    dg[8:16] = float("nan")
    out = tuple(torch.full(s, 7.0, device="cuda") for s in ((24, H, 64), (24, G, 128), (24, G, 128), (24, H)))
    got = rs.conv_prefill(cs, ug, dg, torch.tensor([0, 8, 16, 20], dtype=torch.int32, device="cuda"), out=out)
    for r, (a, e) in enumerate([(0, 8), (16, 20)]):
        o, err, _ = ref.conv(torch.zeros(3, cs.channels), u[a:e], w, b)
        dv, de = ref.dt(d[a:e], db)
        _check_conv([x[a:e] for x in got], o, err, dv, de, F32, H, G, f"row {r}")
    assert all((x[20:] == 7).all() for x in got[:3])
    cs.check_device_errors()


def test_conv_bad_offsets_and_slots_are_flagged(rs):
    H, G = 2, 1
    cs, *_ = _conv(rs, 2, H, G, 4, F32, seed=4)
    _, _, u, d = _rows(_gen(9), (24,), H, G, F32)
    for cu in ([0, 30, 24], [-3, 5, 24], [0, 12, 25]):
        rs.conv_prefill(cs, u, d, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        with pytest.raises(rs.ReplaySSMError, match="offsets"):
            cs.check_device_errors()
        cs.work.zero_()
    rs.conv_step(cs, u[:2], d[:2], slots=torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    with pytest.raises(rs.ReplaySSMError, match="slot"):
        cs.check_device_errors()


def _layer(rs, slots, H, G, dtype, seed, state_format="f32"):
    g = _gen(seed)
    A = -torch.exp(torch.rand(H, generator=g) * math.log(16.0))
    D = torch.randn(H, generator=g)
    ls = rs.LayerState(slots, H, G, A, D, in_dtype=dtype, state_format=state_format, seed=5)
    S0 = 0.1 * torch.randn(slots, H, 64, 128, generator=g)
    rs.load_checkpoint(ls, S0.cuda())
    return ls, A, D, S0


def _scan_inputs(g, total, H, G, dtype):
    x = torch.randn(total, H, 64, generator=g).to(dtype)
    B = torch.randn(total, G, 128, generator=g).to(dtype)
    C = torch.randn(total, G, 128, generator=g).to(dtype)
    dt = torch.nn.functional.softplus(torch.randn(total, H, generator=g) - 2).to(dtype)
    return x, B, C, dt


def _check_scan(y, S, yr, Sr, ym, Sm, what):
    # The framework's bar for fp32 outputs and states, 2e-5 max(1, |ref|); the
    # terms behind a value are bounded by ym / Sm, which covers cancellation.
    tol = lambda r, m: 2e-5 * torch.maximum(torch.ones_like(r), r.abs()) + 64 * ref.U32 * m  # noqa: E731
    ty = tol(yr, ym)
    if y.dtype == BF16:   # one rounding of y; the weights of the terms may be rounded to bf16 as well
        ty = ty + ref.U16 * yr.abs() + ref.U16 * ym
    ref.assert_within(y, yr, ty, what + " y")
    ref.assert_within(S, Sr, tol(Sr, Sm), what + " state")


SCAN_LENGTHS = [[0, 1, 15, 16, 17, 0, 63, 64, 65], [200], [1], [129, 0, 3], [255, 256, 0, 257, 700], [1300]]


@pytest.mark.parametrize("lens", SCAN_LENGTHS)
@pytest.mark.parametrize("H,G,dtype,ydt", [(4, 2, F32, F32), (3, 1, BF16, F32), (4, 2, BF16, BF16), (2, 2, BF16, F32),
                                           (5, 1, F32, BF16), (9, 1, BF16, F32)])
def test_packed_prefill(rs, lens, H, G, dtype, ydt):
    g, n, slots, cu, fresh = _lens_case(lens, 21)
    ls, A, D, S0 = _layer(rs, n + 2, H, G, dtype, 31)
    x, B, C, dt = _scan_inputs(g, sum(lens), H, G, dtype)
    y = rs.prefill_packed(ls, x.cuda(), B.cuda(), C.cuda(), dt.cuda(), cu.cuda(), fresh=fresh.cuda(), y_dtype=ydt,
                          slots=slots.cuda())
    rs.check_device_errors(ls)
    untouched = set(range(n + 2))
    for r in range(n):
        a, e, s = int(cu[r]), int(cu[r + 1]), int(slots[r])
        if e == a:
            continue
        untouched.discard(s)
        start = torch.zeros_like(S0[s]) if fresh[r] else S0[s]
        yr, Sr, ym, Sm = ref.scan(start, x[a:e], B[a:e], C[a:e], dt[a:e], A, D)
        _check_scan(y[a:e], ls.ckpt[s], yr, Sr, ym, Sm, f"row {r} of {e - a}")
        assert int(ls.intv[s]) == 1 and int(ls.pos[s]) == 0
    for s in untouched:
        assert torch.equal(ls.ckpt[s].cpu(), S0[s]) and int(ls.intv[s]) == 0
    assert int(ls.work.abs().sum()) == 0


def test_packed_prefill_of_many_sequences(rs):
    """Sequences of no, whole and broken segments, more of them than are put in order together: each runs once."""
    g = _gen(61)
    lens = torch.randint(0, 30, (520,), generator=g).tolist()
    for at, n in ((3, 256), (100, 700), (255, 512), (256, 257), (400, 255), (519, 1030)):
        lens[at] = n
    H, G = 2, 1
    g, n, slots, cu, fresh = _lens_case(lens, 62)
    ls, A, D, S0 = _layer(rs, n + 2, H, G, BF16, 63)
    x, B, C, dt = _scan_inputs(g, sum(lens), H, G, BF16)
    y = rs.prefill_packed(ls, x.cuda(), B.cuda(), C.cuda(), dt.cuda(), cu.cuda(), fresh=fresh.cuda(), y_dtype=F32,
                          slots=slots.cuda())
    rs.check_device_errors(ls)
    used = torch.zeros(n + 2, dtype=torch.int64)
    used[slots.long()] = torch.tensor([int(v > 0) for v in lens])
    assert torch.equal(ls.intv.cpu().long(), used)
    for r in [3, 4, 99, 100, 101, 254, 255, 256, 257, 399, 400, 401, 518, 519]:
        a, e, s = int(cu[r]), int(cu[r + 1]), int(slots[r])
        if e == a:
            continue
        start = torch.zeros_like(S0[s]) if fresh[r] else S0[s]
        yr, Sr, ym, Sm = ref.scan(start, x[a:e], B[a:e], C[a:e], dt[a:e], A, D)
        _check_scan(y[a:e], ls.ckpt[s], yr, Sr, ym, Sm, f"row {r} of {e - a}")


@pytest.mark.parametrize("fmt", ["split-bf16", "split-e4m3", "shared-fp4", "low-bf16", "low-e4m3"])
def test_packed_prefill_low_precision_states(rs, fmt):
    """Each row equals the row's own replayssm_prefill bit for bit: outputs and stored bytes."""
    lens, H, G = [5, 0, 40], 4, 2
    g, n, slots, cu, _ = _lens_case(lens, 23)
    a, *_ = _layer(rs, n + 2, H, G, BF16, 33, fmt)
    b, *_ = _layer(rs, n + 2, H, G, BF16, 33, fmt)
    ins = [t.cuda() for t in _scan_inputs(g, sum(lens), H, G, BF16)]
    y = rs.prefill_packed(a, *ins, cu.cuda(), slots=slots.cuda())
    for r in range(n):
        lo, hi = int(cu[r]), int(cu[r + 1])
        if lo == hi:
            continue
        yr = rs.prefill(b, *(t[lo:hi][None].contiguous() for t in ins), slots=slots[r:r + 1].cuda())
        assert torch.equal(y[lo:hi], yr[0])
    for k, v in b.tensors().items():
        assert torch.equal(a.tensors()[k], v), k


def test_packed_prefill_states_only_and_errors(rs):
    lens, H, G = [30, 70], 4, 1
    g, n, slots, cu, _ = _lens_case(lens, 25, 0)
    ls, A, D, S0 = _layer(rs, 2, H, G, BF16, 35)
    x, B, C, dt = (t.cuda() for t in _scan_inputs(g, 100, H, G, BF16))
    assert rs.prefill_packed(ls, x, B, None, dt, cu.cuda(), from_zero=True, outputs=False) is None
    for r in range(2):
        a, e = int(cu[r]), int(cu[r + 1])
        _, Sr, _, Sm = ref.scan(torch.zeros_like(S0[r]), *(t[a:e].cpu() for t in (x, B, C, dt)), A, D)
        ref.assert_within(ls.ckpt[r], Sr, 2e-5 * torch.maximum(torch.ones_like(Sr), Sr.abs()) + 64 * ref.U32 * Sm,
                          "state")
    rs.check_device_errors(ls)
    snap = ls.snapshot()
    for bad in ([0, 120, 100], [-1, 30, 100], [0, 30, 101]):
        ls.restore(snap)
        rs.prefill_packed(ls, x, B, C, dt, torch.tensor(bad, dtype=torch.int32, device="cuda"))
        with pytest.raises(rs.ReplaySSMError, match="offsets"):
            rs.check_device_errors(ls)


@pytest.mark.parametrize("rows,dim,groups,yt,zt,before", [
    (5, 512, 1, F32, BF16, False), (3, 6144, 8, F32, BF16, False), (2, 8192, 8, BF16, BF16, True),
    (1, 4096, 1, F32, F32, False), (7, 1000, 8, BF16, BF16, False), (4, 15, 5, F32, BF16, True),
    (2, 10001, 1, F32, F32, True), (3, 2001, 1, BF16, F32, False), (1, 16384, 1, F32, BF16, False),
    (3, 5000, 1, BF16, BF16, False), (130, 64, 1, F32, BF16, False),
])
def test_gated_norm(rs, rows, dim, groups, yt, zt, before):
    g = _gen(dim)
    y = (3 * torch.randn(rows, dim, generator=g)).to(yt)
    zr = torch.randn(rows, dim + 7, generator=g).to(zt)
    z = zr[:, 5:5 + dim]
    w = 1 + 0.1 * torch.randn(dim, generator=g)
    if rows > 2:
        y[1] = 0            # a row of zeros: 0 rsqrt(eps)
        zr[2, :] = -100.0   # a gate that shuts
    got = rs.gated_norm(y.cuda(), zr.cuda()[:, 5:5 + dim], w.cuda(), groups=groups, eps=1e-5, norm_before_gate=before)
    assert got.dtype == zt
    want = ref.gated_norm(y, z, w, groups, 1e-5, before)
    # gate: exp of a rounded argument, sum, reciprocal, product ((2|z| + 10) half steps), once in the value and once
    # (halved by the root) in the norm; a sum of n squares in blocks of 8 a lane and a tree: 8 NV + 14 half steps,
    # halved by the root; root, weight and products.
    zmax = float(z.double().abs().max())
    rel = ref.U32 * (2 * (2 * zmax + 10) + 32)
    u = ref.half_step(zt) if zt != F32 else 0.0
    ref.assert_within(got, want, (rel + u) * want.abs() + 1e-30, "gated norm")


@pytest.mark.parametrize("rows,dim,xt,rt,post,inplace", [
    (1, 4096, BF16, F32, False, False), (3, 2560, BF16, BF16, True, True), (5, 1, F32, F32, True, False),
    (4, 7, F32, BF16, False, True), (2, 5001, BF16, F32, True, False), (2, 16384, F32, F32, True, True),
    (300, 64, BF16, BF16, False, False), (9, 513, F32, F32, False, False), (2, 8192, BF16, BF16, True, False),
])
def test_add_norm(rs, rows, dim, xt, rt, post, inplace):
    g = _gen(dim + 1)
    x = torch.randn(rows, dim, generator=g).to(xt)
    r = (2 * torch.randn(rows, dim, generator=g)).to(rt)
    w, p = 1 + 0.1 * torch.randn(dim, generator=g), 0.5 + 0.1 * torch.randn(dim, generator=g)
    if rows > 2:
        x[1], r[1] = 0, 0
    rg = r.cuda()
    keep = rg.clone()
    out, res = rs.add_norm(x.cuda(), rg, w.cuda(), scale=0.22, post_weight=p.cuda() if post else None, eps=1e-6,
                           residual_out=rg if inplace else None)
    assert (res.data_ptr() == rg.data_ptr()) == inplace and (inplace or torch.equal(rg, keep))
    assert out.dtype == xt and res.dtype == rt
    want, rw = ref.add_norm(x, r, w, 0.22, p if post else None, 1e-6)
    # 0.22 itself is rounded to fp32; f(x) with a norm: sum of squares, root, two products; then the sum
    f = rw - r.double()
    rerr = ref.U32 * (rw.abs() + (28 if post else 3) * f.abs())
    u = ref.half_step(rt) if rt != F32 else 0.0
    ref.assert_within(res, rw, rerr * (1 + u) + u * rw.abs() + 1e-37, "residual")
    # the error of r, scaled as r is, moves the norm by at most its own relative size
    inv = 1 / (rw.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    rel_norm = (rerr.pow(2).mean(-1, keepdim=True) + 0).sqrt() * inv
    u = ref.half_step(xt) if xt != F32 else 0.0
    tol = rerr * inv * w.double().abs() + want.abs() * (rel_norm + 28 * ref.U32 + u)
    ref.assert_within(out, want, tol + 1e-30, "normed")


def test_no_rows_is_a_no_op(rs):
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    assert rs.gated_norm(e, e, w).shape == (0, 64)
    assert rs.add_norm(e, e, w)[0].shape == (0, 64)
    cs, *_ = _conv(rs, 3, 2, 1, 4, F32)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    got = rs.conv_step(cs, torch.empty(0, cs.channels, device="cuda"), torch.empty(0, 2, device="cuda"), slots=none)
    assert got[0].shape == (0, 2, 64)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = rs.conv_prefill(cs, torch.empty(0, cs.channels, device="cuda"), torch.empty(0, 2, device="cuda"), cu)
    assert got[1].shape == (0, 1, 128)
    ls, A, D, S0 = _layer(rs, 3, 2, 1, F32, 3)
    y = rs.prefill_packed(ls, torch.empty(0, 2, 64, device="cuda"), torch.empty(0, 1, 128, device="cuda"),
                          torch.empty(0, 1, 128, device="cuda"), torch.empty(0, 2, device="cuda"), cu)
    assert y.shape == (0, 2, 64) and torch.equal(ls.ckpt.cpu(), S0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
def test_packed_prefill_non_finite_inputs_stay_behind(rs, dtype, what):
    """A non-finite value of a token reaches no earlier token of its sequence and no other sequence; a NaN in x stays
    in its head's row of the state, and a C only in its own token."""
    lens, H, G, bad = [70, 200, 64], 5, 1, 101      # token `bad` of the middle sequence, inside its second chunk
    g, n, slots, cu, _ = _lens_case(lens, 27, 0)
    ls, A, D, S0 = _layer(rs, n, H, G, dtype, 37)
    ins = dict(zip(("x", "B", "C", "dt"), _scan_inputs(g, sum(lens), H, G, dtype)))
    spoilt = {k: v.clone() for k, v in ins.items()}
    at = 70 + bad
    if what == "x":
        spoilt["x"][at, 2, 37] = float("nan")
        spoilt["x"][at + 3, 2, 5] = float("inf")
    else:
        spoilt[what][at] = float("nan")
    y = rs.prefill_packed(ls, *(spoilt[k].cuda() for k in ("x", "B", "C", "dt")), cu.cuda(), slots=slots.cuda())
    rs.check_device_errors(ls)
    for r in range(n):
        a, e, s = int(cu[r]), int(cu[r + 1]), int(slots[r])
        yr, Sr, ym, Sm = ref.scan(S0[s], *(ins[k][a:e] for k in ("x", "B", "C", "dt")), A, D)
        S = ls.ckpt[s]
        if r != 1:
            _check_scan(y[a:e], S, yr, Sr, ym, Sm, f"row {r}")
            continue
        _check_scan(y[a:at], torch.zeros_like(S), yr[:bad], torch.zeros_like(Sr), ym[:bad], Sm, "before")
        rest = y[at:e].float().cpu()
        if what == "x":
            rows = torch.ones(H, 64, dtype=torch.bool)
            rows[2, 37] = rows[2, 5] = False
            ok = rows[None].expand(e - at, -1, -1)
            tol = 2e-5 * yr[bad:].abs().clamp(min=1) + 64 * ref.U32 * ym[bad:]
            assert ((rest.double() - yr[bad:]).abs()[ok] <= tol[ok]).all()
            assert not torch.isfinite(rest[:, 2, 37]).any() and not torch.isfinite(rest[3:, 2, 5]).any()
            assert torch.isfinite(rest[:3, 2, 5]).all()
            Sg = S.cpu()
            assert torch.isfinite(Sg[rows]).all() and not torch.isfinite(Sg[2, 37]).any()
        elif what == "C":
            assert torch.isnan(rest[0]).all() and torch.isfinite(rest[1:]).all()
            ref.assert_within(S, Sr, 2e-5 * Sr.abs().clamp(min=1) + 64 * ref.U32 * Sm, "state")
        else:
            assert torch.isnan(rest).all()
            assert torch.isnan(S).all()


def test_packed_prefill_with_and_without_workspace(rs):
    """Pieces run side by side and sequences run end to end agree to rounding."""
    from state_space_recurrence_amd import mixer
    import ctypes
    lens, H, G = [1500, 3, 900], 4, 1
    g, n, slots, cu, _ = _lens_case(lens, 29, 0)
    ins = [t.cuda() for t in _scan_inputs(g, sum(lens), H, G, BF16)]
    ins[3] = (ins[3].float() * 0.02).to(BF16)          # slow decays: earlier pieces reach into later ones
    a, *_ = _layer(rs, n, H, G, BF16, 39)
    b, *_ = _layer(rs, n, H, G, BF16, 39)
    ya = rs.prefill_packed(a, *ins, cu.cuda())
    d, st, _ = rs._ctx(b, None)
    L = mixer._lib()
    assert L.replayssm_prefill_packed_workspace(ctypes.addressof(d), sum(lens)) > 0
    yb = torch.empty_like(ya)
    x, B, C, dt = ins
    c = cu.cuda()
    rc = L.replayssm_prefill_packed(ctypes.addressof(d), ctypes.addressof(st), sum(lens), c.data_ptr(), 0, None,
                                    x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr(), yb.data_ptr(), 0, None, 0,
                                    torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    f = lambda u, v: float((u.double() - v.double()).norm() / v.double().norm())  # noqa: E731
    assert f(ya, yb) < 2e-6 and f(a.ckpt, b.ckpt) < 2e-6


def _decode_layer(rs, B, H, G, seed):
    cs, *_ = _conv(rs, B, H, G, 4, BF16, seed=seed)
    ls, *_ = _layer(rs, B, H, G, BF16, seed)
    return cs, ls


def _decode(rs, cs, ls, rows, res, w1, w2, H, G, outs):
    """One token through a layer: views of the projection's rows in, normed residual out."""
    Cc = cs.channels
    u, dt = rows[:, 64 * H:64 * H + Cc], rows[:, 64 * H + Cc:]
    x, B, C, d = rs.conv_step(cs, u, dt, out=outs["conv"])
    y = rs.step(ls, x, B, C, d, y=outs["y"])
    o = rs.gated_norm(y, rows[:, :64 * H], w1, groups=G, out=outs["o"])
    return rs.add_norm(o, res, w2, scale=0.5, out=outs["n"], residual_out=res)


def test_decode_token_in_a_graph(rs):
    """A captured layer token replayed 20 times (over a commit), eager work on another layer between the replays,
    equals eager tokens bit for bit."""
    B, H, G = 5, 6, 2
    g = _gen(41)
    w1, w2 = torch.rand(64 * H, generator=g).cuda(), torch.rand(64 * H, generator=g).cuda()
    toks = torch.randn(20, B, 64 * H + 64 * H + 256 * G + H, generator=g).to(BF16).cuda()

    def bufs():
        e = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        return {"conv": (e(B, H, 64), e(B, G, 128), e(B, G, 128), e(B, H)), "y": e(B, H, 64, dt=F32),
                "o": e(B, 64 * H), "n": e(B, 64 * H)}

    cs, ls = _decode_layer(rs, B, H, G, 51)
    cg, lg = _decode_layer(rs, B, H, G, 51)
    oe, og = bufs(), bufs()
    re_, rg = (torch.zeros(B, 64 * H, device="cuda") for _ in range(2))
    static = torch.zeros_like(toks[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm_c, warm_l = _decode_layer(rs, B, H, G, 52)
        _decode(rs, warm_c, warm_l, static, torch.zeros_like(rg), w1, w2, H, G, bufs())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _decode(rs, cg, lg, static, rg, w1, w2, H, G, og)
    for t in range(20):
        _decode(rs, cs, ls, toks[t], re_, w1, w2, H, G, oe)
        static.copy_(toks[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(og["n"], oe["n"]) and torch.equal(rg, re_), t
    for k, v in {**ls.tensors(), **cs.tensors()}.items():
        assert torch.equal(v, {**lg.tensors(), **cg.tensors()}[k]), k


def test_calls_on_another_stream(rs):
    """Outputs allocated by a call on a side stream hold its results once that stream is waited for."""
    H, G = 4, 1
    g = _gen(61)
    _, _, u, d = _rows(g, (200,), H, G, BF16)
    z = torch.randn(200, 64 * H, generator=g).to(BF16).cuda()
    w = torch.rand(64 * H, generator=g).cuda()
    cu = torch.tensor([0, 90, 200], dtype=torch.int32, device="cuda")

    def run(stream):
        cs, *_ = _conv(rs, 2, H, G, 4, BF16, seed=6)
        ls, *_ = _layer(rs, 2, H, G, BF16, 7)
        torch.cuda.synchronize()
        x, B, C, dt = rs.conv_prefill(cs, u, d, cu, stream=stream)
        y = rs.prefill_packed(ls, x, B, C, dt, cu, stream=stream)
        o = rs.gated_norm(y, z, w, groups=G, stream=stream)
        n, r = rs.add_norm(o, z, w, stream=stream)
        torch.cuda.synchronize()
        return x, y, o, n, r, ls.ckpt, cs.ring

    for a, b in zip(run(None), run(torch.cuda.Stream())):
        assert torch.equal(a, b)


def test_example_stack(rs):
    """The example: prompts at once, tokens and drafts against the same tokens one by one.  Every bf16 activation
    between the parts may round the other way (2^-8 each; about ten of them in two blocks, growing with the square
    root), outputs of both ways being right to fp32 before that."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixer_block.py")
    spec = importlib.util.spec_from_file_location("mixer_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(verbose=False) < 10 ** 0.5 * ref.U16
    assert m.main(lengths=(300, 64, 2), tokens=3, seed=1, verbose=False) < 10 ** 0.5 * ref.U16
