"""Packed prefill in the settings of a server: captured graphs, several
streams, and inputs at which the pieces of a long sequence meet."""
import ctypes

import pytest
import torch

import mixer_ref as ref
from state_space_recurrence_amd import mixer
from test_gpu_mixer import BF16, F32, _check_scan, _gen, _layer, _lens_case, _scan_inputs, rs  # noqa: F401

pytestmark = pytest.mark.gpu


def _slow(ins):
    """Slow decays, so that earlier pieces of a sequence reach into later ones."""
    ins[3] = (ins[3].float() * 0.02).to(ins[3].dtype)
    return ins


def test_captured_prefill_beside_larger_eager_calls(rs):  # noqa: F811
    """A prefill captured after an eager one of its size, then a larger eager one on the same layer and tensors that
    may take any memory freed since: every replay gives the eager result bit for bit and writes nothing else."""
    lens, H, G = [1500, 3, 900], 4, 1
    g, n, slots, cu, _ = _lens_case(lens, 71, 0)
    cu = cu.cuda()
    ins = _slow([t.cuda() for t in _scan_inputs(g, sum(lens), H, G, BF16)])
    ls, *_ = _layer(rs, n, H, G, BF16, 73)
    start = ls.snapshot()
    want = rs.prefill_packed(ls, *ins, cu)
    after = ls.snapshot()
    y = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rs.prefill_packed(ls, *ins, cu, y=y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rs.prefill_packed(ls, *ins, cu, y=y)
    big = [3000, 700, 4100]
    more = _slow([t.cuda() for t in _scan_inputs(g, sum(big), H, G, BF16)])
    rs.prefill_packed(ls, *more, torch.tensor([0, *big]).cumsum(0).to(torch.int32).cuda())
    torch.cuda.synchronize()
    guards = [torch.full((k,), 7.0, device="cuda") for k in (1 << 10, 1 << 14, 1 << 17, 1 << 18, 1 << 19, 1 << 20) * 4]
    for i in range(5):
        ls.restore(start)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        for k, v in after.items():
            assert torch.equal(ls.tensors()[k], v), (i, k)
        rs.prefill_packed(ls, *more, torch.tensor([0, *big]).cumsum(0).to(torch.int32).cuda())
        assert all(bool((t == 7).all()) for t in guards), i
    rs.check_device_errors(ls)


def test_prefills_of_one_layer_on_two_streams(rs):  # noqa: F811
    """Calls that overlap on disjoint slots of a layer give what they give one after the other."""
    H, G, halves = 4, 1, ([2000, 1100], [900, 2500])
    g = _gen(81)
    jobs = []
    for lens, slots in zip(halves, ([0, 3], [2, 1])):
        ins = _slow([t.cuda() for t in _scan_inputs(g, sum(lens), H, G, BF16)])
        jobs.append((ins, torch.tensor([0, *lens]).cumsum(0).to(torch.int32).cuda(),
                     torch.tensor(slots, dtype=torch.int32, device="cuda")))
    one, *_ = _layer(rs, 4, H, G, BF16, 83)
    two, *_ = _layer(rs, 4, H, G, BF16, 83)
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for i in range(4):
        want = [rs.prefill_packed(one, *ins, cu, slots=sl) for ins, cu, sl in jobs]
        got = [rs.prefill_packed(two, *ins, cu, slots=sl, stream=s) for (ins, cu, sl), s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        assert torch.equal(one.ckpt, two.ckpt), i
    rs.check_device_errors(two)


def _whole(rs, ls, x, B, C, dt, cu, y):  # noqa: F811
    """The packed call without scratch: every sequence in one piece."""
    d, st, _ = rs._ctx(ls, None)
    rc = mixer._lib().replayssm_prefill_packed(
        ctypes.addressof(d), ctypes.addressof(st), x.shape[0], cu.data_ptr(), 0, None, x.data_ptr(), B.data_ptr(),
        C.data_ptr(), dt.data_ptr(), y.data_ptr(), 1 if y.dtype == BF16 else 0, None, 0,
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0


@pytest.mark.parametrize("what", ["x", "B", "C", "dt", "start"])
@pytest.mark.parametrize("dtype,ydt,lens", [(BF16, BF16, [4000]), (F32, F32, [2100]), (BF16, F32, [900, 5, 1500, 64])])
def test_non_finite_values_cross_the_pieces(rs, dtype, ydt, lens, what):  # noqa: F811
    """A NaN stays in the state and in all later outputs of its sequence however many pieces the sequence is cut into
    and however fast the state decays: the same elements as when each sequence runs in one piece, which is what the
    recurrence makes of them (0 NaN is NaN)."""
    H, G, q = 9, 1, 0 if len(lens) == 1 else 2
    g, n, _, cu, _ = _lens_case(lens, 91, 0)
    x, B, C, dt = _scan_inputs(g, sum(lens), H, G, dtype)
    a, A, D, S0 = _layer(rs, n, H, G, dtype, 93)
    b, *_ = _layer(rs, n, H, G, dtype, 93)
    at, end = int(cu[q]) + 33, int(cu[q + 1])
    state, rows = torch.zeros(H, 64, 128, dtype=torch.bool), torch.zeros(H, 64, dtype=torch.bool)   # which are NaN
    if what == "x":
        x[at, 2, 37] = float("nan")
        x[at, 8, 0] = float("nan")
        rows[2, 37] = rows[8, 0] = True
        state |= rows[..., None]
    elif what == "B":
        B[at, 0, 100] = float("nan")
        state[:, :, 100] = True
        rows[:] = True
    elif what == "C":
        C[at] = float("nan")
    elif what == "dt":
        dt[at, 4] = float("nan")
        state[4] = rows[4] = True
    else:
        for ls in (a, b):
            ls.ckpt[q, 5, 40, 7] = float("nan")
        state[5, 40, 7] = rows[5, 40] = True
        at = int(cu[q])
    ins, cug = [t.cuda() for t in (x, B, C, dt)], cu.cuda()
    assert mixer._lib().replayssm_prefill_packed_workspace(ctypes.addressof(rs._ctx(a, None)[0]), sum(lens)) > 0
    y = rs.prefill_packed(a, *ins, cug, y_dtype=ydt)
    yw = torch.empty_like(y)
    _whole(rs, b, *ins, cug, yw)
    rs.check_device_errors(a)
    nan_y = torch.zeros(sum(lens), H, 64, dtype=torch.bool)
    nan_y[at:end] = rows
    if what == "C":
        nan_y[at] = True
    nan_S = torch.zeros(n, H, 64, 128, dtype=torch.bool)
    nan_S[q] = state
    for way, got_y, got_S in (("whole", yw, b.ckpt), ("in pieces", y, a.ckpt)):
        assert torch.equal(torch.isnan(got_S).cpu(), nan_S), way
        assert torch.equal(torch.isnan(got_y).cpu(), nan_y), way
    # what is finite is right
    near = lambda u, v, t: float((u - v).nan_to_num().norm() / v.nan_to_num().norm()) < t  # noqa: E731
    assert near(a.ckpt, b.ckpt, 2e-6) and near(y.float(), yw.float(), 2e-6 if ydt == F32 else ref.U16)
    a.ckpt.zero_()
    rs.prefill_packed(a, ins[0], ins[1], None, ins[3], cug, outputs=False)
    if what != "start":
        assert torch.equal(torch.isnan(a.ckpt).cpu(), nan_S)


@pytest.mark.parametrize("dtype,ydt", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_decays_past_the_range_of_whole_numbers(rs, dtype, ydt):  # noqa: F811
    """dt so large that a chunk's sum of decays passes 2^31 powers of two: such tokens forget what came before them."""
    H, G, T = 4, 2, 150
    ls, A, D, S0 = _layer(rs, 1, H, G, dtype, 97)
    x, B, C, dt = _scan_inputs(_gen(98), T, H, G, dtype)
    dt[20:24] = 1e9
    dt[70:90:3] = 2e9
    dt[100] = 1e4
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    y = rs.prefill_packed(ls, x.cuda(), B.cuda(), C.cuda(), dt.cuda(), cu, y_dtype=ydt)
    yr, Sr, ym, Sm = ref.scan(S0[0], x, B, C, dt, A, D)
    _check_scan(y, ls.ckpt[0], yr, Sr, ym, Sm, "large dt")


@pytest.mark.parametrize("H,G,dtype", [(16, 2, BF16), (10, 2, BF16), (4, 1, BF16), (3, 1, BF16), (4, 2, BF16),
                                       (2, 2, BF16), (6, 2, F32), (2, 2, F32)])
def test_bf16_outputs_carry_16_bits_before_their_rounding(rs, H, G, dtype):  # noqa: F811
    """Several groups, several workgroups a group and heads that fill none, sequences whole and in pieces.

    Of the values formed in fp32 (M, the state) two bf16 parts are taken: each part is off by half a step, 2^-8 of
    what is left, so 2^-16 of the value.  bf16 inputs are exact operands; all sums are fp32, in about 100 roundings of
    2^-24 of the terms' sizes at most (products of a chunk, its Gram tile, the state over the chunks), less than
    2^-17.  fp32 inputs are taken in two parts as well, and of a product of two pairs the last one is left out: three
    times 2^-16 for C B or S C, as much again for M x.  Then one rounding."""
    lens = [700, 65, 0, 1300, 1]
    g, n, slots, cu, fresh = _lens_case(lens, 101)
    ls, A, D, S0 = _layer(rs, n + 2, H, G, dtype, 103)
    x, B, C, dt = _scan_inputs(g, sum(lens), H, G, dtype)
    y = rs.prefill_packed(ls, x.cuda(), B.cuda(), C.cuda(), dt.cuda(), cu.cuda(), fresh=fresh.cuda(), y_dtype=BF16,
                          slots=slots.cuda())
    rs.check_device_errors(ls)
    parts = (2 if dtype == BF16 else 7) * 2.0 ** -16
    for r in range(n):
        a, e, s = int(cu[r]), int(cu[r + 1]), int(slots[r])
        if e == a:
            continue
        start = torch.zeros_like(S0[s]) if fresh[r] else S0[s]
        yr, Sr, ym, Sm = ref.scan(start, x[a:e], B[a:e], C[a:e], dt[a:e], A, D)
        ref.assert_within(y[a:e], yr, ref.U16 * yr.abs() + (1 + ref.U16) * parts * ym + 1e-30, f"row {r} of {e - a} y")
        _check_scan(torch.zeros(0, H, 64), ls.ckpt[s], yr[:0], Sr, ym[:0], Sm, f"row {r} of {e - a}")


@pytest.mark.parametrize("fmt", ["split-bf16", "split-e4m3", "shared-fp4", "low-bf16", "low-e4m3"])
@pytest.mark.parametrize("dtype,ydt", [(F32, F32), (F32, BF16), (BF16, BF16)])
def test_low_precision_states_over_types_and_fresh_rows(rs, fmt, dtype, ydt):  # noqa: F811
    """Each row equals the row's own replayssm_prefill bit for bit (bf16 outputs: its outputs rounded once)."""
    lens, H, G = [200, 1, 0, 67], 6, 2
    g, n, slots, cu, fresh = _lens_case(lens, 107)
    fresh[0], fresh[3] = 0, 1
    a, *_ = _layer(rs, n + 2, H, G, dtype, 109, fmt)
    b, *_ = _layer(rs, n + 2, H, G, dtype, 109, fmt)
    ins = [t.cuda() for t in _scan_inputs(g, sum(lens), H, G, dtype)]
    y = rs.prefill_packed(a, *ins, cu.cuda(), fresh=fresh.cuda(), y_dtype=ydt, slots=slots.cuda())
    for r in range(n):
        lo, hi = int(cu[r]), int(cu[r + 1])
        if lo == hi:
            continue
        yr = rs.prefill(b, *(t[lo:hi][None].contiguous() for t in ins), from_zero=bool(fresh[r]),
                        slots=slots[r:r + 1].cuda())
        assert torch.equal(y[lo:hi], yr[0].to(ydt)), r
    for k, v in b.tensors().items():
        assert torch.equal(a.tensors()[k], v), k
    rs.check_device_errors(a)
