"""Rows of any alignment: products of bf16 rows that start or end at any element, and of MX rows whose scales start at
any byte, over several tiles, steps and output types."""
import math

import pytest
import torch

import linear_ref as ref
import mixer_ref
from test_gpu_linear import BF16, F32, MX, _check, _cuda, _operands, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rs():
    import state_space_recurrence_amd as rs
    return rs


def _moved(t, by):
    """The same bytes `by` elements behind a multiple of 16 bytes."""
    buf = torch.zeros(t.numel() + by, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device=t.device)
    v = t.view(torch.uint8) if t.element_size() == 1 else t
    buf[by:].copy_(v.flatten())
    return buf[by:].view(v.shape).view(t.dtype)


# rows x outputs x inputs: one and several tiles of 64 in both directions, whole and partial ones; steps of 64 inputs
# (bf16), one to many, and every kind of end within 16 bytes
SIZES = [(130, 224, 1001), (65, 257, 4095), (700, 96, 515), (64, 64, 63), (128, 128, 127), (1, 320, 2049), (200, 1000, 66),
         (63, 65, 130), (129, 192, 1023), (300, 40, 4), (257, 33, 1)]


@pytest.mark.parametrize("rows,n_out,n_in", SIZES)
@pytest.mark.parametrize("out_type,act,res_type", [(BF16, None, None), (F32, "silu", BF16), (MX, "gelu", F32)])
def test_bf16_rows_of_any_length(rs, rows, n_out, n_in, out_type, act, res_type):
    n_out += -n_out % 32 if out_type == MX else 0
    _check(rs, BF16, rows, n_out, n_in, out_type, True, act, res_type, 0.5, seed=41)


@pytest.mark.parametrize("by_x,by_w", [(1, 0), (0, 1), (3, 5), (4, 2), (7, 7)])
@pytest.mark.parametrize("rows,n_out,n_in", [(130, 224, 256), (66, 100, 320), (700, 96, 72)])
def test_bf16_rows_from_any_element(rs, by_x, by_w, rows, n_out, n_in):
    """Rows that would be aligned but for where they start."""
    x, w, xv, wv = _operands(BF16, rows, n_out, n_in, 42)
    want, err = ref.linear(xv, wv, None, None, None, 1.0)
    got = rs.linear(_moved(x.cuda(), by_x), _moved(w.cuda(), by_w), out_dtype=F32)
    mixer_ref.assert_within(got, want, err, f"{by_x}, {by_w} elements behind")


MX_SIZES = [(70, 96, 160), (130, 224, 1056), (200, 64, 2080), (65, 128, 4096), (300, 352, 96), (1, 64, 416), (64, 64, 32)]


@pytest.mark.parametrize("rows,n_out,n_in", MX_SIZES)
@pytest.mark.parametrize("by_x,by_w", [(1, 0), (0, 2), (3, 1), (2, 3)])
@pytest.mark.parametrize("out_type", [BF16, F32, MX])
def test_scales_from_any_byte(rs, rows, n_out, n_in, by_x, by_w, out_type):
    x, w, xv, wv = _operands(MX, rows, n_out, n_in, 43)
    want, err = ref.linear(xv, wv, None, None, None, 1.0)
    (xc, xs), (wc, ws) = _cuda(x), _cuda(w)
    got = rs.linear((xc, _moved(xs, by_x)), (wc, _moved(ws, by_w)), out_dtype=ref.E4M3 if out_type == MX else out_type)
    if out_type == MX:
        ref.assert_mx(got, want, err, "mx output")
    else:
        u = ref.half_step(BF16) if out_type == BF16 else 0.0
        mixer_ref.assert_within(got, want, err * (1 + u) + u * want.abs(), "scales")


SHAPES = [(BF16, 130, 96, 1001), (BF16, 70, 257, 67), (MX, 130, 96, 1056), (MX, 70, 257, 160)]


def _at(x_type, x, w):
    """MX rows with scales of both sides between multiples of 4 bytes (bf16 rows are unaligned by their length)."""
    x, w = _cuda(x), _cuda(w)
    return ((x[0], _moved(x[1], 1)), (w[0], _moved(w[1], 3))) if x_type == MX else (x, w)


@pytest.mark.parametrize("x_type,rows,n_out,n_in", SHAPES)
def test_nothing_around_is_written_or_read(rs, x_type, rows, n_out, n_in):
    x, w, xv, wv = _operands(x_type, rows, n_out, n_in, 44)
    want, err = ref.linear(xv, wv, None, None, None, 1.0)
    x, w = _at(x_type, x, w)
    if x_type == BF16:
        wide = torch.full((rows + 2, n_in + 64), math.nan, dtype=BF16, device="cuda")
        wide[1:-1, 3:3 + n_in] = x
        x = wide[1:-1, 3:3 + n_in]
    buf = torch.full((rows + 4, n_out), 7.0, dtype=F32, device="cuda")
    rs.linear(x, w, out=buf[2:-2])
    assert bool((buf[:2] == 7).all()) and bool((buf[-2:] == 7).all())
    mixer_ref.assert_within(buf[2:-2], want, err, "inside")


@pytest.mark.parametrize("x_type,rows,n_out,n_in", SHAPES)
def test_rows_that_are_not_finite(rs, x_type, rows, n_out, n_in):
    x, w, _, _ = _operands(x_type, rows, n_out, n_in, 45)
    clean = rs.linear(*_at(x_type, x, w), out_dtype=F32)
    if x_type == MX:
        x[0].view(torch.uint8)[1, n_in - 1] = 0x7F
        x[1].view(torch.uint8)[rows - 1, -1] = 255
        w[1].view(torch.uint8)[5, 0] = 255
    else:
        x[1, n_in - 1], x[rows - 1, 0], w[5, n_in - 1] = math.nan, math.inf, math.nan
    got = rs.linear(*_at(x_type, x, w), out_dtype=F32)
    assert bool(torch.isnan(got[1]).all()) and not bool(torch.isfinite(got[-1]).any()) and bool(torch.isnan(got[:, 5]).all())
    got[1], got[-1], got[:, 5] = clean[1], clean[-1], clean[:, 5]
    assert _same(got, clean)
