"""How MX operands are multiplied: exactly unless the caller asks for the fast
products, whatever the output's type, the tile and the address; and how far
both are off, over all outputs as well as at each."""
import math

import pytest
import torch

import linear_ref as ref
import mixer_ref
from test_gpu_linear import BF16, F32, MX, _cuda, _operands, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rs():
    import state_space_recurrence_amd as rs
    return rs


def _out(t):
    return ref.E4M3 if t == MX else t


# Rows and outputs of every tile, the smallest first
TILES = [(3, 100), (5, 64), (200, 544), (20, 4096), (33, 4128), (65, 9024), (200, 9024), (700, 9024), (3000, 4128)]


def _cancelling(rows, n_out, n_in):
    """Codes with scales of 1: among any 16 consecutive inputs the products 2^16 and -2^16 side by side, all others
    whole numbers up to 9.  Every partial sum is a whole number below 2^24, so fp32 sums are exact in any order."""
    g = torch.Generator()
    g.manual_seed(rows + n_out + n_in)
    x = torch.randint(1, 4, (rows, n_in), generator=g).float()
    w = torch.randint(-3, 4, (n_out, n_in), generator=g).float()
    at = torch.arange(0, n_in, 16) + 2 * torch.randint(0, 8, (n_in // 16,), generator=g)
    x[:, at] = x[:, at + 1] = 256.0
    w[:, at], w[:, at + 1] = 256.0, -256.0
    ones = lambda n: torch.full((n, n_in // 32), 127, dtype=torch.uint8).view(ref.E8M0)  # noqa: E731
    return x, w, (x.to(ref.E4M3), ones(rows)), (w.to(ref.E4M3), ones(n_out))


def _moved(pair, by):
    """The same pair with its scales `by` bytes behind a multiple of 4."""
    s = pair[1].view(torch.uint8)
    buf = torch.zeros(s.numel() + by, dtype=torch.uint8, device=s.device)
    buf[by:].copy_(s.flatten())
    return pair[0], buf[by:].view(s.shape).view(ref.E8M0)


@pytest.mark.parametrize("rows,n_out", TILES)
@pytest.mark.parametrize("n_in", [512, 160])
@pytest.mark.parametrize("out_type", [BF16, F32, MX])
@pytest.mark.parametrize("by", [0, 1])
def test_large_products_that_cancel(rs, rows, n_out, n_in, out_type, by):
    if out_type == MX and n_out % 32:
        n_out += 32 - n_out % 32
    xv, wv, x, w = _cancelling(rows, n_out, n_in)
    want = (xv.cuda().double() @ wv.cuda().double().t()).cpu()
    got = rs.linear(_moved(_cuda(x), by), _cuda(w), out_dtype=_out(out_type))
    if out_type == MX:
        ref.assert_mx(got, want, torch.zeros_like(want), "cancelling")
    else:
        mixer_ref.assert_within(got, want, (ref.half_step(BF16) if out_type == BF16 else 0.0) * want.abs(), "cancelling")


# n_in: whole fours of steps and others, few and many
DEPTHS = [512, 4096, 160, 1056]


@pytest.mark.parametrize("rows,n_out", TILES)
@pytest.mark.parametrize("n_in", DEPTHS)
@pytest.mark.parametrize("x_type", [MX, BF16])
def test_error_of_all_outputs(rs, rows, n_out, n_in, x_type):
    """Each of fewer than n_in additions is off by a step (2 U32) of a partial sum at most, in either direction, and
    partial sums are about as large as the root of their terms' squares: the norm of the errors stays within twice
    what independent ones give.  Products cut 13 places below another, which cost 1e-4 and more, would not pass."""
    x, w, xv, wv = _operands(x_type, rows, n_out, n_in, 21)
    xv, wv = xv.cuda().double(), wv.cuda().double()
    got = rs.linear(_cuda(x), _cuda(w), out_dtype=F32)
    size = (xv.square() @ wv.t().square()).sum().sqrt()
    off = (got.double() - xv @ wv.t()).norm()
    assert float(off) <= float(4 * mixer_ref.U32 * math.sqrt(n_in) * size)


@pytest.mark.parametrize("rows,n_out", TILES)
@pytest.mark.parametrize("n_in", DEPTHS)
def test_output_type_only_rounds(rs, rows, n_out, n_in):
    x, w, _, _ = _operands(MX, rows, n_out, n_in, 22)
    x, w = _cuda(x), _cuda(w)
    full = rs.linear(x, w, out_dtype=F32)
    assert _same(rs.linear(x, w), full.to(BF16))
    if n_out % 32 == 0 and (rows, n_out) != (5, 64):      # (MX outputs are whole blocks: no tiles of 16 outputs)
        assert _same(rs.linear(x, w, out_dtype=ref.E4M3), rs.quantize_mx(full))


@pytest.mark.parametrize("rows,n_out", TILES)
@pytest.mark.parametrize("n_in", DEPTHS)
@pytest.mark.parametrize("by", [0, 1])
def test_fast_products_within_their_bound(rs, rows, n_out, n_in, by):
    """Asked for, they are off by 2^-13 of the largest of 16 neighbouring products each, whatever the output's type."""
    if n_in <= 512:
        xv, wv, x, w = _cancelling(rows, n_out, n_in)
        want, err = ref.linear(xv.cuda(), wv.cuda(), None, None, None, 1.0, cut=True)
        x = _moved(_cuda(x), by)
        got = rs.linear(x, _cuda(w), out_dtype=F32, fast_products=True)
        mixer_ref.assert_within(got, want.cpu(), err.cpu(), "cancelling")
    x, w, xv, wv = _operands(MX, rows, n_out, n_in, 23)
    xv, wv, x, w = xv.cuda().double(), wv.cuda().double(), _moved(_cuda(x), by), _cuda(w)
    full = rs.linear(x, w, out_dtype=F32, fast_products=True)
    assert _same(rs.linear(x, w, fast_products=True), full.to(BF16))
    if n_out % 32 == 0 and (rows, n_out) != (5, 64):
        assert _same(rs.linear(x, w, out_dtype=ref.E4M3, fast_products=True), rs.quantize_mx(full))
    # the norm of all errors: of independent sign, each product's at most 2^-13 of its group's largest
    group, rest = torch.zeros(rows, n_out, dtype=torch.float64, device="cuda"), xv.square() @ wv.t().square()
    for k in range(0, n_in, 16):
        for r in range(0, rows, 500):
            group[r:r + 500] += (xv[r:r + 500, None, k:k + 16] * wv[None, :, k:k + 16]).abs().amax(-1).square()
    bound = (16 * group.sum()).sqrt() * 2.0 ** -13 + 4 * mixer_ref.U32 * math.sqrt(n_in) * rest.sum().sqrt()
    assert float((full.double() - xv @ wv.t()).norm()) <= float(bound)


def test_fast_products_leave_bf16_rows_alone(rs):
    x, w, _, _ = _operands(BF16, 200, 9024, 256, 24)
    assert _same(rs.linear(x.cuda(), w.cuda(), fast_products=True), rs.linear(x.cuda(), w.cuda()))
