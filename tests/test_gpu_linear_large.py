"""Offsets of operands and outputs that 32 bits do not hold."""
import pytest
import torch

import linear_ref as ref
import mixer_ref
from test_gpu_linear import BF16, F32, MX, _gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rs():
    import state_space_recurrence_amd as rs
    return rs


def _some(rows):
    return torch.tensor(sorted({0, 1, rows // 3, rows // 2, rows // 2 + 1, rows - 2, rows - 1}))


@pytest.mark.parametrize("n_in", [64, 33])
def test_rows_far_apart(rs, n_in):
    """x rows 2^22 elements apart: 700 of them span 5.9 GB.  Aligned and unaligned lengths."""
    rows, pitch = 700, 1 << 22
    g = _gen(51)
    flat = torch.empty((rows - 1) * pitch + n_in, dtype=BF16, device="cuda")
    x = flat.as_strided((rows, n_in), (pitch, 1))
    xv, wv = torch.randn(rows, n_in, generator=g).to(BF16), torch.randn(96, n_in, generator=g).to(BF16)
    x.copy_(xv)
    want, err = ref.linear(xv, wv, None, None, None, 1.0)
    mixer_ref.assert_within(rs.linear(x, wv.cuda(), out_dtype=F32), want, err, "far rows")
    if n_in % 32 == 0:
        got = ref.mx_values(rs.quantize_mx(x))
        assert torch.equal(got.cpu(), ref.mx_values(tuple(t.cpu() for t in rs.quantize_mx(xv.cuda()))))


@pytest.mark.parametrize("x_type,n_in", [(BF16, 32), (BF16, 31), (MX, 32)])
@pytest.mark.parametrize("out_type", [BF16, MX])
def test_more_than_2_31_outputs(rs, x_type, n_in, out_type):
    """160000 rows of 14432 outputs, 2.3e9: rows from the first to the last, in place of the residual for bf16."""
    rows, n_out = 160000, 14432
    g = torch.Generator(device="cuda")
    g.manual_seed(n_in)
    x = torch.randn(rows, n_in, generator=g, device="cuda").to(BF16)
    w = torch.randn(n_out, n_in, generator=g, device="cuda").to(BF16)
    at = _some(rows).cuda()
    xv, wv = x[at], w
    if x_type == MX:
        x, w = rs.quantize_mx(x), rs.quantize_mx(w)
        xv, wv = ref.mx_values((x[0][at], x[1].view(torch.uint8)[at].view(ref.E8M0))), ref.mx_values(w)
    res = None
    if out_type == BF16:
        out = torch.ones(rows, n_out, dtype=BF16, device="cuda")
        res = torch.ones(len(at), n_out, dtype=BF16, device="cuda")
        rs.linear(x, w, residual=out, out=out)
        got = out[at]
    else:
        codes, scales = rs.linear(x, w, out_dtype=ref.E4M3)
        got = codes[at], scales.view(torch.uint8)[at].view(ref.E8M0)
    want, err = ref.linear(xv, wv, None, None, res, 1.0)
    if out_type == BF16:
        u = ref.half_step(BF16)
        mixer_ref.assert_within(got, want.cpu(), (err * (1 + u) + u * want.abs()).cpu(), "bf16")
    else:
        ref.assert_mx(got, want, err, "mx")


def test_norms_of_more_than_2_31_elements(rs):
    """132000 rows of 16384 elements: the last rows equal the same rows by themselves."""
    rows, dim = 132000, 16384
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(1000, dim, generator=g, device="cuda").to(BF16).repeat(rows // 1000, 1)
    w = torch.ones(dim, device="cuda")
    few = x[:1000]
    for call in (lambda v: rs.quantize_mx(v), lambda v: rs.add_norm_mx(None, v, w)[0],
                 lambda v: rs.gated_norm_mx(v, v, w, groups=2)):
        codes, scales = (t.view(torch.uint8) for t in call(x))
        one = [t.view(torch.uint8) for t in call(few)]
        for i in (0, rows // 2000 * 1000, rows - 1000):
            assert torch.equal(codes[i:i + 1000], one[0]) and torch.equal(scales[i:i + 1000], one[1])
