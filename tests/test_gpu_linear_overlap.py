"""Buffers that a call of the projections may share are shared, others are refused before anything is launched."""
import pytest
import torch

import linear_ref as ref
import mixer_ref
from test_gpu_linear import BF16, F32, _gen, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rs():
    import state_space_recurrence_amd as rs
    return rs


def test_outputs_over_operands_are_refused(rs):
    x, w = torch.ones(70, 128, dtype=BF16, device="cuda"), torch.ones(128, 128, dtype=BF16, device="cuda")
    keep = x.clone()
    r = torch.zeros(70, 128, device="cuda")
    with pytest.raises(rs.ReplaySSMError, match="overlap"):
        rs.linear(x, w, out=x)
    with pytest.raises(rs.ReplaySSMError, match="overlap"):
        rs.linear(x[:60], w, residual=r[:60], out=r[1:61])
    with pytest.raises(rs.ReplaySSMError, match="overlap"):
        rs.quantize_mx(x, out=(x.view(torch.uint8)[:35].view(70, 128).view(ref.E4M3), rs.quantize_mx(x)[1]))
    with pytest.raises(rs.ReplaySSMError, match="overlap"):
        rs.add_norm_mx(x, r, torch.ones(128, device="cuda"), residual_out=r.view(-1)[:70 * 128].view(70, 128),
                       out=(r.view(torch.uint8).view(-1)[:70 * 128].view(70, 128).view(ref.E4M3), rs.quantize_mx(x)[1]))
    assert _same(x, keep)


@pytest.mark.parametrize("rows,n_in,n_out", [(2, 64, 96), (2, 40, 33)])
def test_output_between_two_rows(rs, rows, n_in, n_out):
    """Rows of a wide buffer whose gap holds the whole output."""
    g = _gen(31)
    flat = torch.randn(4096 + n_in, generator=g).to(BF16).cuda()
    x = flat.as_strided((rows, n_in), (4096, 1))
    w = torch.randn(n_out, n_in, generator=g).to(BF16).cuda()
    want, err = ref.linear(x.cpu(), w.cpu(), None, None, None, 1.0)
    out = flat[512:512 + 2 * rows * n_out].view(F32).view(rows, n_out)
    assert rs.linear(x, w, out=out) is out
    mixer_ref.assert_within(out, want, err, "in the gap")


@pytest.mark.parametrize("rows,dim", [(5, 96), (3, 4096), (2, 8224)])
def test_sum_over_either_operand(rs, rows, dim):
    g = _gen(dim)
    x, r = torch.randn(rows, dim, generator=g).cuda(), torch.randn(rows, dim, generator=g).cuda()
    w = torch.ones(dim, device="cuda")
    want, res = rs.add_norm_mx(x, r, w, scale=0.5)
    for over in (0, 1):
        a, b = x.clone(), r.clone()
        got, total = rs.add_norm_mx(a, b, w, scale=0.5, residual_out=(a, b)[over])
        assert _same(got, want) and _same(total, res) and total is (a, b)[over]
