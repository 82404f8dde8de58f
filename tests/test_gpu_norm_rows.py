"""Norms over more units than one axis of a launch can hold threads for."""
import pytest
import torch

import mixer_ref as ref
from test_gpu_mixer import BF16, _gen, rs  # noqa: F401

pytestmark = pytest.mark.gpu


def test_gated_norm_of_many_small_groups(rs):  # noqa: F811
    """Half a wave a unit: 2^27 + 96 units are more than 2^32 threads."""
    rows, dim, groups = (1 << 22) + 3, 32, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    y, z = (torch.randn(rows, dim, generator=g, device="cuda").to(BF16) for _ in range(2))
    w = 1 + 0.1 * torch.randn(dim, generator=_gen(2))
    out = torch.full_like(z, float("nan"))
    rs.gated_norm(y, z, w.cuda(), groups=groups, eps=1e-5, out=out)
    assert not torch.isnan(out).any()
    at = torch.cat([torch.arange(500), torch.randint(0, rows, (3000,), generator=_gen(3)), torch.arange(rows - 500, rows)])
    zs = z[at.cuda()].cpu()
    want = ref.gated_norm(y[at.cuda()].cpu(), zs, w, groups, 1e-5, False)
    # as for the other gated norms: gate and product in the value and in the norm, root, weight; one bf16 rounding
    rel = ref.U32 * (2 * (2 * float(zs.double().abs().max()) + 10) + 32)
    ref.assert_within(out[at.cuda()], want, (rel + ref.U16) * want.abs() + 1e-30, "gated norm")
