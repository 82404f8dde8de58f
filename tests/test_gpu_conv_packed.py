"""Packed convolution at the tiles that real prompts take, and what it leaves alone."""
import pytest
import torch

import mixer_ref as ref
from test_gpu_mixer import BF16, F32, _check_conv, _conv, _gen, _history, _rows, rs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tokens_of_no_row_are_left_alone(rs, dtype):  # noqa: F811
    """Tokens before the first offset, of padding rows and behind the last offset: none of their outputs is written,
    dt as little as x, B and C."""
    H, G = 3, 1
    cs, w, b, db = _conv(rs, 4, H, G, 4, dtype, seed=4)
    total, cu = 90, [5, 20, 41, 41, 70]
    slots = torch.tensor([2, -1, 0, 3], dtype=torch.int32, device="cuda")
    u, d, ug, dg = _rows(_gen(9), (total,), H, G, dtype)
    out = tuple(torch.full(s, 7.0, device="cuda", dtype=dtype)
                for s in ((total, H, 64), (total, G, 128), (total, G, 128), (total, H)))
    got = rs.conv_prefill(cs, ug, dg, torch.tensor(cu, dtype=torch.int32, device="cuda"), slots=slots, out=out)
    taken = torch.zeros(total, dtype=torch.bool)
    for a, e in ((5, 20), (41, 70)):
        taken[a:e] = True
        o, err, _ = ref.conv(torch.zeros(3, cs.channels, dtype=dtype), u[a:e], w, b)
        dv, de = ref.dt(d[a:e], db)
        _check_conv([x[a:e] for x in got], o, err, dv, de, dtype, H, G, f"tokens {a}..{e}")
    for x, name in zip(got, ("x", "B", "C", "dt")):
        assert (x[~taken.cuda()] == 7).all(), name
    cs.check_device_errors()
