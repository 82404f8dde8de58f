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


def _lengths(tile):
    """Prompts from the first, second and last two places of a tile over several tiles, and many within one tile."""
    lens, at = [], 0
    for off in (tile - 2, 1, tile - 1, 0, tile - 2, tile - 1):
        gap = (off - at) % tile
        lens += [gap] if gap else []         # a short prompt up to the place
        at += gap
        n = 2 * tile + 3 + off
        lens.append(n)                       # ... and one over three or four tiles from there
        at += n
    lens += [1, 2, 3, 0, 1, 1, 2, 0, 0, 3, 1] * 3
    lens += [tile, 2 * tile, tile - 1, tile + 1]
    return lens


@pytest.mark.parametrize("tile,blocks_total", [(4, 0), (8, 520), (16, 1056), (32, 2112)])
@pytest.mark.parametrize("W,dtype", [(4, BF16), (3, F32), (2, BF16), (4, F32)])
def test_tiles_of_real_prompts(rs, tile, blocks_total, W, dtype):  # noqa: F811
    """Every tile size, with eight workgroups across the channels: outputs at channels of each workgroup, and all of
    the histories, of prompts that continue a random history or start afresh."""
    H, G = 224, 1
    lens = _lengths(tile)
    lens.append(max(blocks_total - sum(lens), 0))     # to the total that takes this tile
    n, total = len(lens), sum(lens)
    nblk, t = -(-(64 * H + 256 * G) // 2048), 32
    while t > 4 and -(-total // t) * nblk < 512:
        t //= 2
    assert t == tile and nblk == 8
    g = _gen(100 + tile)
    cs, w, b, db = _conv(rs, n + 3, H, G, W, dtype, seed=W)
    Cc = cs.channels
    cs.ring.copy_(torch.randn(cs.ring.shape, generator=g).to(dtype))
    cs.head.copy_(torch.randint(0, cs.ring_rows, (n + 3,), generator=g).to(torch.int32))
    slots = torch.randperm(n + 3, generator=g)[:n].to(torch.int32)
    fresh = (torch.rand(n, generator=g) < 0.3).to(torch.int32)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    chs = torch.cat([torch.arange(k, k + 16) for k in range(0, Cc - 16, 2040)] + [torch.arange(Cc - 300, Cc)]).unique()
    hist = [_history(cs, int(s)) for s in slots]
    for call in range(2):
        u, d, ug, dg = _rows(g, (total,), H, G, dtype, extra=call)
        got = rs.conv_prefill(cs, ug, dg, cu.cuda(), fresh=fresh.cuda() if call else None, slots=slots.cuda())
        flat = torch.cat([got[0].flatten(1), got[1].flatten(1), got[2].flatten(1)], -1)[:, chs.cuda()].cpu()
        for r in range(n):
            a, e = int(cu[r]), int(cu[r + 1])
            if a == e:
                assert torch.equal(_history(cs, int(slots[r])), hist[r]), (call, r)
                continue
            h0 = torch.zeros_like(hist[r]) if call and fresh[r] else hist[r]
            out, err, _ = ref.conv(h0[:, chs], u[a:e, chs], w[chs], b[chs])
            half = ref.half_step(dtype) if dtype != F32 else 0.0
            what = f"call {call} row {r}, tokens {a}..{e}"
            ref.assert_within(flat[a:e], out, err * (1 + half) + half * out.abs() + 1e-37, what)
            dv, de = ref.dt(d[a:e], db)
            ref.assert_within(got[3][a:e], dv, de * (1 + half) + half * dv + 1e-37, what + " dt")
            hist[r] = torch.cat([h0, u[a:e]])[-(W - 1):]
            assert torch.equal(_history(cs, int(slots[r])), hist[r]), what
    cs.check_device_errors()
    assert int(cs.work.abs().sum()) == 0
