"""The product with its epilogue and rows in 8 bits on the GPU, against plain
64-bit forms."""
import math

import pytest
import torch

import linear_ref as ref
import mixer_ref

pytestmark = pytest.mark.gpu

BF16, F32, MX = torch.bfloat16, torch.float32, "mx"


@pytest.fixture(scope="module")
def rs():
    import state_space_recurrence_amd as rs
    return rs


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _cuda(v):
    if v is None:
        return None
    return tuple(t.cuda() for t in v) if isinstance(v, tuple) else v.cuda()


def _same(a, b):
    """Bit for bit."""
    if isinstance(a, tuple):
        return all(_same(x, y) for x, y in zip(a, b))
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _operands(x_type, rows, n_out, n_in, seed, zero_row=True):
    """(x, w as handed over, their values)."""
    g = _gen(seed)
    x = torch.randn(rows, n_in, generator=g) * torch.exp(torch.randn(n_in, generator=g))
    w = torch.randn(n_out, n_in, generator=g) / math.sqrt(n_in)
    if zero_row and rows > 2:
        x[1] = 0
    if x_type == MX:
        x, w = ref.mx_pair(x), ref.mx_pair(w)
        return x, w, ref.mx_values(x), ref.mx_values(w)
    x, w = x.to(BF16), w.to(BF16)
    return x, w, x, w


def _check(rs, x_type, rows, n_out, n_in, out_type, bias, act, res_type, scale, seed=0, at="cpu"):
    x, w, xv, wv = _operands(x_type, rows, n_out, n_in, seed + rows + 7 * n_out + 13 * n_in)
    xv, wv = xv.to(at), wv.to(at)
    g = _gen(seed + 1)
    b = 0.1 * torch.randn(n_out, generator=g) if bias else None
    r = None if res_type is None else (2 * torch.randn(rows, n_out, generator=g)).to(res_type)
    got = rs.linear(_cuda(x), _cuda(w), _cuda(b), activation=act, residual=_cuda(r), scale=scale,
                    out_dtype=ref.E4M3 if out_type == MX else out_type)
    want, err = ref.linear(xv, wv, None if b is None else b.to(at), act, None if r is None else r.to(at), scale,
                           cut=x_type == MX and out_type == BF16)
    want, err = want.cpu(), err.cpu()
    if out_type == MX:
        ref.assert_mx(got, want, err, "mx output")
    else:
        assert got.dtype == out_type and got.shape == (rows, n_out)
        u = ref.half_step(BF16) if out_type == BF16 else 0.0
        mixer_ref.assert_within(got, want, err * (1 + u) + u * want.abs(), "linear")


# ------------------------------------------------------------ rows in 8 bits --

@pytest.mark.parametrize("rows,dim,wide,xt", [(1, 32, 32, F32), (5, 96, 96, BF16), (45, 1056, 1060, F32),
                                              (3, 4096, 4101, BF16), (700, 64, 64, BF16), (2, 16416, 16416, F32)])
def test_quantize(rs, rows, dim, wide, xt):
    """Bit for bit the definition, over the range of scales, ties and values that are not finite."""
    g = _gen(dim)
    v = torch.randn(rows, wide, generator=g) * torch.exp(3 * torch.randn(rows, wide, generator=g))
    line = v[0, :dim].view(-1, 32)
    line[0] = torch.arange(32) * 0.0625 + 446.5                       # around 448, and ties between codes
    if rows > 2:
        v[1, :32] = 0
        v[2, :32] = torch.linspace(-1e-38, 3e-39, 32)                 # scales at their least, subnormal numbers
        v[2, 32:64] = 3e38 * torch.linspace(-1, 1, 32)
        v[2, 5], v[2, 40], v[1, 33], v[1, 63] = math.inf, -math.inf, math.nan, math.inf
    x = v.to(xt).cuda()[:, :dim]
    codes, scales = rs.quantize_mx(x)
    want, power = ref.mx_quantize(x.cpu())
    assert torch.equal(scales.cpu().view(torch.uint8).long() - 127, power.long())
    got = codes.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


def test_quantize_every_code(rs):
    """All of a block's rounding borders: sizes between two codes, the middle, and one step to either side of it."""
    codes = torch.arange(127, dtype=torch.uint8).view(ref.E4M3).double()
    mid = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mid, mid * (1 + 2.0 ** -22), mid * (1 - 2.0 ** -22)])
    v = torch.cat([v, -v])
    v = torch.nn.functional.pad(v, (0, -len(v) % 31)).view(-1, 31)
    v = torch.cat([torch.full((len(v), 1), 448.0, dtype=torch.float64), v], 1).float()
    for scale in (1.0, 2.0 ** -100, 2.0 ** 60):
        c, s = rs.quantize_mx((v * scale).cuda())
        want, power = ref.mx_quantize(v * scale)
        assert torch.equal(s.cpu().view(torch.uint8).long() - 127, power.long())
        assert torch.equal(c.cpu().double(), want)


@pytest.mark.parametrize("rows,dim,groups,yt,zt,before", [
    (1, 6144, 8, F32, BF16, False), (5, 64, 1, F32, F32, False), (33, 512, 2, BF16, BF16, True),
    (4, 1536, 1, BF16, F32, False), (3, 4096, 1, F32, BF16, True), (2, 8192, 1, BF16, BF16, False),
    (2, 16384, 1, F32, F32, False), (300, 256, 8, BF16, BF16, False), (3, 2016, 3, F32, BF16, False),
])
def test_gated_norm_mx(rs, rows, dim, groups, yt, zt, before):
    g = _gen(dim)
    y = (3 * torch.randn(rows, dim, generator=g)).to(yt)
    zr = torch.randn(rows, dim + 7, generator=g).to(zt)
    w = 1 + 0.1 * torch.randn(dim, generator=g)
    if rows > 2:
        y[1] = 0
        zr[2, :] = -100.0
    got = rs.gated_norm_mx(y.cuda(), zr.cuda()[:, 5:5 + dim], w.cuda(), groups=groups, eps=1e-5, norm_before_gate=before)
    z = zr[:, 5:5 + dim]
    want = mixer_ref.gated_norm(y, z, w, groups, 1e-5, before)
    zmax = float(z.double().abs().max())
    rel = mixer_ref.U32 * (2 * (2 * zmax + 10) + 32)      # as for outputs that are numbers
    ref.assert_mx(got, want, rel * want.abs() + 1e-30, "gated norm")


@pytest.mark.parametrize("rows,dim,xt,rt,post,inplace", [
    (1, 4096, BF16, F32, False, False), (3, 2560, BF16, BF16, True, True), (5, 32, F32, F32, True, False),
    (4, 96, F32, BF16, False, True), (2, 5024, BF16, F32, True, False), (2, 16384, F32, F32, True, True),
    (300, 64, BF16, BF16, False, False), (9, 544, F32, F32, False, False), (3, 800, None, F32, False, False),
    (2, 8192, None, BF16, False, False), (1, 16384, None, F32, False, False),
])
def test_add_norm_mx(rs, rows, dim, xt, rt, post, inplace):
    g = _gen(dim + 1)
    r = (2 * torch.randn(rows, dim, generator=g)).to(rt)
    x = None if xt is None else torch.randn(rows, dim, generator=g).to(xt)
    w, p = 1 + 0.1 * torch.randn(dim, generator=g), 0.5 + 0.1 * torch.randn(dim, generator=g)
    if rows > 2:
        r[1] = 0
        if x is not None:
            x[1] = 0
    rg = r.cuda()
    keep = rg.clone()
    out, res = rs.add_norm_mx(_cuda(x), rg, w.cuda(), scale=0.22, post_weight=p.cuda() if post else None, eps=1e-6,
                              residual_out=rg if inplace else None)
    if x is None:
        assert res is rg and torch.equal(rg, keep)
        want, rw = mixer_ref.add_norm(torch.zeros_like(r, dtype=F32), r, w, 1.0, None, 1e-6)
    else:
        assert (res.data_ptr() == rg.data_ptr()) == inplace and (inplace or torch.equal(rg, keep))
        want, rw = mixer_ref.add_norm(x, r, w, 0.22, p if post else None, 1e-6)
    f = rw - r.double()
    rerr = mixer_ref.U32 * (rw.abs() + (28 if post else 3) * f.abs())
    u = mixer_ref.half_step(rt) if rt != F32 else 0.0
    mixer_ref.assert_within(res, rw, rerr * (1 + u) + u * rw.abs() + 1e-37, "residual")
    inv = 1 / (rw.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    rel_norm = (rerr.pow(2).mean(-1, keepdim=True) + 0).sqrt() * inv
    err = rerr * inv * w.double().abs() + want.abs() * (rel_norm + 28 * mixer_ref.U32)
    ref.assert_mx(out, want, err + 1e-30, "normed")


def test_norms_mx_agree_with_quantized_norms(rs):
    """The fp32 output of the plain norm, quantised by a call of its own: the same bits."""
    g = _gen(3)
    y, z = torch.randn(37, 768, generator=g).cuda(), torch.randn(37, 768, generator=g).to(BF16).cuda()
    w = (1 + 0.1 * torch.randn(768, generator=g)).cuda()
    full = torch.empty(37, 768, device="cuda")
    rs.gated_norm(y, z, w, groups=3, out=full)
    assert _same(rs.gated_norm_mx(y, z, w, groups=3), rs.quantize_mx(full))
    rs.add_norm(z, y, w, out=full)
    assert _same(rs.add_norm_mx(z, y, w)[0], rs.quantize_mx(full))


# ---------------------------------------------------------------- products --

# rows x outputs x inputs: single rows, edges of every tile, sums of one step and of many
SIZES = [(1, 1, 1), (1, 33, 64), (2, 16, 8), (3, 100, 63), (5, 7, 251), (16, 48, 128), (17, 130, 192), (31, 64, 1000),
         (33, 96, 640), (64, 64, 64), (65, 257, 128), (100, 300, 320), (128, 128, 256), (129, 200, 72),
         (1, 40, 8), (4, 100, 1000), (20, 200, 2056), (70, 500, 88)]


@pytest.mark.parametrize("rows,n_out,n_in", SIZES)
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_linear_bf16(rs, rows, n_out, n_in, out_type):
    _check(rs, BF16, rows, n_out, n_in, out_type, False, None, None, 1.0)


MX_SIZES = [(1, 1, 32), (1, 33, 64), (2, 16, 96), (3, 100, 128), (5, 7, 256), (16, 48, 1152), (17, 130, 224),
            (31, 64, 1024), (33, 96, 640), (64, 64, 128), (65, 257, 384), (100, 300, 320), (128, 128, 256),
            (129, 200, 160), (1, 40, 1056), (4, 100, 992), (20, 200, 2080), (70, 500, 96)]


@pytest.mark.parametrize("rows,n_out,n_in", MX_SIZES)
@pytest.mark.parametrize("out_type", [BF16, F32])
def test_linear_mx(rs, rows, n_out, n_in, out_type):
    _check(rs, MX, rows, n_out, n_in, out_type, False, None, None, 1.0)


@pytest.mark.parametrize("x_type,rows,n_out,n_in", [
    (BF16, 1, 32, 64), (BF16, 3, 96, 100), (BF16, 40, 160, 256), (BF16, 130, 288, 128), (MX, 1, 64, 128),
    (MX, 7, 32, 96), (MX, 16, 320, 512), (MX, 70, 160, 256), (MX, 200, 544, 128), (BF16, 300, 1024, 64),
    (MX, 270, 1056, 256),
])
@pytest.mark.parametrize("bias,act,res_type,scale,out_type", [
    (True, None, None, 1.0, BF16), (True, "silu", F32, 0.5, F32), (False, "gelu", BF16, -2.0, BF16),
    (True, "relu2", F32, 0.22, MX), (True, "gelu", None, 1.0, MX), (False, None, BF16, 1.0, F32),
])
def test_epilogue(rs, x_type, rows, n_out, n_in, bias, act, res_type, scale, out_type):
    _check(rs, x_type, rows, n_out, n_in, out_type, bias, act, res_type, scale)


# Sizes at which each of the tiles is taken (16 x 16 and 32 x 16 ones by the sizes above): sums of whole fours of steps
# and others, edges in both directions
BY_TILE = [(BF16, 20, 4100, 576), (BF16, 32, 4128, 2048), (BF16, 33, 4100, 1024), (BF16, 64, 9000, 1088),
           (BF16, 65, 9000, 640), (BF16, 128, 9120, 2048), (BF16, 200, 9000, 1088), (BF16, 256, 9120, 2048),
           (BF16, 700, 9000, 1088), (BF16, 700, 9024, 2048),
           (BF16, 2000, 4100, 1088), (BF16, 2048, 4128, 2048), (MX, 20, 4100, 1152), (MX, 33, 4128, 2048),
           (MX, 64, 9000, 4096), (MX, 65, 9000, 1152), (MX, 128, 9120, 2048), (MX, 200, 9000, 1152),
           (MX, 256, 9120, 2048), (MX, 700, 9000, 1152), (MX, 700, 9024, 2048), (MX, 2000, 4100, 1152),
           (MX, 3000, 4128, 2048),
           # rows that end inside a step, and scales that start at any byte
           (BF16, 20, 4100, 1000), (BF16, 33, 4128, 1096), (BF16, 128, 9120, 8), (BF16, 200, 9000, 1048),
           (BF16, 2000, 4128, 1112), (BF16, 2000, 4100, 1064), (MX, 20, 4100, 1184), (MX, 33, 4128, 1120), (MX, 64, 9000, 32),
           (MX, 65, 9120, 1248), (MX, 128, 9000, 1216), (MX, 200, 9120, 1056), (MX, 250, 9000, 96), (MX, 2000, 4128, 1184),
           (MX, 3000, 4128, 1120), (MX, 2000, 4100, 1056), (MX, 3000, 4100, 64),
           (BF16, 700, 9024, 1032), (MX, 700, 9024, 1088), (MX, 690, 9000, 96)]


@pytest.mark.parametrize("x_type,rows,n_out,n_in", BY_TILE)
@pytest.mark.parametrize("out_type,res_type", [(BF16, None), (F32, F32)])
def test_every_tile(rs, x_type, rows, n_out, n_in, out_type, res_type):
    """The 64-bit product is taken on the GPU here."""
    _check(rs, x_type, rows, n_out, n_in, out_type, True, None, res_type, 0.5, at="cuda")


@pytest.mark.parametrize("x_type,rows,n_out,n_in", [c for c in BY_TILE if c[2] % 32 == 0])
def test_every_tile_mx_output(rs, x_type, rows, n_out, n_in):
    _check(rs, x_type, rows, n_out, n_in, MX, True, "gelu", BF16, 0.5, at="cuda")


@pytest.mark.parametrize("act", ["silu", "gelu", "relu2"])
def test_activation_values(rs, act):
    """An identity product: the activation over the range of its argument, large ones and zeros among them."""
    v = torch.cat([torch.linspace(-12, 12, 2000), torch.tensor([0.0, -0.0, 100.0, -100.0, 3e4, -3e4]),
                   torch.zeros(42)]).view(-1, 64).to(BF16)
    eye = torch.eye(64, dtype=BF16)
    got = rs.linear(v.cuda(), eye.cuda(), activation=act, out_dtype=F32)
    want, err = ref.linear(v, eye, None, act, None, 1.0)
    mixer_ref.assert_within(got, want, err, act)


SHAPES_BY_KERNEL = [(BF16, 3, 100, 65), (BF16, 5, 96, 256), (BF16, 40, 160, 256), (BF16, 200, 544, 256), (MX, 5, 96, 256),
                    (MX, 9, 160, 96), (MX, 40, 160, 256), (MX, 200, 544, 256), (BF16, 600, 1000, 192), (MX, 600, 1000, 256),
                    (BF16, 33, 4100, 128), (BF16, 100, 9024, 192), (BF16, 200, 9024, 64), (BF16, 2000, 4128, 64),
                    (MX, 33, 4100, 256), (MX, 200, 9024, 128), (MX, 3000, 4128, 128),
                    (BF16, 5, 96, 72), (BF16, 33, 4100, 136), (BF16, 200, 9024, 88), (BF16, 2000, 4128, 72), (MX, 5, 96, 160),
                    (MX, 33, 4100, 224), (MX, 200, 9024, 96), (MX, 3000, 4128, 160), (BF16, 700, 9024, 72), (MX, 700, 9024, 96)]


@pytest.mark.parametrize("x_type,rows,n_out,n_in", SHAPES_BY_KERNEL)
def test_nothing_else_is_written(rs, x_type, rows, n_out, n_in):
    """Rows before and behind the outputs stay as they were, and what lies between strided rows of x is not read."""
    x, w, xv, wv = _operands(x_type, rows, n_out, n_in, 5)
    xc = _cuda(x)
    if x_type == BF16:
        wide = torch.full((rows + 2, n_in + 64), math.nan, dtype=BF16, device="cuda")
        wide[1:-1, 8:8 + n_in] = xc          # (a multiple of 8 elements: rows stay aligned where n_in is one)
        xc = wide[1:-1, 8:8 + n_in]
    buf = torch.full((rows + 4, n_out), 7.0, dtype=F32, device="cuda")
    rs.linear(xc, _cuda(w), out=buf[2:-2])
    assert bool((buf[:2] == 7).all()) and bool((buf[-2:] == 7).all())
    want, err = ref.linear(xv, wv, None, None, None, 1.0)
    mixer_ref.assert_within(buf[2:-2], want, err, "strided")
    if n_out % 32 == 0:
        codes = torch.full((rows + 32, n_out), 7, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows + 32, n_out // 32), 7, dtype=torch.uint8, device="cuda")
        out = (codes[16:-16].view(ref.E4M3), scales[16:-16].view(ref.E8M0))
        rs.linear(xc, _cuda(w), out=out)
        for t in (codes, scales):
            assert bool((t[:16] == 7).all()) and bool((t[-16:] == 7).all())
        ref.assert_mx(out, want, err, "mx rows")


@pytest.mark.parametrize("x_type,rows,n_out,n_in", SHAPES_BY_KERNEL)
def test_rows_that_are_not_finite_stay_alone(rs, x_type, rows, n_out, n_in):
    x, w, xv, wv = _operands(x_type, rows, n_out, n_in, 6)
    xc = _cuda(x)
    clean = rs.linear(xc, _cuda(w), out_dtype=F32)
    if x_type == MX:
        xc[0].view(torch.uint8)[1, 3] = 0x7F
        xc[1].view(torch.uint8)[2, 0] = 0xFF
    else:
        xc[1, 3] = math.nan
        xc[2, n_in - 1] = math.inf
    got = rs.linear(xc, _cuda(w), out_dtype=F32)
    assert bool(torch.isnan(got[1]).all()) and not bool(torch.isfinite(got[2]).any())
    keep = [i for i in range(rows) if i not in (1, 2)]
    assert _same(got[keep], clean[keep])
    wc = _cuda(w)
    if x_type == MX:
        wc[0].view(torch.uint8)[n_out - 1, 0] = 0x7F
    else:
        wc[n_out - 1, 0] = math.nan
    got = rs.linear(_cuda(x), wc, out_dtype=F32)
    assert bool(torch.isnan(got[:, -1]).all()) and _same(got[:, :-1].contiguous(), clean[:, :-1].contiguous())


@pytest.mark.parametrize("x_type,rows,n_out,n_in", SHAPES_BY_KERNEL)
def test_in_place_repeated_and_equal_rows(rs, x_type, rows, n_out, n_in):
    """The residual may be the output; calls repeat bit for bit; equal rows get equal outputs."""
    x, w, xv, wv = _operands(x_type, rows, n_out, n_in, 8)
    xc, wc = _cuda(x), _cuda(w)
    for t in xc if x_type == MX else (xc,):
        t.view(torch.uint8)[-1] = t.view(torch.uint8)[0]
    r = torch.randn(rows, n_out, generator=_gen(9)).cuda()
    r[-1] = r[0]
    first = rs.linear(xc, wc, residual=r, scale=0.5, out_dtype=F32)
    again = rs.linear(xc, wc, residual=r, scale=0.5, out_dtype=F32)
    assert _same(first, again) and _same(first[0], first[-1])
    rs.linear(xc, wc, residual=r, scale=0.5, out=r)
    assert _same(r, first)


def test_unaligned_rows_agree(rs):
    """The same rows at other addresses: odd element offsets and pitches."""
    x, w, xv, wv = _operands(BF16, 50, 100, 128, 11)
    want, err = ref.linear(xv, wv, None, None, None, 1.0)
    for off, pitch in ((0, 128), (1, 131), (8, 136), (3, 192)):
        flat = torch.zeros(50 * pitch + 16, dtype=BF16, device="cuda")
        view = flat.as_strided((50, 128), (pitch, 1), off)
        view.copy_(x.cuda())
        mixer_ref.assert_within(rs.linear(view, w.cuda(), out_dtype=F32), want, err, f"offset {off}")


@pytest.mark.parametrize("rows,n_out,n_in", [(3, 64, 64), (64, 9000, 160), (200, 9024, 96), (2000, 4128, 64)])
@pytest.mark.parametrize("sx,sw", [(0, 246), (1, 246), (3, 240), (60, 194), (246, 0), (246, 7), (127, 127)])
def test_scales_over_their_range(rs, rows, n_out, n_in, sx, sw):
    """From the least scale to the largest whose values are all finite: products of the codes times a power of two."""
    g = _gen(sx)
    xc, wc = (torch.randn(n, n_in, generator=g).mul(20).to(ref.E4M3) for n in (rows, n_out))
    pair = lambda c, s: (c.cuda(), torch.full((c.shape[0], n_in // 32), s, dtype=torch.uint8, device="cuda").view(ref.E8M0))  # noqa: E731
    for out_type in (F32, BF16):
        got = rs.linear(pair(xc, sx), pair(wc, sw), out_dtype=out_type)
        want, err = ref.linear(xc.cuda(), wc.cuda(), None, None, None, 1.0, cut=out_type == BF16)
        f = 2.0 ** (sx + sw - 254)
        # operands widened to bf16 are multiples of 2^-133, its least subnormal number: off by half of that, which is
        # 2^-7 - s of a code with scale byte s, times the other side's codes; E4M3's codes are multiples of 2^-9, so this
        # is nothing from byte 3 on
        lost = lambda s: 2.0 ** (-7 - s) if s < 3 else 0.0  # noqa: E731
        err = err + lost(sx) * wc.cuda().double().abs().sum(1) + lost(sw) * xc.cuda().double().abs().sum(1)[:, None]
        u = ref.half_step(BF16) if out_type == BF16 else 0.0
        mixer_ref.assert_within(got, (f * want).cpu(), (f * (err * (1 + u) + u * want.abs())).cpu(), "scaled")


@pytest.mark.parametrize("rows,n_out", [(3, 64), (64, 9000), (200, 9024), (700, 9024), (2000, 4128)])
@pytest.mark.parametrize("out_type", [F32, BF16])
def test_not_a_number_scales(rs, rows, n_out, out_type):
    x, w, _, _ = _operands(MX, rows, n_out, 96, 13)
    clean = rs.linear(_cuda(x), _cuda(w), out_dtype=out_type)
    xc, wc = _cuda(x), _cuda(w)
    xc[1].view(torch.uint8)[2, 1] = 255
    wc[1].view(torch.uint8)[5, 2] = 255
    got = rs.linear(xc, wc, out_dtype=out_type)
    assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[:, 5]).all())
    got[2], got[:, 5] = clean[2], clean[:, 5]
    assert _same(got, clean)


def test_scales_at_any_address(rs):
    """MX scales that start between multiples of 4 bytes: the same values, by another kernel."""
    x, w, xv, wv = _operands(MX, 50, 100, 96, 12)
    want, err = ref.linear(xv, wv, None, None, None, 1.0)
    xc, wc = _cuda(x), _cuda(w)
    for off in (0, 1, 2, 3):
        buf = torch.zeros(off + 150, dtype=torch.uint8, device="cuda")
        scales = buf[off:].view(50, 3)
        scales.copy_(xc[1].view(torch.uint8))
        mixer_ref.assert_within(rs.linear((xc[0], scales.view(ref.E8M0)), wc, out_dtype=F32), want, err, f"offset {off}")


def test_no_rows(rs):
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.zeros(96, 64, dtype=BF16, device="cuda")
    assert rs.linear(e, w).shape == (0, 96)
    codes, scales = rs.quantize_mx(e)
    assert codes.shape == (0, 64) and scales.shape == (0, 2)
    one = torch.ones(64, device="cuda")
    assert rs.gated_norm_mx(e, e, one)[0].shape == (0, 64) and rs.add_norm_mx(e, e, one)[0][1].shape == (0, 2)
    assert rs.linear((codes, scales), rs.quantize_mx(w), out_dtype=ref.E4M3)[1].shape == (0, 3)


def _block(rs, x, res, p):
    """A feed-forward block in 8 bits: norm, product with activation, product onto the residual."""
    out, res = rs.add_norm_mx(x, res, p["w"], out=p["n"], residual_out=p["r"])
    up = rs.linear(out, p["up"], p["b"], activation="gelu", out=p["h"])
    return rs.linear(up, p["down"], residual=res, out=p["o"])


def _params(rs, rows, dim, wide, seed):
    g = _gen(seed)
    c = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    e = lambda *s, **k: torch.empty(*s, device="cuda", **k)  # noqa: E731
    mx = lambda n: (e(rows, n, dtype=ref.E4M3), e(rows, n // 32, dtype=ref.E8M0))  # noqa: E731
    return dict(w=1 + 0.1 * c(dim), up=rs.quantize_mx(c(wide, dim) / math.sqrt(dim)), b=0.1 * c(wide),
                down=rs.quantize_mx(c(dim, wide) / math.sqrt(wide)), n=mx(dim), r=e(rows, dim), h=mx(wide), o=e(rows, dim))


@pytest.mark.parametrize("rows", [1, 5, 40, 300])
def test_block_captured_and_replayed(rs, rows):
    """The operators in a row, captured: every replay, between eager work, gives the eager result of its inputs."""
    dim, wide = 256, 1024
    p, q = _params(rs, rows, dim, wide, 1), _params(rs, rows, dim, wide, 1)
    g = _gen(2)
    xs = [torch.randn(rows, dim, generator=g).to(BF16).cuda() for _ in range(4)]
    res = torch.randn(rows, dim, generator=g).cuda()
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _block(rs, x, res, p)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _block(rs, x, res, p)
    for v in xs:
        x.copy_(v)
        graph.replay()
        got = p["o"].clone()
        want = _block(rs, v, res, q).clone()
        torch.cuda.synchronize()
        assert _same(got, want)


def test_two_streams(rs):
    """Calls of the same weights on two streams at once: each the result of its own inputs."""
    g = _gen(4)
    w = torch.randn(512, 256, generator=g).to(BF16).cuda()
    xs = [torch.randn(n, 256, generator=g).to(BF16).cuda() for n in (700, 650)]
    want = [rs.linear(x, w, activation="silu") for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [rs.linear(x, w, activation="silu", stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(got, want))


def test_block_follows_its_formulas(rs):
    """The block's last output against its 64-bit form from the 8-bit rows between its calls."""
    p = _params(rs, 33, 256, 512, 7)
    g = _gen(8)
    x, res = torch.randn(33, 256, generator=g).to(BF16).cuda(), torch.randn(33, 256, generator=g).cuda()
    got = _block(rs, x, res, p)
    hw, he = ref.linear(ref.mx_values(p["n"]), ref.mx_values(p["up"]), p["b"], "gelu", None, 1.0)
    ref.assert_mx(p["h"], hw, he, "hidden rows")
    want, err = ref.linear(ref.mx_values(p["h"]), ref.mx_values(p["down"]), None, None, p["r"], 1.0)
    mixer_ref.assert_within(got, want.cpu(), err.cpu(), "block")


def test_example_in_8_bits():
    """The stack of blocks with its projections in MX: prompts at once, tokens and drafts agree with token by token."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixer_block.py")
    spec = importlib.util.spec_from_file_location("mixer_block_mx", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # five rows of codes lie between the embeddings and the hidden states: the first norm's, and two of each block; where
    # the two ways round differently they are off by a step, 2^-3 of an element at most, as independent as their roundings
    assert m.main(verbose=False, mx=True) < 5 ** 0.5 * 2.0 ** -3
    assert m.main(lengths=(300, 64, 2), tokens=3, seed=1, verbose=False, mx=True) < 5 ** 0.5 * 2.0 ** -3
