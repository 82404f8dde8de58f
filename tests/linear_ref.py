"""Plain 64-bit forms of the products and of rows in 8 bits (OCP MX), and the
error bounds that go with them."""
import math

import torch

from mixer_ref import U32, half_step, silu  # noqa: F401

BLOCK = 32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def mx_power(amax):
    """The power of the least 2^p with amax <= 448 2^p, at least -127 (amax in 64 bits, finite)."""
    m, e = torch.frexp(amax / 448)          # the quotient by 448 = 7 2^6 rounds, but keeps its side of a power of two
    p = torch.where(m > 0.5, e, e - 1)
    return torch.where(amax > 0, p, -127).clamp(min=-127)


def mx_quantize(v):
    """v [rows, dim]: the values of its codes (NaN where v is not finite) and its scales' powers, by the definition."""
    v = v.double()
    b = v.reshape(v.shape[0], -1, BLOCK)
    fine = torch.isfinite(b)
    power = mx_power(torch.where(fine, b.abs(), 0.0).amax(-1))
    u = torch.where(fine, b, 0.0) * torch.exp2(-power.double())[..., None]
    octave = (torch.frexp(u)[1] - 1).clamp(min=-6)
    step = torch.exp2(octave.double() - 3)
    q = torch.round(u / step) * step        # to the nearest, halves to even
    return torch.where(fine, q, math.nan).reshape(v.shape), power


def mx_values(pair):
    """The values that codes and scales stand for, in 64 bits."""
    codes, scales = pair
    s = torch.exp2(scales.view(torch.uint8).double() - 127)
    return codes.double() * s.repeat_interleave(BLOCK, -1)


def mx_pair(v):
    """(codes, scales) of v."""
    q, power = mx_quantize(v)
    return q.to(E4M3), (power + 127).to(torch.uint8).view(E8M0)


def assert_mx(pair, want, err, what):
    """An MX result of values that may be off `want` by `err` before they are quantised: scales between those of the
    block's smallest and largest possible amax, elements off by err and half a step of their octave."""
    got, want, err = mx_values(pair).cpu(), want.cpu(), err.cpu()
    power = pair[1].cpu().view(torch.uint8).long() - 127
    b, e = (t.reshape(t.shape[0], -1, BLOCK) for t in (want.double(), err.double()))
    lo, hi = mx_power((b.abs() - e).clamp(min=0).amax(-1)), mx_power((b.abs() + e).amax(-1))
    assert bool(((power >= lo) & (power <= hi)).all()), f"{what}: scales"
    size = want.abs() + err
    step = torch.maximum(2.0 ** -4 * size, 2.0 ** -10 * torch.exp2(hi.double()).repeat_interleave(BLOCK, -1))
    bad = (got - want).abs() - (err + step) * (1 + 1e-12)
    assert bool((bad <= 0).all()), f"{what}: off by {float(bad.max()):.3g} more than allowed"


def gelu(v):
    return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))


def cut_products(x, w):
    """Error bound of scaled 8-bit products: the matrix units cut a product 13 binary places below the largest of the
    products that they add at once, some of 16 consecutive ones."""
    x, w = (torch.nn.functional.pad(t.double().abs(), (0, -t.shape[1] % 16)) for t in (x, w))
    total = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    for r in range(0, x.shape[0], 64):
        for k in range(0, x.shape[1], 16):
            total[r:r + 64] += (x[r:r + 64, None, k:k + 16] * w[None, :, k:k + 16]).amax(-1)
    return 16 * 2.0 ** -13 * total


def linear(x, w, bias, act, res, scale, cut=False):
    """x [rows,K], w [N,K] (values, any type): outputs in 64 bits and their error bound before the last rounding."""
    x, w = x.double(), w.double()
    v = x @ w.t()
    # K additions into fp32, each off by a step of a partial sum of at most the terms' sum (a half step where the
    # matrix units round to nearest, a whole one where they cut off)
    err = x.shape[1] * 2 * U32 * (x.abs() @ w.abs().t())
    if cut:
        err = err + cut_products(x, w)
    if bias is not None:
        v = v + bias.double()
        err = err + U32 * v.abs()
    if act == "silu":      # |silu'| < 1.1; exp of a rounded argument, sum, reciprocal, product
        out = silu(v)
        err = 1.1 * err + (2 * v.abs() + 10) * U32 * out.abs()
        # sigmoid below the smallest normal number is flushed
        err = err + v.abs() * 2.0 ** -126
    elif act == "gelu":    # |gelu'| < 1.13; 1.5e-7 |v| / 2 from erfc's form, its 12 roundings, exp of a rounded square
        out = gelu(v)
        err = 1.13 * err + 0.75e-7 * v.abs() + (2 * v * v + 24) * U32 * out.abs() + v.abs() * 2.0 ** -126
    elif act == "relu2":
        out = v.clamp(min=0).square()
        err = 2 * v.abs() * err + err * err + U32 * out
    else:
        out = v
    scale = torch.tensor(scale, dtype=torch.float32).double()    # as the call takes it
    out, err = scale * out, scale.abs() * err + U32 * (scale * out).abs()
    if res is not None:
        out = res.double() + out
        err = err + U32 * out.abs()
    return out, err + 1e-37
