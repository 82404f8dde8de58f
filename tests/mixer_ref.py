"""Plain 64-bit forms of the mixer operators, sequence by sequence and token
by token, and the error bounds that go with them."""
import math

import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8     # largest relative error of one rounding: fp32, bf16


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def silu(v):
    return v / (1 + torch.exp(-v))


def conv(history, u, weight, bias, act=True):
    """history [W-1,Cc], u [T,Cc] (any type), weight [Cc,W]: outputs [T,Cc] in
    64 bits, their error bound for fp32 arithmetic, and the new history."""
    W = weight.shape[1]
    line = torch.cat([history, u]).double()
    w = weight.double()
    T = u.shape[0]
    terms = [line[k:k + T] * w[:, k] for k in range(W)]
    b = torch.zeros(w.shape[0], dtype=torch.float64) if bias is None else bias.double()
    c = sum(terms) + b
    size = sum(t.abs() for t in terms) + b.abs()
    # W fused steps, each off by half a step of a partial sum of at most `size`
    err = W * U32 * size
    out = c
    if act:
        out = silu(c)
        # |silu'| < 1.1; exp of a rounded argument (|c| half steps, plus its own two), sum, reciprocal, product
        err = 1.1 * err + (2 * c.abs() + 10) * U32 * out.abs()
    new = torch.cat([history, u])[T:]
    return out, err, new


def dt(raw, bias, lo=0.0, hi=math.inf):
    """softplus(raw + bias) clamped, and its fp32 error bound."""
    v = raw.double() + (0 if bias is None else bias.double())
    sp = v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))
    # the sum's rounding moves softplus by at most its size; exp, log1p and the last sum add a few half steps
    err = U32 * (v.abs() + 8 * sp)
    return sp.clamp(lo, hi), err


def scan(S, x, B, C, dt, A, D):
    """One sequence through the recurrence: S [H,P,N], x [T,H,P], B/C [T,G,N],
    dt [T,H]; y [T,H,P], the final state, and for each the sum of the sizes of
    the terms behind it."""
    H, G = x.shape[1], B.shape[1]
    S, A, D = S.double().clone(), A.double(), D.double()
    M = S.abs()
    ys, ms = [], []
    for t in range(x.shape[0]):
        a = torch.exp(dt[t].double() * A)[:, None, None]
        xt = x[t].double()
        Bt, Ct = (v[t].double().repeat_interleave(H // G, 0) for v in (B, C))
        add = (dt[t].double()[:, None] * xt)[..., None] * Bt[:, None, :]
        S = a * S + add
        M = a * M + add.abs()
        ys.append((S * Ct[:, None, :]).sum(-1) + D[:, None] * xt)
        ms.append((M * Ct[:, None, :].abs()).sum(-1) + (D[:, None] * xt).abs())
    P = x.shape[2]
    stack = lambda v: torch.stack(v) if v else torch.zeros(0, H, P, dtype=torch.float64)  # noqa: E731
    return stack(ys), S, stack(ms), M


def rms(v, eps):
    return v / (v.pow(2).mean(-1, keepdim=True) + eps).sqrt()


def gated_norm(y, z, w, groups, eps, before):
    y, g = y.double().flatten(1), silu(z.double())
    rows, dim = y.shape
    if before:
        return rms(y.view(rows, groups, -1), eps).view(rows, dim) * w.double() * g
    return rms((y * g).view(rows, groups, -1), eps).view(rows, dim) * w.double()


def add_norm(x, res, w, scale, post, eps):
    x = x.double()
    if post is not None:
        x = rms(x, eps) * post.double()
    r = res.double() + scale * x
    return rms(r, eps) * w.double(), r


def assert_within(got, ref, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = (got - ref).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        t = tol[i] if torch.is_tensor(tol) and tol.dim() else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i]} for {ref[i]} "
                             f"(allowed {float(t):.3e})")
