"""Performance cases of the projections around a mixer and of the 8-bit operands they take.

A block's matrix products read normed rows and weights, and end in a bias, an
activation and the residual: ``linear``.  With bf16 operands they are bound by
the weights' bytes (few rows) or the matrix cores (many); in 8 bits both halve.
The 8-bit form is OCP MX: E4M3 codes with one power-of-two scale (E8M0) per 32
consecutive elements of a row.  The norms in front of the products write it
directly (``add_norm_mx``, ``gated_norm_mx``), ``quantize_mx`` makes it of weights
and other rows, and a product can write it for the next one.  ``run`` computes one
pass of one of them, in plain torch operations (``own = False``) or through the
package (``own = True``).
"""
import math

import torch

own = False

P, N, BLOCK = 64, 128, 32     # head dim, state dim, elements that share a scale
EPS = 1e-5
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "mx": E4M3}
BYTES = {"bf16": 2, "f32": 4, "mx": 1 + 1 / BLOCK}


def _projection(heads, groups):
    """Columns of an input projection: z, x, B, C and dt."""
    return 2 * heads * P + 2 * groups * N + heads


def listed():
    wide = _projection(96, 8)
    return [
        # one decoded token through the input projection of a 4B-class layer: the weights' bytes
        dict(name="in projection 1", op="linear", x="bf16", rows=1, n_out=wide, n_in=4096, bias=False, act="none",
             res="none", out="bf16"),
        # a full batch of single tokens, 8-bit weights and rows
        dict(name="in projection 256 mx", op="linear", x="mx", rows=256, n_out=wide, n_in=4096, bias=False, act="none",
             res="none", out="bf16"),
        # the input projection of a prompt batch, 8-bit weights and rows
        dict(name="in projection 16k mx", op="linear", x="mx", rows=16384, n_out=wide, n_in=4096, bias=False,
             act="none", res="none", out="bf16"),
        # the output projection of a prompt batch, added to the residual stream
        dict(name="out projection 16k", op="linear", x="bf16", rows=16384, n_out=4096, n_in=6144, bias=False, act="none",
             res="f32", out="f32"),
        # a feed-forward part of a short prompt: its wider rows leave in 8 bits for the product behind
        dict(name="up projection 333 mx", op="linear", x="mx", rows=333, n_out=16384, n_in=4096, bias=True, act="gelu",
             res="none", out="mx"),
        # a small layer's rows of odd sizes, every part of the epilogue
        dict(name="odd product", op="linear", x="bf16", rows=37, n_out=1543, n_in=251, bias=True, act="silu", res="bf16",
             out="f32"),
        # one token between two blocks
        dict(name="add norm mx 1", op="add_norm", x="bf16", rows=1, dim=4096, res="f32", add=True, post=False),
        # a prompt batch between two blocks
        dict(name="add norm mx 16k", op="add_norm", x="bf16", rows=16384, dim=4096, res="f32", add=True, post=False),
        # behind the replay step: a full batch of single tokens
        dict(name="gated norm mx 256", op="gated_norm", x="bf16", heads=96, groups=8, rows=256, y="f32", before=False),
        # behind the scan of a prompt batch
        dict(name="gated norm mx 16k", op="gated_norm", x="bf16", heads=96, groups=8, rows=16384, y="bf16",
             before=False),
        # a few rows of a small layer, full precision
        dict(name="quantize 45", op="quantize", x="f32", rows=45, dim=1056, wide=1056),
        # the weights of an input projection, as they are loaded
        dict(name="quantize weights", op="quantize", x="bf16", rows=wide, dim=4096, wide=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "add_norm", "gated_norm", "quantize"])
    if op == "linear":
        x = rng.choice(["bf16", "mx"])
        out = rng.choice(["bf16", "bf16", "f32", "mx"])
        n_in = BLOCK * _log(rng, 2, 256) if x == "mx" or rng.random() < 0.8 else _log(rng, 50, 4000)
        n_out = BLOCK * _log(rng, 2, 580) if out == "mx" or rng.random() < 0.7 else _log(rng, 50, 18560)
        most = 16384 * 14432 * 4096 // (n_in * n_out)
        return dict(op=op, x=x, rows=_log(rng, 1, max(1, min(16384, most))), n_out=n_out, n_in=n_in,
                    bias=rng.random() < 0.5, act=rng.choice(["none", "none", "silu", "gelu", "relu2"]),
                    res=rng.choice(["none", "none", "bf16", "f32"]), out=out)
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "add_norm":
        dim, add = BLOCK * _log(rng, 2, 256), rng.random() < 0.7
        return dict(op=op, x=x, rows=_log(rng, 1, min(16384, 16384 * 6144 // dim)), dim=dim, res=rng.choice(["bf16", "f32"]),
                    add=add, post=add and rng.random() < 0.4)
    if op == "gated_norm":
        groups = rng.choice([1, 2, 4, 8])
        heads = groups * _log(rng, 1, 128 // groups)
        return dict(op=op, x=x, heads=heads, groups=groups, rows=_log(rng, 1, min(16384, 16384 * 96 // heads)),
                    y=rng.choice(["bf16", "f32"]), before=rng.random() < 0.3)
    dim = BLOCK * _log(rng, 1, 256)
    return dict(op=op, x=x, rows=_log(rng, 1, min(18560, 16384 * 6144 // dim)), dim=dim,
                wide=dim + rng.choice([0, 0, 8, 40]))


def work(case):
    op, e = case["op"], BYTES[case["x"]]
    if op == "linear":
        m, n, k = case["rows"], case["n_out"], case["n_in"]
        res = 0 if case["res"] == "none" else BYTES[case["res"]]
        return {"bytes": (m + n) * k * e + m * n * (BYTES[case["out"]] + res) + 4 * n * case["bias"],
                "flops": 2 * m * n * k}
    if op == "add_norm":
        n = case["rows"] * case["dim"]
        moved = BYTES["mx"] + BYTES[case["res"]] + (e + BYTES[case["res"]] if case["add"] else 0)
        return {"bytes": n * moved + 4 * case["dim"] * (1 + case["post"]), "flops": n * (12 if case["post"] else 8)}
    if op == "gated_norm":
        dim = case["heads"] * P
        return {"bytes": case["rows"] * dim * (BYTES[case["y"]] + e + BYTES["mx"]) + 4 * dim,
                "flops": 12 * case["rows"] * dim}
    n = case["rows"] * case["dim"]
    return {"bytes": n * (e + BYTES["mx"]), "flops": 2 * n}


# ------------------------------------------------------------------ inputs --

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _plain_quantize(v):
    """Codes and scales of the rows of v (fp32): the smallest power of two that keeps a block within 448."""
    blocks = v.unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(blocks.abs().amax(-1) / 448)
    e = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
    e = torch.where(m == 0, -127, e)
    codes = torch.ldexp(blocks, -e[..., None]).to(E4M3).flatten(-2)
    return codes, torch.ldexp(torch.ones_like(m), e).to(E8M0)


def _values(pair):
    """The values that codes and scales stand for, in fp32."""
    codes, scales = pair
    return (codes.float().unflatten(-1, (-1, BLOCK)) * scales.float()[..., None]).flatten(-2)


def _inputs(case, seed):
    g = _gen(seed)
    op, dtype = case["op"], DTYPES[case["x"]]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {}
    if op == "linear":
        m, n, k = case["rows"], case["n_out"], case["n_in"]
        x, w = rand(m, k) * (1 + rand(k).square()), rand(n, k) / math.sqrt(k)      # some channels are larger
        s["x"], s["w"] = (_plain_quantize(v) if case["x"] == "mx" else v.to(dtype) for v in (x, w))
        s["bias"] = 0.1 * rand(n) if case["bias"] else None
        s["res"] = None if case["res"] == "none" else (2 * rand(m, n)).to(DTYPES[case["res"]])
        s["scale"] = 0.22 if case["res"] != "none" else 1.0
        if case["out"] == "mx":
            s["out"] = (torch.empty(m, n, dtype=E4M3, device="cuda"), torch.empty(m, n // BLOCK, dtype=E8M0, device="cuda"))
        else:
            s["out"] = torch.empty(m, n, dtype=DTYPES[case["out"]], device="cuda")
        return s
    rows = case["rows"]
    dim = case["heads"] * P if op == "gated_norm" else case["dim"]
    s["out"] = (torch.empty(rows, dim, dtype=E4M3, device="cuda"), torch.empty(rows, dim // BLOCK, dtype=E8M0, device="cuda"))
    if op == "quantize":
        s["x"] = (rand(rows, case["wide"]) * torch.exp(rand(case["wide"]))).to(dtype)[:, :dim]
        return s
    s["weight"] = 1 + 0.1 * rand(dim)
    if op == "gated_norm":
        line = rand(rows, _projection(case["heads"], case["groups"])).to(dtype)     # the input projection's rows; z comes first
        s["z"] = line[:, :dim]
        s["y"] = (3 * rand(rows, dim)).to(DTYPES[case["y"]])
        return s
    s["x"] = rand(rows, dim).to(dtype) if case["add"] else None
    s["res"] = (2 * rand(rows, dim)).to(DTYPES[case["res"]])
    s["post"] = 0.5 + 0.1 * rand(dim) if case["post"] else None
    s["scale"] = 0.22
    s["res_out"] = torch.empty_like(s["res"]) if case["add"] else None
    return s


def prepare(case, seed):
    return dict(_inputs(case, seed), case=case)


# -------------------------------------------------------------- plain forms --

def _rms(v):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _plain_linear(s, case):
    x, w = (_values(v) if case["x"] == "mx" else v.float() for v in (s["x"], s["w"]))
    v = torch.matmul(x, w.t())
    if case["bias"]:
        v = v + s["bias"]
    if case["act"] == "silu":
        v = v * torch.sigmoid(v)
    elif case["act"] == "gelu":
        v = 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    elif case["act"] == "relu2":
        v = v.clamp(min=0).square()
    v = s["scale"] * v
    if case["res"] != "none":
        v = s["res"].float() + v
    return _plain_quantize(v) if case["out"] == "mx" else v.to(DTYPES[case["out"]])


def _plain_gated_norm(s, case):
    y, z, G = s["y"].float(), s["z"].float(), case["groups"]
    gate = z * torch.sigmoid(z)
    if case["before"]:
        v = _rms(y.unflatten(-1, (G, -1))).flatten(-2) * s["weight"] * gate
    else:
        v = _rms((y * gate).unflatten(-1, (G, -1))).flatten(-2) * s["weight"]
    return _plain_quantize(v)


def _plain_add_norm(s, case):
    r = s["res"].float()
    if case["add"]:
        x = s["x"].float()
        r = r + s["scale"] * (_rms(x) * s["post"] if case["post"] else x)
    out = _plain_quantize(_rms(r) * s["weight"])
    return (out, r.to(s["res"].dtype)) if case["add"] else (out,)


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        import state_space_recurrence_amd as rs
        if op == "linear":
            return rs.linear(s["x"], s["w"], s["bias"], activation=None if case["act"] == "none" else case["act"],
                             residual=s["res"], scale=s["scale"], out=s["out"])
        if op == "quantize":
            return rs.quantize_mx(s["x"], out=s["out"])
        if op == "gated_norm":
            return rs.gated_norm_mx(s["y"], s["z"], s["weight"], groups=case["groups"], eps=EPS,
                                    norm_before_gate=case["before"], out=s["out"])
        out, res = rs.add_norm_mx(s["x"], s["res"], s["weight"], scale=s["scale"], post_weight=s["post"], eps=EPS,
                                  out=s["out"], residual_out=s["res_out"])
        return (out, res) if case["add"] else (out,)
    if op == "linear":
        return _plain_linear(s, case)
    if op == "quantize":
        return _plain_quantize(s["x"].float())
    return _plain_gated_norm(s, case) if op == "gated_norm" else _plain_add_norm(s, case)


# ------------------------------------------------------------------- exact --

def _exact_quantize(v):
    """From the definitions in 64 bits: the least power of two with amax <= 448 of it, and codes to the nearest even
    of a grid of 8 steps per octave, the lowest octave at 2^-6 (below it the steps stay)."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)
    top = b.abs().max(-1).values
    power = torch.ceil(torch.log2(top / 448))
    for near in (-1, 0, 1):                                   # the logarithm may be off by a little: the least that holds
        fits = torch.exp2(power + near) * 448 >= top
        power = torch.where(fits & (torch.exp2(power) * 448 < top), power + near, power)
        less = torch.exp2(power - 1) * 448 >= top
        power = torch.where(less, power - 1, power)
    power = power.clamp(-127, 127)
    u = b / torch.exp2(power)[..., None]
    octave = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -12))).clamp(min=-6)
    octave = torch.where(torch.exp2(octave) > u.abs().clamp(min=2.0 ** -6), octave - 1, octave)
    octave = torch.where(torch.exp2(octave + 1) <= u.abs(), octave + 1, octave)
    step = torch.exp2(octave - 3)
    return (torch.round(u / step) * step).reshape(v.shape), torch.exp2(power)


def exact(case, seed):
    """The same pass from the operators' definitions in 64 bits."""
    s, op = _inputs(case, seed), case["op"]
    f = lambda v: v.double()  # noqa: E731
    norm = lambda v: v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt()  # noqa: E731
    if op == "quantize":
        return _exact_quantize(f(s["x"]))
    if op == "gated_norm":
        y, gate, shape = f(s["y"]), f(s["z"]) / (1 + torch.exp(-f(s["z"]))), (case["rows"], case["groups"], -1)
        v = norm((y if case["before"] else y * gate).view(shape)).view(case["rows"], -1) * f(s["weight"])
        return _exact_quantize(v * gate if case["before"] else v)
    if op == "add_norm":
        r = f(s["res"])
        if case["add"]:
            r = r + s["scale"] * (norm(f(s["x"])) * f(s["post"]) if case["post"] else f(s["x"]))
        out = _exact_quantize(norm(r) * f(s["weight"]))
        return (out, r) if case["add"] else (out,)
    if case["x"] == "mx":
        x, w = (f(c) * f(e).repeat_interleave(BLOCK, -1) for c, e in (s["x"], s["w"]))
    else:
        x, w = f(s["x"]), f(s["w"])
    v = torch.matmul(x, w.t().contiguous())
    if case["bias"]:
        v += f(s["bias"])
    if case["act"] == "silu":
        v = v / (1 + torch.exp(-v))
    elif case["act"] == "gelu":
        v = v * torch.special.erfc(-v / math.sqrt(2)) / 2
    elif case["act"] == "relu2":
        v = torch.where(v > 0, v * v, 0.0)
    if case["res"] != "none":
        v = f(s["res"]) + s["scale"] * v
    return _exact_quantize(v) if case["out"] == "mx" else v
