"""Performance cases of the mixer operators around the replayed recurrence.

An SSM layer of a hybrid model turns the rows of its input projection,
``[z | x B C | dt]``, into the block's output in four operators: the short
causal convolution with the dt transform (single tokens and drafts from a ring
of recent inputs, or packed prompts), the selective scan of packed prompts
into the checkpoint (single tokens go through the replay step), the gated
group norm behind the recurrence, and the residual add with the norms around
the block.  ``run`` computes one pass of one of them, in plain torch operations
(``own = False``) or through the package (``own = True``).
"""
import math
import random

import torch

own = False

P, N, W = 64, 128, 4          # head dim, state dim, convolution width
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one sequence decoding one token: the latency of the call
        dict(name="conv step 1", op="conv_step", dtype="bf16", heads=96, groups=8, rows=1, drafts=1, advance=True),
        # a full serving batch of single tokens on a larger slot pool
        dict(name="conv step 256", op="conv_step", dtype="bf16", heads=96, groups=8, rows=256, drafts=1, advance=True),
        # speculative verification: five positions a sequence, no history moved
        dict(name="conv verify 512x5", op="conv_step", dtype="bf16", heads=128, groups=8, rows=512, drafts=5,
             advance=False),
        # a few short prompts of odd lengths, full precision
        dict(name="conv prompt ragged", op="conv_prompt", dtype="f32", heads=8, groups=1, seqs=7, tokens=701),
        # a prompt batch of a 4B-class layer, continued from earlier pieces
        dict(name="conv prompt 16k", op="conv_prompt", dtype="bf16", heads=96, groups=8, seqs=6, tokens=16384),
        # short full-precision prompts, one after another
        dict(name="scan ragged f32", op="scan", dtype="f32", heads=8, groups=1, seqs=5, tokens=333, y="f32"),
        # one long prompt alone on the card
        dict(name="scan one 16k", op="scan", dtype="bf16", heads=96, groups=8, seqs=1, tokens=16384, y="bf16"),
        # a prompt batch of a 120B-class layer with fp32 outputs
        dict(name="scan ragged 9k", op="scan", dtype="bf16", heads=128, groups=8, seqs=23, tokens=9001, y="f32"),
        # behind the replay step: a full batch of single tokens
        dict(name="gated norm 256", op="gated_norm", dtype="bf16", heads=96, groups=8, rows=256, y="f32", before=False),
        # behind the scan of a prompt batch
        dict(name="gated norm 16k", op="gated_norm", dtype="bf16", heads=96, groups=8, rows=16384, y="bf16",
             before=False),
        # between two blocks, one token
        dict(name="add norm 1", op="add_norm", dtype="bf16", rows=1, dim=4096, res="f32", post=False),
        # between two blocks of a prompt batch, the block's output normed too
        dict(name="add norm 16k", op="add_norm", dtype="bf16", rows=16384, dim=4096, res="bf16", post=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["conv_step", "conv_prompt", "scan", "gated_norm", "add_norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    groups = rng.choice([1, 2, 4, 8])
    heads = groups * _log(rng, 1, 128 // groups)
    most = 96 * 16384 // heads
    if op == "conv_step":
        drafts = rng.choice([1, 1, 2, 5, 8])
        return dict(op=op, dtype=dtype, heads=heads, groups=groups, rows=_log(rng, 1, 512 if dtype == "bf16" else 256),
                    drafts=drafts, advance=drafts == 1)
    if op == "conv_prompt":
        return dict(op=op, dtype=dtype, heads=heads, groups=groups, seqs=_log(rng, 1, 64),
                    tokens=_log(rng, 1, min(16384 if dtype == "bf16" else 8192, most)))
    if op == "scan":
        # plain fp32 matrix work: full-precision inputs stay at a tenth of the largest prompt batch
        return dict(op=op, dtype=dtype, heads=heads, groups=groups, seqs=_log(rng, 1, 48),
                    tokens=_log(rng, 1, min(16384 if dtype == "bf16" else 1600, most)), y=rng.choice(["bf16", "f32"]))
    if op == "gated_norm":
        return dict(op=op, dtype=dtype, heads=heads, groups=groups,
                    rows=_log(rng, 1, min(16384 if dtype == "bf16" else 4096, most)),
                    y=rng.choice(["bf16", "f32"]), before=rng.random() < 0.3)
    dim = _log(rng, 64, 8192)
    return dict(op=op, dtype=dtype, rows=_log(rng, 1, min(16384, 6144 * 4096 // dim)), dim=dim,
                res=rng.choice(["bf16", "f32"]), post=rng.random() < 0.5)


def _channels(case):
    return case["heads"] * P + 2 * case["groups"] * N


def _ring_rows(case):
    return max(W - 1 + case.get("drafts", 1), 2 * (W - 1))


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "add_norm":
        n = case["rows"] * case["dim"]
        return {"bytes": n * (2 * e + 2 * BYTES[case["res"]]) + 4 * case["dim"] * (1 + case["post"]),
                "flops": n * (10 if case["post"] else 6)}
    H, G = case["heads"], case["groups"]
    if case["op"] == "gated_norm":
        n = case["rows"] * H * P
        return {"bytes": n * (BYTES[case["y"]] + 2 * e) + 4 * H * P, "flops": 10 * n}
    c = _channels(case)
    if case["op"] == "conv_step":
        t = case["rows"] * case["drafts"]
        return {"bytes": e * (3 * t * c + case["rows"] * (W - 1) * c + 2 * t * H) + 4 * (W + 1) * c,
                "flops": t * c * (2 * W + 6)}
    t = case["tokens"]
    n = min(case["seqs"], t)
    if case["op"] == "conv_prompt":
        return {"bytes": e * (2 * t * c + 2 * n * (W - 1) * c + 2 * t * H) + 4 * (W + 1) * c,
                "flops": t * c * (2 * W + 6)}
    return {"bytes": t * (e * (c + H) + BYTES[case["y"]] * H * P) + 8 * n * H * P * N, "flops": 4 * t * H * P * N}


# ------------------------------------------------------------------ inputs --

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _lengths(case, seed):
    """Prompt lengths: ragged, some of a single token, now and then none."""
    n, total = case["seqs"], case["tokens"]
    r = random.Random(seed)
    cuts = sorted(r.randint(0, total) for _ in range(n - 1))
    if n >= 3:
        cuts[1] = min(cuts[0] + 1, total)
        cuts.sort()
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _inputs(case, seed):
    g = _gen(seed)
    dtype = DTYPES[case["dtype"]]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {}
    if case["op"] == "add_norm":
        s["x"] = rand(case["rows"], case["dim"]).to(dtype)
        s["res"] = (2 * rand(case["rows"], case["dim"])).to(DTYPES[case["res"]])
        s["weight"] = 1 + 0.1 * rand(case["dim"])
        s["post"] = 0.5 + 0.1 * rand(case["dim"]) if case["post"] else None
        s["scale"] = 0.22
        s["out"] = torch.empty_like(s["x"])
        s["res_out"] = torch.empty_like(s["res"])
        return s
    H, G = case["heads"], case["groups"]
    c = _channels(case)
    if case["op"] == "gated_norm":
        rows = rand(case["rows"], H * P + c + H).to(dtype)    # the input projection's rows; z comes first
        s["z"] = rows[:, :H * P]
        s["y"] = (3 * rand(case["rows"], H * P)).to(DTYPES[case["y"]])
        s["weight"] = 1 + 0.1 * rand(H * P)
        s["out"] = torch.empty(case["rows"], H * P, dtype=dtype, device="cuda")
        return s
    n = case["rows"] if "rows" in case else case["seqs"]
    S = n + (n + 3) // 4
    s["slots"] = torch.randperm(S, generator=g, device="cuda")[:n].to(torch.int32)
    if "seqs" in case:
        s["cu"] = torch.tensor([0] + _lengths(case, seed)).cumsum(0).to(torch.int32).cuda()
    if case["op"] == "scan":
        t = case["tokens"]
        act = lambda v: (v * torch.sigmoid(v)).to(dtype)  # noqa: E731
        s["x"] = act(rand(t, H, P))
        s["B"] = act(rand(t, G, N))
        s["C"] = act(rand(t, G, N))
        z = rand(t, H) - 2
        s["dt"] = torch.log1p(torch.exp(z)).to(dtype)
        s["A"] = -torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(16.0))
        s["D"] = rand(H)
        s["state"] = 0.1 * rand(S, H, P, N)
        s["y"] = torch.empty(t, H, P, dtype=DTYPES[case["y"]], device="cuda")
        return s
    t = case["rows"] * case["drafts"] if "rows" in case else case["tokens"]
    s["rows"] = rand(t, H * P + c + H).to(dtype)              # the input projection's rows: z, then x B C, then dt
    s["u"] = s["rows"][:, H * P:H * P + c]
    s["dt_raw"] = s["rows"][:, H * P + c:]
    s["weight"] = (torch.rand(c, W, generator=g, device="cuda") * 2 - 1) / math.sqrt(W)
    s["bias"] = 0.1 * rand(c)
    s["dt_bias"] = rand(H) - 2
    s["ring"] = rand(S, _ring_rows(case), c).to(dtype)
    s["head"] = torch.randint(0, _ring_rows(case), (S,), generator=g, device="cuda", dtype=torch.int32)
    s["out"] = (torch.empty(t, H, P, dtype=dtype, device="cuda"), torch.empty(t, G, N, dtype=dtype, device="cuda"),
                torch.empty(t, G, N, dtype=dtype, device="cuda"), torch.empty(t, H, dtype=dtype, device="cuda"))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if "drafts" in case and not case["advance"]:
        n, d = case["rows"], case["drafts"]
        s["u"], s["dt_raw"] = (s[k].unflatten(0, (n, d)) for k in ("u", "dt_raw"))
        s["out"] = tuple(o.unflatten(0, (n, d)) for o in s["out"])
    if own:   # the layer objects that a user's program keeps, over this state's buffers
        import state_space_recurrence_amd as rs
        s["rs"] = rs
        if case["op"].startswith("conv"):
            layer = rs.ConvState(s["ring"].shape[0], case["heads"], case["groups"], s["weight"], s["bias"], s["dt_bias"],
                                 max_draft=case.get("drafts", 1), in_dtype=DTYPES[case["dtype"]])
            layer.ring.copy_(s["ring"])
            layer.head.copy_(s["head"])
            s["layer"], s["ring"], s["head"] = layer, layer.ring, layer.head
        elif case["op"] == "scan":
            layer = rs.LayerState(s["state"].shape[0], case["heads"], case["groups"], s["A"], s["D"],
                                  in_dtype=DTYPES[case["dtype"]])
            rs.load_checkpoint(layer, s["state"])
            s["layer"], s["state"] = layer, layer.ckpt
    return s


# -------------------------------------------------------------- plain forms --

def _conv_out(s, taps, dt_raw, dtype, lead, H, G):
    """The convolution of gathered taps [t, W, channels], split into x, B, C, and dt."""
    v = (taps.float() * s["weight"].t()).sum(-2) + s["bias"]
    v = (v * torch.sigmoid(v)).to(dtype)
    x, B, C = v.split([H * P, G * N, G * N], -1)
    d = dt_raw.float() + s["dt_bias"]
    d = d.clamp(min=0) + torch.log1p(torch.exp(-d.abs()))
    return (x.reshape(*lead, H, P), B.reshape(*lead, G, N), C.reshape(*lead, G, N), d.to(dtype))


def _plain_conv_step(s, case):
    u, ring, head, slots = s["u"], s["ring"], s["head"], s["slots"].long()
    lead, dtype = u.shape[:-1], u.dtype
    u = u.reshape(case["rows"], case["drafts"], -1)
    R = ring.shape[1]
    at = head[slots].long()[:, None]
    back = (at - (W - 1) + torch.arange(W - 1, device="cuda")) % R
    line = torch.cat([ring[slots[:, None], back], u], 1)                       # [rows, W-1+T, channels]
    taps = line.unfold(1, W, 1).transpose(-1, -2).reshape(*lead, W, -1)
    got = _conv_out(s, taps, s["dt_raw"], dtype, lead, case["heads"], case["groups"])
    ring[slots[:, None], (at + torch.arange(case["drafts"], device="cuda")) % R] = u
    if case["advance"]:
        head[slots] = ((at[:, 0] + 1) % R).to(torch.int32)
    return got


def _plain_conv_prompt(s, case):
    u, ring, head, slots, cu = s["u"], s["ring"], s["head"], s["slots"].long(), s["cu"].long()
    t, n, R = u.shape[0], slots.numel(), ring.shape[1]
    lens = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), lens, output_size=t)
    back = (head[slots].long()[:, None] - (W - 1) + torch.arange(W - 1, device="cuda")) % R
    line = torch.cat([ring[slots[:, None], back].reshape(n * (W - 1), -1), u])  # histories, then the tokens
    at = torch.arange(t, device="cuda")[:, None] - (W - 1) + torch.arange(W, device="cuda")
    before = at - cu[seq][:, None]                                              # negative: taken from the history
    index = torch.where(before < 0, seq[:, None] * (W - 1) + W - 1 + before, n * (W - 1) + at)
    got = _conv_out(s, line[index], s["dt_raw"], u.dtype, (t,), case["heads"], case["groups"])
    m = lens.clamp(max=W - 1)
    k = torch.arange(W - 1, device="cuda")
    keep = k < m[:, None]
    rows = (head[slots].long()[:, None] + k) % R
    source = (cu[1:] - m)[:, None] + k
    ring[slots[:, None].expand(n, W - 1)[keep], rows[keep]] = u[source[keep]]
    head[slots] = ((head[slots].long() + m) % R).to(torch.int32)
    return got


def _plain_scan(s, case):
    """Chunks of 64 tokens: masked products inside a chunk, chunk states joined over each prompt."""
    x, B, C, dt, cu, slots = s["x"], s["B"], s["C"], s["dt"], s["cu"].long(), s["slots"].long()
    Q, t, n = 64, x.shape[0], slots.numel()
    H, G = case["heads"], case["groups"]
    lens = cu[1:] - cu[:-1]
    chunks = (lens + Q - 1) // Q
    first = chunks.cumsum(0) - chunks
    nc = int((t + Q - 1) // Q + n)                                              # at least the chunks in use
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), lens, output_size=t)
    place = first[seq] * Q + torch.arange(t, device="cuda") - cu[seq]           # a token's place in padded chunks
    pad = lambda v: v.new_zeros(nc * Q, *v.shape[1:]).index_copy(0, place, v).unflatten(0, (nc, Q))  # noqa: E731
    xf, Bf, Cf, df = (pad(v.float()) for v in (x, B, C, dt))
    grow = (df.double() * s["A"].double()).cumsum(1).permute(0, 2, 1)           # [chunk, head, token]
    chunk = torch.arange(nc, device="cuda")
    owner = (torch.searchsorted(first + chunks, chunk, right=True)).clamp(max=n - 1)
    rel = (grow[..., :, None] - grow[..., None, :]).float()
    low = torch.ones(Q, Q, dtype=torch.bool, device="cuda").tril()
    gram = torch.matmul(Cf.transpose(1, 2), Bf.permute(0, 2, 3, 1).contiguous())  # [chunk, group, t, j]
    gram = gram.repeat_interleave(H // G, 1) * torch.exp(rel.masked_fill(~low, -math.inf))
    xd = (xf * df[..., None]).transpose(1, 2).contiguous()                      # [chunk, head, j, p]
    y = torch.matmul(gram, xd)
    last = grow[..., -1:]
    weighed = xd * torch.exp((last - grow).float())[..., None]
    Bh = Bf.transpose(1, 2).repeat_interleave(H // G, 1).contiguous()
    ends = torch.matmul(weighed.transpose(-1, -2).contiguous(), Bh)             # each chunk's own end state
    total = last[..., 0].cumsum(0)                                              # [chunk, head], over all chunks
    span = (total[:, None] - last[:, None, :, 0] - total[None]).permute(2, 0, 1)  # [head, to, from]: decay between
    same = (owner[:, None] == owner[None]) & (chunk[:, None] > chunk[None])
    join = torch.exp(span.masked_fill(~same, -math.inf).float())
    start = torch.matmul(join, ends.transpose(0, 1).reshape(H, nc, P * N))
    base = total[first.clamp(max=nc - 1)] - last[first.clamp(max=nc - 1), :, 0]  # decay sums before each prompt
    state = s["state"]
    old = state[slots].reshape(n, H, P * N)
    lead = torch.exp((total - last[..., 0] - base[owner]).float())              # from the prompt's start to the chunk's
    start = (start.transpose(0, 1) + lead[..., None] * old[owner]).unflatten(-1, (P, N))
    Ch = Cf.transpose(1, 2).repeat_interleave(H // G, 1).contiguous()
    y = y + torch.exp(grow.float())[..., None] * torch.matmul(Ch, start.transpose(-1, -2).contiguous())
    y = y.transpose(1, 2) + s["D"][:, None] * xf
    end = (first + chunks - 1).clamp(min=0)
    done = torch.exp(last[end, :, 0].float())[..., None, None] * start[end] + ends[end]
    state[slots] = torch.where((lens > 0)[:, None, None, None], done, state[slots])
    return y.flatten(0, 1)[place].to(s["y"].dtype)


def _plain_gated_norm(s, case):
    y, z, G = s["y"].float(), s["z"].float(), case["groups"]
    gate = z * torch.sigmoid(z)
    v = y if case["before"] else y * gate
    parts = v.unflatten(-1, (G, -1))
    v = (parts * torch.rsqrt(parts.square().mean(-1, keepdim=True) + EPS)).flatten(-2) * s["weight"]
    return (v * gate if case["before"] else v).to(s["out"].dtype)


def _plain_add_norm(s, case):
    x, res = s["x"].float(), s["res"].float()
    if case["post"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["post"]
    res = res + s["scale"] * x
    out = res * torch.rsqrt(res.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    return out.to(s["out"].dtype), res.to(s["res"].dtype)


def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        rs = s["rs"]
        if op == "conv_step":
            call = rs.conv_step if case["advance"] else rs.conv_verify
            x, B, C, dt = call(s["layer"], s["u"], s["dt_raw"], out=s["out"], slots=s["slots"])
        elif op == "conv_prompt":
            x, B, C, dt = rs.conv_prefill(s["layer"], s["u"], s["dt_raw"], s["cu"], out=s["out"], slots=s["slots"])
        elif op == "scan":
            y = rs.prefill_packed(s["layer"], s["x"], s["B"], s["C"], s["dt"], s["cu"], y=s["y"], slots=s["slots"])
        elif op == "gated_norm":
            return rs.gated_norm(s["y"], s["z"], s["weight"], groups=case["groups"], eps=EPS,
                                 norm_before_gate=case["before"], out=s["out"])
        else:
            return rs.add_norm(s["x"], s["res"], s["weight"], scale=s["scale"], post_weight=s["post"], eps=EPS,
                               out=s["out"], residual_out=s["res_out"])
    elif op == "conv_step":
        x, B, C, dt = _plain_conv_step(s, case)
    elif op == "conv_prompt":
        x, B, C, dt = _plain_conv_prompt(s, case)
    elif op == "scan":
        y = _plain_scan(s, case)
    elif op == "gated_norm":
        return _plain_gated_norm(s, case)
    else:
        return _plain_add_norm(s, case)
    if op == "scan":
        return {"y": y, "state": s["state"]}
    return {"x": x, "B": B, "C": C, "dt": dt, "ring": s["ring"], "head": s["head"]}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """The same pass from the operators' definitions in 64 bits: token by token, sequence by sequence."""
    s = _inputs(case, seed)
    f = lambda v: v.double()  # noqa: E731
    rms = lambda v: v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt()  # noqa: E731
    silu = lambda v: v / (1 + torch.exp(-v))  # noqa: E731
    if case["op"] == "add_norm":
        x = f(s["x"])
        r = f(s["res"]) + s["scale"] * (rms(x) * f(s["post"]) if case["post"] else x)
        return rms(r) * f(s["weight"]), r
    if case["op"] == "gated_norm":
        y, gate, shape = f(s["y"]), silu(f(s["z"])), (case["rows"], case["groups"], -1)
        if case["before"]:
            return rms(y.view(shape)).view(case["rows"], -1) * f(s["weight"]) * gate
        return rms((y * gate).view(shape)).view(case["rows"], -1) * f(s["weight"])
    slots = s["slots"].tolist()
    H, G = case["heads"], case["groups"]
    if case["op"] == "scan":
        cu = s["cu"].tolist()
        lens = [b - a for a, b in zip(cu, cu[1:])]
        S, L = f(s["state"]), max(lens)
        y = torch.zeros(case["tokens"], H, P, dtype=torch.float64, device="cuda")
        order = sorted(range(len(lens)), key=lambda i: -lens[i])                # the longest first
        starts = torch.tensor([cu[i] for i in order], device="cuda")
        cur = S[torch.tensor([slots[i] for i in order], device="cuda")]
        live = [sum(v > t for v in lens) for t in range(L)]
        x, B, C, dt = f(s["x"]), f(s["B"]), f(s["C"]), f(s["dt"])
        A, D = f(s["A"]), f(s["D"])
        for t in range(L):                                                      # the recurrence, one token at a time
            k = live[t]
            at = starts[:k] + t
            d = dt[at]
            Bt, Ct = (v[at].repeat_interleave(H // G, 1) for v in (B, C))
            xt = x[at]
            now = cur[:k]
            now.mul_(torch.exp(d * A)[..., None, None]).addcmul_((d[..., None] * xt)[..., None], Bt[:, :, None, :])
            y[at] = torch.matmul(now, Ct[..., None])[..., 0] + D[:, None] * xt
        for j, i in enumerate(order):
            S[slots[i]] = cur[j]
        return {"y": y, "state": S}
    ring, head, u, d = f(s["ring"]), s["head"], f(s["u"]), f(s["dt_raw"])
    R, heads = ring.shape[1], head.tolist()
    n = len(slots)
    T = case.get("drafts")
    cu = s["cu"].tolist() if T is None else [i * T for i in range(n + 1)]
    w, out = f(s["weight"]), torch.empty_like(u)
    for i, slot in enumerate(slots):
        a, b = cu[i], cu[i + 1]
        h = heads[slot]
        past = [ring[slot, (h - k) % R] for k in range(W - 1, 0, -1)]
        line = torch.cat([torch.stack(past), u[a:b]])
        out[a:b] = sum(line[k:k + b - a] * w[:, k] for k in range(W)) + f(s["bias"])
        if T is None:
            m = min(b - a, W - 1)
            for k in range(m):
                ring[slot, (h + k) % R] = u[b - m + k]
            head[slot] = (h + m) % R
        else:
            for k in range(T):
                ring[slot, (h + k) % R] = u[a + k]
            if case["advance"]:
                head[slot] = (h + 1) % R
    out = silu(out)
    lead = (n, T) if T is not None and not case["advance"] else (u.shape[0],)
    x, B, C = out.split([H * P, G * N, G * N], -1)
    dt = torch.log(1 + torch.exp(d + f(s["dt_bias"])))
    return {"x": x.reshape(*lead, H, P), "B": B.reshape(*lead, G, N), "C": C.reshape(*lead, G, N),
            "dt": dt.reshape(*lead, H), "ring": ring, "head": head}
