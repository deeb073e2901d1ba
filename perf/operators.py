"""Cases of the operators that stand around the gated delta rule in a recurrent layer: the short
causal convolution in front of it, the gated linear recurrence beside it and the group norm
behind it.

``own`` chooses what ``run`` calls: elementary torch operations in 32 bits or more (the plain
forms), or the library's entry points.  ``exact`` is the operators' definition in 64 bits, token
by token and sequence by sequence.

Every operator sees its tokens packed: rows of one length are sequences of that length.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ---------------------------------------------------------------------------------

def listed():
    return [
        # training step of a recurrent layer: 16 heads of 128, each token with its write gate
        dict(name="scan_fwd_train", op="scan_fwd", B=8, T=4096, D=2048, io="bf16", write="gate"),
        # one long document, continued from a state (prefill in pieces)
        dict(name="scan_fwd_long", op="scan_fwd", B=1, T=131072, D=1024, io="bf16", write="plain",
             h0=True),
        # ragged short sequences in 32 bits, scanned backwards (bidirectional mixers), odd width
        dict(name="scan_fwd_ragged_f32", op="scan_fwd", n=37, T=5003, D=1000, io="f32",
             write="tied", h0=True, reverse=True),
        # backward of the training step
        dict(name="scan_bwd_train", op="scan_bwd", B=8, T=4096, D=2048, io="bf16", write="gate"),
        # backward over packed documents with states handed on, 12 heads of 64
        dict(name="scan_bwd_packed", op="scan_bwd", n=64, T=49157, D=768, io="bf16",
             write="plain", h0=True),
        # one token for each of 256 served sequences, 32 heads of 128
        dict(name="scan_step", op="scan_step", N=256, D=4096, io="bf16", write="plain"),
        # prefill of 64 packed prompts, the q, k and v channels of a layer together
        dict(name="conv_fwd_packed", op="conv_fwd", n=64, T=65537, D=4096, W=4, io="bf16",
             act="silu", state=True),
        # its backward in a training step
        dict(name="conv_bwd_train", op="conv_bwd", B=8, T=4096, D=2048, W=4, io="bf16",
             act="silu", bias=True),
        # the smallest call: one token for each of 8 served sequences
        dict(name="conv_step", op="conv_step", N=8, D=4096, W=4, io="bf16", act="silu"),
        # the norm of every token's heads, gated, behind the recurrence in training
        dict(name="norm_fwd_train", op="norm_fwd", B=8, T=4096, H=16, d=128, io="bf16",
             per="token", center=False, gate=True, act="silu"),
        # its backward
        dict(name="norm_bwd_train", op="norm_bwd", B=8, T=4096, H=16, d=128, io="bf16",
             per="token", center=False, gate=True, act="silu"),
        # group norm of whole segments behind a bidirectional mixer: 16 segments, 12 heads of 64
        dict(name="norm_bwd_segments", op="norm_bwd", n=16, T=32768, H=12, d=64, io="bf16",
             per="sequence", center=True, gate=False, act="silu", bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_bwd", "scan_step", "conv_fwd", "conv_bwd", "conv_step",
                     "norm_fwd", "norm_bwd"])
    c = dict(op=op, io=rng.choice(["bf16", "bf16", "f32"]))
    most = 40_000_000  # elements of one tensor
    if op.startswith("norm"):
        c["H"], c["d"] = _log(rng, 1, 32), rng.choice([32, 48, 64, 96, 128, 200, 256])
        D = c["H"] * c["d"]
        c.update(per=rng.choice(["token", "sequence"]), center=rng.random() < 0.5,
                 gate=rng.random() < 0.5, act=rng.choice(["silu", "silu", "sigmoid", "none"]),
                 bias=rng.random() < 0.5)
    else:
        D = c["D"] = rng.choice([1, 2, 8, 8, 16]) * _log(rng, 48, 320)
    if op.startswith("scan"):
        c["write"] = rng.choice(["plain", "gate", "tied"])
    if op.startswith("conv"):
        c.update(W=rng.choice([2, 3, 4, 4]), act=rng.choice(["silu", "silu", "none"]),
                 bias=rng.random() < 0.5)
    if op.endswith("step"):
        c["N"] = _log(rng, 1, 512)
        return c
    T = _log(rng, 64, min(131072, most // D))
    if rng.random() < 0.5:
        c["B"] = min(T, _log(rng, 1, 32))
        c["T"] = T // c["B"]
    else:
        c["n"], c["T"] = min(T, _log(rng, 1, 128)), T
    if not op.startswith("norm"):
        c["reverse"] = rng.random() < 0.25
        c["h0" if op.startswith("scan") else "state"] = rng.random() < 0.5
    return c


# ---- inputs ------------------------------------------------------------------------------------

def _layout(c, seed):
    """(rows, tokens a row, cu_seqlens or None, starts and ends of every sequence as a list)."""
    if "n" not in c:
        B, T = c["B"], c["T"]
        return B, T, None, [i * T for i in range(B + 1)]
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, c["T"] + 1, (c["n"] - 1,), generator=g).sort().values
    cu = torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([c["T"]])])
    return 1, c["T"], cu.to(torch.int32).cuda(), cu.tolist()


def prepare(c, seed):
    op, io = c["op"], DT[c["io"]]
    gen = torch.Generator("cuda").manual_seed(seed)

    def rn(*shape, dtype=io, mean=0.0, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    s = dict(c=c, op=op)
    if op.endswith("step"):
        N, D = c["N"], c["D"]
        if op == "scan_step":
            s.update(v=rn(N, D), g=-torch.nn.functional.softplus(rn(N, D, mean=-2.0)),
                     beta=torch.sigmoid(rn(N, D)) if c["write"] == "gate" else None,
                     h=rn(N, D, dtype=torch.float32))
            s["h_out"] = torch.empty_like(s["h"])
        else:
            W = c["W"]
            s.update(x=rn(N, D), weight=rn(D, W, dtype=torch.float32, std=W ** -0.5),
                     bias=rn(D, dtype=torch.float32, std=0.1) if c.get("bias") else None,
                     state=rn(N, W - 1, D))
            s["state_out"] = torch.empty_like(s["state"])
        return s
    B, T, cu, ends = _layout(c, seed)
    n = len(ends) - 1
    s.update(cu=cu, n=n, longest=max(b - a for a, b in zip(ends, ends[1:])),
             ends=torch.tensor(ends, device="cuda"))
    if op.startswith("scan"):
        D = c["D"]
        s.update(v=rn(B, T, D), g=-torch.nn.functional.softplus(rn(B, T, D, mean=-2.0)),
                 beta=torch.sigmoid(rn(B, T, D)) if c["write"] == "gate" else None,
                 h0=rn(n, D, dtype=torch.float32) if c.get("h0") else None)
        if op == "scan_bwd":
            s["o"] = _plain_scan_fwd(s)[0]
            s["dO"] = rn(B, T, D)
            s["dh_final"] = rn(n, D, dtype=torch.float32) if c.get("h0") else None
    elif op.startswith("conv"):
        D, W = c["D"], c["W"]
        s.update(x=rn(B, T, D), weight=rn(D, W, dtype=torch.float32, std=W ** -0.5),
                 bias=rn(D, dtype=torch.float32, std=0.1) if c.get("bias") else None,
                 state=rn(n, W - 1, D) if c.get("state") else None)
        if op == "conv_bwd":
            s["dy"] = rn(B, T, D)
    else:
        H, d = c["H"], c["d"]
        s.update(x=rn(B, T, H, d, mean=0.2), weight=rn(H, d, dtype=torch.float32, mean=1.0, std=0.1),
                 bias=rn(H, d, dtype=torch.float32, std=0.1) if c.get("bias") else None,
                 z=rn(B, T, H, d) if c["gate"] else None)
        if op == "norm_bwd":
            s["dy"] = rn(B, T, H, d)
            if c["per"] == "sequence":  # the forward's, as a training step has them
                s["stats"] = _plain_stats(s)
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    if not own:
        return _plain(s)
    import gated_delta_rule_146_b200 as gdr
    c, op = s["c"], s["op"]
    if op == "scan_step":
        o = gdr.linear_scan_step(s["v"], s["g"], s["beta"], s["h"], tied=c["write"] == "tied",
                                 h_out=s["h_out"])
        return o, s["h_out"]
    if op == "conv_step":
        y = gdr.short_conv_step(s["x"], s["weight"], s["bias"], s["state"], activation=c["act"],
                                state_out=s["state_out"])
        return y, s["state_out"]
    if op == "scan_fwd":
        return gdr.linear_scan_fwd(s["v"], s["g"], s["beta"], s["h0"], s["cu"],
                                   tied=c["write"] == "tied", reverse=c.get("reverse", False))
    if op == "scan_bwd":
        return gdr.linear_scan_bwd(s["v"], s["g"], s["beta"], s["o"], s["dO"], s["h0"], s["cu"],
                                   s["dh_final"], tied=c["write"] == "tied",
                                   reverse=c.get("reverse", False), dh0=bool(c.get("h0")))
    if op == "conv_fwd":
        return gdr.short_conv_fwd(s["x"], s["weight"], s["bias"], s["state"], s["cu"],
                                  activation=c["act"], reverse=c.get("reverse", False))
    if op == "conv_bwd":
        return gdr.short_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], s["state"], s["cu"],
                                  activation=c["act"], reverse=c.get("reverse", False))
    kw = dict(per=c["per"], center=c["center"], activation=c["act"], eps=1e-6)
    if op == "norm_fwd":
        return gdr.group_norm_fwd(s["x"], s["weight"], s["bias"], s["z"], s["cu"], **kw)
    return gdr.group_norm_bwd(s["x"], s["weight"], s["bias"], s["z"], s["dy"], s["cu"],
                              stats=s.get("stats"), **kw)


def work(c):
    e = 2 if c["io"] == "bf16" else 4
    op = c["op"]
    if op == "scan_step":
        x = c["N"] * c["D"]
        return {"bytes": x * (8 + e * (4 if c["write"] == "gate" else 3)), "flops": 6 * x}
    if op == "conv_step":
        x = c["N"] * c["D"]
        return {"bytes": x * e * 2 * c["W"] + 4 * c["D"] * (c["W"] + bool(c.get("bias"))),
                "flops": x * (2 * c["W"] + 5)}
    rows = c["T"] * c.get("B", 1)
    n = c.get("n", c.get("B", 1))
    if op.startswith("scan"):
        D = c["D"]
        per = {"scan_fwd": {"plain": 3, "tied": 3, "gate": 4},
               "scan_bwd": {"plain": 5, "tied": 6, "gate": 8}}[op][c["write"]]
        states = n * D * 4 * ((1 + bool(c.get("h0"))) if op == "scan_fwd" else 3 * bool(c.get("h0")))
        return {"bytes": rows * D * e * per + states, "flops": rows * D * (5 if per < 5 else 10)}
    if op.startswith("conv"):
        D, W = c["D"], c["W"]
        st = n * (W - 1) * D * e
        if op == "conv_fwd":
            return {"bytes": rows * D * e * 2 + st * (1 + bool(c.get("state"))) + 4 * D * W,
                    "flops": rows * D * (2 * W + 5)}
        return {"bytes": rows * D * e * 3 + 2 * st * bool(c.get("state")) + 8 * D * W,
                "flops": rows * D * (6 * W + 12)}
    D = c["H"] * c["d"]
    if op == "norm_fwd":
        return {"bytes": rows * D * e * (2 + c["gate"]) + 4 * D, "flops": rows * D * 14}
    return {"bytes": rows * D * e * (3 + 2 * c["gate"]) + 8 * D, "flops": rows * D * 30}


# ---- plain forms: elementary operations in 32 bits or more, rounded once at the end ------------

def _plain(s):
    return {"scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
            "conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
            "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[s["op"]](s)


def _packed(t, reverse=False):
    """[B, T, ...] as fp32 [tokens, D], in scan order (the whole axis flipped)."""
    x = t.reshape(t.shape[0] * t.shape[1], -1).float()
    return x.flip(0) if reverse else x


def _unpacked(x, like, reverse=False):
    return (x.flip(0) if reverse else x).to(like.dtype).reshape(like.shape)


def _order(s):
    """Starts, lengths and the sequence of every token, in scan order."""
    ends, rev = s["ends"], s["c"].get("reverse", False)
    if rev:
        ends = ends[-1] - ends.flip(0)
    start, length = ends[:-1], ends[1:] - ends[:-1]
    seq = torch.repeat_interleave(torch.arange(s["n"], device="cuda"), length,
                                  output_size=s["c"]["T"] * s["c"].get("B", 1))
    return start, length, seq


def _states(t, rev):
    """Per-sequence rows in scan order: reversing the packed axis reverses the sequences too."""
    return t.flip(0) if rev and t is not None else t


def _recurrence(a, b, longest):
    """h_t = a_t h_{t-1} + b_t over the first axis, by doubling; a is 0 where a sequence starts."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _decay_and_write(s, rev):
    g, v = _packed(s["g"], rev), _packed(s["v"], rev)
    a = g.exp()
    if s["c"]["write"] == "gate":
        return a, v, _packed(s["beta"], rev)
    return a, v, -torch.expm1(g) if s["c"]["write"] == "tied" else None


def _plain_scan_fwd(s):
    rev = s["c"].get("reverse", False)
    start, length, _ = _order(s)
    a, v, w = _decay_and_write(s, rev)
    b = v if w is None else w * v
    full = length > 0
    h0 = _states(s["h0"], rev)
    if h0 is not None:
        b = b.index_add(0, start[full], a[start[full]] * h0[full])
    a = a.index_fill(0, start[full], 0.0)
    h = _recurrence(a, b, s["longest"])
    last = h[(start + length - 1).clamp(min=0)]
    hf = torch.where(full[:, None], last, torch.zeros_like(last) if h0 is None else h0)
    return _unpacked(h, s["v"], rev), _states(hf, rev)


def _plain_scan_bwd(s):
    c = s["c"]
    rev = c.get("reverse", False)
    start, length, _ = _order(s)
    a, v, w = _decay_and_write(s, rev)
    full = length > 0
    first, last = start[full], (start + length - 1)[full]
    h, lam = _packed(s["o"], rev), _packed(s["dO"], rev)
    h0, dhf = _states(s["h0"], rev), _states(s["dh_final"], rev)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = 0.0 if h0 is None else h0[full]
    if dhf is not None:
        lam = lam.index_add(0, last, dhf[full])
    nxt = torch.cat([a[1:], torch.zeros_like(a[:1])]).index_fill(0, last, 0.0)
    lam = _recurrence(nxt.flip(0), lam.flip(0), s["longest"]).flip(0)
    m = a * lam
    dh0 = None
    if c.get("h0"):
        dh0 = (torch.zeros_like(h0) if dhf is None else dhf).clone()
        dh0[full] = m[first]
        dh0 = _states(dh0, rev)
    dg = m * ((before - v) if c["write"] == "tied" else before)
    dv = lam if w is None else w * lam
    db = _unpacked(v * lam, s["beta"], rev) if c["write"] == "gate" else None
    return _unpacked(dv, s["v"], rev), _unpacked(dg, s["g"], rev), db, dh0


def _plain_scan_step(s):
    g, v = s["g"].float(), s["v"].float()
    w = s["c"]["write"]
    b = v if w == "plain" else (s["beta"].float() * v if w == "gate" else -torch.expm1(g) * v)
    h = g.exp() * s["h"] + b
    return h.to(s["v"].dtype), h


def _act(u, act):
    return u * torch.sigmoid(u) if act == "silu" else torch.sigmoid(u) if act == "sigmoid" else u


def _act_grad(u, act):
    if act == "none":
        return torch.ones_like(u)
    sg = torch.sigmoid(u)
    return sg * (1 + u * (1 - sg)) if act == "silu" else sg * (1 - sg)


def _tap(x, state, j, start, pos, seq, W):
    """x_{t-j} of every token, from the state where that lies before its sequence."""
    y = torch.cat([torch.zeros_like(x[:j]), x[:max(x.shape[0] - j, 0)]])
    out = pos < j
    if state is None:
        return y * ~out[:, None]
    at = out.nonzero()[:, 0]
    return y.index_copy(0, at, state[seq[at], W - 1 + pos[at] - j])


def _conv_parts(s):
    c, rev = s["c"], s["c"].get("reverse", False)
    start, length, seq = _order(s)
    x = _packed(s["x"], rev)
    st = None if s["state"] is None else _states(s["state"], rev).float()
    pos = torch.arange(x.shape[0], device="cuda") - start[seq]
    taps = [_tap(x, st, j, start, pos, seq, c["W"]) for j in range(c["W"])]
    p = taps[0] * s["weight"][:, -1]
    for j in range(1, c["W"]):
        p = p + taps[j] * s["weight"][:, c["W"] - 1 - j]
    if s["bias"] is not None:
        p = p + s["bias"]
    return start, length, seq, pos, x, st, taps, p


def _plain_conv_fwd(s):
    c, rev = s["c"], s["c"].get("reverse", False)
    W = c["W"]
    start, length, seq, pos, x, st, taps, p = _conv_parts(s)
    # the last W - 1 inputs of every sequence, the state's before them
    k = torch.arange(W - 1, device="cuda")
    at = length[:, None] - (W - 1) + k
    inside = at >= 0
    new = x[(start[:, None] + at).clamp(min=0, max=x.shape[0] - 1)]
    old = torch.zeros_like(new) if st is None else \
        st[torch.arange(s["n"], device="cuda")[:, None], (W - 1 + at).clamp(max=W - 2)]
    sf = torch.where(inside[:, :, None], new, old).to(s["x"].dtype)
    return _unpacked(_act(p, c["act"]), s["x"], rev), _states(sf, rev)


def _plain_conv_bwd(s):
    c, rev = s["c"], s["c"].get("reverse", False)
    W = c["W"]
    start, length, seq, pos, x, st, taps, p = _conv_parts(s)
    dp = _packed(s["dy"], rev) * _act_grad(p, c["act"])
    left = (length[seq] - pos)[:, None]
    dx, dw = dp * s["weight"][:, -1], [None] * W
    dst = None if st is None else torch.zeros_like(st)
    for j in range(W):
        wj = s["weight"][:, W - 1 - j]
        dw[W - 1 - j] = (dp * taps[j]).sum(0, dtype=torch.float64)
        if j:
            dx = dx + torch.cat([dp[j:], torch.zeros_like(dp[:j])]) * wj * (left > j)
            if st is not None:
                at = (pos < j).nonzero()[:, 0]
                dst = dst.index_put((seq[at], W - 1 + pos[at] - j), dp[at] * wj, accumulate=True)
    db = None if s["bias"] is None else dp.sum(0, dtype=torch.float64).float()
    return (_unpacked(dx, s["x"], rev), torch.stack(dw, 1).float(), db,
            None if st is None else _states(dst, rev).to(s["state"].dtype))


def _plain_conv_step(s):
    c = s["c"]
    x = torch.cat([s["state"], s["x"][:, None]], 1)
    p = (x.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        p = p + s["bias"]
    return _act(p, c["act"]).to(s["x"].dtype), x[:, 1:].contiguous()


def _group_mean(t, s):
    """Mean over a group's values: of every token's head, or of a sequence's tokens in it."""
    if s["c"]["per"] == "token":
        return t.mean(-1, keepdim=True)
    _, length, seq = _order(s)
    upto = t.sum(-1, dtype=torch.float64).t().contiguous().cumsum(1)
    upto = torch.cat([torch.zeros_like(upto[:, :1]), upto], 1)
    ends = s["ends"]
    m = (upto[:, ends[1:]] - upto[:, ends[:-1]]) / (length.clamp(min=1) * t.shape[-1])
    return m.float().t()[seq][:, :, None]


def _tokens(t):
    return t.reshape(-1, t.shape[2], t.shape[3]).float()


def _mean_rstd(s):
    x = _tokens(s["x"])
    mean = _group_mean(x, s) if s["c"]["center"] else torch.zeros_like(x[:, :, :1])
    xc = x - mean
    return xc, mean, torch.rsqrt(_group_mean(xc * xc, s) + 1e-6)


def _plain_stats(s):
    """[sequences, heads, 2] mean and 1 / deviation; an empty sequence has 0 and eps^-1/2."""
    _, mean, r = _mean_rstd(s)
    start, length, _ = _order(s)
    at = start.clamp(max=max(mean.shape[0] - 1, 0))
    st = torch.cat([mean[at], r[at]], -1)
    none = torch.tensor([0.0, 1e-6 ** -0.5], device="cuda")
    return torch.where((length > 0)[:, None, None], st, none).contiguous()


def _norm_parts(s):
    xc, _, r = _mean_rstd(s)
    n = xc * r
    u = n * s["weight"]
    if s["bias"] is not None:
        u = u + s["bias"]
    return n, r, u


def _plain_norm_fwd(s):
    _, _, u = _norm_parts(s)
    act = s["c"]["act"]
    y = _act(u, act) if s["z"] is None else u * _act(_tokens(s["z"]), act)
    return y.to(s["x"].dtype).reshape(s["x"].shape)


def _plain_norm_bwd(s):
    c, x = s["c"], s["x"]
    n, r, u = _norm_parts(s)
    dy = _tokens(s["dy"])
    dz = None
    if s["z"] is None:
        du = dy * _act_grad(u, c["act"])
    else:
        z = _tokens(s["z"])
        du = dy * _act(z, c["act"])
        dz = (dy * u * _act_grad(z, c["act"])).to(x.dtype).reshape(x.shape)
    q = du * s["weight"]
    dx = q - n * _group_mean(q * n, s)
    if c["center"]:
        dx = dx - _group_mean(q, s)
    dw = (du * n).sum(0, dtype=torch.float64).float()
    db = None if s["bias"] is None else du.sum(0, dtype=torch.float64).float()
    return (dx * r).to(x.dtype).reshape(x.shape), dw, db, dz


# ---- the definitions in 64 bits, one token or one sequence after the other ---------------------

def exact(c, seed):
    s = prepare(c, seed)
    f = {k: (t.double() if torch.is_tensor(t) and t.is_floating_point() else t)
         for k, t in s.items()}
    op = c["op"]
    if op == "scan_step":
        al = torch.exp(f["g"])
        wr = {"plain": lambda: 1.0, "gate": lambda: f["beta"], "tied": lambda: 1.0 - al}[c["write"]]()
        h = al * f["h"] + wr * f["v"]
        return h, h
    if op == "conv_step":
        win = torch.cat([f["state"], f["x"].unsqueeze(1)], dim=1)
        p = torch.einsum("nkd,dk->nd", win, f["weight"])
        p = p if f["bias"] is None else p + f["bias"]
        return (p / (1 + torch.exp(-p)) if c["act"] == "silu" else p), win[:, 1:]
    ends = s["ends"].tolist()
    rev = c.get("reverse", False)
    spans = list(zip(ends, ends[1:]))
    if op.startswith("scan"):
        return _exact_scan(c, f, spans, rev)
    if op.startswith("conv"):
        return _exact_conv(c, f, spans, rev)
    return _exact_norm(c, f, spans)


def _exact_scan(c, f, spans, rev):
    """Token by token; the sequences of one length (rows) go side by side."""
    D = c["D"]
    flat = {k: f[k].reshape(-1, D) for k in ("v", "g", "beta", "o", "dO") if f.get(k) is not None}
    if "n" in c:
        groups = [(torch.arange(i, i + 1), a, b) for i, (a, b) in enumerate(spans)]
        pick = lambda k, i, t: flat[k][spans[i[0]][0] + t][None]  # noqa: E731
    else:
        groups = [(torch.arange(len(spans)), 0, c["T"])]
        pick = lambda k, i, t: flat[k].view(len(spans), -1, D)[:, t]  # noqa: E731
    al, wv = torch.exp(flat["g"]), flat["v"]
    flat["al"] = al
    if c["write"] == "gate":
        wv = flat["beta"] * flat["v"]
    elif c["write"] == "tied":
        wv = (1 - al) * flat["v"]
    flat["b"] = wv
    names = ["o"] if c["op"] == "scan_fwd" else ["dv", "dg"] + ["dbeta"] * (c["write"] == "gate")
    out = {k: torch.zeros_like(flat["v"]) for k in names}

    def put(k, i, t, val):
        if "n" in c:
            out[k][spans[i[0]][0] + t] = val[0]
        else:
            out[k].view(len(spans), -1, D)[:, t] = val

    state = torch.zeros(len(spans), D, dtype=torch.float64, device="cuda")
    for i, a, b in groups:
        L = b - a
        order = range(L - 1, -1, -1) if rev else range(L)
        zero = torch.zeros(len(i), D, dtype=torch.float64, device="cuda")
        h0 = zero if f["h0"] is None else f["h0"][i.to("cuda")]
        if c["op"] == "scan_fwd":
            h = h0
            for t in order:
                h = torch.addcmul(pick("b", i, t), pick("al", i, t), h)
                put("o", i, t, h)
            state[i.to("cuda")] = h
            continue
        m = zero if f["dh_final"] is None else f["dh_final"][i.to("cuda")]
        step = -1 if rev else 1
        for t in reversed(order):
            lam = pick("dO", i, t) + m
            m = pick("al", i, t) * lam
            before = pick("o", i, t - step) if 0 <= t - step < L else h0
            if c["write"] == "tied":
                put("dg", i, t, m * (before - pick("v", i, t)))
                put("dv", i, t, lam - m)
            else:
                put("dg", i, t, m * before)
                put("dv", i, t, lam if c["write"] == "plain" else pick("beta", i, t) * lam)
            if c["write"] == "gate":
                put("dbeta", i, t, pick("v", i, t) * lam)
        state[i.to("cuda")] = m
    shape = f["v"].shape
    res = {k: t.reshape(shape) for k, t in out.items()}
    if c["op"] == "scan_fwd":
        return res["o"], state
    return res["dv"], res["dg"], res.get("dbeta"), state if c.get("h0") else None


def _exact_conv(c, f, spans, rev):
    W, D = c["W"], c["D"]
    x = f["x"].reshape(-1, D)
    back = c["op"] == "conv_bwd"
    y = torch.zeros_like(x)
    sf = torch.zeros(len(spans), W - 1, D, dtype=torch.float64, device="cuda")
    w = f["weight"].clone().requires_grad_(back)
    bias = None if f["bias"] is None else f["bias"].clone().requires_grad_(back)
    dst = torch.zeros_like(sf)
    for i, (a, b) in enumerate(spans):
        seg = x[a:b].flip(0) if rev else x[a:b]
        past = sf.new_zeros(W - 1, D) if f["state"] is None else f["state"][i]
        win = torch.cat([past, seg]).requires_grad_(back)
        sf[i] = win[win.shape[0] - (W - 1):].detach()
        if a == b:
            continue
        p = torch.nn.functional.conv1d(win.t()[None], w[:, None], bias, groups=D)[0].t()
        r = p / (1 + torch.exp(-p)) if c["act"] == "silu" else p
        if back:
            up = f["dy"].reshape(-1, D)[a:b]
            r.backward(up.flip(0) if rev else up)
            dst[i] = win.grad[:W - 1]
            r = win.grad[W - 1:]
        y[a:b] = (r.flip(0) if rev else r).detach()
    y = y.reshape(f["x"].shape)
    if not back:
        return y, sf
    return y, w.grad, None if bias is None else bias.grad, None if f["state"] is None else dst


def _exact_norm(c, f, spans):
    shape = f["x"].shape
    H, d = shape[2:]
    back = c["op"] == "norm_bwd"
    w = f["weight"].clone().requires_grad_(back)
    bias = None if f["bias"] is None else f["bias"].clone().requires_grad_(back)
    flat = {k: f[k].reshape(-1, H, d) for k in ("x", "z", "dy") if f.get(k) is not None}
    y, dz = torch.zeros_like(flat["x"]), torch.zeros_like(flat["x"])
    if c["per"] == "token":  # groups of any length may go side by side: a few thousand at a time
        spans = [(a, min(a + 4096, spans[-1][1])) for a in range(0, spans[-1][1], 4096)]
    dims = (2,) if c["per"] == "token" else (0, 2)
    act = {"silu": lambda t: t / (1 + torch.exp(-t)), "sigmoid": lambda t: 1 / (1 + torch.exp(-t)),
           "none": lambda t: t}[c["act"]]
    for a, b in spans:
        if a == b:
            continue
        x = flat["x"][a:b].clone().requires_grad_(back)
        xc = x - x.mean(dims, keepdim=True) if c["center"] else x
        u = xc / torch.sqrt(xc.square().mean(dims, keepdim=True) + 1e-6) * w
        u = u if bias is None else u + bias
        z = flat["z"][a:b].clone().requires_grad_(back) if c["gate"] else None
        r = act(u) if z is None else u * act(z)
        if back:
            r.backward(flat["dy"][a:b])
            r = x.grad
            if z is not None:
                dz[a:b] = z.grad
        y[a:b] = r.detach()
    y = y.reshape(shape)
    if not back:
        return y
    return y, w.grad, None if bias is None else bias.grad, dz.reshape(shape) if c["gate"] else None
