"""Short causal convolution on the GPU against its 64-bit definition."""
import pytest
import torch

import gated_delta_rule_146_b200 as gdr
from gated_delta_rule_146_b200 import _abi
from layer_helpers import E, check, conv_tol
from oracle import layer as ol

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(lengths, D, W=4, io="f32", bias=True, state=True, act="silu", seed=0, rows=False):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T, n = sum(lengths), len(lengths)
    shape = (n, lengths[0], D) if rows else (1, T, D)
    cu = [0]
    for length in lengths:
        cu.append(cu[-1] + length)
    return dict(x=rn(*shape).to(DT[io]), w=rn(D, W) * 0.6, bias=rn(D) * 0.3 if bias else None,
                state=rn(n, W - 1, D).to(DT[io]) if state else None, dy=rn(*shape).to(DT[io]),
                cu=cu, act=act, rows=rows)


def dev(x):
    d = {k: t.cuda() if torch.is_tensor(t) else t for k, t in x.items()}
    d["cu_t"] = None if x["rows"] else torch.tensor(x["cu"], dtype=torch.int32, device="cuda")
    return d


def flat(t):
    return t.reshape(-1, t.shape[-1])


def forward(d, reverse=False, **kw):
    return gdr.short_conv_fwd(d["x"], d["w"], d["bias"], d["state"], d["cu_t"],
                              activation=d["act"], reverse=reverse, **kw)


def backward(d, reverse=False, **kw):
    return gdr.short_conv_bwd(d["x"], d["w"], d["bias"], d["dy"], d["state"], d["cu_t"],
                              activation=d["act"], reverse=reverse, **kw)


def compare(x, reverse=False):
    d = dev(x)
    xs, dys = flat(x["x"]), flat(x["dy"])
    tol = conv_tol(xs, x["w"], x["bias"], dys, x["state"], x["cu"], x["act"], reverse)
    y, st = forward(d, reverse)
    wy, wst, _ = ol.conv(xs, x["w"], x["bias"], x["state"], x["cu"], x["act"], reverse)
    check("y", flat(y), wy, tol[0], y.dtype)
    check("state_out", st, wst, 0.0)
    dx, dw, db, ds = backward(d, reverse)
    want = ol.conv_backward(xs, x["w"], x["bias"], dys, x["state"], x["cu"], x["act"], reverse)
    check("dx", flat(dx), want[0], tol[1], dx.dtype)
    check("dw", dw, want[1], tol[2])
    assert (db is None) == (x["bias"] is None) and (ds is None) == (x["state"] is None)
    if db is not None:
        check("dbias", db, want[2], tol[3])
    if ds is not None:
        check("dstate", ds, want[3], tol[4], ds.dtype)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_types_and_widths(W, io, act):
    compare(make([70, 0, 1, 200, 2, 3, 0], 72, W, io, act=act, seed=W))


@pytest.mark.parametrize("lengths", [[1], [2], [3], [31], [64], [257], [1000], [0, 5], [5, 0],
                                     [1] * 70, [2, 1, 0, 3] * 9])
@pytest.mark.parametrize("reverse", [False, True])
def test_lengths(lengths, reverse):
    compare(make(lengths, 24, seed=len(lengths)), reverse)


@pytest.mark.parametrize("D", [1, 2, 3, 31, 64, 130, 132, 260])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_channels(D, io):
    compare(make([40, 9], D, 4, io, seed=D))


@pytest.mark.parametrize("B,T", [(1, 1), (4, 2), (3, 70), (2, 513)])
@pytest.mark.parametrize("reverse", [False, True])
def test_rows(B, T, reverse):
    compare(make([T] * B, 36, 3, seed=T, rows=True), reverse)


def test_without_bias_or_state():
    compare(make([50, 1, 20], 40, bias=False, state=False, seed=1))
    compare(make([33] * 2, 40, bias=False, state=False, seed=2, rows=True))


def test_thousands_of_sequences():
    lengths = torch.randint(0, 5, (2500,), generator=torch.Generator().manual_seed(9)).tolist()
    compare(make(lengths, 36, 4, "bf16", seed=9))
    compare(make(lengths, 33, 3, "f32", seed=10), True)


def test_long_runs():
    """More tokens than the runs of one wave of warps: the partial sums span many blocks."""
    compare(make([9000, 3001], 8, 4, "f32", seed=3))


def test_a_sequence_does_not_see_another_ones_nan():
    x = make([40, 3, 50, 1, 9], 64, seed=4)
    d = dev(x)
    y, st = forward(d)
    dx = backward(d)[0]
    bad = {k: t.clone() if torch.is_tensor(t) else t for k, t in d.items()}
    b, e = x["cu"][2], x["cu"][3]
    bad["x"][0, b:e] = float("nan")
    bad["dy"][0, b:e] = float("inf")
    bad["state"][2] = float("nan")
    y2, st2 = forward(bad)
    dx2, _, _, ds2 = backward(bad)
    keep = torch.ones(x["cu"][-1], dtype=torch.bool, device="cuda")
    keep[b:e] = False
    assert torch.equal(y2[0, keep], y[0, keep]) and torch.equal(dx2[0, keep], dx[0, keep])
    assert torch.equal(st2[[0, 1, 3, 4]], st[[0, 1, 3, 4]])
    assert torch.isfinite(ds2[[0, 1, 3, 4]]).all() and y2[0, b:e].isnan().all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("N,D", [(1, 1), (1, 520), (5, 33), (300, 64)])
def test_step(N, D, W, io):
    x = make([1] * N, D, W, io, seed=N + D)
    d = dev(x)
    wy, wst, _ = ol.conv(x["x"][0], x["w"], x["bias"], x["state"], x["cu"])
    tol = conv_tol(x["x"][0], x["w"], x["bias"], None, x["state"], x["cu"], "silu", False)
    out = torch.empty_like(d["state"])
    y = gdr.short_conv_step(d["x"][0], d["w"], d["bias"], d["state"], state_out=out)
    check("y", y, wy, tol, y.dtype)
    check("state_out", out, wst, 0.0)
    assert torch.equal(d["state"].cpu(), x["state"])
    y2 = gdr.short_conv_step(d["x"][0], d["w"], d["bias"], d["state"])
    assert torch.equal(y, y2) and torch.equal(d["state"], out)


def test_steps_continue_the_sequence():
    x = make([12] * 3, 40, 4, "bf16", seed=5, rows=True)
    d = dev(x)
    y, st = forward(d)
    s = d["state"].clone()
    outs = [gdr.short_conv_step(d["x"][:, t].contiguous(), d["w"], d["bias"], s) for t in range(12)]
    assert torch.equal(torch.stack(outs, 1), y) and torch.equal(s, st)
    p, q = d["x"][:, :5].contiguous(), d["x"][:, 5:].contiguous()
    ya, sa = gdr.short_conv_fwd(p, d["w"], d["bias"], d["state"])
    yb, sb = gdr.short_conv_fwd(q, d["w"], d["bias"], sa)
    assert torch.equal(torch.cat([ya, yb], 1), y) and torch.equal(sb, st)


def test_heads_and_empty_calls():
    x = torch.randn(2, 30, 3, 16, device="cuda")
    w = torch.randn(3, 16, 4, device="cuda")
    y, st = gdr.short_conv_fwd(x, w)
    y2, st2 = gdr.short_conv_fwd(x.view(2, 30, 48), w.view(48, 4))
    assert st.shape == (2, 3, 3, 16)
    assert torch.equal(y.view(2, 30, 48), y2) and torch.equal(st.view(2, 3, 48), st2)
    e = x[:, :0].contiguous()
    s = torch.randn(2, 3, 3, 16, device="cuda")
    y, st = gdr.short_conv_fwd(e, w, None, s)
    assert y.shape == e.shape and torch.equal(st, s)
    dx, dw, db, ds = gdr.short_conv_bwd(e, w, None, e, s)
    assert not dw.any() and not ds.any() and db is None
    assert gdr.short_conv_step(x[:0, 0], w, None, s[:0]).shape == (0, 3, 16)


def test_bad_cu_seqlens_is_reported_and_stays_inside():
    D, T, W = 64, 100, 4
    for cu in ([0, 60, 40, 100], [0, 50, 99], [1, 50, 100], [0, -7, 100], [0, 200, 100]):
        n = len(cu) - 1
        d = dev(make([T], D, seed=6))
        buf = torch.full((T + 8, D), 7.0, device="cuda")
        sbuf = torch.full((n + 2, W - 1, D), 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        s = torch.zeros(n, W - 1, D, device="cuda")
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        gdr.short_conv_fwd(d["x"], d["w"], None, s, c, y=buf[None, :T], state_out=sbuf[:n],
                           status=status)
        assert status.item() == _abi.GDR_ERR_DEVICE_CHECK, cu
        status.zero_()
        gdr.short_conv_bwd(d["x"], d["w"], None, d["dy"], s, c, status=status)
        assert status.item() == _abi.GDR_ERR_DEVICE_CHECK, cu
        assert (buf[T:] == 7).all() and (sbuf[n:] == 7).all()


def test_streams_graphs_and_repeats():
    x, y = make([300, 40], 64, 4, "bf16", seed=7), make([300, 40], 64, 4, "bf16", seed=8)
    d, e = dev(x), dev(y)
    want = [(forward(t), backward(t)) for t in (d, e)]
    again = backward(d)
    assert all(torch.equal(a, b) for a, b in zip(again, want[0][1]))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = forward(d, stream=side), backward(d, stream=side)
    side.synchronize()
    for a, b in zip(got, want[0]):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(d), backward(d)
    for src, w in zip((x, y), want):
        for k in ("x", "w", "bias", "state", "dy"):
            d[k].copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, w):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_activation_in_fp32_at_large_sums():
    """One weight of one leaves p exact: what is left is the activation's own error, 8 E of y (its
    exponential, sum, reciprocal and product), and 24 E of the terms of its slope s (1 + p (1 - s)).
    (An exponent rounded before the exponential would be off by |p| E.)"""
    p = torch.cat([torch.linspace(-80, 80, 40001), torch.linspace(-3, 3, 4097)])
    x = p.view(1, 1, -1).cuda()
    D = p.numel()
    w = torch.zeros(D, 4)
    w[:, 3] = 1.0
    y = gdr.short_conv_fwd(x, w.cuda())[0]
    dx = gdr.short_conv_bwd(x, w.cuda(), None, torch.ones_like(x))[0]
    z = torch.zeros(1, 3, D, device="cuda")
    step = gdr.short_conv_step(x[0], w.cuda(), None, z)
    assert torch.equal(step, y[0])
    q = p.double()
    s = 1 / (1 + torch.exp(-q))
    rest = 1 / (1 + torch.exp(q))
    check("y", y[0], (q * s)[None].numpy(), (8 * E * (q * s).abs())[None].numpy())
    check("dx", dx[0], (s * (1 + q * rest))[None].numpy(), (24 * E * s * (1 + q.abs() * rest))[None].numpy())
