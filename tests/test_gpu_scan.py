"""Gated linear recurrence on the GPU against its 64-bit definition."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_146_b200 as gdr
from gated_delta_rule_146_b200 import _abi
from layer_helpers import check, scan_bwd_tol, scan_fwd_tol
from oracle import layer as ol

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(lengths, D, io="f32", gate=None, write="plain", h0=True, seed=0, rows=False, long=False):
    """Inputs on the CPU.  rows: equal lengths as rows of one tensor, without cu_seqlens."""
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lengths), len(lengths)
    shape = (n, lengths[0], D) if rows else (1, T, D)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    gd = DT[gate or io]
    # long: decays near one, so that states reach far back
    raw = -torch.nn.functional.softplus(rn(*shape) - (6.0 if long else 2.0))
    x = dict(v=rn(*shape).to(DT[io]), g=raw.to(gd), beta=None, h0=None, dhf=None,
             dO=rn(*shape).to(DT[io]), cu=[0], write=write, rows=rows)
    for length in lengths:
        x["cu"].append(x["cu"][-1] + length)
    if write == "gate":
        x["beta"] = torch.sigmoid(rn(*shape)).to(gd)
    if h0:
        x["h0"], x["dhf"] = rn(n, D), rn(n, D)
    return x


def dev(x):
    d = {k: t.cuda() if torch.is_tensor(t) else t for k, t in x.items()}
    d["cu_t"] = None if x["rows"] else torch.tensor(x["cu"], dtype=torch.int32, device="cuda")
    return d


def flat(t):
    return None if t is None else t.reshape(-1, t.shape[-1])


def forward(d, reverse=False, **kw):
    return gdr.linear_scan_fwd(d["v"], d["g"], d["beta"], d["h0"], d["cu_t"],
                               tied=d["write"] == "tied", reverse=reverse, **kw)


def backward(d, o, reverse=False, **kw):
    return gdr.linear_scan_bwd(d["v"], d["g"], d["beta"], o, d["dO"], d["h0"], d["cu_t"], d["dhf"],
                               tied=d["write"] == "tied", reverse=reverse, **kw)


def compare(x, reverse=False):
    d = dev(x)
    tied = x["write"] == "tied"
    f = {k: flat(x[k]) for k in ("v", "g", "beta", "dO")}
    o, hf = forward(d, reverse)
    want = ol.scan(f["v"], f["g"], f["beta"], x["h0"], x["cu"], tied, reverse)
    tol = scan_fwd_tol(f["v"], f["g"], f["beta"], x["h0"], x["cu"], tied, reverse)
    check("o", flat(o), want[0], tol[0], o.dtype)
    check("h_final", hf, want[1], tol[1])
    got = backward(d, o, reverse)
    args = (f["v"], f["g"], f["beta"], flat(o).cpu(), f["dO"], x["h0"], x["dhf"], x["cu"], tied,
            reverse)
    want, tol = ol.scan_backward(*args), scan_bwd_tol(*args)
    for name, a, b, t in zip(("dv", "dg", "dbeta", "dh0"), got, want, tol):
        assert (a is None) == (b is None), name
        if a is not None:
            check(name, flat(a), b, t, None if name == "dh0" else a.dtype)


@pytest.mark.parametrize("write", ["plain", "gate", "tied"])
@pytest.mark.parametrize("io,gate", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                     ("f32", "bf16")])
def test_types_and_writes(io, gate, write):
    compare(make([70, 0, 1, 200, 3, 0], 72, io, gate, write, seed=1))


@pytest.mark.parametrize("lengths", [[1], [2], [63], [64], [65], [129], [1000], [0, 0, 5], [5, 0],
                                     [1] * 70, [31, 33, 64, 128, 1]])
@pytest.mark.parametrize("reverse", [False, True])
def test_lengths(lengths, reverse):
    compare(make(lengths, 40, seed=len(lengths)), reverse)


@pytest.mark.parametrize("D", [1, 2, 3, 31, 33, 64, 65, 130])
def test_widths(D):
    compare(make([90, 17], D, "bf16", write="gate", seed=D))


@pytest.mark.parametrize("D", [8, 24, 50, 77, 96, 200, 520, 1032])
@pytest.mark.parametrize("io,write", [("bf16", "gate"), ("f32", "tied"), ("bf16", "plain")])
def test_layouts(D, io, write):
    """Widths that are laid out as clusters of other sizes and groups, over several steps, with
    bounds of sequences at odd places."""
    r = np.random.default_rng(D)
    cuts = np.sort(r.integers(0, 2500, 9))
    lengths = np.diff(np.concatenate([[0], cuts, [2500]])).tolist()
    compare(make(lengths, D, io, write=write, seed=D), reverse=D % 3 == 0)
    compare(make([1300, 1300], D, io, write=write, seed=D, rows=True), reverse=D % 3 == 1)


def test_thousands_of_sequences():
    """More sequences than the kernels keep bounds of, many of them empty."""
    r = np.random.default_rng(5)
    compare(make(r.integers(0, 4, 2500).tolist(), 72, "bf16", write="gate", seed=6))
    compare(make(r.integers(0, 3, 1500).tolist(), 33, "f32", seed=7), True)


@pytest.mark.parametrize("B,T", [(1, 1), (3, 7), (2, 63), (2, 64), (5, 200), (1, 4099)])
@pytest.mark.parametrize("reverse", [False, True])
def test_rows(B, T, reverse):
    compare(make([T] * B, 34, write="tied", seed=T, rows=True), reverse)


def test_no_initial_state():
    compare(make([100, 0, 30], 66, h0=False, seed=3))
    compare(make([100] * 2, 66, h0=False, seed=3, rows=True))


def test_long_memory():
    """States that reach back over thousands of tokens and over every join of the walk."""
    compare(make([6000], 64, "f32", long=True, seed=4))
    compare(make([2900] * 2, 34, "bf16", write="gate", long=True, seed=5, rows=True), True)


def test_growing_decays():
    x = make([300], 64, seed=6)
    x["g"] = x["g"].abs() * 0.2  # products stay below e^30
    compare(x)


def test_a_decay_of_zero_drops_the_state():
    x = make([200, 50], 64, seed=7)
    for t in (0, 13, 64, 199, 200, 210):
        x["g"][0, t] = -float("inf")
    x["g"][0, 100] = torch.finfo(torch.float32).min
    for w in ("plain", "tied"):
        x["write"] = w
        compare(x)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("rows", [False, True])
def test_a_sequence_does_not_see_another_ones_nan(rows, reverse):
    """Infinities and NaN in one sequence leave the others' results as they are."""
    lengths = [100] * 4 if rows else [70, 1, 130, 64]
    x = make(lengths, 64, seed=8, rows=rows)
    clean = dev(x)
    o, hf = forward(clean, reverse)
    grads = backward(clean, o, reverse)
    bad = {k: t.clone() if torch.is_tensor(t) else t for k, t in clean.items()}
    b, e = x["cu"][2], x["cu"][3]
    for k, v in (("v", float("nan")), ("dO", float("inf"))):
        flat(bad[k])[b:e] = v
    bad["h0"][2] = float("inf")
    bad["dhf"][2] = float("nan")
    o2, hf2 = forward(bad, reverse)
    keep = torch.ones(x["cu"][-1], dtype=torch.bool, device="cuda")
    keep[b:e] = False
    assert torch.equal(flat(o2)[keep], flat(o)[keep])
    rest = [0, 1, 3]
    assert torch.equal(hf2[rest], hf[rest])
    assert not torch.isfinite(flat(o2)[b:e]).any()
    g2 = backward(bad, o2, reverse)
    for a, c in zip(grads[:2], g2[:2]):
        assert torch.equal(flat(a)[keep], flat(c)[keep])
    assert torch.equal(grads[3][rest], g2[3][rest])


def test_states_in_place_and_repeated_calls():
    x = make([300, 0, 7, 90], 128, "bf16", write="gate", seed=9)
    d = dev(x)
    o, hf = forward(d)
    d2 = dict(d, h0=d["h0"].clone())
    o2, hf2 = forward(d2, h_final=d2["h0"])
    assert hf2.data_ptr() == d2["h0"].data_ptr()
    assert torch.equal(o, o2) and torch.equal(hf, hf2)
    a, b = backward(d, o), backward(d, o)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a = make([500] * 3, 64, seed=10, rows=True)
    d = dev(a)
    _, hf = forward(d)
    _, hf2 = forward(d, h_final=d["h0"])
    assert torch.equal(hf, hf2)


def test_pieces_continue_one_another():
    x = make([257], 64, seed=11)
    d = dev(x)
    o, hf = forward(d)
    cut = 100
    p = {k: d[k][:, :cut].contiguous() for k in ("v", "g")}
    q = {k: d[k][:, cut:].contiguous() for k in ("v", "g")}
    oa, ha = gdr.linear_scan_fwd(p["v"], p["g"], None, d["h0"])
    ob, hb = gdr.linear_scan_fwd(q["v"], q["g"], None, ha)
    tol = scan_fwd_tol(flat(x["v"]), flat(x["g"]), None, x["h0"], x["cu"], False, False)
    check("o", flat(torch.cat([oa, ob], 1)), ol.f64(flat(o)), 2 * tol[0])
    check("h_final", hb, ol.f64(hf), 2 * tol[1])


@pytest.mark.parametrize("io,gate", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("write", ["plain", "gate", "tied"])
@pytest.mark.parametrize("N,D", [(1, 1), (1, 64), (3, 50), (7, 33), (257, 96)])
def test_step(N, D, write, io, gate):
    x = make([1] * N, D, io, gate, write, seed=N + D)
    d = dev(x)
    s = {k: None if d[k] is None else d[k][0] for k in ("v", "g", "beta")}
    f = {k: None if x[k] is None else x[k][0] for k in ("v", "g", "beta")}
    tied = write == "tied"
    want = ol.scan(f["v"], f["g"], f["beta"], x["h0"], x["cu"], tied)
    tol = scan_fwd_tol(f["v"], f["g"], f["beta"], x["h0"], x["cu"], tied, False)
    out = torch.empty_like(d["h0"])
    o = gdr.linear_scan_step(s["v"], s["g"], s["beta"], d["h0"], tied=tied, h_out=out)
    check("o", o, want[0], tol[0], o.dtype)
    check("h_out", out, want[1], tol[1])
    assert torch.equal(d["h0"].cpu(), x["h0"])
    o2 = gdr.linear_scan_step(s["v"], s["g"], s["beta"], d["h0"], tied=tied)
    assert torch.equal(o, o2) and torch.equal(d["h0"], out)


def test_step_continues_the_scan():
    x = make([40] * 3, 32, write="gate", seed=12, rows=True)
    d = dev(x)
    o, hf = forward(d)
    h = d["h0"].clone()
    outs = [gdr.linear_scan_step(*(d[k][:, t].contiguous() for k in ("v", "g", "beta")), h)
            for t in range(40)]
    tol = scan_fwd_tol(flat(x["v"]), flat(x["g"]), flat(x["beta"]), x["h0"], x["cu"], False, False)
    check("o", flat(torch.stack(outs, 1)), ol.f64(flat(o)), 2 * tol[0])
    check("h", h, ol.f64(hf), 2 * tol[1])


def test_heads_and_empty_calls():
    v, g = torch.randn(2, 70, 3, 16, device="cuda"), -torch.rand(2, 70, 3, 16, device="cuda")
    o, hf = gdr.linear_scan_fwd(v, g)
    o2, hf2 = gdr.linear_scan_fwd(v.view(2, 70, 48), g.view(2, 70, 48))
    assert o.shape == v.shape and hf.shape == (2, 3, 16)
    assert torch.equal(o.view(2, 70, 48), o2) and torch.equal(hf.view(2, 48), hf2)
    e = v[:, :0].contiguous()
    h0 = torch.randn(2, 3, 16, device="cuda")
    o, hf = gdr.linear_scan_fwd(e, e, None, h0)
    assert o.shape == e.shape and torch.equal(hf, h0)
    _, hf = gdr.linear_scan_fwd(e, e)
    assert not hf.any()
    out = gdr.linear_scan_bwd(e, e, None, e, e, h0, dh_final=h0)
    assert torch.equal(out[3], h0)
    n = gdr.linear_scan_step(v[:0, 0], g[:0, 0], None, h0[:0])
    assert n.shape == (0, 3, 16)


def test_bad_cu_seqlens_is_reported_and_stays_inside():
    """Bounds that decrease or miss the ends: the status word says so; a guard behind the
    outputs keeps its values."""
    D, T = 64, 100
    for cu in ([0, 60, 40, 100], [0, 50, 99], [1, 50, 100], [0, -7, 100], [0, 200, 100]):
        n = len(cu) - 1
        x = make([T], D, seed=13)
        d = dev(x)
        buf = torch.full((T + 8, D), 7.0, device="cuda")
        hbuf = torch.full((n + 4, D), 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        h0 = torch.zeros(n, D, device="cuda")
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        gdr.linear_scan_fwd(d["v"], d["g"], None, h0, c, o=buf[None, :T], h_final=hbuf[:n],
                            status=status)
        gdr.linear_scan_bwd(d["v"], d["g"], None, d["v"], d["dO"], h0, c, h0, status=status)
        torch.cuda.synchronize()
        assert status.item() == _abi.GDR_ERR_DEVICE_CHECK, cu
        assert (buf[T:] == 7).all() and (hbuf[n:] == 7).all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = torch.tensor([0, 30, 100], dtype=torch.int32, device="cuda")
    gdr.linear_scan_fwd(d["v"], d["g"], None, None, c, status=status)
    assert status.item() == _abi.GDR_OK


def test_streams_and_graphs():
    """On a side stream, and captured into a graph that is replayed on new inputs."""
    x, y = make([300, 40], 64, "bf16", seed=14), make([300, 40], 64, "bf16", seed=15)
    d, e = dev(x), dev(y)
    want, want_g = forward(d), None
    want_g = backward(d, want[0])
    want2 = forward(e)
    want_g2 = backward(e, want2[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = forward(d, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(d)
        grads = backward(d, out[0])
    for src, w, wg in ((x, want, want_g), (y, want2, want_g2)):
        for k in ("v", "g", "h0", "dO", "dhf"):
            d[k].copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(grads, wg))


# ---- single blocks -------------------------------------------------------------------------------
# At most 148 clusters of one block are resident, so more slabs of 64 channels (times rows) than
# that are always laid out as single blocks, whose walk is another one than the clusters'.

def single(write, io="bf16", gate=None, D=4864, packed=False, seed=0, T=330):
    """Inputs for single blocks, over six steps in bf16 and eleven in fp32."""
    if packed:
        D += 4864
    units = -(-D // 64) * (1 if packed else 2)
    assert units > 148
    lengths = [T // 5, 0, 1, T - T // 5 - 5, 3, 1, 0] if packed else [T] * 2
    return make(lengths, D, io, gate, write, seed=seed, rows=not packed)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("write", ["plain", "gate", "tied"])
@pytest.mark.parametrize("io,gate", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                     ("f32", "bf16")])
def test_single_blocks(io, gate, write, packed):
    compare(single(write, io, gate, packed=packed, seed=20), reverse=packed)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("D", [4866, 4865])
@pytest.mark.parametrize("io,write", [("bf16", "gate"), ("bf16", "tied"), ("f32", "plain")])
def test_single_blocks_of_odd_widths(io, write, D, packed):
    """Rows that are copied two channels and one channel at a time."""
    compare(single(write, io, D=D, packed=packed, seed=D), reverse=not packed)


@pytest.mark.parametrize("T", [64, 65, 127, 128, 129, 192, 257])
def test_single_blocks_of_other_lengths(T):
    compare(single("tied", T=T, seed=T), reverse=T % 2 == 0)
    compare(single("plain", T=T, packed=True, seed=T), reverse=T % 2 == 1)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_single_blocks_keep_sequences_apart(packed, reverse):
    """Infinities and NaN of one sequence (the longest) leave the others' results as they are."""
    x = single("gate", packed=packed, seed=21)
    s = 3 if packed else 0
    d = dev(x)
    o, hf = forward(d, reverse)
    grads = backward(d, o, reverse)
    bad = {k: t.clone() if torch.is_tensor(t) else t for k, t in d.items()}
    b, e = x["cu"][s], x["cu"][s + 1]
    for k, v in (("v", float("nan")), ("dO", float("inf"))):
        flat(bad[k])[b:e] = v
    bad["h0"][s] = float("inf")
    bad["dhf"][s] = float("nan")
    o2, hf2 = forward(bad, reverse)
    g2 = backward(bad, o2, reverse)
    keep = torch.ones(x["cu"][-1], dtype=torch.bool, device="cuda")
    keep[b:e] = False
    rest = [i for i in range(len(x["cu"]) - 1) if i != s]
    assert not torch.isfinite(flat(o2)[b:e]).any()
    for a, c in zip((o, *grads[:3]), (o2, *g2[:3])):
        assert torch.equal(flat(a)[keep], flat(c)[keep])
    assert torch.equal(hf2[rest], hf[rest]) and torch.equal(g2[3][rest], grads[3][rest])


def raw_backward(d, o, dv, dg, dh0, dhf, status=None, n=None):
    """gdr_scan_bwd of a plain write on outputs of the caller's."""
    B, T, D = d["v"].shape
    a = _abi.ScanArgs(B, T, D, n or len(d["cu"]) - 1, _abi.F32 if d["v"].dtype == torch.float32 else
                      _abi.BF16, _abi.F32 if d["g"].dtype == torch.float32 else _abi.BF16,
                      _abi.WRITE_PLAIN, 0, None if status is None else status.data_ptr())
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _abi.check(_abi.lib().gdr_scan_bwd(
        ctypes.byref(a), p(d["v"]), p(d["g"]), None, p(o), p(d["dO"]), p(d["h0"]), p(d["cu_t"]),
        p(dhf), p(dv), p(dg), None, p(dh0), torch.cuda.current_stream().cuda_stream))


def test_backward_reports_bad_cu_seqlens_and_stays_inside():
    D, T = 64, 100
    for cu in ([0, 60, 40, 100], [0, 50, 99], [1, 50, 100], [0, -7, 100], [0, 200, 100]):
        n = len(cu) - 1
        d = dev(make([T], D, seed=13))
        d["cu_t"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        d["h0"], dhf = torch.zeros(n, D, device="cuda"), torch.zeros(n, D, device="cuda")
        dv, dg = (torch.full((T + 8, D), 7.0, device="cuda") for _ in range(2))
        dh0 = torch.full((n + 4, D), 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        raw_backward(d, d["v"], dv, dg, dh0, dhf, status, n)
        assert status.item() == _abi.GDR_ERR_DEVICE_CHECK, cu
        assert (dv[T:] == 7).all() and (dg[T:] == 7).all() and (dh0[n:] == 7).all()


@pytest.mark.parametrize("case", ["clusters", "clusters packed", "blocks", "blocks packed",
                                  "empty", "one by one"])
def test_states_in_place_in_every_layout(case):
    """h_final in h0's place and dh0 in dh_final's give the bits of arrays of their own."""
    packed = "packed" in case
    x = (single("plain", packed=packed, seed=22) if "blocks" in case else
         make([40, 0, 300, 1, 0], 65, seed=23) if case == "one by one" else
         make([0, 0], 64, seed=24) if case == "empty" else
         make([500, 0, 1, 700] if packed else [600] * 3, 200, "bf16", seed=25, rows=not packed))
    d = dev(x)
    o, hf = forward(d)
    for _ in range(3):
        d2 = dict(d, h0=d["h0"].clone())
        o2, hf2 = forward(d2, h_final=d2["h0"])
        assert hf2.data_ptr() == d2["h0"].data_ptr()
        assert torch.equal(o2, o) and torch.equal(hf2, hf)
    dv, dg, _, dh0 = backward(d, o)
    for _ in range(3):
        state = d["dhf"].clone()
        dv2, dg2 = torch.empty_like(dv), torch.empty_like(dg)
        raw_backward(d, o, dv2, dg2, state, state)
        assert torch.equal(dv2, dv) and torch.equal(dg2, dg) and torch.equal(state, dh0)
