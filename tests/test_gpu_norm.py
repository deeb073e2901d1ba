"""Group norm on the GPU against its 64-bit definition."""
import numpy as np
import pytest
import torch

import gated_delta_rule_146_b200 as gdr
from gated_delta_rule_146_b200 import _abi
from layer_helpers import E, check, norm_tol
from oracle import layer as ol

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(lengths, H, d, io="f32", gate=True, affine="own", bias=True, seed=0, rows=False,
         mean=0.3):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T, n = sum(lengths), len(lengths)
    shape = (n, lengths[0], H, d) if rows else (1, T, H, d)
    wshape = (d,) if affine == "shared" else (H, d)
    cu = [0]
    for length in lengths:
        cu.append(cu[-1] + length)
    return dict(x=(rn(*shape) + mean).to(DT[io]), z=rn(*shape).to(DT[io]) if gate else None,
                dy=rn(*shape).to(DT[io]), w=1 + 0.2 * rn(*wshape) if affine != "none" else None,
                b=0.2 * rn(*wshape) if bias else None, cu=cu, rows=rows)


def dev(x):
    d = {k: t.cuda() if torch.is_tensor(t) else t for k, t in x.items()}
    d["cu_t"] = None if x["rows"] else torch.tensor(x["cu"], dtype=torch.int32, device="cuda")
    return d


def flat(t):
    return None if t is None else t.reshape(-1, *t.shape[2:])


def compare(x, per="token", center=True, act="silu", eps=1e-5):
    d = dev(x)
    H = x["x"].shape[2]
    xs, zs, dys = flat(x["x"]), flat(x["z"]), flat(x["dy"])
    kw = dict(per=per, center=center, activation=act, eps=eps)
    out = gdr.group_norm_fwd(d["x"], d["w"], d["b"], d["z"], d["cu_t"],
                             output_stats=per == "sequence", **kw)
    y, stats = out if per == "sequence" else (out, None)
    eps = float(np.float32(eps))
    wy, wst = ol.norm(xs, x["w"], x["b"], zs, x["cu"], per, center, act, eps)
    tol = norm_tol(xs, x["w"], x["b"], zs, dys, x["cu"], per, center, act, eps)
    check("y", flat(y), wy, tol[0], y.dtype)
    if stats is not None:
        for i, (b, e) in enumerate(zip(x["cu"], x["cu"][1:])):
            mu = np.abs(ol.f64(xs)[b:e]).mean((0, 2)) if e > b else np.zeros(H)
            r = wst[i, :, 1]
            check("mean", stats[i, :, 0], wst[i, :, 0], 100 * E * mu + 1e-30)
            check("rstd", stats[i, :, 1], r, E * r * (108 + 100 * mu * r))
    dx, dw, db, dz = gdr.group_norm_bwd(d["x"], d["w"], d["b"], d["z"], d["dy"], d["cu_t"],
                                        stats=stats, **kw)
    want = ol.norm_backward(xs, x["w"], x["b"], zs, dys, x["cu"], per, center, act, eps)
    check("dx", flat(dx), want[0], tol[1], dx.dtype)
    for name, got, w, t, given in (("dw", dw, want[1], tol[2], x["w"]),
                                   ("db", db, want[2], tol[3], x["b"])):
        assert (got is None) == (given is None), name
        if got is not None:
            if given.dim() == 1:
                w, t = w.sum(0), t.sum(0)
            check(name, got, w, t)
    assert (dz is None) == (x["z"] is None)
    if dz is not None:
        check("dz", flat(dz), want[3], tol[4], dz.dtype)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("per", ["token", "sequence"])
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("act", ["silu", "sigmoid", "none"])
def test_forms(per, center, gate, act, io):
    compare(make([40, 0, 1, 77, 0], 3, 64, io, gate, seed=1), per, center, act)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("per", ["token", "sequence"])
@pytest.mark.parametrize("d", [1, 2, 3, 4, 8, 12, 31, 32, 40, 48, 64, 100, 128, 200, 256, 264, 512,
                               520, 1024])
def test_group_sizes(d, per, io):
    if io == "bf16" and d % 8 and d > 256 or io == "f32" and d % 4 and d > 256:
        pytest.skip("refused (see the refusals' test)")
    # a group of one channel has no variance: eps alone
    compare(make([9, 30], 2, d, io, seed=d), per, center=d > 2, eps=1e-2)


@pytest.mark.parametrize("per", ["token", "sequence"])
@pytest.mark.parametrize("H,d", [(1, 128), (5, 64), (16, 128), (17, 128), (33, 32), (100, 16)])
def test_heads(H, d, per):
    compare(make([50, 33], H, d, "bf16", seed=H), per, False)
    compare(make([50, 33], H, d, "f32", affine="shared", seed=H + 1), per, True)


@pytest.mark.parametrize("per", ["token", "sequence"])
def test_affine_forms(per):
    for affine, bias in (("none", False), ("own", False), ("shared", True), ("none", True)):
        compare(make([20, 5], 4, 32, affine=affine, bias=bias, seed=2), per)


@pytest.mark.parametrize("lengths", [[1], [1] * 40, [700], [0, 0, 3], [300, 1, 0, 2, 513, 64]])
def test_sequence_lengths(lengths):
    compare(make(lengths, 2, 48, seed=3), "sequence")
    compare(make(lengths, 2, 48, "bf16", gate=False, seed=4), "sequence", False)


def test_thousands_of_sequences():
    lengths = torch.randint(0, 4, (1500,), generator=torch.Generator().manual_seed(15)).tolist()
    compare(make(lengths, 2, 32, "bf16", seed=15), "sequence")


def test_rows_and_many_tokens():
    compare(make([130] * 3, 4, 64, "bf16", seed=5, rows=True), "sequence")
    compare(make([130] * 3, 4, 64, "bf16", seed=6, rows=True), "token")
    compare(make([5000], 3, 32, "f32", seed=7), "token")
    compare(make([5000, 3000], 3, 32, "f32", seed=8), "sequence")


def test_a_mean_far_from_zero():
    """The variance is taken about the mean: no squares of the mean cancel."""
    compare(make([400, 30], 2, 64, seed=9, mean=50.0), "sequence")
    compare(make([20, 30], 2, 64, seed=9, mean=50.0), "token")


def test_constant_groups_and_zero():
    x = make([6, 4], 2, 32, seed=10)
    x["x"][:] = 0
    for per in ("token", "sequence"):
        compare(x, per, True)
        compare(x, per, False)


@pytest.mark.parametrize("per", ["token", "sequence"])
def test_groups_do_not_see_another_ones_nan(per):
    x = make([10, 50, 7], 3, 64, seed=11)
    d = dev(x)
    kw = dict(per=per, output_stats=per == "sequence")
    ref = gdr.group_norm_fwd(d["x"], d["w"], d["b"], d["z"], d["cu_t"], **kw)
    bad = d["x"].clone()
    bad[0, 10:60, 1] = float("nan")
    got = gdr.group_norm_fwd(bad, d["w"], d["b"], d["z"], d["cu_t"], **kw)
    y, y2 = (t[0] if per == "sequence" else t for t in (ref, got))
    keep = torch.ones(67, 3, dtype=torch.bool, device="cuda")
    keep[10:60, 1] = False
    assert torch.equal(y2[0][keep], y[0][keep]) and y2[0][~keep].isnan().all()
    stats = [t[1] if per == "sequence" else None for t in (ref, got)]
    g = [gdr.group_norm_bwd(t, d["w"], d["b"], d["z"], d["dy"], d["cu_t"], per=per, stats=s)
         for t, s in zip((d["x"], bad), stats)]
    assert torch.equal(g[1][0][0][keep], g[0][0][0][keep])
    assert torch.equal(g[1][3][0][keep], g[0][3][0][keep])


def test_empty_calls():
    e = torch.zeros(2, 0, 3, 16, device="cuda")
    w = torch.ones(3, 16, device="cuda")
    assert gdr.group_norm_fwd(e, w).shape == e.shape
    y, st = gdr.group_norm_fwd(e, w, per="sequence", output_stats=True, eps=0.25)
    assert torch.equal(st, torch.tensor([0.0, 2.0], device="cuda").expand(2, 3, 2))
    for per in ("token", "sequence"):
        dx, dw, db, dz = gdr.group_norm_bwd(e, w, None, None, e, per=per, stats=st)
        assert dx.shape == e.shape and not dw.any() and db is None and dz is None


def test_bad_cu_seqlens_is_reported_and_stays_inside():
    H, dd, T = 2, 32, 100
    for cu in ([0, 60, 40, 100], [0, 50, 99], [1, 50, 100], [0, -7, 100], [0, 200, 100]):
        d = dev(make([T], H, dd, seed=12))
        buf = torch.full((T + 8, H, dd), 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        _, st = gdr.group_norm_fwd(d["x"], d["w"], None, None, c, per="sequence", y=buf[None, :T],
                                   output_stats=True, status=status)
        assert status.item() == _abi.GDR_ERR_DEVICE_CHECK, cu
        status.zero_()
        gdr.group_norm_bwd(d["x"], d["w"], None, None, d["dy"], c, per="sequence", stats=st,
                           status=status)
        assert status.item() == _abi.GDR_ERR_DEVICE_CHECK, cu
        assert (buf[T:] == 7).all()


@pytest.mark.parametrize("per", ["token", "sequence"])
def test_streams_graphs_and_repeats(per):
    x, y = make([300, 40], 4, 64, "bf16", seed=13), make([300, 40], 4, 64, "bf16", seed=14)
    d, e = dev(x), dev(y)

    def both(t, **kw):
        out = gdr.group_norm_fwd(t["x"], t["w"], t["b"], t["z"], t["cu_t"], per=per,
                                 output_stats=per == "sequence", **kw)
        out = out if per == "sequence" else (out, None)
        return out[:1] + gdr.group_norm_bwd(t["x"], t["w"], t["b"], t["z"], t["dy"], t["cu_t"],
                                            per=per, stats=out[1], **kw)

    want = [both(d), both(e)]
    assert all(torch.equal(a, b) for a, b in zip(both(d), want[0]))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = both(d)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(d)
    for src, w in zip((x, y), want):
        for k in ("x", "w", "b", "z", "dy"):
            d[k].copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))
