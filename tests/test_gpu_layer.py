"""The operators together, as a recurrent layer uses them: convolution, recurrence, gated norm,
with gradients through all three, and one token at a time behind a prefill."""
import numpy as np
import pytest
import torch

import gated_delta_rule_146_b200 as gdr
from gated_delta_rule_146_b200 import _abi
from oracle import layer as ol

pytestmark = pytest.mark.gpu


def layer_inputs(T, H, d, n, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    D = H * d
    return dict(x=rn(1, T, D).to(dtype), w=0.5 * rn(D, 4), b=0.2 * rn(D),
                g=(-torch.nn.functional.softplus(rn(1, T, D) - 2)).to(dtype),
                z=rn(1, T, H, d).to(dtype), nw=1 + 0.1 * rn(d), dy=rn(1, T, H, d).to(dtype),
                st=rn(n, 3, D).to(dtype), h0=rn(n, D))


def reference(x, cu, H, d):
    f = {k: ol.f64(t) for k, t in x.items()}
    flat = {k: f[k].reshape(-1, H * d) for k in ("x", "g")}
    v, st, _ = ol.conv(flat["x"], f["w"], f["b"], f["st"], cu)
    h, hf = ol.scan(v, flat["g"], None, f["h0"], cu, tied=True)
    z, dy = (f[k].reshape(-1, H, d) for k in ("z", "dy"))
    y, _ = ol.norm(h.reshape(-1, H, d), f["nw"], None, z, cu, center=False)
    dh, dnw, _, dz = ol.norm_backward(h.reshape(-1, H, d), f["nw"], None, z, dy, cu, center=False)
    dv, dg, _, dh0 = ol.scan_backward(v, flat["g"], None, h, dh.reshape(-1, H * d), f["h0"], None,
                                      cu, tied=True)
    dx, dw, db, dst = ol.conv_backward(flat["x"], f["w"], f["b"], dv, f["st"], cu)
    return dict(y=y, st=st, hf=hf, dnw=dnw.sum(0), dz=dz, dg=dg, dh0=dh0, dx=dx, dw=dw, db=db, dst=dst)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_layer_with_its_gradients(dtype):
    H, d, lengths = 3, 64, [70, 0, 1, 130]
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    x = layer_inputs(cu[-1], H, d, len(lengths), dtype, 1)
    t = {k: v.cuda() for k, v in x.items()}
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    v, st = gdr.short_conv_fwd(t["x"], t["w"], t["b"], t["st"], c)
    h, hf = gdr.linear_scan_fwd(v, t["g"], None, t["h0"], c, tied=True)
    hh = h.view(1, -1, H, d)
    y = gdr.group_norm_fwd(hh, t["nw"], None, t["z"], center=False)
    dh, dnw, _, dz = gdr.group_norm_bwd(hh, t["nw"], None, t["z"], t["dy"], center=False)
    dv, dg, _, dh0 = gdr.linear_scan_bwd(v, t["g"], None, h, dh.view_as(v), t["h0"], c, tied=True)
    dx, dw, db, dst = gdr.short_conv_bwd(t["x"], t["w"], t["b"], dv, t["st"], c)
    got = dict(y=y, st=st, hf=hf, dnw=dnw, dz=dz, dg=dg, dh0=dh0, dx=dx, dw=dw, db=db, dst=dst)
    want = reference(x, cu, H, d)
    # Relative to the tensor's 2-norm.  fp32: each operator is within a few hundred steps of its
    # inputs' precision (layer_helpers), 6e-8 each.  bf16: at most six tensors rounded on the
    # way (v, h, dh, dv and the result, v and h taken twice), each off by 2^-8 at most and a
    # third of a step's square on average, 2^-8 / sqrt(3); the norm's division by small groups
    # can double a share.
    tol = 3e-5 if dtype == torch.float32 else 2 * 6 ** 0.5 * 2.0 ** -8
    for k, w in want.items():
        a = ol.f64(got[k]).reshape(w.shape)
        off = np.linalg.norm(a - w) / np.linalg.norm(w)
        assert off <= (0 if k == "st" else tol), (k, off)


def test_prefill_then_tokens():
    """A prompt through the sequence forms, then single tokens from the states they leave, equal
    the whole sequence through the sequence forms."""
    N, T, extra, H, d = 3, 33, 6, 2, 64
    x = layer_inputs(N * (T + extra), H, d, N, torch.bfloat16, 2)
    t = {k: v.cuda() for k, v in x.items()}
    D = H * d
    rows = {k: t[k].view(N, T + extra, D) for k in ("x", "g", "z")}

    def sequence(lo, hi, st, h):
        part = {k: v[:, lo:hi].contiguous() for k, v in rows.items()}
        v, st = gdr.short_conv_fwd(part["x"], t["w"], t["b"], st)
        o, h = gdr.linear_scan_fwd(v, part["g"], None, h, tied=True)
        return gdr.group_norm_fwd(o.view(N, hi - lo, H, d), t["nw"], None,
                                  part["z"].view(N, hi - lo, H, d), center=False), st, h

    whole, st_w, h_w = sequence(0, T + extra, t["st"], t["h0"])
    y, st, h = sequence(0, T, t["st"], t["h0"])
    outs = [y]
    for i in range(T, T + extra):
        tok = {k: v[:, i].contiguous() for k, v in rows.items()}
        v = gdr.short_conv_step(tok["x"], t["w"], t["b"], st)
        o = gdr.linear_scan_step(v, tok["g"], None, h, tied=True)
        outs.append(gdr.group_norm_fwd(o.view(N, 1, H, d), t["nw"], None,
                                       tok["z"].view(N, 1, H, d), center=False))
    assert torch.equal(st, st_w)
    # the scan joins its runs in another order than the tokens one by one: fp32 states differ by
    # a few steps, and a bf16 value next to a border by one step of bf16, twice (o and y)
    assert (h - h_w).abs().max() <= 1e-5 * h_w.abs().max()
    got, want = torch.cat(outs, 1).float(), whole.float()
    assert ((got - want).abs() <= 2.0 ** -6 * want.abs() + 1e-3).all()
    assert (got != want).float().mean() < 0.02


def test_the_norm_behind_the_delta_rule():
    """The output norm of the decode step's epilogue, for whole sequences behind chunk_fwd."""
    H, d, T = 2, 64, 100
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    q, k, v, z = (rn(1, T, H, d) for _ in range(4))
    gate, beta = -torch.nn.functional.softplus(rn(1, T, H) - 2), torch.sigmoid(rn(1, T, H))
    w = 1 + 0.1 * rn(d)
    o, _ = gdr.chunk_fwd(q, k, v, gate, beta)
    y = gdr.group_norm_fwd(o, w, None, z, center=False, eps=1e-6)
    S = torch.zeros(1, H, d, d, device="cuda")
    for t in range(T):
        step = gdr.decode_step(*(a[:, t].clone() for a in (q, k, v, gate, beta)), S,
                               norm_z=z[:, t].clone(), norm_weight=w, norm_eps=1e-6)
        # both within 1e-4 of the recurrence (the bound of its fp32 form), times the norm's gain
        scale = 1 / o[:, t].square().mean(-1, keepdim=True).sqrt()
        assert ((step - y[:, t]).abs() <= 3e-4 * (1 + scale) * (1 + z[:, t].abs())).all()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one GPU")
def test_tensors_of_another_device_than_the_current_one():
    x = torch.randn(1, 70, 64, device="cuda:1")
    w = torch.randn(64, 4, device="cuda:1")
    with torch.cuda.device(0):
        a, _ = gdr.short_conv_fwd(x, w)
        b, _ = gdr.linear_scan_fwd(x, -x.abs())
    with torch.cuda.device(1):
        assert torch.equal(a, gdr.short_conv_fwd(x, w)[0])
        assert torch.equal(b, gdr.linear_scan_fwd(x, -x.abs())[0])


def _tail(t, n):
    return t[:, -n:].contiguous()


def test_offsets_beyond_31_bits():
    """More than 2^31 elements a tensor: the last tokens, cut off from the others by the
    operators' own means, equal the same tokens in a short call."""
    D, n = 4096, 700
    T = (1 << 31) // D + 1000
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    g = torch.empty_like(x).uniform_(-1.0, -0.1, generator=gen)
    close = lambda a, b: ((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 1e-3).all()  # noqa: E731
    o, hf = gdr.linear_scan_fwd(x, g, None, None, cu)
    os_, hs = gdr.linear_scan_fwd(_tail(x, n), _tail(g, n), None, None, one)
    assert close(_tail(o, n), os_) and (hf[1] - hs[0]).abs().max() < 1e-4
    dv, dg, _, _ = gdr.linear_scan_bwd(x, g, None, o, x, None, cu)
    a = gdr.linear_scan_bwd(_tail(x, n), _tail(g, n), None, _tail(o, n), _tail(x, n), None, one)
    assert close(_tail(dv, n), a[0]) and close(_tail(dg, n), a[1])
    del dv, dg, g
    w = torch.randn(D, 4, device="cuda", generator=gen)
    y, st = gdr.short_conv_fwd(x, w, cu_seqlens=cu)
    ys, ss = gdr.short_conv_fwd(_tail(x, n), w, cu_seqlens=one)
    assert torch.equal(_tail(y, n), ys) and torch.equal(st[1:], ss)
    dx = gdr.short_conv_bwd(x, w, None, o, None, cu)[0]
    assert torch.equal(_tail(dx, n), gdr.short_conv_bwd(_tail(x, n), w, None, _tail(o, n), None, one)[0])
    del dx, y
    h = (1, T, 32, 128)
    nw = torch.rand(32, 128, device="cuda", generator=gen) + 0.5
    for per in ("token", "sequence"):
        big = gdr.group_norm_fwd(x.view(h), nw, None, o.view(h), cu, per=per, output_stats=per == "sequence")
        small = gdr.group_norm_fwd(_tail(x, n).view(1, n, 32, 128), nw, None,
                                   _tail(o, n).view(1, n, 32, 128), one, per=per,
                                   output_stats=per == "sequence")
        big, st = big if per == "sequence" else (big, None)
        small, ss = small if per == "sequence" else (small, None)
        assert close(_tail(big, n), small)
        a = gdr.group_norm_bwd(x.view(h), nw, None, None, o.view(h), cu, per=per, stats=st)[0]
        b = gdr.group_norm_bwd(_tail(x, n).view(1, n, 32, 128), nw, None, None,
                               _tail(o, n).view(1, n, 32, 128), one, per=per, stats=ss)[0]
        assert close(_tail(a, n), b)
        del big, a


def run_layer(t, c, H, d, **kw):
    """Forward and backward of all operators, the norm per token and per sequence."""
    v, st = gdr.short_conv_fwd(t["x"], t["w"], t["b"], t["st"], c, **kw)
    h, hf = gdr.linear_scan_fwd(v, t["g"], None, t["h0"], c, tied=True, **kw)
    hh = h.view(1, -1, H, d)
    y = gdr.group_norm_fwd(hh, t["nw"], None, t["z"], center=False, **kw)
    ys, stats = gdr.group_norm_fwd(hh, t["nw"], None, t["z"], c, per="sequence", output_stats=True,
                                   **kw)
    dh, dnw, _, dz = gdr.group_norm_bwd(hh, t["nw"], None, t["z"], t["dy"], center=False, **kw)
    sh, snw, _, sz = gdr.group_norm_bwd(hh, t["nw"], None, t["z"], t["dy"], c, per="sequence",
                                        stats=stats, **kw)
    dv, dg, _, dh0 = gdr.linear_scan_bwd(v, t["g"], None, h, dh.view_as(v), t["h0"], c, tied=True,
                                         **kw)
    dx, dw, db, dst = gdr.short_conv_bwd(t["x"], t["w"], t["b"], dv, t["st"], c, **kw)
    return [st, h, hf, y, ys, stats, dh, dnw, dz, sh, snw, sz, dv, dg, dh0, dx, dw, db, dst]


def test_calls_that_overlap_on_two_streams():
    """Two layers' calls at once, eagerly and as two graphs' replays, give the bits of calls one
    after the other.  Clusters' walks (few slabs) and single blocks' (many) meet."""
    sizes = [(4, 64, [900, 0, 1, 300]), (64, 128, [500, 77])]
    cases, want = [], []
    for i, (H, d, lengths) in enumerate(sizes):
        cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
        t = {k: v.cuda() for k, v in layer_inputs(cu[-1], H, d, len(lengths), torch.bfloat16,
                                                  20 + i).items()}
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        cases.append((t, c, H, d))
        want.append(run_layer(*cases[-1]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(6):
        for i, case in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(run_layer(*case))
    torch.cuda.synchronize()
    graphs, out = [], []
    for case in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out.append(run_layer(*case))
        graphs.append(g)
    for _ in range(6):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        for r in got[i] + [out[i]]:
            assert all(torch.equal(a, b) for a, b in zip(r, w)), i


def test_bad_bounds_of_no_tokens_are_reported():
    """A row of no tokens has bounds to check too: [0, 5] does not end at 0, [3, 0] neither
    starts there nor rises.  The results are those of empty sequences all the same."""
    e = torch.empty(1, 0, 4, 16, device="cuda")
    h0 = torch.randn(1, 4, 16, device="cuda")
    w = torch.randn(4, 16, 4, device="cuda")
    past = torch.randn(1, 3, 4, 16, device="cuda")
    stats = torch.ones(1, 4, 2, device="cuda")
    calls = dict(
        scan_fwd=lambda **k: gdr.linear_scan_fwd(e, e, None, h0, **k)[1],
        scan_bwd=lambda **k: gdr.linear_scan_bwd(e, e, None, e, e, None, dh_final=h0, **k)[3],
        conv_fwd=lambda **k: gdr.short_conv_fwd(e, w, None, past, **k)[1],
        conv_bwd=lambda **k: gdr.short_conv_bwd(e, w, None, e, past, **k)[1],
        norm_fwd=lambda **k: gdr.group_norm_fwd(e, per="sequence", eps=0.25, output_stats=True, **k)[1],
        norm_bwd=lambda **k: gdr.group_norm_bwd(e, w[..., 0].contiguous(), None, None, e, stats=stats,
                                                per="sequence", **k)[1])
    want = dict(scan_fwd=h0, scan_bwd=h0, conv_fwd=past, conv_bwd=torch.zeros_like(w),
                norm_fwd=torch.tensor([0.0, 2.0], device="cuda").expand(1, 4, 2),
                norm_bwd=torch.zeros(4, 16, device="cuda"))
    for cu, st in (([0, 0], _abi.GDR_OK), ([0, 5], _abi.GDR_ERR_DEVICE_CHECK),
                   ([3, 0], _abi.GDR_ERR_DEVICE_CHECK), ([-1, 0], _abi.GDR_ERR_DEVICE_CHECK)):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for name, call in calls.items():
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = call(cu_seqlens=c, status=status)
            assert status.item() == st, (name, cu)
            assert torch.equal(got, want[name]), (name, cu)
            assert torch.equal(call(cu_seqlens=c), want[name]), (name, cu)


def test_calls_of_no_tokens_in_a_graph():
    """Captured as a graph's first node, and behind one that is no kernel."""
    e = torch.empty(2, 0, 3, 16, device="cuda")
    w = torch.ones(3, 16, device="cuda")
    for first in (False, True):
        g = torch.cuda.CUDAGraph()
        other = torch.ones(8, device="cuda")
        with torch.cuda.graph(g):
            if not first:
                other.zero_()
            _, st = gdr.group_norm_fwd(e, w, per="sequence", output_stats=True, eps=0.25)
            other.zero_()
            _, dw, _, _ = gdr.group_norm_bwd(e, w, None, None, e, per="sequence", stats=st)
        dw.fill_(1.0)
        g.replay()
        assert torch.equal(st, torch.tensor([0.0, 2.0], device="cuda").expand(2, 3, 2))
        assert not dw.any() and not other.any()


def test_neighbouring_arrays_of_one_buffer():
    """Inputs, outputs and states that touch without sharing a byte go through, with the results
    of arrays of their own."""
    n, T, D = 2, 70, 64
    gen = torch.Generator("cuda").manual_seed(5)
    flat_, state = n * T * D, n * D
    buf = torch.empty(4 * flat_ + 2 * state, device="cuda").normal_(generator=gen)
    v, g, o, y = (buf[i * flat_:(i + 1) * flat_].view(n, T, D) for i in range(4))
    h0, hf = (buf[4 * flat_ + i * state:4 * flat_ + (i + 1) * state].view(n, D) for i in range(2))
    g.abs_().neg_()
    w = torch.randn(D, 4, device="cuda", generator=gen)
    want = gdr.linear_scan_fwd(v.clone(), g.clone(), None, h0.clone())
    gdr.linear_scan_fwd(v, g, None, h0, o=o, h_final=hf)
    assert torch.equal(o, want[0]) and torch.equal(hf, want[1])
    assert torch.equal(gdr.short_conv_fwd(o, w, y=y)[0], gdr.short_conv_fwd(o.clone(), w)[0])
    x4, y4 = o.view(n, T, 1, D), y.view(n, T, 1, D)
    assert torch.equal(gdr.group_norm_fwd(x4, y=y4), gdr.group_norm_fwd(x4.clone()))


def test_outputs_that_begin_inside_an_input_are_refused():
    T, D = 70, 64
    buf = torch.randn(1, T + 1, D, device="cuda")
    x, later = buf[:, :T], buf[:, 1:]
    w = torch.randn(D, 4, device="cuda")
    rows, states = torch.randn(2, T, D, device="cuda"), torch.zeros(3, D, device="cuda")
    for call in (lambda: gdr.linear_scan_fwd(x, -torch.ones_like(x), o=later),
                 lambda: gdr.linear_scan_fwd(rows, -rows.abs(), None, states[:2], h_final=states[1:]),
                 lambda: gdr.short_conv_fwd(x, w, y=later),
                 lambda: gdr.group_norm_fwd(x.view(1, T, 1, D), y=later.view(1, T, 1, D))):
        with pytest.raises(gdr.GdrError):
            call()
