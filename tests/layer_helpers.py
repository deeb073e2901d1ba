"""Tolerances of the operators around the recurrence, derived from their arithmetic.

E = 2^-24 is half a step of fp32; a result written in bf16 is off by half a step of bf16 more,
2^-8 of its size.  CUDA's expf and expm1f are off by at most one step, 2 E.

scan.  Per token alpha is off by 2 E (tied: 1 + expm1(g) by 2 E |1 - alpha| + E, absolute, at
most 3 E max(1, alpha)) and the multiply-add rounds once; joining runs multiplies decays (one
rounding per token) and adds one multiply-add.  So a state's error grows per token by at most
4 E max(1, alpha) M, with M the same recurrence over |b| and |h0|, and is carried on with alpha:
    N_t = alpha N_{t-1} + max(1, alpha) M_{t-1} + 2 |b_t|,     |error_t| <= 4 E (N_t + M_t).
The backward's m runs the same recurrence over dO; the products behind it round up to four times.

conv.  p: W + 1 roundings of sums not above P = |bias| + sum |w x|.  Activation: slope at most
1.1, own roundings at most 8 E |y| (exponential 2, sum, division, products, each one or two).
dp = dy act'(p): act' changes by at most 0.5 per unit of p and is formed within 24 E.  dx adds
W + 1 roundings; dw and dbias add up to K = 300 terms one after the other (a run of at most 256
tokens, then the block's runs, then the rows in eight parts).

norm.  A lane adds at most 32 values, a group's lanes add in 5 steps, a sequence's pieces in up
to 60 more: K = 100 additions, each E of the sum of magnitudes.  With mu = mean |x| of a group
the centred value is off by E (|x - mean| + K mu), rstd by (K + 8) E relative to within K E mu
rstd, so |dn| <= E ((K + 10) |n| + 2 K rstd mu (1 + |n|)).  The rest follows as for conv.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import layer as ol

E = 2.0 ** -24
HALF = {torch.float32: E, torch.bfloat16: 2.0 ** -8}


def check(name, got, want, tol, dtype=None):
    """|got - want| <= tol, plus the rounding to dtype where the result is written in one."""
    g = ol.f64(got)
    assert g.shape == want.shape, (name, g.shape, want.shape)
    assert np.array_equal(np.isfinite(g), np.isfinite(want)), name
    assert np.array_equal(np.isnan(g), np.isnan(want)), name
    fine = np.isfinite(want)
    allowed = np.broadcast_to(tol, want.shape) + (HALF[dtype] * (np.abs(want) + tol) if dtype else 0)
    err = np.abs(g - want)[fine]
    bad = err > allowed[fine]
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} beyond the bound, worst "
                           f"{(err / np.maximum(allowed[fine], 1e-300)).max():.3g} of it")


def scan_tol(al, b, start, cu, reverse=False):
    """(bound per token, bound of the state behind each sequence) of x <- al x + b from
    ``start`` (None: zero)."""
    al, b = np.nan_to_num(al, posinf=0.0), np.abs(np.nan_to_num(b, posinf=0.0, neginf=0.0))
    tol = np.zeros_like(b)
    end = np.zeros((len(cu) - 1, b.shape[1]))
    for s, toks in enumerate(ol.spans(cu, reverse)):
        M = np.zeros(b.shape[1]) if start is None else np.abs(ol.f64(start)[s])
        N = np.zeros(b.shape[1])
        for t in toks:
            N = al[t] * N + np.maximum(1.0, al[t]) * M + 2 * b[t]
            M = al[t] * M + b[t]
            tol[t] = 4 * E * (N + M)
        end[s] = 4 * E * (N + M)
    return tol, end


def scan_fwd_tol(v, g, beta, h0, cu, tied, reverse):
    v, g, beta = ol.f64(v), ol.f64(g), ol.f64(beta)
    al, w = ol.writes(v, g, beta, tied)
    return scan_tol(al, w * v, h0, cu, reverse)


def scan_bwd_tol(v, g, beta, o, dO, h0, dhf, cu, tied, reverse):
    """Bounds of (dv, dg, dbeta, dh0)."""
    v, g, beta, o, dO = (ol.f64(t) for t in (v, g, beta, o, dO))
    al, w = ol.writes(v, g, beta, tied)
    # m_t = alpha_t (m_{t+1} + dO_t): the recurrence over alpha dO, the other way round
    m_tol, end = scan_tol(al, np.abs(al * dO), dhf, cu, not reverse)
    big = np.zeros_like(v)   # |m_{t+1}| and its bound, beside |dO_t|
    lam_tol, before = np.zeros_like(v), np.zeros_like(v)
    for s, toks in enumerate(ol.spans(cu, reverse)):
        M = np.zeros(v.shape[1]) if dhf is None else np.abs(ol.f64(dhf)[s])
        T = np.zeros(v.shape[1])
        for i in range(len(toks) - 1, -1, -1):
            t = toks[i]
            big[t] = M + np.abs(dO[t])
            lam_tol[t] = T + E * big[t]
            T, M = m_tol[t], al[t] * big[t]
            before[t] = np.abs(o[toks[i - 1]]) if i else (0 if h0 is None else np.abs(ol.f64(h0)[s]))
    reach = before + (np.abs(v) if tied else 0)
    dv = np.abs(w) * lam_tol + 4 * E * np.abs(w) * big
    dg = m_tol * reach + 4 * E * al * big * reach
    return dv, dg, np.abs(v) * (lam_tol + 4 * E * big), end


def conv_tol(x, w, bias, dy, state, cu, name, reverse):
    """Bounds of (y, dx, dw, dbias, dstate); those of the gradients only with dy."""
    W = w.shape[1]
    y, _, p = ol.conv(x, w, bias, state, cu, name, reverse)
    a = lambda t: None if t is None else np.abs(ol.f64(t))  # noqa: E731
    P = ol.conv(a(x), a(w), a(bias), a(state), cu, "none", reverse)[0]
    dp_err = (W + 1) * E * P
    yt = 1.1 * dp_err + 8 * E * np.abs(y)
    if dy is None:
        return yt
    ady = a(dy)
    ddp = ady * (0.5 * dp_err + 24 * E)
    top = ady * 1.1
    per = [ol.conv_backward(a(x), a(w), None, t, a(state), cu, "none", reverse) for t in (ddp, top)]
    K = 300
    return (yt, per[0][0] + (W + 1) * E * per[1][0], per[0][1] + K * E * per[1][1],
            per[0][2] + K * E * per[1][2], per[0][3] + (W + 1) * E * per[1][3])


def norm_tol(x, w, b, z, dy, cu, per, center, name, eps):
    """Bounds of (y, dx, dw, db, dz); those of the gradients only with dy."""
    K = 100
    x, z, dy = ol.f64(x), ol.f64(z), ol.f64(dy)
    H, d = x.shape[1:]
    w = np.ones((H, d)) if w is None else np.broadcast_to(ol.f64(w), (H, d))
    b = np.zeros((H, d)) if b is None else np.broadcast_to(ol.f64(b), (H, d))
    _, stats = ol.norm(x, w, b, z, cu, per, center, name, eps)
    out = [np.zeros_like(x), np.zeros_like(x), np.zeros((H, d)), np.zeros((H, d)), np.zeros_like(x)]
    for i, t in enumerate(ol.groups(cu, x.shape[0], per)):
        if not len(t):
            continue
        mean, rstd = stats[i, :, 0][None, :, None], stats[i, :, 1][None, :, None]
        n = (x[t] - mean) * rstd
        mu = np.abs(x[t]).mean((0, 2), keepdims=True) * center
        dn = E * ((K + 10) * np.abs(n) + 2 * K * rstd * mu * (1 + np.abs(n)))
        u = n * w + b
        du_ = np.abs(w) * dn + 2 * E * (np.abs(n * w) + np.abs(b))
        if z is None:
            y = ol.act(u, name)
            out[0][t] = 1.1 * du_ + 8 * E * np.abs(y)
        else:
            az = np.abs(ol.act(z[t], name))
            out[0][t] = du_ * az + 9 * E * np.abs(u) * az
        if dy is None:
            continue
        g = np.abs(dy[t])
        if z is None:
            G = g * np.abs(ol.act_grad(u, name))
            e = g * (0.5 * du_ + 24 * E)
        else:
            G = g * az
            e = 9 * E * G
            out[4][t] = g * (1.1 * du_ + 24 * E * np.abs(u))
        out[2] += (e * np.abs(n) + G * dn + 300 * E * G * np.abs(n)).sum(0)
        out[3] += (e + 300 * E * G).sum(0)
        q, qe = G * np.abs(w), (e + E * G) * np.abs(w)
        m = lambda v: v.mean((0, 2), keepdims=True)  # noqa: E731
        an = np.abs(n)
        size = q + m(q) + an * m(q * an)
        err = (qe + m(qe) + K * E * m(q) + an * (m(qe * an) + m(q * dn) + K * E * m(q * an))
               + dn * m(q * an))
        out[1][t] = rstd * (err + size * ((K + 12) * E + 2 * K * E * rstd * mu))
    return out[0] if dy is None else out
