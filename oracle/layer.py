"""fp64 definitions of the operators around the recurrence (NumPy, token by token): the gated
linear recurrence, the short causal convolution and the group norm, each with its gradient.

Tensors are [tokens, channels] (norm: [tokens, heads, d]); ``cu`` holds the sequences' bounds.
Every function takes anything NumPy can view as float64 and returns float64.  With ``reverse``
a sequence runs from its last token to its first.
"""
from __future__ import annotations

import numpy as np


def f64(t):
    if t is None:
        return None
    return np.asarray(t.detach().double().cpu().numpy() if hasattr(t, "detach") else t,
                      dtype=np.float64)


def spans(cu, reverse):
    """The token numbers of every sequence, in scan order."""
    return [np.arange(b, e)[::-1] if reverse else np.arange(b, e) for b, e in zip(cu, cu[1:])]


def writes(v, g, beta, tied):
    """(alpha, factor on v)"""
    al = np.exp(g)
    return al, -np.expm1(g) if tied else np.ones_like(v) if beta is None else beta


def scan(v, g, beta, h0, cu, tied=False, reverse=False):
    """(o, h_final): h_t = alpha_t h_{t-1} + w_t v_t."""
    v, g, beta, h0 = f64(v), f64(g), f64(beta), f64(h0)
    al, w = writes(v, g, beta, tied)
    o = np.zeros_like(v)
    hf = np.zeros((len(cu) - 1, v.shape[1])) if h0 is None else h0.copy()
    for s, toks in enumerate(spans(cu, reverse)):
        h = hf[s]
        for t in toks:
            h = al[t] * h + w[t] * v[t]
            o[t] = h
        hf[s] = h
    return o, hf


def scan_backward(v, g, beta, o, dO, h0, dhf, cu, tied=False, reverse=False):
    """(dv, dg, dbeta, dh0) with h_{t-1} taken from o."""
    v, g, beta, o, dO, h0, dhf = (f64(t) for t in (v, g, beta, o, dO, h0, dhf))
    al, w = writes(v, g, beta, tied)
    dv, dg, db = np.zeros_like(v), np.zeros_like(v), np.zeros_like(v)
    dh0 = np.zeros((len(cu) - 1, v.shape[1])) if dhf is None else dhf.copy()
    for s, toks in enumerate(spans(cu, reverse)):
        m = dh0[s]
        for i in range(len(toks) - 1, -1, -1):
            t = toks[i]
            lam = dO[t] + m
            m = al[t] * lam
            before = o[toks[i - 1]] if i else (0.0 if h0 is None else h0[s])
            dv[t] = w[t] * lam
            dg[t] = m * (before - v[t] if tied else before)
            db[t] = v[t] * lam
        dh0[s] = m
    return dv, dg, None if beta is None else db, dh0


def act(u, name):
    sg = 0.5 * (1.0 + np.tanh(0.5 * u))
    return u if name == "none" else sg if name == "sigmoid" else u * sg


def act_grad(u, name):
    sg = 0.5 * (1.0 + np.tanh(0.5 * u))
    return np.ones_like(u) if name == "none" else sg * (1 - sg) if name == "sigmoid" \
        else sg * (1 + u * (1 - sg))


def conv(x, w, bias, state, cu, name="silu", reverse=False):
    """(y, state_out, p): the last inputs of every sequence, and the sums before the
    activation."""
    x, w, bias, state = f64(x), f64(w), f64(bias), f64(state)
    W = w.shape[1]
    p = np.zeros_like(x)
    out = np.zeros((len(cu) - 1, W - 1, x.shape[1]))
    for s, toks in enumerate(spans(cu, reverse)):
        past = np.zeros((W - 1, x.shape[1])) if state is None else state[s]
        seq = np.concatenate([past, x[toks]])
        for i, t in enumerate(toks):
            p[t] = (seq[i:i + W] * w.T).sum(0) + (0.0 if bias is None else bias)
        out[s] = seq[len(seq) - (W - 1):]
    return act(p, name), out, p


def conv_backward(x, w, bias, dy, state, cu, name="silu", reverse=False):
    """(dx, dw, dbias, dstate)"""
    _, _, p = conv(x, w, bias, state, cu, name, reverse)
    x, w, dy, state = f64(x), f64(w), f64(dy), f64(state)
    W = w.shape[1]
    dp = dy * act_grad(p, name)
    dx, dw = np.zeros_like(x), np.zeros_like(w)
    ds = np.zeros((len(cu) - 1, W - 1, x.shape[1]))
    for s, toks in enumerate(spans(cu, reverse)):
        past = np.zeros((W - 1, x.shape[1])) if state is None else state[s]
        seq = np.concatenate([past, x[toks]])
        dseq = np.zeros_like(seq)
        for i, t in enumerate(toks):
            dw += (seq[i:i + W] * dp[t]).T
            dseq[i:i + W] += w.T * dp[t]
        ds[s], dx[toks] = dseq[:W - 1], dseq[W - 1:]
    return dx, dw, dp.sum(0), ds


def groups(cu, tokens, per):
    return [np.arange(t, t + 1) for t in range(tokens)] if per == "token" else spans(cu, False)


def norm(x, w, b, z, cu, per="token", center=True, name="silu", eps=1e-6):
    """(y, stats [sequences or tokens, heads, 2])"""
    x, w, b, z = f64(x), f64(w), f64(b), f64(z)
    y = np.zeros_like(x)
    gr = groups(cu, x.shape[0], per)
    stats = np.zeros((len(gr), x.shape[1], 2))
    for i, toks in enumerate(gr):
        if not len(toks):
            stats[i, :, 1] = eps ** -0.5
            continue
        mean = x[toks].mean((0, 2), keepdims=True) * center
        rstd = 1 / np.sqrt(((x[toks] - mean) ** 2).mean((0, 2), keepdims=True) + eps)
        stats[i, :, 0], stats[i, :, 1] = mean[0, :, 0], rstd[0, :, 0]
        u = (x[toks] - mean) * rstd * (1.0 if w is None else w) + (0.0 if b is None else b)
        y[toks] = act(u, name) if z is None else u * act(z[toks], name)
    return y, stats


def norm_backward(x, w, b, z, dy, cu, per="token", center=True, name="silu", eps=1e-6):
    """(dx, dw, db, dz), dw and db per head"""
    _, stats = norm(x, w, b, z, cu, per, center, name, eps)
    x, w, b, z, dy = f64(x), f64(w), f64(b), f64(z), f64(dy)
    w = np.ones(x.shape[1:]) if w is None else np.broadcast_to(w, x.shape[1:])
    b = np.zeros(x.shape[1:]) if b is None else b
    dx, dz = np.zeros_like(x), np.zeros_like(x)
    dw, db = np.zeros(x.shape[1:]), np.zeros(x.shape[1:])
    for i, toks in enumerate(groups(cu, x.shape[0], per)):
        if not len(toks):
            continue
        mean, rstd = stats[i, :, 0][None, :, None], stats[i, :, 1][None, :, None]
        n = (x[toks] - mean) * rstd
        u = n * w + b
        if z is None:
            du = dy[toks] * act_grad(u, name)
        else:
            du = dy[toks] * act(z[toks], name)
            dz[toks] = dy[toks] * u * act_grad(z[toks], name)
        dw += (du * n).sum(0)
        db += du.sum(0)
        q = du * w
        dx[toks] = rstd * (q - center * q.mean((0, 2), keepdims=True)
                           - n * (q * n).mean((0, 2), keepdims=True))
    return dx, dw, db, dz
