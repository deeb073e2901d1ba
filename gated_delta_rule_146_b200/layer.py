"""The operators around the delta rule: gated linear recurrence, short causal convolution and
group norm (include/gdr.h, "Operators around the recurrence").

As in the package's other entry points, every computation runs in libgdr.so's kernels; this
module checks and marshals torch CUDA tensors and allocates outputs and workspaces.  A call runs
on the tensors' device, on ``stream`` or that device's current stream.  What a call allocates
belongs to the stream it runs on; tensors of other streams are the caller's to order.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext

import torch

from . import _abi
from ._abi import ConvArgs, NormArgs, ScanArgs

_DTYPES = {torch.float32: _abi.F32, torch.bfloat16: _abi.BF16}
_ACTS = {"none": _abi.ACT_NONE, "silu": _abi.ACT_SILU, "sigmoid": _abi.ACT_SIGMOID}


def _code(t):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32") from None


def _check(first, *others):
    """Every given tensor is a contiguous CUDA tensor, all on one device; returns its index."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("gdr kernels take CUDA tensors only (there is no CPU path)")
    if not first.is_contiguous():
        raise ValueError("gdr kernels take contiguous tensors")
    for t in others:
        if t is None:
            continue
        if t.get_device() != dev:
            if t.get_device() < 0:
                raise ValueError("gdr kernels take CUDA tensors only (there is no CPU path)")
            raise ValueError(f"tensors on devices {dev} and {t.get_device()}: one call uses one")
        if not t.is_contiguous():
            raise ValueError("gdr kernels take contiguous tensors")
    return dev


def _expect(name, t, shape, dtype):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:  # (torch.Size is a tuple)
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _expect_channels(name, t, count, dtype=torch.float32):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.numel() != count:
        raise ValueError(f"{name} must hold {count} values, not {t.numel()}")


_HERE = nullcontext()


def _on(dev, stream):
    """(context, raw stream) of a call on device ``dev``: the context makes the device current if
    it is not, and what is allocated in it belongs to the stream."""
    here = dev == torch.cuda.current_device()
    if stream is None:
        return (_HERE if here else torch.cuda.device(dev)), _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"a stream of device {stream.device_index} for tensors on {dev}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _raw_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


# the same without the Stream object: a third of a short call's time otherwise
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _status(status, dev):
    if status is None:
        return None
    if status.dtype != torch.int32 or not status.is_cuda or status.numel() < 1:
        raise TypeError("status must be an int32 CUDA tensor")
    if status.get_device() != dev:
        raise ValueError("status is on another device")
    return status.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _fits(*sizes):
    """ctypes would keep the low 32 bits of a larger size."""
    if max(sizes) > 0x7fffffff:
        raise ValueError("every size must be below 2^31")


def _rows(x, cu_seqlens):
    """(B, T, number of sequences) of a [B, T, ...] tensor."""
    if x.dim() < 3:
        raise ValueError("expected [B, T, channels...]")
    B, T = x.shape[:2]
    _fits(B, T)
    if cu_seqlens is None:
        return B, T, B
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise TypeError("cu_seqlens must be int32 [n_seqs + 1]")
    _fits(cu_seqlens.numel())
    return B, T, cu_seqlens.numel() - 1


def _workspace(size, given, dev):
    if size == 0:
        return None, 0
    if given is None or given.numel() * given.element_size() < size:
        given = torch.empty(size, dtype=torch.uint8, device=dev)
    return given, given.numel() * given.element_size()


def _count(shape):
    n = shape[0] if len(shape) == 1 else shape.numel()
    _fits(n)
    return n


# ---- gated linear recurrence ---------------------------------------------------------------------

def _write(v, g, beta, tied):
    if tied and beta is not None:
        raise ValueError("tied takes the place of beta")
    if g.shape != v.shape:
        raise ValueError("g has the shape of v")
    _code(g)
    if beta is not None:
        _expect("beta", beta, v.shape, g.dtype)
    return _abi.WRITE_TIED if tied else _abi.WRITE_PLAIN if beta is None else _abi.WRITE_GATE


def linear_scan_fwd(v, g, beta=None, h0=None, cu_seqlens=None, *, tied=False, reverse=False,
                    o=None, output_final_state=True, h_final=None, stream=None, status=None):
    """Gated linear recurrence over whole sequences (gdr_scan_fwd):
    h_t = exp(g_t) h_{t-1} + b_t with b = v, beta v, or with ``tied`` (1 - exp(g)) v; o_t = h_t.

    v, g and beta are [B, T, ...] with the same channel axes ([B, T, D] or [B, T, H, d]); h0 is
    [n_seqs, ...] fp32 or None for zero.  With cu_seqlens (int32 [n_seqs + 1], B == 1) the row
    holds packed sequences, else each row is one.  ``reverse`` runs every sequence from its last
    token to its first, in place.  ``status``: an optional int32 CUDA tensor the caller zeroes,
    where a bad cu_seqlens is reported.  h_final may be h0.  Returns (o, h_final [n_seqs, ...]
    fp32, or None)."""
    dev = _check(v, g, beta, h0, cu_seqlens, o, h_final)
    B, T, n = _rows(v, cu_seqlens)
    chan = v.shape[2:]
    a = ScanArgs(B, T, _count(chan), n, _code(v), _code(g), _write(v, g, beta, tied),
                 bool(reverse), _status(status, dev))
    _expect("h0", h0, (n, *chan), torch.float32)
    _expect("o", o, v.shape, v.dtype)
    _expect("h_final", h_final, (n, *chan), torch.float32)
    ctx, raw = _on(dev, stream)
    with ctx:
        if o is None:
            o = torch.empty_like(v)
        if h_final is None and output_final_state:
            h_final = torch.empty((n, *chan), dtype=torch.float32, device=dev)
        _abi.check(_abi.lib().gdr_scan_fwd(
            ctypes.byref(a), v.data_ptr(), g.data_ptr(), _ptr(beta), _ptr(h0), _ptr(cu_seqlens),
            o.data_ptr(), _ptr(h_final), raw))
    return o, h_final


def linear_scan_bwd(v, g, beta, o, dO, h0=None, cu_seqlens=None, dh_final=None, *, tied=False,
                    reverse=False, dh0=True, stream=None, status=None):
    """Backward of ``linear_scan_fwd`` (gdr_scan_bwd): the gradients of <dO, o> +
    <dh_final, h_final>.  ``o`` is the forward's output (the states, read for dg).  Without beta
    and ``tied`` v is not read.  Returns (dv, dg, dbeta, dh0): dbeta None without beta, dh0 fp32
    [n_seqs, ...], None when ``dh0=False``."""
    dev = _check(v, g, beta, o, dO, h0, cu_seqlens, dh_final)
    B, T, n = _rows(v, cu_seqlens)
    chan = v.shape[2:]
    a = ScanArgs(B, T, _count(chan), n, _code(v), _code(g), _write(v, g, beta, tied),
                 bool(reverse), _status(status, dev))
    _expect("o", o, v.shape, v.dtype)
    _expect("dO", dO, v.shape, v.dtype)
    _expect("h0", h0, (n, *chan), torch.float32)
    _expect("dh_final", dh_final, (n, *chan), torch.float32)
    ctx, raw = _on(dev, stream)
    with ctx:
        dv, dg = torch.empty_like(v), torch.empty_like(g)
        dbeta = None if beta is None else torch.empty_like(beta)
        dh = torch.empty((n, *chan), dtype=torch.float32, device=dev) if dh0 else None
        _abi.check(_abi.lib().gdr_scan_bwd(
            ctypes.byref(a), v.data_ptr(), g.data_ptr(), _ptr(beta), o.data_ptr(), dO.data_ptr(),
            _ptr(h0), _ptr(cu_seqlens), _ptr(dh_final), dv.data_ptr(), dg.data_ptr(), _ptr(dbeta),
            _ptr(dh), raw))
    return dv, dg, dbeta, dh


def linear_scan_step(v, g, beta, h, *, tied=False, h_out=None, o=None, stream=None):
    """One token for each of N sequences (gdr_scan_step): v, g, beta [N, ...]; h [N, ...] fp32,
    updated in place, or left as it is with the new state in ``h_out``.  Returns o [N, ...]."""
    dev = _check(v, g, beta, h, h_out, o)
    if v.dim() < 2:
        raise ValueError("expected [N, channels...]")
    N, chan = v.shape[0], v.shape[1:]
    _fits(N)
    a = ScanArgs(N, 1, _count(chan), N, _code(v), _code(g), _write(v, g, beta, tied), 0, None)
    _expect("h", h, v.shape, torch.float32)
    _expect("h_out", h_out, v.shape, torch.float32)
    _expect("o", o, v.shape, v.dtype)
    ctx, raw = _on(dev, stream)
    with ctx:
        if o is None:
            o = torch.empty_like(v)
        if N:
            _abi.check(_abi.lib().gdr_scan_step(
                ctypes.byref(a), v.data_ptr(), g.data_ptr(), _ptr(beta), h.data_ptr(),
                (h if h_out is None else h_out).data_ptr(), o.data_ptr(), raw))
    return o


# ---- short convolution ----------------------------------------------------------------------------

def _activation(name):
    try:
        return _ACTS[name]
    except KeyError:
        raise ValueError(f"unknown activation {name!r}; use {', '.join(_ACTS)}") from None


def _conv_weights(weight, bias, D):
    if weight.dim() < 2 or weight.numel() != D * weight.shape[-1]:
        raise ValueError(f"weight must be [channels, width] for {D} channels")
    _expect_channels("weight", weight, D * weight.shape[-1])
    _expect_channels("bias", bias, D)
    _fits(weight.shape[-1])
    return weight.shape[-1]


def short_conv_fwd(x, weight, bias=None, state=None, cu_seqlens=None, *, activation="silu",
                   reverse=False, y=None, output_final_state=True, state_out=None, stream=None,
                   status=None):
    """Short causal depthwise convolution with an activation (gdr_conv_fwd):
    y_t = act(bias + sum_j weight[:, W-1-j] x_{t-j}), W = 2, 3 or 4, act "silu" or "none".

    x is [B, T, ...]; weight [channels..., W] and bias [channels...] fp32; state
    [n_seqs, W - 1, ...] of x's dtype holds the inputs before every sequence, oldest first (None:
    zeros).  cu_seqlens, ``reverse`` and ``status`` as in ``linear_scan_fwd``.  Returns (y,
    state_out [n_seqs, W - 1, ...], the inputs to continue from, or None)."""
    dev = _check(x, weight, bias, state, cu_seqlens, y, state_out)
    B, T, n = _rows(x, cu_seqlens)
    chan = x.shape[2:]
    D = _count(chan)
    W = _conv_weights(weight, bias, D)
    a = ConvArgs(B, T, D, n, W, _code(x), _activation(activation), bool(reverse),
                 _status(status, dev))
    _expect("state", state, (n, W - 1, *chan), x.dtype)
    _expect("state_out", state_out, (n, W - 1, *chan), x.dtype)
    _expect("y", y, x.shape, x.dtype)
    ctx, raw = _on(dev, stream)
    with ctx:
        if y is None:
            y = torch.empty_like(x)
        if state_out is None and output_final_state:
            state_out = torch.empty((n, W - 1, *chan), dtype=x.dtype, device=dev)
        _abi.check(_abi.lib().gdr_conv_fwd(
            ctypes.byref(a), x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state),
            _ptr(cu_seqlens), y.data_ptr(), _ptr(state_out), raw))
    return y, state_out


def short_conv_bwd(x, weight, bias, dy, state=None, cu_seqlens=None, *, activation="silu",
                   reverse=False, workspace=None, stream=None, status=None):
    """Backward of ``short_conv_fwd`` (gdr_conv_bwd): the gradients of <dy, y>.  Returns (dx,
    dweight, dbias, dstate): fp32 for the weights; dbias and dstate None without bias and
    state."""
    dev = _check(x, weight, bias, dy, state, cu_seqlens, workspace)
    B, T, n = _rows(x, cu_seqlens)
    chan = x.shape[2:]
    D = _count(chan)
    W = _conv_weights(weight, bias, D)
    a = ConvArgs(B, T, D, n, W, _code(x), _activation(activation), bool(reverse),
                 _status(status, dev))
    _expect("dy", dy, x.shape, x.dtype)
    _expect("state", state, (n, W - 1, *chan), x.dtype)
    ctx, raw = _on(dev, stream)
    lib = _abi.lib()
    with ctx:
        ws, size = _workspace(lib.gdr_conv_bwd_workspace_size(ctypes.byref(a)), workspace, dev)
        dx, dw = torch.empty_like(x), torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        ds = None if state is None else torch.empty_like(state)
        _abi.check(lib.gdr_conv_bwd(
            ctypes.byref(a), x.data_ptr(), weight.data_ptr(), _ptr(bias), dy.data_ptr(),
            _ptr(state), _ptr(cu_seqlens), dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(ds),
            _ptr(ws), size, raw))
    return dx, dw, db, ds


def short_conv_step(x, weight, bias, state, *, activation="silu", state_out=None, y=None,
                    stream=None):
    """One token for each of N sequences (gdr_conv_step): x [N, ...]; state [N, W - 1, ...],
    x appended in place, or left as it is with the new one in ``state_out``.  Returns y."""
    dev = _check(x, weight, bias, state, state_out, y)
    if x.dim() < 2:
        raise ValueError("expected [N, channels...]")
    N, chan = x.shape[0], x.shape[1:]
    _fits(N)
    D = _count(chan)
    W = _conv_weights(weight, bias, D)
    a = ConvArgs(N, 1, D, N, W, _code(x), _activation(activation), 0, None)
    _expect("state", state, (N, W - 1, *chan), x.dtype)
    _expect("state_out", state_out, (N, W - 1, *chan), x.dtype)
    _expect("y", y, x.shape, x.dtype)
    ctx, raw = _on(dev, stream)
    with ctx:
        if y is None:
            y = torch.empty_like(x)
        if N:
            _abi.check(_abi.lib().gdr_conv_step(
                ctypes.byref(a), x.data_ptr(), weight.data_ptr(), _ptr(bias), state.data_ptr(),
                (state if state_out is None else state_out).data_ptr(), y.data_ptr(), raw))
    return y


# ---- group norm -----------------------------------------------------------------------------------

def _norm_args(x, weight, bias, z, cu_seqlens, per, center, activation, eps, status, dev):
    if x.dim() != 4:
        raise ValueError("expected x [B, T, H, d]")
    if per not in ("token", "sequence"):
        raise ValueError('per is "token" or "sequence"')
    H, d = x.shape[2:]
    _fits(H, d)
    cu = cu_seqlens if per == "sequence" else None
    B, T, n = _rows(x, cu)
    shape = next((tuple(t.shape) for t in (weight, bias) if t is not None), (H, d))
    if shape not in ((H, d), (d,)):
        raise ValueError(f"weight and bias are [{H}, {d}] or [{d}]")
    _expect("weight", weight, shape, torch.float32)
    _expect("bias", bias, shape, torch.float32)
    _expect("z", z, x.shape, x.dtype)
    a = NormArgs(B, T, H, d, n, _code(x), per == "sequence", bool(center),
                 _activation(activation), len(shape) == 1, float(eps), _status(status, dev))
    return a, cu, (n, H, 2)


def group_norm_fwd(x, weight=None, bias=None, z=None, cu_seqlens=None, *, per="token",
                   center=True, activation="silu", eps=1e-6, y=None, output_stats=False,
                   workspace=None, stream=None, status=None):
    """Group norm with an activation, channels last (gdr_norm_fwd); the groups are the heads of x
    [B, T, H, d].  n = (x - mean) / sqrt(var + eps), or x / sqrt(mean(x^2) + eps) without
    ``center``; u = n weight + bias; y = u act(z) with a gate z, act(u) without; act "silu",
    "sigmoid" or "none".

    The statistics are over each token's d channels (``per="token"``) or over all tokens of a
    sequence (``per="sequence"``: rows, or the packed sequences of cu_seqlens).  weight and bias
    are fp32 [H, d], or [d] for all heads.  Returns y, or with ``output_stats`` (per sequence)
    (y, stats [n_seqs, H, 2]), which the backward takes."""
    dev = _check(x, weight, bias, z, cu_seqlens, y, workspace)
    a, cu, stats_shape = _norm_args(x, weight, bias, z, cu_seqlens, per, center, activation, eps,
                                    status, dev)
    if output_stats and per != "sequence":
        raise ValueError('stats go with per="sequence"')
    _expect("y", y, x.shape, x.dtype)
    ctx, raw = _on(dev, stream)
    lib = _abi.lib()
    with ctx:
        if y is None:
            y = torch.empty_like(x)
        stats = torch.empty(stats_shape, dtype=torch.float32, device=dev) if output_stats else None
        ws, size = None, 0
        if per == "sequence":
            ws, size = _workspace(lib.gdr_norm_fwd_workspace_size(ctypes.byref(a)), workspace, dev)
        _abi.check(lib.gdr_norm_fwd(
            ctypes.byref(a), x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(z), _ptr(cu),
            y.data_ptr(), _ptr(stats), _ptr(ws), size, raw))
    return (y, stats) if output_stats else y


def group_norm_bwd(x, weight, bias, z, dy, cu_seqlens=None, *, per="token", center=True,
                   activation="silu", eps=1e-6, stats=None, workspace=None, stream=None,
                   status=None):
    """Backward of ``group_norm_fwd`` (gdr_norm_bwd): the gradients of <dy, y>.  ``stats``: the
    forward's, required with ``per="sequence"``.  Returns (dx, dweight, dbias, dz), None for
    what was not given."""
    dev = _check(x, weight, bias, z, dy, cu_seqlens, stats, workspace)
    a, cu, stats_shape = _norm_args(x, weight, bias, z, cu_seqlens, per, center, activation, eps,
                                    status, dev)
    _expect("dy", dy, x.shape, x.dtype)
    if per == "sequence" and stats is None:
        raise ValueError('per="sequence" takes the forward\'s stats')
    _expect("stats", stats, stats_shape, torch.float32)
    ctx, raw = _on(dev, stream)
    lib = _abi.lib()
    with ctx:
        ws, size = _workspace(lib.gdr_norm_bwd_workspace_size(ctypes.byref(a)), workspace, dev)
        dx = torch.empty_like(x)
        dw = None if weight is None else torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        dz = None if z is None else torch.empty_like(z)
        _abi.check(lib.gdr_norm_bwd(
            ctypes.byref(a), x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(z), dy.data_ptr(),
            _ptr(cu), _ptr(stats), dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(dz), _ptr(ws), size,
            raw))
    return dx, dw, db, dz
