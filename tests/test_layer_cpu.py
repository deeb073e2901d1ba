"""Host-side validation of the operators around the recurrence: nothing here reaches a GPU.
Every call is refused before a launch (the addresses are never read)."""
import ctypes

import pytest
import torch

import gated_delta_rule_146_b200 as gdr
from gated_delta_rule_146_b200 import _abi, build
from gated_delta_rule_146_b200._abi import ConvArgs, NormArgs, ScanArgs

P = 0x10000
INV, UNS, ALI, WS = (_abi.GDR_ERR_INVALID_ARG, _abi.GDR_ERR_UNSUPPORTED, _abi.GDR_ERR_ALIGNMENT,
                     _abi.GDR_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.lib()


def args(cls, base, kw):
    return ctypes.byref(cls(**{**base, **kw}))


SCAN = dict(B=2, T=100, D=64, n_seqs=2, io_dtype=1, gate_dtype=1, write=0, reverse=0)
CONV = dict(B=2, T=100, D=64, n_seqs=2, width=4, io_dtype=1, activation=1, reverse=0)
NORM = dict(B=2, T=100, H=4, d=64, n_seqs=2, io_dtype=1, per_sequence=0, center=0, activation=1,
            shared_weight=0, eps=1e-6)

BAD_SIZES = [(dict(B=0), INV), (dict(T=-1), INV), (dict(n_seqs=3), INV), (dict(n_seqs=0), INV),
             (dict(B=1 << 16, n_seqs=1 << 16, T=1 << 15), INV), (dict(io_dtype=2), INV)]


@pytest.mark.parametrize("kw,st", BAD_SIZES + [
    (dict(D=0), INV), (dict(D=(1 << 20) + 1), UNS), (dict(gate_dtype=9), INV), (dict(write=3), INV),
    (dict(reverse=2), INV), (dict(status=P + 2), ALI)])
def test_scan_refusals(lib, kw, st):
    a = args(ScanArgs, SCAN, kw)
    assert lib.gdr_scan_fwd(a, P, P, None, None, None, P, None, None) == st
    assert lib.gdr_scan_bwd(a, P, P, None, P, P, None, None, None, P, P, None, None, None) == st


def test_scan_pointers(lib):
    a, gate = args(ScanArgs, SCAN, {}), args(ScanArgs, SCAN, dict(write=1))
    tied = args(ScanArgs, SCAN, dict(write=2))
    f, b, s = lib.gdr_scan_fwd, lib.gdr_scan_bwd, lib.gdr_scan_step
    assert f(None, P, P, None, None, None, P, None, None) == INV
    assert f(a, None, P, None, None, None, P, None, None) == INV
    assert f(a, P, P, P, None, None, P, None, None) == INV          # beta without its write
    assert f(gate, P, P, None, None, None, P, None, None) == INV    # and the write without beta
    assert f(a, P, P, None, None, P, P, None, None) == INV          # packed with B = 2
    for i in (0, 1, 5):
        ptr = [P, P, None, None, None, P, None]
        ptr[i] = P + 8
        assert f(a, *ptr, None) == ALI
    assert f(a, P, P, None, P + 4, None, P, None, None) == ALI
    assert b(gate, P, P, P, P, P, None, None, None, P, P, None, None, None) == INV  # no dbeta
    assert b(tied, None, P, None, P, P, None, None, None, P, P, None, None, None) == INV
    assert b(a, P, P, None, P, P, None, None, None, P, P + 2, None, None, None) == ALI
    one = args(ScanArgs, SCAN, dict(T=1))
    assert s(a, P, P, None, P, P, P, None) == INV                   # more than a token
    assert s(args(ScanArgs, SCAN, dict(T=1, reverse=1)), P, P, None, P, P, P, None) == INV
    assert s(one, P, P, None, None, P, P, None) == INV
    assert s(one, P, P, None, P, P + 4, P, None) == ALI


@pytest.mark.parametrize("kw,st", BAD_SIZES + [
    (dict(D=0), INV), (dict(width=0), INV), (dict(width=1), UNS), (dict(width=5), UNS),
    (dict(activation=2), UNS), (dict(activation=3), INV), (dict(reverse=-1), INV)])
def test_conv_refusals(lib, kw, st):
    a = args(ConvArgs, CONV, kw)
    assert lib.gdr_conv_fwd(a, P, P, None, None, None, P, None, None) == st
    assert lib.gdr_conv_bwd(a, P, P, None, P, None, None, P, P, None, None, P, 1 << 40, None) == st
    assert "n_seqs" in kw and kw["n_seqs"] == 3 or lib.gdr_conv_bwd_workspace_size(a) == 0


def test_conv_pointers(lib):
    a = args(ConvArgs, CONV, {})
    f, b, s = lib.gdr_conv_fwd, lib.gdr_conv_bwd, lib.gdr_conv_step
    assert f(a, P, None, None, None, None, P, None, None) == INV
    assert f(a, P, P, None, P, None, P, P, None) == INV             # the state over itself
    assert f(a, P, P + 2, None, None, None, P, None, None) == ALI
    assert f(a, P + 8, P, None, None, None, P, None, None) == ALI
    need = lib.gdr_conv_bwd_workspace_size(a)
    assert need > 0 and need % 256 == 0
    call = lambda *p, ws=P, size=need: b(a, *p, ws, size, None)  # noqa: E731
    ok = [P, P, None, P, None, None, P, P, None, None]
    assert call(*ok, size=need - 1) == WS and call(*ok, ws=None) == WS
    assert call(*ok, ws=P + 16) == ALI
    assert call(*(ok[:7] + [None] + ok[8:])) == INV                 # dw is required
    assert s(a, P, P, None, P, P, P, None) == INV                   # more than a token
    assert s(args(ConvArgs, CONV, dict(T=1)), P, P, None, P, None, P, None) == INV


@pytest.mark.parametrize("kw,st", BAD_SIZES + [
    (dict(H=0), INV), (dict(d=0), INV), (dict(d=1032), UNS), (dict(d=260), UNS),
    (dict(d=516, io_dtype=0), _abi.GDR_OK), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(center=2), INV), (dict(activation=4), INV), (dict(H=70000, d=8), UNS)])
def test_norm_refusals(lib, kw, st):
    a = args(NormArgs, NORM, kw)
    if st == _abi.GDR_OK:
        assert lib.gdr_norm_bwd_workspace_size(a) > 0
        return
    assert lib.gdr_norm_fwd(a, P, P, None, None, None, P, None, None, 0, None) == st
    assert lib.gdr_norm_bwd(a, P, P, None, None, P, None, None, P, P, None, None, P, 1 << 40,
                            None) == st


def test_norm_pointers(lib):
    a, seq = args(NormArgs, NORM, {}), args(NormArgs, NORM, dict(per_sequence=1))
    f, b = lib.gdr_norm_fwd, lib.gdr_norm_bwd
    assert lib.gdr_norm_fwd_workspace_size(a) == 0
    need = lib.gdr_norm_fwd_workspace_size(seq)
    assert need > 0 and need % 256 == 0
    assert f(a, None, P, None, None, None, P, None, None, 0, None) == INV
    assert f(a, P, P, None, None, None, P, P, None, 0, None) == INV       # stats of tokens
    assert f(a, P + 8, P, None, None, None, P, None, None, 0, None) == ALI
    assert f(seq, P, P, None, None, None, P, None, P, need - 1, None) == WS
    assert f(seq, P, P, None, None, None, P, None, P + 64, need, None) == ALI
    need = lib.gdr_norm_bwd_workspace_size(a)
    assert b(a, P, P, None, P, P, None, None, P, P, None, None, P, need, None) == INV  # no dz
    assert b(a, P, P, None, None, P, None, None, P, P, None, None, P, need - 1, None) == WS
    need = lib.gdr_norm_bwd_workspace_size(seq)
    assert b(seq, P, P, None, None, P, None, None, P, P, None, None, P, need, None) == INV


def test_struct_layouts_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    if not shutil.which("gcc"):
        pytest.skip("no host C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    fields = {"gdr_scan_args": ScanArgs, "gdr_conv_args": ConvArgs, "gdr_norm_args": NormArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gdr.h"', "int main(void) {"]
    want = []
    for c, py in fields.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        want.append(ctypes.sizeof(py))
        for f, _ in py._fields_:
            lines.append(f'printf("%zu\\n", offsetof({c}, {f}));')
            want.append(getattr(py, f).offset)
    (tmp_path / "l.c").write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", inc, str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in out.split()] == want


def test_the_binding_refuses_before_it_calls():
    """CPU tensors, and shapes and types that do not belong together."""
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.linear_scan_fwd(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.short_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        gdr.group_norm_fwd(x.view(1, 4, 2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        gdr.linear_scan_step(x[0], x[0], None, x[0])


class Fake:
    """Stands for a CUDA tensor where only checks run."""

    def __init__(self, t, device="cuda:0", contiguous=True):
        self.t, self.device, self._c = t, torch.device(device), contiguous
        self.is_cuda, self.dtype, self.shape = True, t.dtype, t.shape

    def __getattr__(self, name):
        return getattr(self.t, name)

    def is_contiguous(self):
        return self._c

    def get_device(self):
        return self.device.index


def test_the_binding_checks_shapes_types_and_devices():
    F = lambda *s, dtype=torch.float32, **k: Fake(torch.zeros(*s, dtype=dtype), **k)  # noqa: E731
    v = F(2, 4, 8)
    bad = [
        (ValueError, lambda: gdr.linear_scan_fwd(v, F(2, 4, 7))),
        (ValueError, lambda: gdr.linear_scan_fwd(v, F(2, 4, 8, device="cuda:1"))),
        (ValueError, lambda: gdr.linear_scan_fwd(v, F(2, 4, 8, contiguous=False))),
        (ValueError, lambda: gdr.linear_scan_fwd(v, v, v, tied=True)),
        (TypeError, lambda: gdr.linear_scan_fwd(v, v, F(2, 4, 8, dtype=torch.bfloat16))),
        (TypeError, lambda: gdr.linear_scan_fwd(F(2, 4, 8, dtype=torch.float16), v)),
        (ValueError, lambda: gdr.linear_scan_fwd(v, v, None, F(3, 8))),
        (TypeError, lambda: gdr.linear_scan_fwd(v, v, None, F(2, 8, dtype=torch.float64))),
        (TypeError, lambda: gdr.linear_scan_fwd(v, v, cu_seqlens=F(3, dtype=torch.int64))),
        (TypeError, lambda: gdr.linear_scan_fwd(v, v, cu_seqlens=F(1, dtype=torch.int32))),
        (ValueError, lambda: gdr.linear_scan_fwd(F(4, 8), F(4, 8))),
        (ValueError, lambda: gdr.linear_scan_bwd(v, v, None, v, F(2, 4, 9))),
        (ValueError, lambda: gdr.linear_scan_step(F(4, 8), F(4, 8), None, F(5, 8))),
        (ValueError, lambda: gdr.short_conv_fwd(v, F(7, 4))),
        (TypeError, lambda: gdr.short_conv_fwd(v, F(8, 4, dtype=torch.bfloat16))),
        (ValueError, lambda: gdr.short_conv_fwd(v, F(8, 4), F(9))),
        (ValueError, lambda: gdr.short_conv_fwd(v, F(8, 4), None, F(2, 4, 8))),
        (ValueError, lambda: gdr.short_conv_fwd(v, F(8, 4), activation="relu")),
        (ValueError, lambda: gdr.short_conv_step(F(4, 8), F(8, 4), None, F(4, 2, 8))),
        (ValueError, lambda: gdr.group_norm_fwd(v)),
        (ValueError, lambda: gdr.group_norm_fwd(F(1, 2, 3, 8), F(4, 8))),
        (ValueError, lambda: gdr.group_norm_fwd(F(1, 2, 3, 8), F(8), F(3, 8))),
        (ValueError, lambda: gdr.group_norm_fwd(F(1, 2, 3, 8), per="batch")),
        (ValueError, lambda: gdr.group_norm_fwd(F(1, 2, 3, 8), output_stats=True)),
        (TypeError, lambda: gdr.group_norm_fwd(F(1, 2, 3, 8), z=F(1, 2, 3, 8, dtype=torch.bfloat16))),
        (ValueError, lambda: gdr.group_norm_bwd(F(1, 2, 3, 8), None, None, None, F(1, 2, 3, 8),
                                                per="sequence")),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            raise AssertionError(f"call {i} went through")


def test_sizes_beyond_32_bits_are_refused():
    """The C structs hold sizes in 32 bits: 2^32 + 5 tokens or channels must not become 5."""
    n = (1 << 32) + 5
    big = lambda *s, dtype=torch.float32: Fake(torch.zeros((), dtype=dtype).expand(*s))  # noqa: E731
    row, many, wide = big(1, n, 1), big(n, 1, 1), big(1, 1, n)
    bounds = big(n, dtype=torch.int32)
    for call in (
            lambda: gdr.linear_scan_fwd(row, row), lambda: gdr.linear_scan_fwd(many, many),
            lambda: gdr.linear_scan_fwd(wide, wide),
            lambda: gdr.linear_scan_fwd(big(1, 4, 8), big(1, 4, 8), cu_seqlens=bounds),
            lambda: gdr.linear_scan_bwd(row, row, None, row, row),
            lambda: gdr.linear_scan_step(big(n, 1), big(n, 1), None, big(n, 1)),
            lambda: gdr.linear_scan_step(big(1, n), big(1, n), None, big(1, n)),
            lambda: gdr.short_conv_fwd(row, big(1, 4)), lambda: gdr.short_conv_fwd(wide, big(n, 4)),
            lambda: gdr.short_conv_fwd(big(1, 4, 1), big(1, n)),
            lambda: gdr.short_conv_bwd(row, big(1, 4), None, row),
            lambda: gdr.short_conv_step(big(n, 1), big(1, 4), None, big(n, 3, 1)),
            lambda: gdr.group_norm_fwd(big(1, n, 1, 1)), lambda: gdr.group_norm_fwd(big(1, 1, n, 1)),
            lambda: gdr.group_norm_fwd(big(1, 1, 1, n)),
            lambda: gdr.group_norm_bwd(big(1, n, 1, 1), None, None, None, big(1, n, 1, 1))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_an_output_in_an_inputs_place_is_refused(lib):
    """Every pointer of its own is fine for the checks before, so INV is the overlap's."""
    q = [P + 0x1000 * i for i in range(16)]

    def each(fn, a, ptrs, pairs, tail=(None,)):
        for out, other in pairs:
            p = list(ptrs)
            p[out] = p[other]
            assert fn(a, *p, *tail) == INV, (fn.__name__, out, other)

    gate = args(ScanArgs, SCAN, dict(write=1))
    # v g beta h0 cu o h_final
    each(lib.gdr_scan_fwd, gate, [*q[:4], None, q[5], q[6]], [(5, 0), (5, 1), (5, 2), (5, 3), (6, 5), (6, 0)])
    # v g beta o dO h0 cu dh_final dv dg dbeta dh0
    each(lib.gdr_scan_bwd, gate, [*q[:6], None, *q[7:12]],
         [(8, 0), (8, 4), (9, 1), (10, 2), (9, 8), (10, 9), (8, 3), (11, 5), (8, 7)])
    # v g beta h h_out o
    each(lib.gdr_scan_step, args(ScanArgs, SCAN, dict(write=1, T=1)), q[:6],
         [(5, 0), (5, 3), (4, 1), (5, 4)])
    conv = args(ConvArgs, CONV, {})
    # x w bias state cu y state_out
    each(lib.gdr_conv_fwd, conv, [*q[:4], None, q[5], q[6]], [(5, 0), (5, 3), (6, 0), (6, 5), (5, 1)])
    need = lib.gdr_conv_bwd_workspace_size(conv)
    # x w bias dy state cu dx dw dbias dstate workspace
    each(lib.gdr_conv_bwd, conv, [*q[:5], None, *q[6:11]],
         [(6, 0), (6, 3), (9, 4), (7, 1), (8, 2), (8, 7), (10, 6), (10, 0)], (need, None))
    each(lib.gdr_conv_step, args(ConvArgs, CONV, dict(T=1)), q[:6], [(5, 0), (5, 3), (4, 0), (5, 4)])
    for kw in ({}, dict(per_sequence=1)):
        norm = args(NormArgs, NORM, kw)
        seq = bool(kw)
        need = lib.gdr_norm_fwd_workspace_size(norm)
        # x w bias z cu y stats workspace
        each(lib.gdr_norm_fwd, norm, [*q[:4], None, q[5], q[6] if seq else None, q[7]],
             [(5, 0), (5, 3), (5, 1)] + ([(6, 0), (7, 5)] if seq else []), (need, None))
        need = lib.gdr_norm_bwd_workspace_size(norm)
        # x w bias z dy cu stats dx dw dbias dz workspace
        each(lib.gdr_norm_bwd, norm, [*q[:5], None, *q[6:12]],
             [(7, 0), (7, 4), (10, 3), (8, 1), (9, 8), (10, 7), (11, 7)], (need, None))


def test_an_output_that_shares_bytes_with_another_array_is_refused(lib):
    """An output whose first or last 16 bytes lie in an input's or another output's; in place,
    only the whole array will do."""
    x, h, w, b, cs = 2 * 100 * 64 * 2, 2 * 64 * 4, 64 * 4 * 4, 64 * 4, 2 * 3 * 64 * 2
    nx, nw, ns = 2 * 100 * 4 * 64 * 2, 4 * 64 * 4, 2 * 4 * 2 * 4

    def each(fn, a, sizes, outs, absent=(), in_place=(), tail=(None,)):
        q = [None if i in absent else P + (i + 1 << 32) for i in range(len(sizes))]
        for o in outs:
            for i in range(len(sizes)):
                if i == o or q[i] is None:
                    continue
                places = [q[i] + sizes[i] - 16, q[i] - sizes[o] + 16]
                if (o, i) not in in_place:
                    places.append(q[i])
                for at in places:
                    if at == q[i] and (o, i) in in_place:
                        continue  # arrays of 16 bytes
                    assert fn(a, *(at if j == o else v for j, v in enumerate(q)), *tail) == INV, \
                        (fn.__name__, o, i, at - q[i])

    def sequences(a, cls, base):
        """Packed: B = 1 and bounds (of two sequences)."""
        return args(cls, {**base, **a}, dict(B=1, T=200))

    scan = sequences(dict(write=1), ScanArgs, SCAN)
    each(lib.gdr_scan_fwd, scan, [x, x, x, h, 16, x, h], (5, 6), in_place=[(6, 3)])
    each(lib.gdr_scan_bwd, scan, [x, x, x, x, x, h, 16, h, x, x, x, h], (8, 9, 10, 11),
         in_place=[(11, 7)])
    one = args(ScanArgs, SCAN, dict(write=1, T=1))
    each(lib.gdr_scan_step, one, [x // 100] * 3 + [h, h, x // 100], (4, 5), in_place=[(4, 3)])
    conv = sequences({}, ConvArgs, CONV)
    each(lib.gdr_conv_fwd, conv, [x, w, b, cs, 16, x, cs], (5, 6))
    need = lib.gdr_conv_bwd_workspace_size(conv)
    each(lib.gdr_conv_bwd, conv, [x, w, b, x, cs, 16, x, w, b, cs], (6, 7, 8, 9),
         tail=(P + (20 << 32), need, None))
    each(lib.gdr_conv_step, args(ConvArgs, CONV, dict(T=1)), [x // 100, w, b, cs, cs, x // 100], (4, 5),
         in_place=[(4, 3)])
    for per in (0, 1):
        norm = sequences(dict(per_sequence=per), NormArgs, NORM) if per else args(NormArgs, NORM, {})
        need = lib.gdr_norm_fwd_workspace_size(norm)
        each(lib.gdr_norm_fwd, norm, [nx, nw, nw, nx, 16, nx, ns], (5, 6) if per else (5,),
             absent=() if per else (4, 6), tail=(P + (20 << 32), need, None))
        need = lib.gdr_norm_bwd_workspace_size(norm)
        each(lib.gdr_norm_bwd, norm, [nx, nw, nw, nx, nx, 16, ns, nx, nw, nw, nx], (7, 8, 9, 10),
             absent=() if per else (5, 6), tail=(P + (20 << 32), need, None))
        # the workspace in an input's place, 256-byte aligned: its last bytes over x's first
        q = [P + (i + 1 << 32) for i in range(11)]
        if not per:
            q[5] = q[6] = None
        assert lib.gdr_norm_bwd(norm, *q, q[0] - need + 256, need, None) == INV
