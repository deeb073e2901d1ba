"""A cluster of the gated linear recurrence whose wait for a block's run comes to its limit: what
misses the run is NaN, everything else is right, and the kernel ends."""
import ctypes
import subprocess
import os

import numpy as np
import pytest
import torch

from gated_delta_rule_146_b200 import build

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "scan_late.cu")
WAIT_NS = 2_000_000


def compiled(folder):
    out = os.path.join(str(folder), "scan_late.so")
    subprocess.run([build._nvcc(), *build.NVCC_FLAGS, f"-DGDR_SCAN_WAIT_NS={WAIT_NS}ull", "-I",
                    build.INCLUDE, "-I", build.CSRC, "-shared", "-o", out, SOURCE], check=True)
    return out


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    return ctypes.CDLL(compiled(tmp_path_factory.mktemp("late"))).scan_late


def walk(late, steps, mute, start):
    """(o, state, ok, the recurrence in 64 bits, tokens that start a sequence)"""
    r = np.random.default_rng(steps)
    T = 4 * steps
    a, b = r.uniform(0.2, 0.9, (T, 64)).astype(np.float32), r.normal(size=(T, 64)).astype(np.float32)
    starts = np.arange(T) % 11 == 7
    a[starts] = -1.0
    x, want = np.ones(64), np.zeros((T, 64))
    for t in range(T):
        x = want[t] = b[t] if starts[t] else a[t].astype(np.float64) * x + b[t]
    dev = [torch.from_numpy(v).cuda() for v in (a, b)]
    o, state = torch.zeros(T, 64, device="cuda"), torch.zeros(2, 64, device="cuda")
    ok = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    err = late(p(dev[0]), p(dev[1]), p(o), p(state), p(ok), steps, mute, start,
               ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    end.record()
    assert err == 0
    torch.cuda.synchronize()
    return o.cpu().numpy(), state.cpu().numpy(), ok.tolist(), want, starts, begin.elapsed_time(end)


# a state is a sum of decaying terms, each rounded a few times: off by a few 2^-24 of their size,
# which is below 10 here
TOL = 10 * 16 * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [1, 2, 3, 8, 37])
def test_every_run_comes(late, steps):
    o, state, ok, want, _, _ = walk(late, steps, 0, steps)
    assert ok == [1, 1]
    assert np.abs(o - want).max() <= TOL and np.abs(state - want[-1]).max() <= TOL


@pytest.mark.gpu
@pytest.mark.parametrize("mute", [0, 1])
@pytest.mark.parametrize("steps,start", [(1, 0), (4, 3), (9, 1), (37, 6), (37, 35)])
def test_a_run_that_never_comes(late, steps, start, mute):
    o, state, ok, want, starts, ms = walk(late, steps, mute, start)
    assert ok == [0, 0] and np.isnan(state).all()
    # right: the tiles before, the starts of sequences, and what the block itself knows to follow one
    fine = np.arange(4 * steps) < 4 * start
    fine |= starts
    fine[1::2] |= starts[::2]
    assert np.abs(o - want)[fine].max(initial=0.0) <= TOL
    assert np.isnan(o[~fine]).all()
    assert ms < 200
