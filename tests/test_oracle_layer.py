"""The 64-bit definitions of the operators around the recurrence: gradients against central
differences of the forward, and properties that do not depend on how either is written."""
import numpy as np
import pytest

from oracle import layer as ol

CU = [0, 3, 3, 4, 9]  # ragged: an empty sequence and one of a single token


def differences(loss, arrays, h=1e-6):
    """Central differences of loss() with respect to every element of every array."""
    out = []
    for a in arrays:
        g = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            x = a[i]
            a[i] = x + h
            up = loss()
            a[i] = x - h
            g[i] = (up - loss()) / (2 * h)
            a[i] = x
        out.append(g)
    return out


def close(got, want):
    assert got.shape == want.shape
    # truncation h^2 and cancellation 1e-16 / h of a loss of order 10
    assert np.abs(got - want).max() <= 1e-7 * max(1.0, np.abs(want).max())


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("write", ["plain", "gate", "tied"])
def test_scan_gradient_against_differences(write, reverse):
    r = np.random.default_rng(1)
    v, g = r.normal(size=(9, 2)), -np.exp(r.normal(size=(9, 2)))
    beta = r.normal(size=(9, 2)) if write == "gate" else None
    h0, dO, dhf = r.normal(size=(4, 2)), r.normal(size=(9, 2)), r.normal(size=(4, 2))

    def loss():
        o, hf = ol.scan(v, g, beta, h0, CU, write == "tied", reverse)
        return (dO * o).sum() + (dhf * hf).sum()

    o, _ = ol.scan(v, g, beta, h0, CU, write == "tied", reverse)
    dv, dg, db, dh0 = ol.scan_backward(v, g, beta, o, dO, h0, dhf, CU, write == "tied", reverse)
    want = differences(loss, [v, g, h0] + ([beta] if write == "gate" else []))
    for got, w in zip([dv, dg, dh0] + ([db] if write == "gate" else []), want):
        close(got, w)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_gradient_against_differences(W, reverse):
    r = np.random.default_rng(2)
    x, w, b = r.normal(size=(9, 2)), r.normal(size=(2, W)), r.normal(size=2)
    st, dy = r.normal(size=(4, W - 1, 2)), r.normal(size=(9, 2))
    got = ol.conv_backward(x, w, b, dy, st, CU, "silu", reverse)
    want = differences(lambda: (dy * ol.conv(x, w, b, st, CU, "silu", reverse)[0]).sum(),
                       [x, w, b, st])
    for g, v in zip(got, want):
        close(g, v)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("per,name", [("token", "silu"), ("sequence", "sigmoid"),
                                      ("sequence", "silu"), ("token", "none")])
def test_norm_gradient_against_differences(per, name, center, gate):
    r = np.random.default_rng(3)
    x, w, b = r.normal(size=(9, 2, 3)), r.normal(size=(2, 3)), r.normal(size=(2, 3))
    z, dy = r.normal(size=(9, 2, 3)) if gate else None, r.normal(size=(9, 2, 3))
    got = ol.norm_backward(x, w, b, z, dy, CU, per, center, name, 0.1)
    want = differences(lambda: (dy * ol.norm(x, w, b, z, CU, per, center, name, 0.1)[0]).sum(),
                       [x, w, b] + ([z] if gate else []))
    for g, v in zip(got if gate else got[:3], want):
        close(g, v)


def test_scan_closed_forms():
    """Without decay a cumulative sum; without memory the write itself; tied keeps a constant
    input's fixed point; a sequence continued from its state is the whole sequence."""
    r = np.random.default_rng(4)
    v = r.normal(size=(7, 3))
    o, hf = ol.scan(v, np.zeros_like(v), None, None, [0, 7])
    assert np.allclose(o, np.cumsum(v, 0)) and np.array_equal(hf[0], o[-1])
    o, _ = ol.scan(v, np.full_like(v, -np.inf), None, np.ones((1, 3)), [0, 7])
    assert np.array_equal(o, v)
    one = np.ones_like(v)
    o, _ = ol.scan(one, -np.exp(v), None, one[:1], [0, 7], tied=True)
    assert np.allclose(o, 1.0)
    g = -np.exp(v)
    o, hf = ol.scan(v, g, None, None, [0, 7])
    a, ha = ol.scan(v[:4], g[:4], None, None, [0, 4])
    b, hb = ol.scan(v[4:], g[4:], None, ha, [0, 3])
    assert np.allclose(np.concatenate([a, b]), o) and np.allclose(hb, hf)


def test_reverse_is_the_flipped_sequence():
    r = np.random.default_rng(5)
    v, g, w = r.normal(size=(6, 2)), -np.exp(r.normal(size=(6, 2))), r.normal(size=(2, 3))
    o, hf = ol.scan(v, g, None, None, [0, 6], reverse=True)
    f, ff = ol.scan(v[::-1], g[::-1], None, None, [0, 6])
    assert np.array_equal(o, f[::-1]) and np.array_equal(hf, ff)
    y, st, _ = ol.conv(v, w, None, None, [0, 6], reverse=True)
    f, sf, _ = ol.conv(v[::-1], w, None, None, [0, 6])
    assert np.array_equal(y, f[::-1]) and np.array_equal(st, sf)


def test_conv_closed_forms():
    """A unit tap shifts; the state is the shifted-in past; pieces continue one another."""
    r = np.random.default_rng(6)
    x, w = r.normal(size=(5, 2)), np.array([[1.0, 0, 0], [0, 0, 1.0]])
    st = r.normal(size=(1, 2, 2))
    y, out, _ = ol.conv(x, w, None, st, [0, 5], "none")
    assert np.array_equal(y[:, 1], x[:, 1])
    assert np.array_equal(y[:, 0], np.concatenate([st[0, :, 0], x[:3, 0]]))
    assert np.array_equal(out[0], x[3:])
    a, sa, _ = ol.conv(x[:1], w, None, st, [0, 1])
    b, sb, _ = ol.conv(x[1:], w, None, sa, [0, 4])
    assert np.allclose(np.concatenate([a, b]), ol.conv(x, w, None, st, [0, 5])[0])
    assert np.array_equal(sb, out)


def test_norm_closed_forms():
    """Shifting x changes nothing with centering, scaling nothing at eps 0; one token per
    sequence is the per-token norm."""
    r = np.random.default_rng(7)
    x, cu = r.normal(size=(4, 2, 8)), [0, 1, 2, 3, 4]
    y, _ = ol.norm(x, None, None, None, cu, eps=0.0)
    assert np.allclose(ol.norm(3 * x + 5, None, None, None, cu, eps=0.0)[0], y)
    assert np.allclose(ol.norm(x, None, None, None, cu, per="sequence", eps=0.0)[0], y)
    n, st = ol.norm(x, None, None, None, [0, 4], per="sequence", name="none", eps=0.0)
    assert np.allclose(n.mean((0, 2)), 0) and np.allclose((n ** 2).mean((0, 2)), 1)
    assert np.allclose(st[0, :, 0], x.mean((0, 2)))
