"""The layer oracle's gradients against central differences of its forwards, and its forward forms
against independent statements."""
import numpy as np
import pytest

from oracle import block as OB
from oracle import layers as OL


def _difference(f, value, dout):
    """Central differences of sum(f(value) * dout) by every entry of value."""
    grad = np.zeros_like(value)
    for i in np.ndindex(value.shape):
        step = 1e-6 * max(1.0, abs(value[i]))
        v = value.copy()
        v[i] += step
        up = sum((a * b).sum() for a, b in zip(f(v), dout))
        v[i] -= 2 * step
        down = sum((a * b).sum() for a, b in zip(f(v), dout))
        grad[i] = (up - down) / (2 * step)
    return grad


def _close(a, b, what):
    # central differences of step 1e-6: 1e-12 of curvature and 1e-16 / 1e-6 of rounding, times the sums' sizes
    assert np.max(np.abs(a - b)) <= 1e-7 * max(1.0, np.max(np.abs(b))), what


@pytest.mark.parametrize("gate,softplus", [(True, True), (False, True), (True, False)])
def test_scan_gradients_are_differences(gate, softplus):
    rng = np.random.default_rng(0)
    T, C, N = 5, 3, 4
    v = dict(x=rng.normal(size=(T, C)), dt=rng.normal(size=(T, C)) * 0.5, A=-np.exp(rng.normal(size=(C, N)) * 0.3),
             Bm=rng.normal(size=(T, N)), Cm=rng.normal(size=(T, N)), D=rng.normal(size=C),
             z=rng.normal(size=(T, C)) if gate else None, dt_bias=rng.normal(size=C), S0=rng.normal(size=(C, N)))
    dy, dS = rng.normal(size=(T, C)), rng.normal(size=(C, N))
    g = OL.ssm_backward(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], dy, v["D"], v["z"], v["dt_bias"], v["S0"], dS,
                        with_softplus=softplus)
    for name, value in v.items():
        if value is None:
            continue
        d = _difference(lambda w: OL.ssm_scan(**{**v, name: w}, with_softplus=softplus)[:2], value, (dy, dS))
        _close(g["d" + name], d, name)


@pytest.mark.parametrize("l2", [True, False])
@pytest.mark.parametrize("T", [1, 2, 6])
def test_conv_gradients_are_differences(l2, T):
    rng = np.random.default_rng(1)
    H, d, W = 2, 3, 4
    x, w, s = rng.normal(size=(T, H, d)), rng.normal(size=(H * d, W)), rng.normal(size=(W - 1, H, d))
    dy, dso = rng.normal(size=(T, H, d)), rng.normal(size=(W - 1, H, d))

    def f(x_=x, w_=w, s_=s):
        y, _ = OB.short_conv_silu(x_.reshape(1, T, H * d), w_, s_.reshape(1, W - 1, H * d), l2norm=l2, heads=H, eps=1e-2)
        after = np.concatenate([s_, x_], 0)[T:]
        return np.asarray(y).reshape(T, H, d), after

    g = OL.conv_backward(x, w, dy, s, dso, l2norm=l2, eps=1e-2)
    _close(g["dx"], _difference(lambda v: f(x_=v), x, (dy, dso)), "dx")
    _close(g["dweight"], _difference(lambda v: f(w_=v), w, (dy, dso)), "dweight")
    _close(g["dstate"], _difference(lambda v: f(s_=v), s, (dy, dso)), "dstate")


@pytest.mark.parametrize("norm", ["rms", "l2", None])
@pytest.mark.parametrize("interleaved", [True, False])
def test_head_norm_rope_gradients_are_differences(norm, interleaved):
    rng = np.random.default_rng(2)
    x, w, dy = rng.normal(size=(3, 2, 8)), rng.normal(size=8), rng.normal(size=(3, 2, 8))
    ang = rng.normal(size=(7, 2))
    table, pos = np.concatenate([np.cos(ang), np.sin(ang)], 1), np.array([5, 0, 6])
    kw = dict(cos_sin=table, positions=pos, norm=norm, eps=1e-2, interleaved=interleaved)
    dx, dw = OL.head_norm_rope_backward(x, dy, w, **kw)
    _close(dx, _difference(lambda v: (OL.head_norm_rope(v, w, **kw),), x, (dy,)), "dx")
    _close(dw, _difference(lambda v: (OL.head_norm_rope(x, v, **kw),), w, (dy,)), "dweight")


def test_rotation_keeps_lengths_and_composes():
    """Turning by p and then by q is turning by p + q; the scores of two rotated rows depend on
    the distance of their positions alone; position 0 is the identity."""
    rng = np.random.default_rng(3)
    freq = 10000.0 ** (-np.arange(4) / 4.0)
    ang = np.arange(40)[:, None] * freq
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x, y = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8))
    for il in (False, True):
        r = lambda v, p: OL.head_norm_rope(v, None, table, np.array([p]), norm=None, interleaved=il)  # noqa: E731
        np.testing.assert_allclose(r(r(x, 7), 11), r(x, 18), atol=1e-12)
        np.testing.assert_allclose(r(x, 0), x)
        np.testing.assert_allclose((r(x, 9) * r(y, 4)).sum(), (r(x, 30) * r(y, 25)).sum(), atol=1e-12)


def test_scan_closed_forms():
    """Constant decay and input give the geometric sum; A = 0 the running sum; a far step forgets."""
    T, C, N = 9, 2, 3
    one = np.ones((T, C))
    A = -np.ones((C, N)) * 0.7
    _, S, _ = OL.ssm_scan(one, one, A, np.ones((T, N)), np.ones((T, N)), with_softplus=False)
    a = np.exp(-0.7)
    np.testing.assert_allclose(S, (1 - a ** T) / (1 - a))
    y, S, _ = OL.ssm_scan(one, one, 0 * A, np.ones((T, N)), np.ones((T, N)), with_softplus=False)
    np.testing.assert_allclose(y, N * np.arange(1, T + 1)[:, None] * one)
    x = np.random.default_rng(4).normal(size=(T, C))
    _, S, _ = OL.ssm_scan(x, 1000 * one, A, np.ones((T, N)), np.ones((T, N)), S0=np.ones((C, N)), with_softplus=False)
    np.testing.assert_allclose(S, 1000 * x[-1][:, None] * np.ones((1, N)))
