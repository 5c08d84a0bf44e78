"""fp64 oracle of the layers around the mixer (test infrastructure): the selective state-space
scan, the short convolution's gradients and the per-head norm with rotation.

Every function is its definition, token by token or written out. With ``absolute`` the gradients and
the scan return, for each output, the sum of the absolute values of the terms that form it
(decays stay as they are, they are positive): the scale that a rounding error of one term is
relative to, for the tests' bounds. Shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * np.asarray(v, dtype=np.float64)))


def softplus(v):
    return np.logaddexp(0.0, np.asarray(v, dtype=np.float64))


def silu_slope(u, absolute=False):
    s = sigmoid(u)
    return s * (1.0 + (np.abs(u) if absolute else u) * (1.0 - s))


def _f(*arrays):
    return [None if a is None else np.asarray(a, dtype=np.float64) for a in arrays]


def ssm_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, S0=None, *, with_softplus=True, absolute=False):
    """x, dt, z [T, C]; Bm, Cm [T, N]; A, S0 [C, N]: one sequence. Returns (y, S_T, all states [T + 1, C, N])."""
    x, dt, A, Bm, Cm, D, z, dt_bias, S0 = _f(x, dt, A, Bm, Cm, D, z, dt_bias, S0)
    step = dt + (0.0 if dt_bias is None else dt_bias)
    step = softplus(step) if with_softplus else step
    m = np.abs if absolute else (lambda v: v)
    T, C = x.shape
    h = np.zeros((T + 1,) + A.shape)
    if S0 is not None:
        h[0] = m(S0)
    y = np.zeros((T, C))
    for t in range(T):
        h[t + 1] = np.exp(step[t][:, None] * A) * h[t] + m(step[t] * x[t])[:, None] * m(Bm[t])[None, :]
        y[t] = (h[t + 1] * m(Cm[t])[None, :]).sum(1)
    if D is not None:
        y = y + m(D * x)
    if z is not None:
        y = y * m(z * sigmoid(z))
    return y, h[T], h


def ssm_backward(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, S0=None, dS_T=None, *, with_softplus=True,
                 absolute=False):
    """Gradients of <y, dy> + <S_T, dS_T> for one sequence (the layouts of ssm_scan)."""
    _, _, h = ssm_scan(x, dt, A, Bm, Cm, D, None, dt_bias, S0, with_softplus=with_softplus, absolute=absolute)
    pre, _, _ = ssm_scan(x, dt, A, Bm, Cm, D, None, dt_bias, S0, with_softplus=with_softplus, absolute=absolute)
    x, dt, A, Bm, Cm, dy, D, z, dt_bias, dS_T = _f(x, dt, A, Bm, Cm, dy, D, z, dt_bias, dS_T)
    m = np.abs if absolute else (lambda v: v)
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    step = softplus(raw) if with_softplus else raw
    T, C = x.shape
    out = {}
    g = m(dy)
    if z is not None:
        out["dz"] = g * pre * silu_slope(z, absolute)
        g = g * m(z * sigmoid(z))
    dx, ddt = np.zeros((T, C)), np.zeros((T, C))
    dB, dC, dA = np.zeros_like(Bm), np.zeros_like(Cm), np.zeros_like(A)
    e = np.zeros_like(A) if dS_T is None else m(dS_T)
    for t in reversed(range(T)):
        a = np.exp(step[t][:, None] * A)
        dh = e + g[t][:, None] * m(Cm[t])[None, :]
        dC[t] = (g[t][:, None] * h[t + 1]).sum(0)
        dB[t] = (m(step[t] * x[t])[:, None] * dh).sum(0)
        du = (dh * m(Bm[t])[None, :]).sum(1)
        dx[t] = m(step[t]) * du + (0.0 if D is None else m(D) * g[t])
        e = a * dh
        q = e * h[t]
        ddt[t] = m(x[t]) * du + (m(A) * q).sum(1)
        dA += m(step[t])[:, None] * q
    if with_softplus:
        ddt = ddt * sigmoid(raw)
    out.update(dx=dx, ddt=ddt, dBm=dB, dCm=dC, dA=dA, dS0=e)
    if D is not None:
        out["dD"] = (g * m(x)).sum(0)
    if dt_bias is not None:
        out["ddt_bias"] = ddt.sum(0)
    return out


def conv_backward(x, weight, dy, state=None, dstate_out=None, *, l2norm=False, eps=1e-6, absolute=False):
    """Gradients of block.short_conv_silu for x, dy [T, H, d], weight [H * d, W], state [W - 1, H, d]."""
    x, weight, dy, state, dstate_out = _f(x, weight, dy, state, dstate_out)
    T, H, d = x.shape
    W = weight.shape[1]
    w = weight.reshape(H, d, W)
    m = np.abs if absolute else (lambda v: v)
    xp = np.concatenate([np.zeros((W - 1, H, d)) if state is None else state, x], 0)
    u = np.zeros((T, H, d))
    for i in range(W):
        u += w[:, :, i] * xp[i:i + T]
    y = u * sigmoid(u)
    ds = m(dy)
    if l2norm:
        r = np.sqrt((y * y).sum(-1, keepdims=True) + eps)
        yh = m(y / r)
        sign = 1.0 if absolute else -1.0
        ds = (ds + sign * yh * (yh * ds).sum(-1, keepdims=True)) / r
    du = ds * silu_slope(u, absolute)
    dxp, dw = np.zeros_like(xp), np.zeros_like(w)
    for i in range(W):
        dxp[i:i + T] += m(w[:, :, i]) * du
        dw[:, :, i] = (du * m(xp[i:i + T])).sum(0)
    if dstate_out is not None and W > 1:
        dxp[T:] += m(dstate_out)
    return {"dx": dxp[W - 1:], "dweight": dw.reshape(H * d, W), "dstate": dxp[:W - 1]}


def _turn(v, cos, sin, interleaved, absolute):
    R = 2 * cos.shape[-1]
    out = v.copy()
    for j in range(R // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
        c, s = cos[..., j], sin[..., j]
        if absolute:
            c, s = np.abs(c), np.abs(s)
            out[..., a], out[..., b] = v[..., a] * c + v[..., b] * s, v[..., b] * c + v[..., a] * s
        else:
            out[..., a], out[..., b] = v[..., a] * c - v[..., b] * s, v[..., b] * c + v[..., a] * s
    return out


def _angles(cos_sin, positions):
    row = np.asarray(cos_sin, dtype=np.float64)[np.asarray(positions)]
    half = row.shape[-1] // 2
    return row[..., None, :half], row[..., None, half:]


def head_norm_rope(x, weight=None, cos_sin=None, positions=None, *, norm="rms", eps=1e-6, interleaved=False,
                   absolute=False):
    """x [..., H, d] with positions [...]."""
    x, weight = _f(x, weight)
    r = 1.0 if norm is None else np.sqrt((x * x).sum(-1, keepdims=True) / (x.shape[-1] if norm == "rms" else 1) + eps)
    v = x / r * (1.0 if weight is None else weight)
    v = np.abs(v) if absolute else v
    return v if cos_sin is None else _turn(v, *_angles(cos_sin, positions), interleaved, absolute)


def head_norm_rope_backward(x, dy, weight=None, cos_sin=None, positions=None, *, norm="rms", eps=1e-6,
                            interleaved=False, absolute=False):
    """(dx, dweight) of <head_norm_rope(x), dy>."""
    x, dy, weight = _f(x, dy, weight)
    m = np.abs if absolute else (lambda v: v)
    k = 1.0 if norm == "l2" else 1.0 / x.shape[-1]
    r = 1.0 if norm is None else np.sqrt((x * x).sum(-1, keepdims=True) * k + eps)
    xh, g = m(x / r), m(dy)
    if cos_sin is not None:
        c, s = _angles(cos_sin, positions)
        g = _turn(g, c, -s, interleaved, absolute)
    dw = (g * xh).reshape(-1, x.shape[-1]).sum(0)
    g = g * (1.0 if weight is None else m(weight))
    if norm is None:
        return g, dw
    sign = 1.0 if absolute else -1.0
    return (g + sign * xh * (xh * g).sum(-1, keepdims=True) * k) / r, dw
