"""Plain sequential float64 forms of the recurrent block's operators, with error bounds.

TEST INFRASTRUCTURE ONLY, written from the formulas in include/ss_scan.h: the gated linear
recurrence, the layer norm with its residual add and the causal depthwise convolution, their
gradients and their one-token forms.  Every result is a ``Bounded``: .v is the float64 value and
.e bounds what float32 arithmetic may be off (before any rounding to the io dtype).  Arrays are
float64 numpy; optional ones None.
"""
from __future__ import annotations

import numpy as np

from .rounding import (Bounded, U, exp, one_minus_square, rcp, sigmoid, sqrt, stack, where)


def _silu(z):
    return z * sigmoid(z)


def _silu_grad(z):
    s = sigmoid(z)
    return s * (z * (1.0 - s) + 1.0)


def _bias(v, b):
    """v + b.  It may be formed as fma(v, c, c b) with c = -log2(e): c b then rounds by itself,
    which is U |b| in v + b."""
    if b is None:
        return Bounded(v)
    s = Bounded(v) + b
    return Bounded(s.v, s.e + U * np.abs(b))


def gates(x, r, i, A, r_bias=None, i_bias=None):
    rg, ig = sigmoid(_bias(r, r_bias)), sigmoid(_bias(i, i_bias))
    l = Bounded(A) * rg
    a = exp(l)
    s = sqrt(one_minus_square(Bounded(2.0 * l.v, 2.0 * l.e), a))
    return rg, ig, a, s


def gated_fwd(x, r, i, A, r_bias=None, i_bias=None, z=None, starts=None, h0=None):
    """(out, h): h (batch, L, d) holds every state."""
    rg, ig, a, s = gates(x, r, i, A, r_bias, i_bias)
    b = s * ig * Bounded(x)
    batch, L, d = x.shape
    h = Bounded(np.zeros((batch, d)) if h0 is None else h0)
    hs = []
    for t in range(L):
        step = a[:, t] * h + b[:, t]
        if starts is not None:
            step = where(starts[:, t, None] != 0, b[:, t], step)
        h = step
        hs.append(h)
    hs = stack(hs, 1) if L else Bounded(np.zeros((batch, 0, d)))
    out = hs if z is None else hs * _silu(Bounded(z))
    return out, hs


def gated_bwd(x, r, i, A, dout, r_bias=None, i_bias=None, z=None, starts=None, h0=None,
              dh_last=None):
    batch, L, d = x.shape
    rg, ig, a, s = gates(x, r, i, A, r_bias, i_bias)
    _, h = gated_fwd(x, r, i, A, r_bias, i_bias, z, starts, h0)
    X, g, dz = Bounded(x), Bounded(dout), None
    if z is not None:
        dz = g * h * _silu_grad(Bounded(z))
        g = g * _silu(Bounded(z))
    carry = Bounded(np.zeros((batch, d)) if dh_last is None else dh_last)
    lams = [None] * L
    for t in range(L - 1, -1, -1):
        lams[t] = g[:, t] + carry
        carry = a[:, t] * lams[t]
        if starts is not None:
            carry = where(starts[:, t, None] != 0, 0.0, carry)
    depth = 64 + batch * (L // 64 + 1)
    if not L:
        zero = Bounded(np.zeros(d))
        e = Bounded(np.zeros((batch, 0, d)))
        return dict(dx=e, dr=e, di=e, dz=e if z is not None else None, dA=zero, dr_bias=zero,
                    di_bias=zero, dh0=carry)
    lam = stack(lams, 1)
    first = np.zeros((batch, d)) if h0 is None else h0
    prev = stack([Bounded(first)] + [h[:, t] for t in range(L - 1)], 1)
    if starts is not None:
        prev = where(starts[..., None] != 0, 0.0, prev)
    live = s.v > 0.0
    slope = where(live, a * a * rcp(where(live, s, 1.0)), 0.0)
    dl = lam * (a * prev - ig * X * slope)
    dr = dl * Bounded(A) * rg * (1.0 - rg)
    di = lam * s * X * ig * (1.0 - ig)
    return dict(dx=lam * s * ig, dr=dr, di=di, dz=dz, dA=(dl * rg).sum((0, 1), depth),
                dr_bias=dr.sum((0, 1), depth), di_bias=di.sum((0, 1), depth), dh0=carry)


def gated_step(state, x, r, i, A, r_bias=None, i_bias=None, z=None):
    out, h = gated_fwd(x[:, None], r[:, None], i[:, None], A, r_bias, i_bias,
                       None if z is None else z[:, None], None, state)
    return out[:, 0], h[:, 0]


def norm_fwd(x, weight=None, bias=None, residual=None, eps=1e-5):
    """(out, sum, mean, rstd, xhat)"""
    s = Bounded(x) if residual is None else Bounded(x) + residual
    n = x.shape[1]
    depth = 24 + n / 64
    mean = s.sum(1, depth) * (1.0 / n)
    c = s - mean[:, None]
    var = (c * c).sum(1, depth) * (1.0 / n)
    rstd = rcp(sqrt(var + eps))
    xh = c * rstd[:, None]
    out = xh if weight is None else xh * weight
    out = out + (0.0 if bias is None else bias)
    return out, s, mean, rstd, xh


def norm_bwd(dout, x, weight=None, residual=None, dsum=None, eps=1e-5):
    _, _, _, rstd, xh = norm_fwd(x, weight, None, residual, eps)
    rows, n = x.shape
    depth = 24 + n / 64
    dy = Bounded(dout)
    g = dy if weight is None else dy * weight
    c1, c2 = g.sum(1, depth) * (1.0 / n), (g * xh).sum(1, depth) * (1.0 / n)
    ds = rstd[:, None] * (g - c1[:, None] - xh * c2[:, None])
    if dsum is not None:
        ds = ds + dsum
    return dict(ds=ds, dweight=(dy * xh).sum(0, rows + 8), dbias=dy.sum(0, rows + 8))


def _window(x, x_prev, starts, k):
    """taps[j] (batch, L, d): the input tap j sees (0 across a start), and which it sees at all."""
    batch, L, d = x.shape
    taps, seen = np.zeros((k, batch, L, d)), np.zeros((k, batch, L), dtype=bool)
    for b in range(batch):
        for t in range(L):
            for lag in range(k):
                if starts is not None and any(starts[b, t - q] for q in range(lag) if t >= q):
                    continue
                src = t - lag
                if src >= 0:
                    taps[k - 1 - lag, b, t] = x[b, src]
                elif x_prev is not None:
                    taps[k - 1 - lag, b, t] = x_prev[b, k - 1 + src]
                seen[k - 1 - lag, b, t] = True
    return taps, seen


def conv_fwd(x, weight, bias=None, x_prev=None, starts=None, silu=True):
    """(out, pre-activation)"""
    k = weight.shape[1]
    taps, _ = _window(x, x_prev, starts, k)
    p = Bounded(np.zeros_like(x) if bias is None else np.broadcast_to(bias, x.shape))
    for j in range(k):
        p = p + Bounded(weight[:, j]) * taps[j]
    return (_silu(p) if silu else p), p


def conv_bwd(x, weight, dout, bias=None, x_prev=None, starts=None, silu=True):
    batch, L, d = x.shape
    k = weight.shape[1]
    taps, seen = _window(x, x_prev, starts, k)
    _, p = conv_fwd(x, weight, bias, x_prev, starts, silu)
    g = Bounded(dout) * _silu_grad(p) if silu else Bounded(dout)
    depth = 64 + batch * (L // 16 + 1)
    dpad = Bounded(np.zeros((batch, L + k - 1, d)))
    for j in range(k):
        add = where(seen[j][..., None], g * weight[:, j], 0.0)
        v, e = dpad.v.copy(), dpad.e.copy()
        new = dpad[:, j:j + L] + add
        v[:, j:j + L], e[:, j:j + L] = new.v, new.e
        dpad = Bounded(v, e)
    dw = stack([(g * taps[j]).sum((0, 1), depth) for j in range(k)], 1)
    return dict(dx=dpad[:, k - 1:], dx_prev=dpad[:, :k - 1], dweight=dw,
                dbias=g.sum((0, 1), depth))


def conv_step(conv_state, x, weight, bias=None, silu=True):
    out, _ = conv_fwd(x[:, None], weight, bias, conv_state, None, silu)
    window = np.concatenate([conv_state, x[:, None]], 1)
    return out[:, 0], window[:, 1:]
