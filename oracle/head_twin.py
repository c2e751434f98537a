"""Plain float64 forms of the operators around the multi-head scan, with error bounds.

TEST INFRASTRUCTURE ONLY, written from the formulas in include/ss_scan.h: one token of the scan and
its convolution, the scan's gradients step by step, the RMS norm with the scaled and dropped-out
residual add, the gated norm, and dropout's mask.  Results are ``Bounded`` (float64 value, bound on
what float32 arithmetic may be off before any rounding to the io dtype).  Arrays are float64 numpy;
optional ones None.
"""
from __future__ import annotations

import numpy as np

from . import block_twin as bt
from .block_twin import _silu, _silu_grad
from .rounding import Bounded, U, exp, rcp, sqrt, where

M32 = 0xFFFFFFFF


def philox(counter, key):
    """Philox4x32-10 of Python integers: four 32-bit words for four counter and two key words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & M32, (a >> 32) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def drop_cut(p):
    return round(p * 65536)


def keep_mask(rng, rows, dim, p):
    """(rows, dim) bool: which elements dropout keeps."""
    seed, offset = (int(v) & ((1 << 64) - 1) for v in rng)
    keep, cut = np.zeros((rows, dim), dtype=bool), drop_cut(p)
    for r in range(rows):
        for c8 in range((dim + 7) // 8):
            w = philox((c8, r, offset & M32, offset >> 32), (seed & M32, seed >> 32))
            bits = [h for v in w for h in (v & 0xFFFF, v >> 16)]
            for j in range(min(8, dim - 8 * c8)):
                keep[r, 8 * c8 + j] = bits[j] >= cut
    return keep


def drop(v, keep, p):
    """Bounded v / (1 - q) where kept, 0 elsewhere."""
    if keep is None:
        return v
    cut = drop_cut(p)
    up = 65536.0 / (65536 - cut) if cut < 65536 else 0.0
    return where(keep, v * Bounded(up, U * up), 0.0)


# ---------------------------------------------------------------------------------------- norms


def _rstd(v, eps, axis):
    n = v.shape[axis]
    ms = (v * v).sum(axis, 24 + n / 64) * (1.0 / n)
    return rcp(sqrt(ms + eps))


def rms_fwd(x, weight=None, residual=None, scale=None, norm_branch=False, keep=None, p=0.0,
            eps=1e-5):
    """(out, sum, rstd, branch_rstd, b): b is x or its norm."""
    b, rb = Bounded(x), None
    if norm_branch:
        rb = _rstd(b, eps, 1)
        b = b * rb[:, None]
    v = b if scale is None else b * scale
    v = drop(v, keep, p)
    if residual is not None:
        v = v + residual
    r = _rstd(v, eps, 1)
    out = v * r[:, None]
    return (out if weight is None else out * weight), v, r, rb, b


def rms_bwd(dout, x, weight=None, residual=None, scale=None, norm_branch=False, keep=None, p=0.0,
            dsum=None, eps=1e-5):
    _, v, r, rb, b = rms_fwd(x, weight, residual, scale, norm_branch, keep, p, eps)
    rows, n = x.shape
    depth = 24 + n / 64
    dy, vh = Bounded(dout), v * r[:, None]
    g = dy if weight is None else dy * weight
    m = (g * vh).sum(1, depth) * (1.0 / n)
    ds = r[:, None] * (g - vh * m[:, None])
    if dsum is not None:
        ds = ds + dsum
    db = drop(ds, keep, p)
    dh = db if scale is None else db * scale
    dx = dh
    if norm_branch:
        m2 = (dh * b).sum(1, depth) * (1.0 / n)
        dx = rb[:, None] * (dh - b * m2[:, None])
    return dict(dx=dx, dresidual=ds, dweight=(dy * vh).sum(0, rows + 8),
                dscale=(db * b).sum(0, rows + 8))


def _parts(v, groups):
    return Bounded(v.v.reshape(v.shape[0], groups, -1),
                   np.broadcast_to(v.e, v.shape).reshape(v.shape[0], groups, -1))


def _whole(v):
    return Bounded(v.v.reshape(v.shape[0], -1), v.e.reshape(v.shape[0], -1))


def gated_fwd(x, z=None, weight=None, groups=1, gate_first=True, eps=1e-5):
    """(out, rstd)"""
    x = _parts(Bounded(x), groups)
    gate = None if z is None else _silu(_parts(Bounded(z), groups))
    u = x * gate if gate is not None and gate_first else x
    r = _rstd(u, eps, 2)
    y = u * r[..., None]
    if weight is not None:
        y = y * weight.reshape(groups, -1)
    if gate is not None and not gate_first:
        y = y * gate
    return _whole(y), r


def gated_bwd(dout, x, z=None, weight=None, groups=1, gate_first=True, eps=1e-5):
    rows, n = x.shape[0], x.shape[1] // groups
    do, x = _parts(Bounded(dout), groups), _parts(Bounded(x), groups)
    w = 1.0 if weight is None else weight.reshape(groups, -1)
    gate = slope = Bounded(1.0)
    if z is not None:
        zz = _parts(Bounded(z), groups)
        gate, slope = _silu(zz), _silu_grad(zz)
    u = x * gate if gate_first else x
    r = _rstd(u, eps, 2)
    hat = u * r[..., None]
    after = do if gate_first else do * gate
    g = after * w
    m = (g * hat).sum(2, 24 + n / 64) * (1.0 / n)
    du = r[..., None] * (g - hat * m[..., None])
    dx = du * gate if gate_first else du
    dz = (du * x if gate_first else do * hat * w) * slope
    dw = (after * hat).sum(0, rows + 8)
    return dict(dx=_whole(dx), dz=_whole(dz) if z is not None else None,
                dweight=Bounded(dw.v.reshape(-1), dw.e.reshape(-1)))


# ------------------------------------------------------------------------------ the scan's token


def _softplus(v):
    """max(v, 0) + log1p(e^-|v|) in float32: at most 8 roundings of the result, and what v is off
    (its slope is at most 1)."""
    s = np.maximum(v.v, 0.0) + np.log1p(np.exp(-np.abs(v.v)))
    slope = 1.0 / (1.0 + np.exp(-(v.v + v.e)))
    return Bounded(s, slope * v.e + 8 * U * s)


def steps(dt, dt_bias=None, softplus=True):
    raw = Bounded(dt) if dt_bias is None else Bounded(dt) + dt_bias
    return _softplus(raw) if softplus else raw


def step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True):
    """(out, state); x (batch, H, P), B, C (batch, G, N) may be Bounded already."""
    x, B, C = Bounded.of(x), Bounded.of(B), Bounded.of(C)
    H, G = x.shape[1], B.shape[1]
    rep = lambda t: Bounded(np.repeat(t.v, H // G, 1), np.repeat(t.e, H // G, 1))  # noqa: E731
    B, C = rep(B), rep(C)
    s = steps(dt, dt_bias, softplus)
    a = exp(s * Bounded(A))
    S = a[..., None, None] * Bounded(state) + \
        (s[..., None] * B)[..., None] * x[:, :, None, :]
    N = state.shape[2]
    y = (C[..., None] * S).sum(2, N + 8)
    if D is not None:
        y = y + x * D[:, None]
    if z is not None:
        y = y * _silu(Bounded(z))
    return y, S


def step_conv(state, conv_state, xbc, weight, bias, dt, A, G, D=None, z=None, dt_bias=None,
              softplus=True):
    """(out, state, conv_state)"""
    batch, H, N, P = state.shape
    act, _ = bt.conv_fwd(xbc[:, None], weight, bias, conv_state, None, True)
    act, d = act[:, 0], H * P
    cut = lambda a, b, *s: Bounded(act.v[:, a:b].reshape(batch, *s),  # noqa: E731
                                   act.e[:, a:b].reshape(batch, *s))
    out, S = step(state, cut(0, d, H, P), dt, A, cut(d, d + G * N, G, N),
                  cut(d + G * N, d + 2 * G * N, G, N), D,
                  None if z is None else z.reshape(batch, H, P), dt_bias, softplus)
    window = np.concatenate([conv_state, xbc[:, None]], 1)
    return out, S, window[:, 1:]


# ----------------------------------------------------------------------------- the scan's gradients


def _scan2_bwd(x, dt, a, A, B, C, gy, D, h0, dh_last):
    """The recurrence and its adjoint, one step after the other.  dt: step sizes, a: decays
    (batch, L, H); B, C per head (batch, L, H, N)."""
    batch, L, H, P = x.shape
    N = B.shape[3]
    S, states = h0, []
    for t in range(L):
        states.append(S)
        S = a[:, t, :, None, None] * S + (dt[:, t, :, None] * B[:, t])[..., None] * x[:, t, :, None]
    last = S
    y, v = np.zeros_like(x), np.zeros_like(x)
    dl, dB, dC = np.zeros_like(dt), np.zeros_like(B), np.zeros_like(C)
    lam = dh_last
    for t in range(L - 1, -1, -1):
        prev = states[t]
        S = states[t + 1] if t + 1 < L else last
        y[:, t] = (C[:, t][..., None] * S).sum(2)
        lam = lam + C[:, t][..., None] * gy[:, t, :, None]
        v[:, t] = (B[:, t][..., None] * lam).sum(2)
        dB[:, t] = dt[:, t, :, None] * (lam * x[:, t, :, None]).sum(3)
        dC[:, t] = (S * gy[:, t, :, None]).sum(3)
        dl[:, t] = a[:, t] * (lam * prev).sum((2, 3))
        lam = a[:, t, :, None, None] * lam
    return dict(y=y, v=v, dl=dl, dB=dB, dC=dC, dh0=lam, h_last=last)


def scan2_bwd(x, dt, A, B, C, dout, D=None, z=None, dt_bias=None, softplus=True, h0=None,
              dh_last=None):
    """All gradients as Bounded, and y (before the gate) under "y".

    Every value is a sum of products, evaluated in float32 in an order of the kernel's choice.  Its
    bound is kappa U times the sum of the products' absolute values (the same formulas with all
    factors made positive), kappa counting the roundings on the way of one product: sums over the
    states, channels, three chunk-long ones and two per chunk that a state passes through; 64 for
    the products, exponentials, gates and step sizes themselves; and the exponents, which are
    differences of two sums of up to 64 log decays, c: each is off by 8 U c at most (six additions
    in a tree, the product and its constant), so what they scale by 16 U c.  dl takes the
    pairs of steps of its chunk as a difference of sums of all of them, so those stand in its sum.
    """
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    per = lambda t: np.repeat(t, H // G, 2)  # noqa: E731
    back = lambda t: t.reshape(batch, L, G, H // G, N).sum(3)  # noqa: E731
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    s = np.maximum(raw, 0.0) + np.log1p(np.exp(-np.abs(raw))) if softplus else raw
    a = np.exp(s * A)
    Dv = np.zeros(H) if D is None else D
    sig = 1.0 if z is None else 1.0 / (1.0 + np.exp(-z))
    gate = 1.0 if z is None else z * sig
    gy = dout * gate
    zero = np.zeros((batch, H, N, P))
    h0 = zero if h0 is None else h0
    dl_last = zero if dh_last is None else dh_last
    f = _scan2_bwd(x, s, a, A, per(B), per(C), gy, Dv, h0, dl_last)
    m = _scan2_bwd(np.abs(x), np.abs(s), a, A, np.abs(per(B)), np.abs(per(C)), np.abs(gy),
                   np.abs(Dv), np.abs(h0), np.abs(dl_last))
    log2 = np.abs(s * A) * np.log2(np.e)
    c = max([log2[:, i:i + 64].sum(1).max() for i in range(0, L, 64)], default=0.0)
    pairs = np.zeros_like(m["dl"])
    for i in range(0, L, 64):
        part = slice(i, min(i + 64, L))
        w = np.abs(gy[:, part]).transpose(0, 2, 1, 3) @ np.abs(x[:, part]).transpose(0, 2, 3, 1)
        g = np.abs(per(C)[:, part]).transpose(0, 2, 1, 3) @ \
            np.abs(per(B)[:, part]).transpose(0, 2, 3, 1)
        cum = np.cumsum(s[:, part] * A, 1).transpose(0, 2, 1)
        n = cum.shape[2]
        seg = np.where(np.tril(np.ones((n, n), bool), -1), cum[..., None] - cum[:, :, None], -np.inf)
        e = w * g * np.exp(seg) * np.abs(s[:, part]).transpose(0, 2, 1)[:, :, None]
        pairs[:, part] = e.sum((2, 3))[:, None]
    m["dl"] = m["dl"] + pairs
    kappa = (N + P + 192 + 2 * (L // 64 + 1) + 64 + 16 * c) * U
    sums = 8 + batch * (L // 64 + 1)      # further additions of a sum over tokens

    def total(value, mass, axes):
        return Bounded(value.sum(axes), (kappa + sums * U) * mass.sum(axes))

    D4 = Dv[:, None]
    xv, mxv = (x * f["v"]).sum(3), (np.abs(x) * m["v"]).sum(3)
    up = 1.0 / (1.0 + np.exp(-raw)) if softplus else np.ones_like(raw)
    ddt = (A * f["dl"] + xv) * up
    mddt = (np.abs(A) * m["dl"] + mxv) * up
    y, my = f["y"] + D4 * x, m["y"] + np.abs(D4 * x)
    dz = None
    if z is not None:
        slope, mslope = sig * (1.0 + z * (1.0 - sig)), sig * (1.0 + np.abs(z) * (1.0 - sig))
        dz = Bounded(dout * y * slope, kappa * np.abs(dout) * my * mslope)
    b = lambda v, mass: Bounded(v, kappa * mass)  # noqa: E731
    return dict(
        y=b(y, my), h_last=b(f["h_last"], m["h_last"]),
        dx=b(D4 * gy + s[..., None] * f["v"], np.abs(D4 * gy) + np.abs(s)[..., None] * m["v"]),
        ddt=b(ddt, mddt), dz=dz, dB=b(back(f["dB"]), back(m["dB"])),
        dC=b(back(f["dC"]), back(m["dC"])), dA=total(s * f["dl"], np.abs(s) * m["dl"], (0, 1)),
        dD=total(gy * x, np.abs(gy * x), (0, 1, 3)), ddt_bias=total(ddt, mddt, (0, 1)),
        dh0=b(f["dh0"], m["dh0"]))
