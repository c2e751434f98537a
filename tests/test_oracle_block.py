"""The float64 forms of the recurrent block's operators: gradients against differences of the
forward pass, the sequence forms against the one-token forms, starts against separate calls, and
the error bounds against a float32 evaluation."""
import numpy as np
import pytest

from oracle import block_twin as bt


def numeric(loss, args, name, h=1e-6):
    """Central differences of loss(**args) in every element of args[name]."""
    base = args[name]
    g = np.zeros_like(base)
    for k in np.ndindex(base.shape):
        vals = []
        for s in (1.0, -1.0):
            p = base.copy()
            p[k] += s * h
            vals.append(loss(**{**args, name: p}))
        g[k] = (vals[0] - vals[1]) / (2 * h)
    return g


def close(got, want, what):
    # central differences: h^2 f''' / 6 + 2^-52 |f| / h, both near 1e-9 for sums of some tens
    np.testing.assert_allclose(got, want, rtol=2e-6, atol=2e-7, err_msg=what)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_recurrence_gradients_are_differences(gate, packed):
    rng = np.random.default_rng(1)
    b, L, d = 2, 7, 3
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    args = dict(x=n(b, L, d), r=n(b, L, d), i=n(b, L, d), A=-np.exp(n(d)), r_bias=n(d),
                i_bias=n(d), z=n(b, L, d) if gate else None, h0=n(b, d))
    starts = None
    if packed:
        starts = np.zeros((b, L), dtype=bool)
        starts[0, 3] = starts[0, 4] = starts[1, 0] = True
    dout, dlast = n(b, L, d), n(b, d)

    def loss(**kw):
        out, h = bt.gated_fwd(**kw, starts=starts)
        return float((out.v * dout).sum() + (h.v[:, -1] * dlast).sum())

    g = bt.gated_bwd(**args, dout=dout, dh_last=dlast, starts=starts)
    for name in ("x", "r", "i", "A", "r_bias", "i_bias", "h0") + (("z",) if gate else ()):
        key = {"r_bias": "dr_bias", "i_bias": "di_bias"}.get(name, "d" + name)
        close(g[key].v, numeric(loss, args, name), name)


@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradients_are_differences(residual):
    rng = np.random.default_rng(2)
    rows, dim = 3, 9
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    args = dict(x=n(rows, dim), weight=n(dim), bias=n(dim),
                residual=n(rows, dim) if residual else None)
    dout, dsum = n(rows, dim), n(rows, dim)

    def loss(**kw):
        out, s, *_ = bt.norm_fwd(**kw)
        return float((out.v * dout).sum() + (s.v * dsum).sum())

    g = bt.norm_bwd(dout, args["x"], args["weight"], args["residual"], dsum)
    close(g["ds"].v, numeric(loss, args, "x"), "x")
    if residual:
        close(g["ds"].v, numeric(loss, args, "residual"), "residual")
    close(g["dweight"].v, numeric(loss, args, "weight"), "weight")
    close(g["dbias"].v, numeric(loss, args, "bias"), "bias")


@pytest.mark.parametrize("k", [1, 2, 4])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_conv_gradients_are_differences(k, silu, packed):
    rng = np.random.default_rng(3)
    b, L, d = 2, 6, 2
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    args = dict(x=n(b, L, d), weight=n(d, k), bias=n(d), x_prev=n(b, k - 1, d))
    starts = None
    if packed:
        starts = np.zeros((b, L), dtype=bool)
        starts[0, 2] = starts[0, 3] = starts[1, 0] = True
    dout = n(b, L, d)

    def loss(**kw):
        return float((bt.conv_fwd(**kw, starts=starts, silu=silu)[0].v * dout).sum())

    g = bt.conv_bwd(args["x"], args["weight"], dout, args["bias"], args["x_prev"], starts, silu)
    for name, key in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"),
                      ("x_prev", "dx_prev")):
        close(g[key].v, numeric(loss, args, name), name)


def test_starts_are_separate_calls():
    rng = np.random.default_rng(4)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    x, r, i, A, w = n(1, 9, 4), n(1, 9, 4), n(1, 9, 4), -np.exp(n(4)), n(4, 3)
    starts = np.zeros((1, 9), dtype=bool)
    starts[0, 5] = True
    whole = bt.gated_fwd(x, r, i, A, starts=starts, h0=n(1, 4))[0].v[:, 5:]
    np.testing.assert_array_equal(whole, bt.gated_fwd(x[:, 5:], r[:, 5:], i[:, 5:], A)[0].v)
    np.testing.assert_array_equal(bt.conv_fwd(x, w, starts=starts)[0].v[:, 5:],
                                  bt.conv_fwd(x[:, 5:], w)[0].v)


def test_one_token_forms_repeat_the_sequence():
    rng = np.random.default_rng(5)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    x, r, i, z = (n(2, 5, 3) for _ in range(4))
    A, w, bias = -np.exp(n(3)), n(3, 4), n(3)
    h, win = n(2, 3), n(2, 3, 3)
    out, hs = bt.gated_fwd(x, r, i, A, z=z, h0=h)
    conv = bt.conv_fwd(x, w, bias, win)[0]
    for t in range(5):
        o, h = bt.gated_step(getattr(h, "v", h), x[:, t], r[:, t], i[:, t], A, z=z[:, t])
        c, win = bt.conv_step(win, x[:, t], w, bias)
        np.testing.assert_allclose(o.v, out.v[:, t], rtol=1e-13)
        np.testing.assert_allclose(c.v, conv.v[:, t], rtol=1e-13)


def test_bounds_hold_for_float32():
    """numpy's float32 evaluation stays inside the bounds, and they are not loose beyond use."""
    rng = np.random.default_rng(6)
    f = np.float32
    n = lambda *s: rng.standard_normal(s).astype(f)  # noqa: E731
    x, r, i, A = n(2, 50, 8), n(2, 50, 8), n(2, 50, 8), -np.exp(n(8))
    out, _ = bt.gated_fwd(*(v.astype(np.float64) for v in (x, r, i, A)))
    sig = lambda v: f(1) / (f(1) + np.exp(-v))  # noqa: E731
    l = A * sig(r)
    a, s = np.exp(l), np.sqrt(-np.expm1(f(2) * l))
    b = s * sig(i) * x
    h, got = np.zeros((2, 8), f), np.zeros_like(x)
    for t in range(50):
        h = a[:, t] * h + b[:, t]
        got[:, t] = h
    err = np.abs(got - out.v)
    assert (err <= out.e).all()
    assert np.median(out.e / np.abs(out.v)) < 1e-5
