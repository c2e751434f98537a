"""CPU checks of the float64 references of the block around the multi-head scan: the generator
against published vectors, every gradient against differences of the forward."""
import numpy as np
import pytest

from oracle import head_twin as ht


def test_philox_known_answers():
    """The known answers published with the generator (Random123, philox4x32 of 10 rounds)."""
    ones = 0xFFFFFFFF
    assert ht.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ht.philox((ones,) * 4, (ones,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ht.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
                     (0xA4093822, 0x299F31D0)) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_the_mask_drops_its_share():
    keep = ht.keep_mask((7, 11), 40, 203, 0.25)
    n = keep.size
    assert abs(keep.mean() - 0.75) < 5 * (0.25 * 0.75 / n) ** 0.5
    assert not np.array_equal(keep, ht.keep_mask((7, 12), 40, 203, 0.25))
    assert ht.keep_mask((7, 11), 3, 9, 0.0).all() and not ht.keep_mask((7, 11), 3, 9, 1.0).any()


def differences(f, args, name, weights, h=1e-5):
    """d (sum of weights * f) / d args[name] by central differences."""
    base = args[name]
    g = np.zeros_like(base)
    for k in np.ndindex(base.shape):
        v = []
        for sign in (1, -1):
            moved = base.copy()
            moved[k] += sign * h
            v.append(sum((w * o).sum() for w, o in zip(weights, f(**{**args, name: moved}))
                         if w is not None))
        g[k] = (v[0] - v[1]) / (2 * h)
    return g


def close(got, want):
    np.testing.assert_allclose(got, want, rtol=2e-6, atol=2e-7 * max(1.0, np.abs(want).max()))


@pytest.mark.parametrize("branch", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_rms_norm_gradients(branch, p):
    r = np.random.default_rng(1)
    n = r.standard_normal
    keep = ht.keep_mask((3, 5), 4, 11, p) if p else None
    args = dict(x=n((4, 11)), weight=n(11), residual=n((4, 11)), scale=n(11))
    dout, dsum = n((4, 11)), n((4, 11))

    def f(**a):
        out, s, *_ = ht.rms_fwd(**a, norm_branch=branch, keep=keep, p=p, eps=1e-3)
        return out.v, s.v

    g = ht.rms_bwd(dout, **args, norm_branch=branch, keep=keep, p=p, dsum=dsum, eps=1e-3)
    for name, grad in (("x", "dx"), ("weight", "dweight"), ("residual", "dresidual"),
                       ("scale", "dscale")):
        close(g[grad].v, differences(f, args, name, (dout, dsum)))


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("groups", [1, 3])
def test_gated_norm_gradients(first, groups):
    n = np.random.default_rng(2).standard_normal
    args = dict(x=n((3, 12)), z=n((3, 12)), weight=n(12))
    dout = n((3, 12))

    def f(**a):
        return (ht.gated_fwd(**a, groups=groups, gate_first=first, eps=1e-3)[0].v,)

    g = ht.gated_bwd(dout, **args, groups=groups, gate_first=first, eps=1e-3)
    for name in args:
        close(g["d" + name].v, differences(f, args, name, (dout,)))


@pytest.mark.parametrize("softplus", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_scan_gradients(softplus, gate):
    """Of the scan step by step (head_twin.step, which has no gradient of its own)."""
    r = np.random.default_rng(3)
    n = r.standard_normal
    batch, L, H, P, G, N = 2, 4, 2, 3, 1, 2
    args = dict(x=n((batch, L, H, P)), dt=n((batch, L, H)) * 0.3, A=-r.uniform(0.5, 2, H),
                B=n((batch, L, G, N)), C=n((batch, L, G, N)), D=n(H), dt_bias=n(H) * 0.2,
                h0=n((batch, H, N, P)))
    if gate:
        args["z"] = n((batch, L, H, P))
    dout, dh_last = n((batch, L, H, P)), n((batch, H, N, P))

    def f(x, dt, A, B, C, D, dt_bias, h0, z=None):
        S, outs = h0, []
        for t in range(L):
            out, S = ht.step(S, x[:, t], dt[:, t], A, B[:, t], C[:, t], D,
                             None if z is None else z[:, t], dt_bias, softplus)
            outs.append(out.v)
            S = S.v
        return np.stack(outs, 1), S

    g = ht.scan2_bwd(**args, dout=dout, softplus=softplus, dh_last=dh_last)
    for name in args:
        close(g["d" + name].v, differences(f, args, name, (dout, dh_last)))


def test_the_bounds_are_not_loose():
    """A thousandth of the upstream gradient moves every gradient out of its bound somewhere (the
    sums over tokens: a hundredth, or a twentieth where they take sums of pairs)."""
    r = np.random.default_rng(4)
    n = r.standard_normal
    a = dict(x=n((2, 70, 3, 8)), dt=n((2, 70, 3)) * 0.5, dt_bias=np.full(3, -3.0),
             A=-np.array([1.0, 2.0, 4.0]), B=n((2, 70, 1, 8)), C=n((2, 70, 1, 8)),
             dout=n((2, 70, 3, 8)), h0=n((2, 3, 8, 8)))
    g = ht.scan2_bwd(**a)
    for k, by in (("dx", 1e-3), ("dB", 1e-3), ("dC", 1e-3), ("ddt", 1e-3), ("dh0", 1e-3),
                  ("dD", 1e-2), ("dA", 5e-2), ("ddt_bias", 5e-2)):
        wrong = ht.scan2_bwd(**{**a, "dout": a["dout"] * (1 + by)})
        assert (np.abs(wrong[k].v - g[k].v) > g[k].e).any(), k
