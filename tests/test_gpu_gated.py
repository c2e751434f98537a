"""The gated linear recurrence on the GPU (forward, saved states, gradients, one token) against
its sequential float64 form, within error bounds carried through the formula."""
import numpy as np
import pytest

from oracle import block_twin as bt
from oracle.rounding import Bounded
from tests.block_helpers import Guarded, check, draw_starts, gpu, starts_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# A product of decays is formed in pieces (per wave, per tile) that are then multiplied, and each
# piece's end state is added to the carried one: at most twice the roundings of the plain order.
SPLIT = 2.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_36_amd import ops
    ops.lib()
    yield


def ops():
    from selective_state_space_36_amd import ops as o
    return o


class Case:
    def __init__(self, seed, batch, L, d, io, gate=False, packed=False, h0=False, bias=True,
                 offset=0):
        print(f"  case batch={batch} L={L} d={d} {io} gate={gate} packed={packed} h0={h0} "
              f"offset={offset}", flush=True)
        rng = np.random.default_rng(seed)
        n = lambda *s: rng.standard_normal(s)  # noqa: E731
        self.io = io
        g, v = {}, {}
        shape = (batch, L, d)
        for name in ("x", "r", "i", "dout"):
            g[name], v[name] = gpu(n(*shape), io, offset)
        g["z"], v["z"] = gpu(n(*shape) if gate else None, io, offset)
        g["A"], v["A"] = gpu(8.0 * np.log(rng.uniform(0.9, 0.999, d)))
        for name in ("r_bias", "i_bias"):
            g[name], v[name] = gpu(0.5 * n(d) if bias else None)
        g["h0"], v["h0"] = gpu(n(batch, d) if h0 else None)
        g["dh_last"], v["dh_last"] = gpu(n(batch, d) if h0 else None)
        v["starts"] = draw_starts(rng, batch, L) if packed and L else None
        g["starts"] = starts_gpu(v["starts"])
        self.g, self.v = g, v

    def kw(self, which):
        return {k: which[k] for k in ("r_bias", "i_bias", "z", "starts", "h0")}

    def args(self, which):
        return tuple(which[k] for k in ("x", "r", "i", "A"))

    def fwd(self):
        return ops().gated_scan_fwd_states(*self.args(self.g), **self.kw(self.g),
                                           return_last_state=True)

    def bwd(self, states):
        return ops().gated_scan_bwd(*self.args(self.g), self.g["dout"], **self.kw(self.g),
                                    dh_last=self.g["dh_last"], states=states)

    def reference(self):
        out, h = bt.gated_fwd(*self.args(self.v), **self.kw(self.v))
        return out, h

    def check_fwd(self):
        out, states, last = self.fwd()
        torch.cuda.synchronize()
        ref, h = self.reference()
        check(out, ref, self.io, "out", SPLIT)
        L = h.shape[1]
        ends = [min(t + 64, L) - 1 for t in range(0, L, 64)]
        check(states, h[:, ends], "f32", "states", SPLIT)
        check(last, h[:, -1], "f32", "h_last", SPLIT)
        return states

    def check_bwd(self, states):
        g = self.bwd(states)
        torch.cuda.synchronize()
        ref = bt.gated_bwd(*self.args(self.v), self.v["dout"], **self.kw(self.v),
                           dh_last=self.v["dh_last"])
        for name, want in ref.items():
            if want is None:
                assert g[name] is None
                continue
            io = self.io if name in ("dx", "dr", "di", "dz") else "f32"
            check(g[name], want, io, name, SPLIT)


SIZES = [(1, 1, 1), (1, 1, 64), (2, 2, 5), (2, 7, 33), (1, 63, 64), (2, 64, 130), (1, 65, 66),
         (3, 127, 128), (2, 129, 70), (1, 513, 257), (2, 1000, 20)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,d", SIZES)
def test_forward_and_gradients(batch, L, d, io):
    c = Case(L * 1000 + d, batch, L, d, io, gate=True, packed=True, h0=True)
    c.check_bwd(c.check_fwd())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("h0", [False, True])
def test_every_option(gate, packed, h0, io):
    c = Case(11, 2, 150, 68, io, gate=gate, packed=packed, h0=h0, bias=h0)
    c.check_bwd(c.check_fwd())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_sequence(io):
    c = Case(5, 1, 5000, 34, io, h0=True)
    c.check_bwd(c.check_fwd())


@pytest.mark.parametrize("batch", [8, 11, 15])
def test_chains_that_the_counters_share_unevenly(batch):
    c = Case(batch, batch, 700, 40, "bf16", gate=True, packed=True, h0=True)
    c.check_bwd(c.check_fwd())


def test_one_chain_of_many_tiles():
    """A single chain, so that most tiles of it are at work at the same time and look far back."""
    c = Case(7, 1, 40000, 8, "f32", packed=False, h0=True)
    c.check_bwd(c.check_fwd())


@pytest.mark.parametrize("d", [512, 1090, 1030])
def test_more_tiles_than_run_at_once(d):
    """A call of 768 (backward 1504) tiles, one of 1728 in 72 chains and one of 1632 in 68, which
    eight counters do not share evenly, equal their rows one by one, of a quarter as many."""
    c = Case(16, 4, 3000, d, "bf16", gate=True, packed=True, h0=True)
    out, states, last = c.fwd()
    g = c.bwd(states)
    for b in range(4):
        row = {k: (t[b:b + 1].contiguous() if t is not None and t.dim() > 1 else t)
               for k, t in c.g.items()}
        o, s, l = ops().gated_scan_fwd_states(*c.args(row), **c.kw(row), return_last_state=True)
        assert torch.equal(out[b:b + 1], o) and torch.equal(states[b:b + 1], s)
        assert torch.equal(last[b:b + 1], l)
        r = ops().gated_scan_bwd(*c.args(row), row["dout"], **c.kw(row), dh_last=row["dh_last"],
                                 states=s)
        for name in ("dx", "dr", "di", "dz", "dh0"):
            assert torch.equal(g[name][b:b + 1], r[name]), name


@pytest.mark.parametrize("io,gate,d", [("bf16", True, 3402), ("f32", False, 2303),
                                       ("bf16", True, 3392), ("f32", False, 2304)])
def test_a_call_that_outgrows_the_cache(io, gate, d):
    """Above 256 MB rows of whole cache lines are accessed non-temporally: the call equals its
    batch rows one by one, which stay below."""
    o, dt = ops(), torch.bfloat16 if io == "bf16" else torch.float32
    shape = (4, 2049, d)
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda: torch.randn(shape, device="cuda", generator=gen).to(dt)  # noqa: E731
    x, rr, ii, z, dout = r(), r(), r(), r() if gate else None, r()
    A = -torch.rand(shape[2], device="cuda", generator=gen)
    starts = torch.rand(shape[:2], device="cuda", generator=gen) < 0.003
    moved = x.numel() * x.element_size()
    assert moved * (5 if gate else 4) > 256 << 20 > moved * (9 if gate else 7) // 4
    out, states, last = o.gated_scan_fwd_states(x, rr, ii, A, z=z, starts=starts,
                                                return_last_state=True)
    g = o.gated_scan_bwd(x, rr, ii, A, dout, z=z, starts=starts, states=states)
    for b in range(4):
        c = lambda t: None if t is None else t[b:b + 1].contiguous()  # noqa: E731
        p = o.gated_scan_fwd_states(c(x), c(rr), c(ii), A, z=c(z), starts=c(starts),
                                    return_last_state=True)
        q = o.gated_scan_bwd(c(x), c(rr), c(ii), A, c(dout), z=c(z), starts=c(starts),
                             states=p[1])
        for whole, alone in zip((out, states, last), p):
            assert torch.equal(whole[b:b + 1], alone)
        for name in ("dx", "dr", "di", "dh0") + (("dz",) if gate else ()):
            assert torch.equal(g[name][b:b + 1], q[name]), name


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_arrays_that_start_inside_a_wider_alignment(offset, io):
    c = Case(offset, 2, 70, 66, io, gate=True, packed=True, offset=offset)
    c.check_bwd(c.check_fwd())


def test_states_recomputed_equal_states_given():
    c = Case(3, 2, 300, 130, "bf16", gate=True, packed=True, h0=True)
    _, states, _ = c.fwd()
    a, b = c.bwd(states), c.bwd(None)
    for name in a:
        assert torch.equal(a[name], b[name]), name


def test_two_runs_agree_bit_for_bit():
    c = Case(4, 3, 3000, 300, "bf16", gate=True, packed=True, h0=True)
    first = (c.fwd(), c.bwd(None))
    for _ in range(3):
        again = (c.fwd(), c.bwd(None))
        for p, q in zip(first[0], again[0]):
            assert torch.equal(p, q)
        for name in first[1]:
            assert torch.equal(first[1][name], again[1][name]), name


def test_result_does_not_depend_on_the_rest_of_the_batch():
    """A row, and a channel range, come out the same alone as within the whole call."""
    c = Case(6, 3, 700, 256, "bf16", gate=True, packed=True)
    whole = c.fwd()[0]
    row = {k: (t[1:2].contiguous() if t is not None and t.dim() > 1 else t)
           for k, t in c.g.items()}
    alone = ops().gated_scan_fwd(*c.args(row), **c.kw(row))
    assert torch.equal(whole[1:2], alone)


@pytest.mark.parametrize("L", [40, 400])
def test_nothing_crosses_a_start(L):
    """Infinities and NaN before a start reach no step behind it, nor a gradient before it."""
    rng = np.random.default_rng(8)
    d, cut = 70, L // 2 + 3
    mk = lambda: rng.standard_normal((1, L, d))  # noqa: E731
    x, r, i, z, dout = mk(), mk(), mk(), mk(), mk()
    x[0, 3, :20], x[0, 5, 20:40], r[0, 4, 40:50], z[0, 2, 50:60] = np.inf, np.nan, np.nan, -np.inf
    t = {k: gpu(a, "f32")[0] for k, a in dict(x=x, r=r, i=i, z=z, dout=dout).items()}
    A = gpu(-rng.uniform(0.01, 1.0, d))[0]
    starts = np.zeros((1, L), dtype=bool)
    starts[0, cut] = True
    s = starts_gpu(starts, torch.uint8)
    out, h = ops().gated_scan_fwd(t["x"], t["r"], t["i"], A, z=t["z"], starts=s,
                                  return_last_state=True)
    tail = {k: a[:, cut:].contiguous() for k, a in t.items()}
    ref, hr = ops().gated_scan_fwd(tail["x"], tail["r"], tail["i"], A, z=tail["z"],
                                   return_last_state=True)
    assert torch.isfinite(out[:, cut:]).all() and torch.isfinite(h).all()
    # the cut falls elsewhere in a tile here than in the separate call: the same up to rounding
    torch.testing.assert_close(out[:, cut:], ref, rtol=1e-4, atol=1e-5)
    g = ops().gated_scan_bwd(t["x"], t["r"], t["i"], A, t["dout"], z=t["z"], starts=s)
    gt = ops().gated_scan_bwd(tail["x"], tail["r"], tail["i"], A, tail["dout"], z=tail["z"])
    for name in ("dx", "dr", "di", "dz"):
        torch.testing.assert_close(g[name][:, cut:], gt[name], rtol=1e-4, atol=1e-5)
    # a NaN gradient behind the start does not flow back over it
    bad = t["dout"].clone()
    bad[:, cut + 1] = float("nan")
    clean = {k: gpu(rng.standard_normal((1, L, d)))[0] for k in ("x", "r", "i")}
    g = ops().gated_scan_bwd(clean["x"], clean["r"], clean["i"], A, bad, starts=s)
    assert torch.isfinite(g["dx"][:, :cut]).all()
    assert torch.isnan(g["dx"][:, cut:cut + 2]).all()


def test_a_nan_stays_in_its_channel_to_the_end_of_its_sequence():
    c = Case(9, 1, 900, 130, "f32")
    c.g["x"][0, 5, 7] = float("nan")
    c.g["x"][0, 6, 9] = float("inf")
    out, h = ops().gated_scan_fwd(*c.args(c.g), **c.kw(c.g), return_last_state=True)
    assert torch.isnan(out[0, 5:, 7]).all() and torch.isfinite(out[0, :5, 7]).all()
    assert torch.isinf(out[0, 6:, 9]).all() and torch.isfinite(out[0, :6, 9]).all()
    rest = [k for k in range(130) if k not in (7, 9)]
    assert torch.isfinite(out[0][:, rest]).all()


@pytest.mark.parametrize("A,r", [(0.0, 0.0), (-1e-30, 0.0), (-1e-4, 3.0), (-40.0, 5.0),
                                 (-200.0, 9.0), (-1.0, -200.0), (-1.0, 200.0), (-0.5, -15.0),
                                 (-0.01, -84.0), (-0.5, -87.0), (-0.01, -88.0)])
def test_extreme_gates(A, r):
    """Decays of exactly 1, nearly 1, underflowing, and gates that saturate."""
    rng = np.random.default_rng(10)
    L, d = 150, 66
    x, i, dout = (rng.standard_normal((1, L, d)) for _ in range(3))
    rr = np.full((1, L, d), r) + 1e-3 * rng.standard_normal((1, L, d))
    gs, vs = zip(*(gpu(a) for a in (x, rr, i, np.full(d, A), dout, rng.standard_normal((1, d)))))
    out, states = ops().gated_scan_fwd_states(*gs[:4], h0=gs[5])
    ref, _ = bt.gated_fwd(*vs[:4], h0=vs[5])
    check(out, ref, "f32", "out", SPLIT)
    g = ops().gated_scan_bwd(*gs[:4], gs[4], h0=gs[5], states=states)
    want = bt.gated_bwd(*vs[:4], vs[4], h0=vs[5])
    for name in ("dx", "dr", "di", "dh0"):
        check(g[name], want[name], "f32", name, SPLIT)
        assert torch.isfinite(g[name]).all(), name
    assert torch.isfinite(g["dA"]).all()


def test_a_positive_A_is_a_nan():
    c = Case(12, 1, 20, 64, "f32")
    c.g["A"][3] = 0.5
    out = ops().gated_scan_fwd(*c.args(c.g), **c.kw(c.g))
    assert torch.isnan(out[..., 3]).all() and torch.isfinite(out[..., 4:]).all()


@pytest.mark.parametrize("batch,d", [(1, 1), (1, 5120), (3, 77), (128, 256), (5, 1027)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
def test_one_token(batch, d, io, gate):
    rng = np.random.default_rng(d)
    g, v = {}, {}
    for name in ("x", "r", "i", "z"):
        g[name], v[name] = gpu(rng.standard_normal((batch, d)), io)
    if not gate:
        g["z"] = v["z"] = None
    A, vA = gpu(-rng.uniform(0.01, 2.0, d))
    rb, vrb = gpu(rng.standard_normal(d))
    state, vs = gpu(rng.standard_normal((batch, d)))
    out = ops().gated_state_update(state, g["x"], g["r"], g["i"], A, r_bias=rb, z=g["z"])
    ref, h = bt.gated_step(vs, v["x"], v["r"], v["i"], vA, vrb, None, v["z"])
    check(out, ref, io, "out")
    check(state, h, "f32", "state")


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
def test_one_token_misaligned(offset):
    rng = np.random.default_rng(offset)
    mk = lambda: gpu(rng.standard_normal((3, 64)), "bf16", offset)  # noqa: E731
    (x, vx), (r, vr), (i, vi) = mk(), mk(), mk()
    A, vA = gpu(-rng.uniform(0.01, 2.0, 64), "f32", offset)
    state, vs = gpu(rng.standard_normal((3, 64)), "f32", offset)
    out = ops().gated_state_update(state, x, r, i, A)
    ref, h = bt.gated_step(vs, vx, vr, vi, vA)
    check(out, ref, "bf16", "out")
    check(state, h, "f32", "state")


def test_prefill_then_tokens_repeat_the_whole_sequence():
    c = Case(13, 2, 200, 96, "f32", gate=True)
    whole = c.fwd()[0]
    cut = 130
    part = {k: (t[:, :cut].contiguous() if t is not None and t.dim() == 3 else t)
            for k, t in c.g.items()}
    out, state = ops().gated_scan_fwd(*c.args(part), **c.kw(part), return_last_state=True)
    outs = [out]
    for t in range(cut, 200):
        tok = {k: c.g[k][:, t].contiguous() for k in ("x", "r", "i", "z")}
        outs.append(ops().gated_state_update(state, tok["x"], tok["r"], tok["i"], c.g["A"],
                                             c.g["r_bias"], c.g["i_bias"], tok["z"])[:, None])
    ref, _ = c.reference()
    check(torch.cat(outs, 1), ref, "f32", "resumed", SPLIT)
    check(whole, ref, "f32", "whole", SPLIT)


@pytest.mark.parametrize("batch,L,d", [(2, 77, 65), (1, 130, 30), (2, 5, 200)])
def test_writes_stay_inside_the_outputs(batch, L, d):
    c = Case(14, batch, L, d, "bf16", gate=True, packed=True)
    out, last = Guarded((batch, L, d), torch.bfloat16), Guarded((batch, d), torch.float32)
    states = Guarded((batch, -(-L // 64), d), torch.float32)
    o = ops()
    n = o.lib().ss_gated_scan_fwd_workspace_bytes(batch, L, d, o.SS_BF16)
    ws = Guarded((max(n, 16),), torch.uint8)
    o.gated_scan_fwd_states(*c.args(c.g), **c.kw(c.g), return_last_state=True, out=out.t,
                            h_last=last.t, states=states.t, workspace=ws.t)
    for given in (states.t, None):
        n = o.lib().ss_gated_scan_bwd_workspace_bytes(batch, L, d, o.SS_BF16, given is not None)
        wb = Guarded((max(n, 16),), torch.uint8)
        o.gated_scan_bwd(*c.args(c.g), c.g["dout"], **c.kw(c.g), states=given, workspace=wb.t)
        torch.cuda.synchronize()
        assert wb.intact()
    assert out.intact() and last.intact() and states.intact() and ws.intact()
    ref, h = c.reference()
    check(out.t, ref, "bf16", "out", SPLIT)
    check(last.t, h[:, -1], "f32", "h_last", SPLIT)


def test_a_workspace_needs_no_preparation():
    c = Case(15, 1, 900, 80, "f32", packed=True)
    o = ops()
    want = c.fwd()[0]
    n = max(16, o.lib().ss_gated_scan_fwd_workspace_bytes(1, 900, 80, o.SS_F32))
    for fill in (0, 0xFF, 0x80):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            assert torch.equal(o.gated_scan_fwd(*c.args(c.g), **c.kw(c.g), workspace=ws), want)


def test_empty_sizes():
    o = ops()
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    A, h0 = -torch.ones(8, device="cuda"), torch.randn(2, 8, device="cuda")
    out, last = o.gated_scan_fwd(e(2, 0, 8), e(2, 0, 8), e(2, 0, 8), A, h0=h0,
                                 return_last_state=True)
    assert out.shape == (2, 0, 8) and torch.equal(last, h0)
    _, last = o.gated_scan_fwd(e(2, 0, 8), e(2, 0, 8), e(2, 0, 8), A, return_last_state=True)
    assert not last.any()
    g = o.gated_scan_bwd(e(2, 0, 8), e(2, 0, 8), e(2, 0, 8), A, e(2, 0, 8), h0=h0, dh_last=h0)
    assert not g["dA"].any() and not g["dr_bias"].any() and torch.equal(g["dh0"], h0)
    g = o.gated_scan_bwd(e(0, 3, 8), e(0, 3, 8), e(0, 3, 8), A, e(0, 3, 8))
    assert not g["dA"].any() and g["dh0"].shape == (0, 8)
    assert o.gated_scan_fwd(e(1, 4, 0), e(1, 4, 0), e(1, 4, 0), e(0)).shape == (1, 4, 0)
    assert o.gated_state_update(e(0, 8), e(0, 8), e(0, 8), e(0, 8), A).shape == (0, 8)


@pytest.mark.parametrize("lo,hi", [(37, 200), (64, 65), (130, 256), (0, 63)])
@pytest.mark.parametrize("L", [100, 700])
def test_a_channel_range_comes_out_the_same_alone(lo, hi, L):
    """Also one that begins inside a group of 64 channels, and one that ends in another."""
    c = Case(17, 3, L, 256, "bf16", gate=True, packed=True, h0=True)
    whole = (*c.fwd(), c.bwd(None))
    part = {k: t if t is None or k == "starts" else t[..., lo:hi].contiguous()
            for k, t in c.g.items()}
    alone = ops().gated_scan_fwd_states(*c.args(part), **c.kw(part), return_last_state=True)
    g = ops().gated_scan_bwd(*c.args(part), part["dout"], **c.kw(part), dh_last=part["dh_last"])
    for p, q in zip(whole, alone):
        assert torch.equal(p[..., lo:hi], q)
    for name in g:
        assert torch.equal(whole[3][name][..., lo:hi], g[name]), name


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("batch,L,d", [(2, 77, 65), (1, 130, 30), (2, 5, 200), (1, 1, 1),
                                       (3, 300, 129)])
def test_gradients_stay_inside_their_arrays(batch, L, d, given, io):
    """Every array that the backward writes, between marker bytes; and the one-token form's."""
    o = ops()
    c = Case(18, batch, L, d, io, gate=True, packed=True, h0=True)
    states = c.fwd()[1] if given else None
    want, v = c.bwd(states), c.g
    dt, f32 = v["x"].dtype, torch.float32
    g = {k: Guarded((batch, L, d), dt) for k in ("dx", "dr", "di", "dz")}
    g.update({k: Guarded((d,), f32) for k in ("dA", "dr_bias", "di_bias")},
             dh0=Guarded((batch, d), f32))
    code = o.SS_BF16 if io == "bf16" else o.SS_F32
    n = o.lib().ss_gated_scan_bwd_workspace_bytes(batch, L, d, code, given)
    ws = Guarded((n,), torch.uint8)
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    o._check(o.lib().ss_gated_scan_bwd(
        *(p(v[k]) for k in ("x", "r", "i", "A", "r_bias", "i_bias", "z", "starts", "h0", "dout",
                            "dh_last")), p(states),
        *(p(g[k].t) for k in ("dx", "dr", "di", "dz", "dA", "dr_bias", "di_bias", "dh0")),
        batch, L, d, code, p(ws.t), n, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    for k, buf in g.items():
        assert torch.equal(buf.t, want[k]) and buf.intact(), k
    assert ws.intact()
    tok = {k: v[k][:, 0].contiguous() for k in ("x", "r", "i", "z")}
    state, out = Guarded((batch, d), f32), Guarded((batch, d), dt)
    state.t.copy_(v["h0"])
    h = v["h0"].clone()
    rest = (tok["x"], tok["r"], tok["i"], v["A"], v["r_bias"], v["i_bias"], tok["z"])
    ref = o.gated_state_update(h, *rest)
    o.gated_state_update(state.t, *rest, out=out.t)
    assert torch.equal(out.t, ref) and torch.equal(state.t, h)
    assert out.intact() and state.intact()


@pytest.mark.parametrize("A,r", [(0.0, 0.0), (-1e-30, 0.0), (-1e-4, 3.0), (-40.0, 5.0),
                                 (-200.0, 9.0), (-1.0, -200.0), (-1.0, 200.0), (-0.5, -15.0),
                                 (-0.01, -84.0), (-0.5, -87.0), (-0.01, -88.0)])
def test_parameter_gradients_of_extreme_gates(A, r):
    rng = np.random.default_rng(10)
    L, d = 150, 66
    x, i, dout = (rng.standard_normal((2, L, d)) for _ in range(3))
    rr = np.full((2, L, d), r) + 1e-3 * rng.standard_normal((2, L, d))
    gs, vs = zip(*(gpu(a) for a in (x, rr, i, np.full(d, A), dout, rng.standard_normal((2, d)))))
    g = ops().gated_scan_bwd(*gs[:4], gs[4], h0=gs[5])
    want = bt.gated_bwd(*vs[:4], vs[4], h0=vs[5])
    check(g["di_bias"], want["di_bias"], "f32", "di_bias", SPLIT)
    for name in ("dA", "dr_bias"):
        if r > -80.0:
            check(g[name], want[name], "f32", name, SPLIT)
            continue
        # 1 - a^2 = 2 |A| rg nears or passes the smallest normal number, and its reciprocal root
        # has no useful bound; but a token adds lam (a h rg - ig x a^2 rg / s) with
        # rg / s = (rg / 2 |A|)^(1/2) < 4.1e-18, or without the second term, where |lam| < 2 L 5,
        # |x| and |h| < 5 and rg < 4e-37: 2 L tokens of 2 L 25 4.1e-18 are below 1e-11.
        assert abs(want[name].v).max() < 1e-11 and (g[name].abs() < 1e-11).all(), name
