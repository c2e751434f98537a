"""One token of the multi-head scan on the GPU, with and without the convolution, against float64."""
import numpy as np
import pytest

from oracle import head_twin as ht
from tests.block_helpers import Guarded, check, gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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
    """Inputs of one token; the rows of xbc, dt and z are parts of a projection's."""

    def __init__(self, seed, batch, H, P, N, G, io, k=0, gate=True, extra=0):
        print(f"  case batch={batch} H={H} P={P} N={N} G={G} {io} k={k} gate={gate}", flush=True)
        r = np.random.default_rng(seed)
        n = r.standard_normal
        self.io, self.G, self.k, self.shape = io, G, k, (batch, H, P)
        self.A, self.vA = gpu(-r.uniform(0.5, 8.0, H))
        self.D, self.vD = gpu(n(H))
        self.bias, self.vbias = gpu(n(H) - 2.0)
        self.state, self.vstate = gpu(n((batch, H, N, P)))
        d, bc = H * P, G * N
        row, v = gpu(n((batch, 2 * d + 2 * bc + H + extra)), io)
        self.z, self.vz = (row[:, :d], v[:, :d]) if gate else (None, None)
        self.xbc, self.vxbc = row[:, d:2 * d + 2 * bc], v[:, d:2 * d + 2 * bc]
        self.dt, self.vdt = (t[:, 2 * d + 2 * bc:2 * d + 2 * bc + H] for t in (row, v))
        if k:
            self.w, self.vw = gpu(0.5 * n((d + 2 * bc, k)))
            self.cb, self.vcb = gpu(0.2 * n(d + 2 * bc))
            self.cs, self.vcs = gpu(n((batch, k - 1, d + 2 * bc)), io)

    def plain(self):
        batch, H, P = self.shape
        d, bc, G = H * P, self.xbc.shape[1] // 2 - H * P // 2, self.G
        cut = lambda t, a, b, *s: t[:, a:b].reshape(batch, *s)  # noqa: E731
        N = bc // G
        parts = [(0, d, H, P), (d, d + bc, G, N), (d + bc, d + 2 * bc, G, N)]
        return ([cut(self.xbc, *q).contiguous() for q in parts],
                [cut(self.vxbc, *q) for q in parts])

    def check(self):
        o, batch, H, P = ops(), *self.shape
        kw = dict(D=self.D, dt_bias=self.bias)
        if self.k:
            out = o.scan2_state_update_conv(self.state, self.cs, self.xbc, self.w, self.cb,
                                            self.dt, self.A, ngroups=self.G, z=self.z, **kw)
            want, S, window = ht.step_conv(self.vstate, self.vcs, self.vxbc, self.vw, self.vcb,
                                           self.vdt, self.vA, self.G, self.vD, self.vz,
                                           self.vbias)
            assert np.array_equal(self.cs.double().cpu().numpy(), window)
        else:
            (x, B, C), (vx, vB, vC) = self.plain()
            z = self.z.reshape(batch, H, P).contiguous() if self.z is not None else None
            vz = self.vz.reshape(batch, H, P) if self.z is not None else None
            out = o.scan2_state_update(self.state, x, self.dt.contiguous(), self.A, B, C, z=z,
                                       **kw)
            want, S = ht.step(self.vstate, vx, self.vdt, self.vA, vB, vC, self.vD, vz, self.vbias)
        check(out, want, self.io, "out", 2.0)
        check(self.state, S, "f32", "state", 2.0)


SHAPES = [(1, 1, 1, 1, 1), (1, 80, 64, 128, 1), (3, 4, 64, 64, 2), (2, 6, 40, 48, 3),
          (5, 3, 17, 33, 1), (2, 2, 130, 256, 1), (3, 2, 4, 7, 2), (300, 2, 64, 16, 1),
          (600, 1, 20, 9, 1), (601, 1, 19, 70, 1), (7, 80, 64, 128, 8)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_token(shape, io):
    Case(sum(shape), *shape, io).check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1, 2, 3, 4])
@pytest.mark.parametrize("shape", SHAPES[1:6] + SHAPES[7:10], ids=str)
def test_token_behind_the_convolution(shape, k, io):
    Case(k + sum(shape), *shape, io, k=k, gate=k != 2, extra=k).check()


def test_without_optional_arguments():
    o = ops()
    c = Case(5, 2, 4, 16, 8, 2, "f32", gate=False)
    (x, B, C), (vx, vB, vC) = c.plain()
    out = o.scan2_state_update(c.state, x, c.dt.contiguous(), c.A, B, C, dt_softplus=False)
    want, S = ht.step(c.vstate, vx, c.vdt, c.vA, vB, vC, softplus=False)
    check(out, want, "f32", "out", 2.0)
    check(c.state, S, "f32", "state", 2.0)


def test_a_state_of_unaligned_rows():
    """A state that starts off a 16-byte boundary takes the one-channel lanes."""
    c = Case(6, 2, 4, 64, 32, 1, "bf16")
    buf = torch.empty(c.state.numel() + 1, device="cuda")
    view = buf[1:].view(c.state.shape)
    view.copy_(c.state)
    c.state = view
    c.check()


def test_writes_stay_inside():
    o = ops()
    for k, shape in ((0, (3, 2, 17, 33, 1)), (4, (600, 1, 20, 9, 1)), (3, (2, 80, 64, 128, 1))):
        c = Case(7, *shape, "bf16", k=k)
        batch, H, P = c.shape
        st, out = Guarded(c.state.shape, torch.float32), Guarded(c.shape, torch.bfloat16)
        st.t.copy_(c.state)
        if k:
            cs = Guarded(c.cs.shape, torch.bfloat16)
            cs.t.copy_(c.cs)
            ws = Guarded((batch * c.xbc.shape[1],), torch.float32)
            o.scan2_state_update_conv(st.t, cs.t, c.xbc, c.w, c.cb, c.dt, c.A, ngroups=c.G, z=c.z,
                                      out=out.t, workspace=ws.t)
            assert cs.intact() and ws.intact()
        else:
            (x, B, C), _ = c.plain()
            o.scan2_state_update(st.t, x, c.dt.contiguous(), c.A, B, C, out=out.t)
        assert st.intact() and out.intact()


def test_many_states_past_the_cache():
    """States above 128 MB are accessed non-temporally: each batch row equals a call on it alone."""
    o = ops()
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    batch, H, P, N = 70, 80, 64, 128
    x, dt, B, C = (r(*s).bfloat16() for s in ((batch, H, P), (batch, H), (batch, 1, N),
                                              (batch, 1, N)))
    A, state = -r(H).abs(), r(batch, H, N, P)
    alone = state[[0, 37, 69]].clone()
    out = o.scan2_state_update(state, x, dt, A, B, C)
    for i, b in enumerate((0, 37, 69)):
        one = slice(b, b + 1)
        s1 = alone[i:i + 1].contiguous()
        o1 = o.scan2_state_update(s1, x[one].contiguous(), dt[one].contiguous(), A,
                                  B[one].contiguous(), C[one].contiguous())
        torch.testing.assert_close(s1, state[one], rtol=0, atol=0)
        # the sums over the states run over other lanes where few heads are cut into blocks
        torch.testing.assert_close(o1.float(), out[one].float(), rtol=2 ** -7, atol=1e-4)


def test_extreme_steps():
    """A step so large that the decay is 0, one of 0, infinite and NaN states beside finite ones."""
    o = ops()
    state = torch.ones(3, 1, 2, 4, device="cuda")
    state[1, 0, 1, 2] = float("inf")
    state[2, 0, 0, 1] = float("nan")
    x, B, C = (torch.ones(3, 1, w, device="cuda") for w in (4, 2, 2))
    dt = torch.tensor([[1e4], [0.0], [1.0]], device="cuda")
    out = o.scan2_state_update(state, x, dt, -torch.ones(1, device="cuda"), B, C,
                               dt_softplus=False)
    assert torch.all(state[0] == 1e4) and torch.all(out[0] == 2e4)
    assert state[1, 0, 1, 2] == float("inf") and out[1, 0, 2] == float("inf")
    assert out[1].isinf().sum() == 1 and out[2].isnan().sum() == 1 and state[2].isnan().sum() == 1


def test_prompt_then_tokens():
    """A prompt through scan2_fwd and tokens one by one equal the whole sequence at once."""
    o = ops()
    r = np.random.default_rng(9)
    n = r.standard_normal
    batch, L, H, P, G, N, cut = 2, 90, 4, 64, 2, 64, 70
    x, _ = gpu(n((batch, L, H, P)))
    B, _ = gpu(n((batch, L, G, N)))
    C, _ = gpu(n((batch, L, G, N)))
    dt, _ = gpu(0.5 * n((batch, L, H)))
    z, _ = gpu(n((batch, L, H, P)))
    A, D, bias = (gpu(v)[0] for v in (-r.uniform(1, 8, H), n(H), n(H) - 3))
    kw = dict(D=D, dt_bias=bias)
    whole, last = o.scan2_fwd(x, dt, A, B, C, z=z, return_last_state=True, **kw)
    part = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    _, state = o.scan2_fwd(part(x, 0, cut), part(dt, 0, cut), A, part(B, 0, cut),
                           part(C, 0, cut), z=part(z, 0, cut), return_last_state=True, **kw)
    for t in range(cut, L):
        out = o.scan2_state_update(state, x[:, t].contiguous(), dt[:, t].contiguous(), A,
                                   B[:, t].contiguous(), C[:, t].contiguous(),
                                   z=z[:, t].contiguous(), **kw)
        torch.testing.assert_close(out, whole[:, t], rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(state, last, rtol=1e-4, atol=1e-4)


def test_the_binding_refuses():
    o = ops()
    c = Case(8, 2, 4, 8, 4, 1, "f32", k=4)
    good = dict(state=c.state, conv_state=c.cs, xbc=c.xbc, conv_weight=c.w, conv_bias=c.cb,
                dt=c.dt, A=c.A, z=c.z)
    o.scan2_state_update_conv(**good)
    for kw, err in ((dict(xbc=c.xbc[:, :-1]), "shape"), (dict(ngroups=2), "shape"),
                    (dict(dt=c.dt.bfloat16()), "must be"), (dict(conv_state=c.cs[:, :2]), "shape"),
                    (dict(z=c.z.t().contiguous().t()), "contiguous"),
                    (dict(xbc=c.xbc[:1].expand(2, -1)), "overlap"),
                    (dict(state=c.state.bfloat16()), "must be")):
        with pytest.raises((ValueError, TypeError), match=err):
            o.scan2_state_update_conv(**{**good, **kw})
    with pytest.raises(o.SSError):
        o.scan2_state_update_conv(**{**good, "out": c.state.view(-1)[:64].view(2, 4, 8)})
