"""Gradients of the multi-head scan on the GPU against the float64 recurrence and its adjoint."""
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
    def __init__(self, seed, batch, L, H, P, G, N, io, gate=True, carry=True, softplus=True,
                 step=-3.0, offset=0):
        print(f"  case batch={batch} L={L} H={H} P={P} G={G} N={N} {io} gate={gate} "
              f"carry={carry}", flush=True)
        r = np.random.default_rng(seed)
        n = r.standard_normal
        self.io, self.softplus = io, softplus
        g = {}
        g["x"] = gpu(n((batch, L, H, P)), io, offset)
        g["dt"] = gpu(0.5 * n((batch, L, H)) if softplus else r.uniform(0, 0.1, (batch, L, H)), io,
                      offset)
        g["A"] = gpu(-r.uniform(1.0, 8.0, H))
        g["B"] = gpu(n((batch, L, G, N)), io, offset)
        g["C"] = gpu(n((batch, L, G, N)), io, offset)
        g["dout"] = gpu(n((batch, L, H, P)), io, offset)
        g["D"] = gpu(n(H))
        g["z"] = gpu(n((batch, L, H, P)) if gate else None, io, offset)
        g["dt_bias"] = gpu(n(H) * 0.3 + step if softplus else None)
        g["h0"] = gpu(n((batch, H, N, P)) if carry else None)
        g["dh_last"] = gpu(n((batch, H, N, P)) if carry else None)
        self.t = {k: v[0] for k, v in g.items()}
        self.v = {k: v[1] for k, v in g.items()}

    def run(self, **kw):
        return ops().scan2_bwd(**self.t, dt_softplus=self.softplus, **kw)

    def check(self):
        got = self.run()
        want = ht.scan2_bwd(**self.v, softplus=self.softplus)
        for name in ("dx", "ddt", "dz", "dB", "dC"):
            if want[name] is not None:
                check(got[name], want[name], self.io, name)
        for name in ("dA", "dD", "ddt_bias", "dh0"):
            check(got[name], want[name], "f32", name)
        return got


SHAPES = [(1, 1, 1, 1, 1, 1), (1, 1, 2, 64, 1, 128), (2, 2, 2, 5, 2, 3), (1, 63, 2, 64, 1, 64),
          (2, 64, 3, 64, 1, 128), (1, 65, 4, 64, 2, 128), (2, 130, 6, 40, 3, 48),
          (1, 200, 2, 17, 1, 33), (1, 129, 2, 130, 1, 20), (1, 70, 2, 9, 2, 130),
          (2, 67, 2, 64, 1, 200), (1, 66, 2, 70, 1, 256), (3, 100, 5, 64, 1, 64)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, io):
    Case(sum(shape), *shape, io).check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("N", [64, 128, 24])
def test_gate_and_carried_state(gate, carry, N, io):
    Case(N, 2, 150, 4, 64, 2, N, io, gate=gate, carry=carry).check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_raw_steps(io):
    Case(3, 2, 100, 4, 64, 1, 64, io, softplus=False).check()


@pytest.mark.parametrize("step", [-8.0, 0.0, 4.0])
def test_slow_and_fast_decays(step):
    """Steps from 3e-4 to 4: decays near 1 and of e^-16 a step, where the exponents of a chunk reach
    e^-2000 and the products of the dual form underflow."""
    Case(4, 1, 140, 4, 64, 1, 64, "f32", step=step).check()


@pytest.mark.parametrize("offset", [1, 3])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_misaligned(offset, io):
    Case(offset, 2, 70, 2, 64, 1, 64, io, offset=offset).check()


@pytest.mark.parametrize("H,G,batch", [(80, 1, 1), (7, 1, 2), (12, 4, 1)])
def test_runs_of_heads(H, G, batch):
    """Few chunks: the heads of a group are cut into runs whose parts of dB and dC are added."""
    Case(H, batch, 80, H, 16, G, 16, "f32").check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 300, 40, 64, 1, 64), (1, 270, 70, 16, 2, 24),
                                   (3, 256, 2, 64, 1, 128), (1, 1100, 3, 64, 3, 64),
                                   (1, 700, 2, 70, 1, 20)], ids=str)
def test_walks_whole_and_cut(shape, io):
    """Many heads walk the chunks whole, few are cut into chunks and joined."""
    Case(sum(shape), *shape, io).check()


def test_two_runs_agree_bit_for_bit():
    c = Case(11, 2, 300, 8, 64, 1, 128, "bf16")
    a, b = c.run(), c.run()
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_optional_outputs():
    c = Case(12, 2, 70, 4, 64, 1, 64, "f32", gate=False, carry=False)
    full = c.run()
    some = c.run(want_dD=False, want_ddt_bias=False, want_dh0=False)
    assert some["dD"] is None and some["ddt_bias"] is None and some["dh0"] is None
    assert some["dz"] is None
    for k in ("dx", "ddt", "dA", "dB", "dC"):
        assert torch.equal(full[k], some[k]), k


def test_empty():
    o = ops()
    for batch, L, P in ((0, 5, 8), (2, 0, 8), (2, 5, 0)):
        z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
        dh = torch.randn(batch, 4, 8, P, device="cuda")
        g = o.scan2_bwd(z(batch, L, 4, P), z(batch, L, 4), -torch.ones(4, device="cuda"),
                        z(batch, L, 1, 8), z(batch, L, 1, 8), z(batch, L, 4, P), dh_last=dh)
        for k in ("dA", "dD", "ddt_bias", "ddt", "dB", "dC"):
            assert torch.all(g[k] == 0), k
        if L == 0:
            assert torch.equal(g["dh0"], dh)


@pytest.mark.parametrize("shape,io", [((2, 70, 3, 17, 1, 33), "bf16"), ((1, 65, 4, 64, 2, 128), "bf16"),
                                      ((2, 130, 4, 64, 1, 64), "bf16"),
                                      ((1, 3, 2, 130, 1, 200), "f32")])
def test_writes_stay_inside(shape, io):
    from selective_state_space_36_amd import ops as o
    batch, L, H, P, G, N = shape
    c = Case(13, *shape, io)
    dt = torch.float32 if io == "f32" else torch.bfloat16
    f32 = torch.float32
    l, code = o.lib(), o.SS_F32 if io == "f32" else o.SS_BF16
    outs = dict(dx=(c.t["x"].shape, dt), ddt=((batch, L, H), dt), dz=(c.t["x"].shape, dt),
                dA=((H,), f32), dB=((batch, L, G, N), dt), dC=((batch, L, G, N), dt),
                dD=((H,), f32), ddt_bias=((H,), f32), dh0=((batch, H, N, P), f32))
    b = {k: Guarded(*v) for k, v in outs.items()}
    n = l.ss_scan2_bwd_workspace_bytes(batch, L, H, P, G, N, code)
    ws = Guarded((n,), torch.uint8)
    t = {k: v.data_ptr() for k, v in c.t.items()}
    assert l.ss_scan2_bwd(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["z"], t["dt_bias"],
                          1, t["h0"], t["dout"], t["dh_last"],
                          *[b[k].t.data_ptr() for k in outs], batch, L, H, P, G, N, code,
                          ws.t.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    want = c.run()
    for k in outs:
        assert b[k].intact() and torch.equal(b[k].t, want[k]), k
    assert ws.intact()


def test_forward_is_what_is_differentiated():
    """Differences of scan2_fwd in float32 along one direction of every input."""
    c = Case(14, 1, 100, 2, 8, 1, 8, "f32")
    g = c.run()
    o, t = ops(), c.t
    gen = torch.Generator(device="cuda").manual_seed(1)

    def loss(v):
        out, last = o.scan2_fwd(v["x"], v["dt"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"],
                                dt_bias=v["dt_bias"], h0=v["h0"], return_last_state=True)
        return float((out.double() * t["dout"].double()).sum()
                     + (last.double() * t["dh_last"].double()).sum())

    for name in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0"):
        way = torch.randn(t[name].shape, device="cuda", generator=gen)
        h = 1e-2
        up, down = ({**t, name: t[name] + s * h * way} for s in (1, -1))
        diff = (loss(up) - loss(down)) / (2 * h)
        slope = float((g["d" + name].double() * way.double()).sum())
        # differences: third derivatives times h^2, and the float32 forward's rounding over h
        size = float((g["d" + name].double() * way.double()).square().sum().sqrt())
        assert abs(diff - slope) <= 0.02 * abs(slope) + 0.02 * size, (name, diff, slope)


def test_offsets_past_32_bits():
    """Rows past 2^31 elements: the last batch rows of a large call equal a call on them alone."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    batch, L, H, P, N = 2, 2100, 2048, 256, 4
    r = lambda *s: torch.randn(s, device="cuda", generator=gen, dtype=torch.bfloat16)  # noqa: E731
    t = dict(x=r(batch, L, H, P), dt=r(batch, L, H), A=-torch.ones(H, device="cuda"),
             B=r(batch, L, 1, N), C=r(batch, L, 1, N), dout=r(batch, L, H, P),
             dt_bias=torch.full((H,), -3.0, device="cuda"))
    assert t["x"].numel() > 1 << 31
    g = ops().scan2_bwd(**t)
    one = {k: v[1:].contiguous() if v.dim() > 1 else v for k, v in t.items()}
    alone = ops().scan2_bwd(**one)
    assert torch.equal(g["dx"][1], alone["dx"][0]) and torch.equal(g["ddt"][1], alone["ddt"][0])
    assert torch.equal(g["dh0"][1], alone["dh0"][0])
