"""What the multi-head scan's gradients keep of float32: sums that cancel, exponents, and the sums
over all tokens (dA, dD, ddt_bias), against float64 on the same inputs."""
import numpy as np
import pytest

from oracle import head_twin as ht
from oracle.rounding import U
from tests.block_helpers import DTYPES, check, gpu

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


@pytest.mark.parametrize("N", [64, 128, 16])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_steps_of_unlike_size(io, N):
    """Step 0 reaches step 1 with 2^26 and step 5 with 1.  At steps 2 to 5 only the second passes,
    from step 6 on nothing does: ddt there is A e^{5 A} and 0, though the first is 2^26 times as
    large.  One product passes: its exponential is off by the exponent's rounding (|c| < 1, so 2 U),
    one ulp of exp2 (2 U) and the sum of log decays (2 U), the products by A, dt and 1 / (1 + ...)
    by U each: 10 U."""
    o, dt = ops(), DTYPES[io]
    L, P, A = 16, 64, -2.0 ** -4
    z = lambda *s: torch.zeros(s, device="cuda", dtype=dt)  # noqa: E731
    x, B, C, dout = z(1, L, 1, P), z(1, L, 1, N), z(1, L, 1, N), z(1, L, 1, P)
    B[..., 0] = C[..., 0] = 1
    x[0, 0, 0, 0], x[0, 0, 0, 1] = 2 ** 13, 1
    dout[0, 1, 0, 0], dout[0, 5, 0, 1] = 2 ** 13, 1
    g = o.scan2_bwd(x, torch.ones(1, L, 1, device="cuda", dtype=dt),
                    torch.full((1,), A, device="cuda"), B, C, dout, dt_softplus=False)
    ddt = g["ddt"][0, :, 0].double().cpu()
    want = A * float(torch.tensor(5 * A, dtype=torch.float64).exp())
    tol = 10 * U + (2 ** -8 if io == "bf16" else 0)
    for t in range(2, 6):
        assert abs(float(ddt[t]) - want) <= tol * abs(want), (t, float(ddt[t]), want)
    assert torch.all(ddt[6:] == 0), ddt


@pytest.mark.parametrize("low", [torch.finfo(torch.float32).min, -1e38, -1e9])
@pytest.mark.parametrize("io,shape", [("f32", (2, 150, 4, 64, 2, 64)), ("bf16", (2, 150, 4, 64, 2, 64)),
                                      ("bf16", (1, 70, 3, 64, 1, 128)), ("f32", (1, 300, 2, 17, 1, 9)),
                                      ("bf16", (4, 320, 40, 64, 1, 64))], ids=str)
def test_heads_that_forget_at_once(io, shape, low):
    """An A down to the type's lowest value lets no state through: the head's gradients are those of
    single steps, the other heads' are what they are.  (The reference and its bound with A = -1e5,
    whose decays of e^-1000 and less are 0 as well.)"""
    batch, L, H, P, G, N = shape
    r = np.random.default_rng(L + N)
    n = r.standard_normal
    A = -r.uniform(1.0, 8.0, H)
    A[1] = -1e5
    v, t = {}, {}
    for k, a, dt in (("x", n((batch, L, H, P)), io), ("dt", 0.5 * n((batch, L, H)), io), ("A", A, "f32"),
                     ("B", n((batch, L, G, N)), io), ("C", n((batch, L, G, N)), io),
                     ("dout", n((batch, L, H, P)), io), ("D", n(H), "f32"),
                     ("z", n((batch, L, H, P)), io), ("dt_bias", 0.3 * n(H) - 1.0, "f32"),
                     ("h0", n((batch, H, N, P)), "f32"), ("dh_last", n((batch, H, N, P)), "f32")):
        t[k], v[k] = gpu(a, dt)
    t["A"][1] = low
    got, want = ops().scan2_bwd(**t), ht.scan2_bwd(**v)
    # (A dl, of that head: its dl is 0, and the reference's exponents stand in the bound of all)
    quiet = dict(v, A=np.where(np.arange(H) == 1, -8.0, v["A"]))
    bound = ht.scan2_bwd(**quiet)
    for k in ("dx", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dh0"):
        want[k].e = bound[k].e
        check(got[k], want[k], io if k in ("dx", "ddt", "dz", "dB", "dC") else "f32", k)
    assert torch.all(got["dh0"][:, 1] == 0) and float(got["dA"][1]) == 0


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_what_only_exponents_scale(io):
    """64 steps of one chunk with one product on every way, scaled by 2^{c}, c to -64: the state's
    adjoint arriving from behind in dh0 (and, in float32, in dx), one step's dout in the dx of all, the
    state before in dC.  Off are exp2 by one ulp (2 U), the correction by U, and up to five products
    and conversions by U each: 8 U, however large the exponent (rounded to float32 it would be 44 U)."""
    o, dt = ops(), DTYPES[io]
    L, H, P, N = 64, 12, 64, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    z = lambda *s, d=dt: torch.zeros(s, device="cuda", dtype=d)  # noqa: E731
    step = (0.5 + 0.25 * torch.rand(1, L, H, device="cuda", generator=g)).to(dt)
    A = -torch.linspace(0.3, 1.2, H, device="cuda")
    c = torch.cumsum(step.double() * A.double(), 1)[0]                       # (L, H)
    assert float(c[-1].min()) < -40
    B, C, x, dout, S = z(1, L, 1, N), z(1, L, 1, N), z(1, L, H, P), z(1, L, H, P), z(1, H, N, P, d=A.dtype)
    B[..., 0] = C[..., 0] = 1
    S[:, :, 0] = 1 + torch.rand(1, H, P, device="cuda", generator=g)
    tol = 8 * U

    def same(got, want, what, tol=tol):
        assert torch.all((got.double() - want).abs() <= tol * want.abs()), what

    r = o.scan2_bwd(x, step, A, B, C, dout, dt_softplus=False, dh_last=S)
    same(r["dh0"][0, :, 0], S[0, :, 0].double() * torch.exp(c[-1])[:, None], "dh0")
    if io == "bf16":
        return
    same(r["dx"][0], step[0, :, :, None].double() * torch.exp(c[-1] - c)[:, :, None]
         * S[0, :, 0].double(), "dx from behind")
    dout[0, -1] = S[0, :, 0]
    r = o.scan2_bwd(x, step, A, B, C, dout, dt_softplus=False)
    same(r["dx"][0], step[0, :, :, None].double() * torch.exp(c[-1] - c)[:, :, None]
         * S[0, :, 0].double(), "dx from the last step")
    dout.zero_()
    dout[..., 0] = 1
    one = slice(0, 1)       # (dC is a sum over the heads: one of them)
    r = o.scan2_bwd(x[:, :, one].contiguous(), step[:, :, one].contiguous(), A[one], B, C,
                    dout[:, :, one].contiguous(), dt_softplus=False, h0=S[:, one].contiguous())
    same(r["dC"][0, :, 0, 0], torch.exp(c[:, 0]) * S[0, 0, 0, 0].double(), "dC")


def _sums(t):
    """In float64: dh0, and of dA and ddt_bias the values and the root of the sum of their terms'
    squares (a term per step)."""
    d = {k: v.double() for k, v in t.items()}
    x, A, B, C, dout, h0 = (d[k] for k in ("x", "A", "B", "C", "dout", "h0"))
    batch, L, H, P = x.shape
    raw = d["dt"] + d["dt_bias"]
    s = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    a = torch.exp(s * A)
    gy = dout * d["z"] * torch.sigmoid(d["z"]) if "z" in d else dout
    per = lambda v: v.repeat_interleave(H // B.shape[2], 1)  # noqa: E731
    S = torch.empty(L + 1, *h0.shape, device="cuda", dtype=torch.float64)
    S[0] = h0
    for k in range(L):
        S[k + 1] = a[:, k, :, None, None] * S[k] + \
            (s[:, k, :, None] * per(B[:, k]))[..., None] * x[:, k, :, None]
    lam, dl, xv = d["dh_last"], torch.empty_like(s), torch.empty_like(s)
    for k in range(L - 1, -1, -1):
        lam = lam + per(C[:, k])[..., None] * gy[:, k, :, None]
        xv[:, k] = ((per(B[:, k])[..., None] * lam).sum(2) * x[:, k]).sum(2)
        dl[:, k] = a[:, k] * (lam * S[k]).sum((2, 3))
        lam = a[:, k, :, None, None] * lam
    terms = dict(dA=s * dl, ddt_bias=(A * dl + xv) * torch.sigmoid(raw))
    return lam, {k: (v.sum((0, 1)), v.square().sum((0, 1)).sqrt()) for k, v in terms.items()}


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("io,shape", [("bf16", (16, 1000, 5, 64, 1, 128)),
                                      ("bf16", (16, 1000, 5, 64, 1, 64)),
                                      ("bf16", (8, 1000, 6, 64, 2, 128)),
                                      ("bf16", (2, 300, 8, 64, 1, 128)),
                                      ("bf16", (16, 1000, 6, 32, 1, 16)),
                                      ("f32", (16, 1000, 6, 32, 1, 130))], ids=str)
def test_many_heads_a_workgroup(io, shape, gate):
    """In all but the fourth shape (few walks, cut) the chunks number the card's CUs, so that one
    workgroup walks all heads of a group: 5, 5, 3, and at the end 6 in the kernel for any shape.  The
    last batch row's gradients against the bounds of float32 products; what is
    float32 by more: a term of it is a product of about ten factors, each off by one rounding or by the
    two U of a hardware function, and the terms' errors differ, so that dh0 is within 16 U of its
    norm and the sums over all tokens within 16 U of the root of their squares (with operands of
    bf16 pairs, 2^-18 each, they were 40 U off)."""
    o = ops()
    batch, L, H, P, G, N = shape
    g = torch.Generator(device="cuda").manual_seed(N + L + H)
    n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    b = lambda *s: n(*s).to(DTYPES[io])  # noqa: E731
    t = dict(x=b(batch, L, H, P), dt=(0.5 * n(batch, L, H)).to(DTYPES[io]),
             A=-1 - 7 * torch.rand(H, device="cuda", generator=g), B=b(batch, L, G, N),
             C=b(batch, L, G, N), dout=b(batch, L, H, P), D=n(H), dt_bias=0.3 * n(H) - 3,
             h0=n(batch, H, N, P), dh_last=n(batch, H, N, P))
    if gate:
        t["z"] = b(batch, L, H, P)
    got = o.scan2_bwd(**t)
    dh0, sums = _sums(t)
    assert float((got["dh0"] - dh0).norm() / dh0.norm()) <= 16 * U
    for k, (want, size) in sums.items():
        assert float((got[k] - want).norm() / size.norm()) <= 16 * U, k
    last = {k: (v[-1:] if v.dim() > 1 else v).double().cpu().numpy() for k, v in t.items()}
    want = ht.scan2_bwd(**last)
    for k in ("dx", "ddt", "dz", "dB", "dC"):
        if want[k] is not None:
            check(got[k][-1:], want[k], io, k)
    again = o.scan2_bwd(**t)
    for k, v in got.items():
        assert v is None or torch.equal(v, again[k]), k


def test_no_heads(monkeypatch):
    """Without heads nothing reaches B and C: their gradients are 0, not what the memory held."""
    o = ops()
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    like = torch.empty_like
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: like(t, **kw).fill_(7))
    g = o.scan2_bwd(z(2, 5, 0, 8), z(2, 5, 0), z(0), z(2, 5, 1, 8), z(2, 5, 1, 8), z(2, 5, 0, 8))
    assert torch.all(g["dB"] == 0) and torch.all(g["dC"] == 0)
    assert g["dB"].shape == (2, 5, 1, 8) and g["dx"].numel() == 0 and g["dA"].numel() == 0
