"""The operators of the multi-head block together, as a model uses them: a training step, a prompt and
the tokens after it, on streams of their own and from a captured graph."""
import numpy as np
import pytest

from oracle import head_twin as ht

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


class Block:
    """norm(residual + scale * dropout(x)) -> [z | x B C | dt] -> convolution -> scan -> gated norm
    -> projection, with the gradients of everything for an upstream gradient of the output and of
    the residual stream."""

    H, P, G, N, k, dm = 4, 16, 2, 8, 4, 24

    def __init__(self, seed, batch=2, L=150, p=0.25, dtype=torch.float32, heads=None):
        if heads:
            self.H, self.P, self.N = heads
        r = np.random.default_rng(seed)
        n = lambda *s: torch.from_numpy(r.standard_normal(s))  # noqa: E731
        self.batch, self.L, self.p, self.dtype = batch, L, p, dtype
        d, bc = self.H * self.P, self.G * self.N
        self.d, self.bc, width = d, bc, 2 * d + 2 * bc + self.H
        self.leaves = dict(
            x=n(batch, L, self.dm), residual=n(batch, L, self.dm), scale=0.5 + 0.1 * n(self.dm),
            weight=1 + 0.1 * n(self.dm), w_in=n(self.dm, width) * self.dm ** -0.5,
            conv_w=0.5 * n(d + 2 * bc, self.k), conv_b=0.1 * n(d + 2 * bc),
            A=-(0.5 + n(self.H).abs()), D=n(self.H), dt_bias=n(self.H) * 0.3 - 2,
            gated_w=1 + 0.1 * n(d), w_out=n(d, self.dm) * d ** -0.5)
        self.up = dict(out=n(batch, L, self.dm), s=n(batch, L, self.dm))
        self.seed = (seed + 1, 77)
        io = ("x", "w_in", "w_out")
        self.t = {k: v.to(dtype if k in io else torch.float32).cuda()
                  for k, v in self.leaves.items()}
        self.dout = self.up["out"].to(dtype).cuda()
        self.ds = self.up["s"].float().cuda()
        self.rng = torch.tensor(self.seed, dtype=torch.int64, device="cuda")

    def step(self):
        """One training step: (out, gradients of every leaf)."""
        o, t = ops(), self.t
        batch, L, d, bc, H, P, G, N = (self.batch, self.L, self.d, self.bc, self.H, self.P, self.G,
                                       self.N)
        drop = dict(scale=t["scale"], p=self.p, rng=self.rng)
        nrm, s, rstd, _ = o.rms_norm_fwd(t["x"], t["weight"], residual=t["residual"],
                                         return_stats=True, **drop)
        proj = nrm.view(-1, self.dm) @ t["w_in"]
        z, xbc, dt = proj.split([d, d + 2 * bc, H], 1)
        xbc = xbc.reshape(batch, L, -1).contiguous()
        act = o.causal_conv_fwd(xbc, t["conv_w"], t["conv_b"])
        xs, B, C = act.split([d, bc, bc], 2)
        scan = dict(x=xs.reshape(batch, L, H, P).contiguous(),
                    dt=dt.reshape(batch, L, H).contiguous(), A=t["A"],
                    B=B.reshape(batch, L, G, N).contiguous(),
                    C=C.reshape(batch, L, G, N).contiguous(), D=t["D"], dt_bias=t["dt_bias"])
        y = o.scan2_fwd(**scan).view(batch * L, d)
        gn, grstd = o.gated_norm_fwd(y, z, t["gated_w"], groups=G, return_stats=True)
        out = (gn @ t["w_out"]).view(batch, L, self.dm)

        do = self.dout.view(-1, self.dm)
        g = dict(w_out=gn.t().contiguous() @ do)
        q = o.gated_norm_bwd(do @ t["w_out"].t().contiguous(), y, z, t["gated_w"], grstd, groups=G)
        g["gated_w"] = q["dweight"]
        b = o.scan2_bwd(dout=q["dx"].view(batch, L, H, P), want_dh0=False, **scan)
        g.update(A=b["dA"], D=b["dD"], dt_bias=b["ddt_bias"])
        dact = torch.cat([b["dx"].view(batch, L, d), b["dB"].view(batch, L, bc),
                          b["dC"].view(batch, L, bc)], 2)
        c = o.causal_conv_bwd(xbc, t["conv_w"], dact, t["conv_b"])
        g.update(conv_w=c["dweight"], conv_b=c["dbias"])
        dproj = torch.cat([q["dz"], c["dx"].view(batch * L, -1), b["ddt"].view(-1, H)], 1)
        g["w_in"] = nrm.view(-1, self.dm).t().contiguous() @ dproj
        m = o.rms_norm_bwd((dproj @ t["w_in"].t().contiguous()).view(batch, L, self.dm), s,
                           t["weight"], rstd, x=t["x"], dsum=self.ds, want_dresidual=True, **drop)
        g.update(x=m["dx"], residual=m["dresidual"], weight=m["dweight"], scale=m["dscale"])
        return out, g

    def exact(self):
        """The same in float64 by autograd, on the CPU."""
        v = {k: t.double().cpu().requires_grad_(True) for k, t in self.t.items()}
        batch, L, d, bc, H, P, G, N = (self.batch, self.L, self.d, self.bc, self.H, self.P, self.G,
                                       self.N)
        silu = lambda a: a * torch.sigmoid(a)  # noqa: E731
        up = 65536 / (65536 - ht.drop_cut(self.p))
        keep = torch.from_numpy(ht.keep_mask(self.seed, batch * L, self.dm, self.p))
        s = v["residual"] + v["scale"] * v["x"] * keep.view(batch, L, -1) * up
        nrm = s / (s.square().mean(-1, keepdim=True) + 1e-5).sqrt() * v["weight"]
        z, xbc, dt = (nrm @ v["w_in"]).split([d, d + 2 * bc, H], 2)
        pad = torch.cat([xbc.new_zeros(batch, self.k - 1, d + 2 * bc), xbc], 1)
        act = silu(v["conv_b"] + sum(v["conv_w"][:, j] * pad[:, j:j + L] for j in range(self.k)))
        xs, B, C = act.split([d, bc, bc], 2)
        xs = xs.view(batch, L, H, P)
        per = lambda a: a.view(batch, L, G, N).repeat_interleave(H // G, 2)  # noqa: E731
        B, C = per(B), per(C)
        step = torch.nn.functional.softplus(dt + v["dt_bias"])
        S, ys = xs.new_zeros(batch, H, N, P), []
        for i in range(L):
            S = torch.exp(step[:, i] * v["A"])[..., None, None] * S + \
                (step[:, i, :, None] * B[:, i])[..., None] * xs[:, i, :, None]
            ys.append((C[:, i][..., None] * S).sum(2) + v["D"][:, None] * xs[:, i])
        u = (torch.stack(ys, 1).view(batch, L, d) * silu(z)).view(batch, L, G, -1)
        gn = (u / (u.square().mean(-1, keepdim=True) + 1e-5).sqrt()).view(batch, L, d) \
            * v["gated_w"]
        out = gn @ v["w_out"]
        ((out * self.dout.double().cpu()).sum() + (s * self.ds.double().cpu()).sum()).backward()
        return out.detach(), {k: a.grad for k, a in v.items()}


def off(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


def test_training_step():
    """Against float64 autograd.  A gradient has passed at most seven of the operators and four
    matrix products, each off by at most some 300 float32 roundings of its terms: 1e-4 of its norm
    is more than ten such operators make."""
    b = Block(1)
    out, g = b.step()
    want, grads = b.exact()
    assert off(out, want) < 1e-4
    for k in b.leaves:
        assert off(g[k], grads[k]) < 1e-4, (k, off(g[k], grads[k]))


def test_training_step_bf16():
    """bfloat16 rounds every activation on the way to half a step, 2^-8, and the matrix products' own
    outputs likewise: some ten roundings in a row, of independent signs, stay below ten half steps."""
    b = Block(2, heads=(4, 64, 64), dtype=torch.bfloat16)
    out, g = b.step()
    want, grads = b.exact()
    assert off(out, want) < 10 * 2 ** -8
    for k in b.leaves:
        assert off(g[k], grads[k]) < 10 * 2 ** -8, (k, off(g[k], grads[k]))


def test_two_steps_agree_bit_for_bit_and_draw_anew():
    b = Block(3)
    _, g1 = b.step()
    _, g2 = b.step()
    for k in g1:
        assert torch.equal(g1[k], g2[k]), k
    b.rng[1] += 1
    _, g3 = b.step()
    assert not torch.equal(g1["x"], g3["x"])


@pytest.mark.parametrize("dtype,heads", [(torch.float32, (4, 16, 8)),
                                         (torch.bfloat16, (4, 64, 128))])
def test_captured_step(dtype, heads):
    """A graph of the whole step, whose last node advances the dropout's offset: every replay equals
    the eager step at that offset, with eager steps and synchronizations between the replays."""
    b, e = (Block(4, dtype=dtype, heads=heads) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, g = b.step()
        b.rng[1:].add_(1)
    for k in range(4):
        graph.replay()
        eager, ge = e.step()
        e.rng[1:].add_(1)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), k
        for name in g:
            assert torch.equal(g[name], ge[name]), (k, name)


def test_two_streams_at_once():
    blocks = [Block(5, dtype=torch.bfloat16, heads=(4, 64, 128), L=700) for _ in range(2)]
    want = blocks[0].step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(blocks[i].step())
    torch.cuda.synchronize()
    for runs in got:
        for out, g in runs:
            assert torch.equal(out, want[0])
            for k in g:
                assert torch.equal(g[k], want[1][k]), k


def test_stream_argument():
    """stream= is as if the call stood under that stream."""
    o, s = ops(), torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *n: torch.randn(*n, device="cuda", generator=g)  # noqa: E731
    x, z, w = r(500, 640), r(500, 640), r(640)
    rng = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    B, C, dt, A = r(2, 40, 1, 16), r(2, 40, 1, 16), r(2, 40, 4), -r(4).abs()
    xs, state = r(2, 40, 4, 8), r(2, 4, 16, 8)
    calls = [lambda **k: o.dropout(x, 0.3, rng, **k),
             lambda **k: o.rms_norm_fwd(x, w, residual=z, scale=w, p=0.3, rng=rng, **k)[1],
             lambda **k: o.gated_norm_fwd(x, z, w, groups=5, **k),
             lambda **k: o.gated_norm_bwd(x, x, z, w, r(500, 5).abs() * 0 + 1, groups=5,
                                          **k)["dweight"],
             lambda **k: o.rms_norm_bwd(x, x, w, x[:, 0].abs().contiguous(), **k)["dx"],
             lambda **k: o.scan2_bwd(xs, dt, A, B, C, xs, **k)["dB"],
             lambda **k: o.scan2_state_update(state.clone(), xs[:, 0].contiguous(),
                                              dt[:, 0].contiguous(), A, B[:, 0].contiguous(),
                                              C[:, 0].contiguous(), **k)]
    want = [f() for f in calls]
    s.wait_stream(torch.cuda.current_stream())
    got = [f(stream=s) for f in calls]
    s.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_then_tokens(dtype):
    """The convolution and the scan over a prompt, then token by token through
    scan2_state_update_conv, against the whole sequence at once.  float32: the orders of a few
    hundred additions differ.  bfloat16: the convolution's output is rounded on the way to the scan
    in the prompt and not for a token, half a step of each of x, B and C."""
    o = ops()
    gen = torch.Generator(device="cuda").manual_seed(7)
    batch, L, cut, H, P, G, N, k = 3, 80, 66, 4, 64, 2, 64, 4
    d, bc = H * P, G * N
    width = d + 2 * bc
    r = lambda *n: torch.randn(*n, device="cuda", generator=gen)  # noqa: E731
    proj = r(batch, L, d + width + H).to(dtype)
    z, xbc, dt = proj.split([d, width, H], 2)
    w, cb, A, D, bias = 0.5 * r(width, k), 0.1 * r(width), -r(H).abs() - 0.5, r(H), r(H) - 3
    kw = dict(D=D, dt_bias=bias)

    def prompt(n):
        act = o.causal_conv_fwd(xbc[:, :n].contiguous(), w, cb)
        x, B, C = act.split([d, bc, bc], 2)
        return o.scan2_fwd(x.reshape(batch, n, H, P).contiguous(), dt[:, :n].contiguous(), A,
                           B.reshape(batch, n, G, N).contiguous(),
                           C.reshape(batch, n, G, N).contiguous(),
                           z=z[:, :n].reshape(batch, n, H, P).contiguous(),
                           return_last_state=True, **kw)

    whole, last = prompt(L)
    _, state = prompt(cut)
    window = xbc[:, cut - k + 1:cut].contiguous()
    tol = 1e-5 if dtype is torch.float32 else 3 * 2 ** -8
    for t in range(cut, L):
        out = o.scan2_state_update_conv(state, window, xbc[:, t], w, cb, dt[:, t], A, ngroups=G,
                                        z=z[:, t], **kw)
        assert float((out - whole[:, t]).norm() / whole[:, t].norm()) < tol
    assert float((state - last).norm() / last.norm()) < tol
    assert torch.equal(window, xbc[:, L - k + 1:])


def test_captured_tokens():
    """A captured token step advances state and window on every replay as eager calls do."""
    o = ops()
    gen = torch.Generator(device="cuda").manual_seed(8)
    H, P, N, k = 8, 64, 128, 4
    width = H * P + 2 * N
    r = lambda *n: torch.randn(*n, device="cuda", generator=gen)  # noqa: E731
    xbc, dt, w, A = r(2, width).bfloat16(), r(2, H).bfloat16(), r(width, k), -r(H).abs()
    states = [r(2, H, N, P)]
    windows = [r(2, k - 1, width).bfloat16()]
    states.append(states[0].clone())
    windows.append(windows[0].clone())
    call = lambda i: o.scan2_state_update_conv(states[i], windows[i], xbc, w, None, dt, A)  # noqa: E731
    s0, w0 = states[0].clone(), windows[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(0)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(0)
    states[0].copy_(s0)
    windows[0].copy_(w0)
    for n in range(4):
        xbc.copy_(r(2, width))
        graph.replay()
        want = call(1)
        torch.cuda.synchronize()
        assert torch.equal(out, want), n
        assert torch.equal(states[0], states[1]) and torch.equal(windows[0], windows[1])
