"""The recurrent block's operators together, as a model uses them: a block norm -> projection ->
convolution -> gate projections -> recurrence -> projection on a residual stream, trained, prefilled
and run token by token; on streams of their own, in captured graphs, and next to the selective
scan.  The projections are plain float32 matrix products."""
import numpy as np
import pytest

from tests.block_helpers import draw_starts, starts_gpu

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


D, W = 24, 40       # model width, width inside the block


def weights(seed, double=False):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    w = dict(nw=1 + 0.1 * n(D), nb=0.1 * n(D), w_in=n(D, W) / D ** 0.5, w_z=n(D, W) / D ** 0.5,
             cw=0.5 * n(W, 4), cb=0.1 * n(W), w_r=n(W, W) / W ** 0.5, w_i=n(W, W) / W ** 0.5,
             A=8 * np.log(rng.uniform(0.9, 0.999, W)), rb=n(W), ib=n(W),
             w_out=n(W, D) / W ** 0.5)
    return {k: torch.from_numpy(v.astype(np.float32)).cuda() if not double else
            torch.from_numpy(v.astype(np.float32)).double() for k, v in w.items()}


def block(o, w, x, stream, starts=None, conv_prev=None, h0=None):
    """(y, new residual stream, what the backward and the next tokens need)"""
    n, s, mean, rstd = o.layer_norm_fwd(x, w["nw"], w["nb"], residual=stream, return_stats=True)
    u, z = n @ w["w_in"], n @ w["w_z"]
    c = o.causal_conv_fwd(u, w["cw"], w["cb"], x_prev=conv_prev, starts=starts, silu=False)
    r, i = c @ w["w_r"], c @ w["w_i"]
    h, states, last = o.gated_scan_fwd_states(c, r, i, w["A"], w["rb"], w["ib"], z=z,
                                              starts=starts, h0=h0, return_last_state=True)
    return h @ w["w_out"], s, dict(n=n, s=s, mean=mean, rstd=rstd, u=u, z=z, c=c, r=r, i=i, h=h,
                                   states=states, last=last, starts=starts)


def block_bwd(o, w, k, dy, ds):
    """Gradients of block for dy of y and ds of the new residual stream."""
    flat = lambda a, b: a.reshape(-1, a.shape[-1]).t() @ b.reshape(-1, b.shape[-1])  # noqa: E731
    g = dict(w_out=flat(k["h"], dy))
    b = o.gated_scan_bwd(k["c"], k["r"], k["i"], w["A"], (dy @ w["w_out"].t()).contiguous(),
                         w["rb"], w["ib"], z=k["z"], starts=k["starts"], states=k["states"])
    g.update(A=b["dA"], rb=b["dr_bias"], ib=b["di_bias"], w_r=flat(k["c"], b["dr"]),
             w_i=flat(k["c"], b["di"]))
    dc = b["dx"] + b["dr"] @ w["w_r"].t() + b["di"] @ w["w_i"].t()
    v = o.causal_conv_bwd(k["u"], w["cw"], dc, w["cb"], starts=k["starts"], silu=False)
    g.update(cw=v["dweight"], cb=v["dbias"], w_in=flat(k["n"], v["dx"]),
             w_z=flat(k["n"], b["dz"]))
    dn = v["dx"] @ w["w_in"].t() + b["dz"] @ w["w_z"].t()
    m = o.layer_norm_bwd(dn, k["s"], w["nw"], k["mean"], k["rstd"], dsum=ds, want_dresidual=True)
    g.update(nw=m["dweight"], nb=m["dbias"])
    return m["dx"], m["dresidual"], g


def block64(w, x, stream, starts):
    """The same block in float64 by torch's own differentiable operations on the CPU."""
    s = x + stream
    n = (s - s.mean(-1, keepdim=True)) / (s.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    n = n * w["nw"] + w["nb"]
    u, z = n @ w["w_in"], n @ w["w_z"]
    B, L, _ = x.shape
    cs = []
    for b in range(B):
        window = []
        for t in range(L):
            if starts[b, t]:
                window = []
            window = (window + [u[b, t]])[-4:]
            cs.append(w["cb"] + sum(w["cw"][:, 3 - q] * window[-1 - q]
                                    for q in range(len(window))))
    c = torch.stack(cs).view(B, L, W)
    rg, ig = torch.sigmoid(c @ w["w_r"] + w["rb"]), torch.sigmoid(c @ w["w_i"] + w["ib"])
    a = torch.exp(w["A"] * rg)
    inp = torch.sqrt(1 - a * a) * ig * c
    hs = []
    for b in range(B):
        h = torch.zeros(W, dtype=torch.float64)
        for t in range(L):
            h = inp[b, t] if starts[b, t] else a[b, t] * h + inp[b, t]
            hs.append(h)
    h = torch.stack(hs).view(B, L, W)
    return (h * torch.nn.functional.silu(z)) @ w["w_out"], s


def test_training_step_of_two_blocks():
    """Outputs and every gradient of two stacked blocks on packed sequences against float64
    autograd.  float32 throughout: about 2^-24 a step, some 150 dependent roundings and sums of 80
    to 150 products, so 1e-4 of the largest value of each tensor is far above what they add up
    to and far below a dropped term."""
    o = ops()
    B, L = 2, 75
    rng = np.random.default_rng(0)
    starts = draw_starts(rng, B, L, 20)
    x0 = rng.standard_normal((B, L, D)).astype(np.float32)
    st0 = rng.standard_normal((B, L, D)).astype(np.float32)
    dy0, ds0 = (rng.standard_normal((B, L, D)).astype(np.float32) for _ in range(2))
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    w1, w2 = weights(1), weights(2)
    sg = starts_gpu(starts)
    y1, s1, k1 = block(o, w1, dev(x0), dev(st0), sg)
    y2, s2, k2 = block(o, w2, y1, s1, sg)
    dx2, dr2, g2 = block_bwd(o, w2, k2, dev(dy0), dev(ds0))
    dx1, dr1, g1 = block_bwd(o, w1, k1, dx2, dr2)

    leaf = lambda d: {k: v.requires_grad_() for k, v in d.items()}  # noqa: E731
    v1, v2 = leaf(weights(1, True)), leaf(weights(2, True))
    x = torch.from_numpy(x0).double().requires_grad_()
    st = torch.from_numpy(st0).double().requires_grad_()
    r1, t1 = block64(v1, x, st, starts)
    r2, t2 = block64(v2, r1, t1, starts)
    ((r2 * torch.from_numpy(dy0)).sum() + (t2 * torch.from_numpy(ds0)).sum()).backward()

    def same(got, want, what):
        err = (got.double().cpu() - want).abs().max() / want.abs().max()
        assert err < 1e-4, (what, float(err))

    same(y2, r2.detach(), "out")
    same(s2, t2.detach(), "stream")
    same(dx1, x.grad, "dx")
    same(dr1, st.grad, "dstream")
    for which, g, v in (("block 1", g1, v1), ("block 2", g2, v2)):
        assert set(g) == set(v)
        for name in v:
            same(g[name].view(v[name].shape), v[name].grad, f"{which} d{name}")


def test_prefill_then_tokens():
    o = ops()
    w = weights(3)
    x = torch.randn(2, 90, D, device="cuda")
    stream = torch.randn(2, 90, D, device="cuda")
    y, s, _ = block(o, w, x, stream)
    cut = 70
    c = lambda t, sl: t[:, sl].contiguous()  # noqa: E731
    y0, s0, k = block(o, w, c(x, slice(0, cut)), c(stream, slice(0, cut)))
    window, state = k["u"][:, cut - 3:].contiguous(), k["last"]
    ys = [y0]
    for t in range(cut, 90):
        n, st = o.layer_norm_fwd(x[:, t].contiguous(), w["nw"], w["nb"],
                                 residual=stream[:, t].contiguous())
        u, z = n @ w["w_in"], n @ w["w_z"]
        v = o.causal_conv_update(window, u, w["cw"], w["cb"], silu=False)
        h = o.gated_state_update(state, v, v @ w["w_r"], v @ w["w_i"], w["A"], w["rb"], w["ib"],
                                 z=z)
        ys.append((h @ w["w_out"])[:, None])
        assert torch.equal(st, s[:, t])
    torch.testing.assert_close(torch.cat(ys, 1), y, rtol=1e-4, atol=1e-4)


def test_on_another_stream():
    """stream= runs everything there, after what that stream was made to wait for."""
    o = ops()
    side = torch.cuda.Stream()
    x, r, i = (torch.randn(2, 300, 70, device="cuda") for _ in range(3))
    A = -torch.rand(70, device="cuda")
    want, states = o.gated_scan_fwd_states(x, r, i, A)
    gw = o.gated_scan_bwd(x, r, i, A, x, states=states)
    w = torch.randn(70, 4, device="cuda")
    cw, nw = o.causal_conv_fwd(x, w), o.layer_norm_fwd(x)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got, st = o.gated_scan_fwd_states(x, r, i, A, stream=side)
        gb = o.gated_scan_bwd(x, r, i, A, x, states=st, stream=side)
        cb, nb = o.causal_conv_fwd(x, w, stream=side), o.layer_norm_fwd(x, stream=side)
        tok = o.gated_state_update(st[:, 0].contiguous(), x[:, 0].contiguous(),
                                   r[:, 0].contiguous(), i[:, 0].contiguous(), A)
        side.synchronize()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want) and torch.equal(cb, cw) and torch.equal(nb, nw)
        assert tok.shape == (2, 70)
        for k in gw:
            if gw[k] is not None:
                assert torch.equal(gb[k], gw[k]), k


def test_two_streams_at_once():
    """Two recurrences with workspaces of their own at the same time on two streams."""
    o = ops()
    streams = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for seed in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x, r, i = (torch.randn(2, 6000, 320, device="cuda", generator=g).bfloat16()
                   for _ in range(3))
        A = -torch.rand(320, device="cuda", generator=g)
        cases.append((x, r, i, A, o.gated_scan_fwd(x, r, i, A), o.gated_scan_bwd(x, r, i, A, x)))
    torch.cuda.synchronize()
    for _ in range(4):
        res = [(o.gated_scan_fwd(*c[:4], stream=s), o.gated_scan_bwd(*c[:4], c[0], stream=s))
               for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for (out, g), c in zip(res, cases):
            assert torch.equal(out, c[4])
            for k in ("dx", "dr", "di", "dA"):
                assert torch.equal(g[k], c[5][k])


def test_captured_graph_replays():
    """A training step of all three operators and their one-token forms captured once and replayed
    on new inputs, with eager work between the replays, against the eager results.  Two graphs
    share one workspace."""
    o = ops()
    B, L, d = 2, 400, 96
    x, r, i, z, dout = (torch.randn(B, L, d, device="cuda").bfloat16() for _ in range(5))
    A, nw = -torch.rand(d, device="cuda"), torch.randn(d, device="cuda")
    cw = torch.randn(d, 4, device="cuda")
    starts = torch.rand(B, L, device="cuda") < 0.02
    ws = torch.empty(max(o.lib().ss_gated_scan_fwd_workspace_bytes(B, L, d, o.SS_BF16),
                         o.lib().ss_gated_scan_bwd_workspace_bytes(B, L, d, o.SS_BF16, 1)),
                     dtype=torch.uint8, device="cuda")
    state, window = torch.randn(B, d, device="cuda"), torch.zeros(B, 3, d, device="cuda").bfloat16()

    def step(workspace):
        n, mean, rstd = o.layer_norm_fwd(x, nw, return_stats=True)
        c = o.causal_conv_fwd(n, cw, starts=starts)
        out, states = o.gated_scan_fwd_states(c, r, i, A, z=z, starts=starts, workspace=workspace)
        g = o.gated_scan_bwd(c, r, i, A, dout, z=z, starts=starts, states=states,
                             workspace=workspace)
        v = o.causal_conv_bwd(n, cw, g["dx"], starts=starts)
        m = o.layer_norm_bwd(v["dx"], x, nw, mean, rstd)
        tok = o.causal_conv_update(window, x[:, 0].contiguous(), cw)
        tok = o.gated_state_update(state, tok, r[:, 0].contiguous(), i[:, 0].contiguous(), A)
        return (out, g["dr"], g["di"], g["dz"], g["dA"], v["dweight"], v["dbias"], m["dx"],
                m["dweight"], m["dbias"], tok)

    def fresh(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, r, i, z, dout):
            t.copy_(torch.randn(t.shape, device="cuda", generator=gen))
        state.copy_(torch.randn(state.shape, device="cuda", generator=gen))
        window.zero_()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step(ws)
        graphs.append((g, res))
    for seed in range(3):
        for g, res in graphs:
            fresh(seed)
            want = [t.clone() for t in step(None)]
            fresh(seed)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for k, (p, q) in enumerate(zip(res, want)):
                assert torch.equal(p, q), (seed, k)


def test_next_to_the_selective_scan():
    """One workspace tensor, used in turn by the selective scan's time split and by the gated
    recurrence on one stream: neither needs what the other left."""
    from selective_state_space_36_amd import workloads as wl
    from tests.helpers import dev
    o = ops()
    p = {k: dev(v) for k, v in wl.make_prefill(wl.WORKLOADS[0], batch=1, seqlen=3000, d_inner=32,
                                               seed=1).items()}
    args = (p["u"], p["delta"], p["A"], p["B"], p["C"])
    x = torch.randn(1, 3000, 32, device="cuda")
    A = -torch.rand(32, device="cuda")
    n = max(o.workspace_bytes(1, 3000, 32, 16, torch.float32),
            o.lib().ss_gated_scan_fwd_workspace_bytes(1, 3000, 32, o.SS_F32))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    want = o.scan_fwd(*args, delta_bias=p["delta_bias"]), o.gated_scan_fwd(x, x, x, A)
    for _ in range(3):
        assert torch.equal(o.scan_fwd(*args, delta_bias=p["delta_bias"], workspace=ws), want[0])
        assert torch.equal(o.gated_scan_fwd(x, x, x, A, workspace=ws), want[1])


def test_refusals_of_the_binding():
    o = ops()
    x, A = torch.randn(1, 6, 8, device="cuda"), -torch.rand(8, device="cuda")
    good = (x, x, x, A)
    w = torch.randn(8, 4, device="cuda")
    cases = [
        (TypeError, lambda: o.gated_scan_fwd(x.half(), x.half(), x.half(), A)),
        (TypeError, lambda: o.gated_scan_fwd(x, x.bfloat16(), x, A)),
        (TypeError, lambda: o.gated_scan_fwd(x, x, x, A.double())),
        (ValueError, lambda: o.gated_scan_fwd(x, x[:, :5], x, A)),
        (ValueError, lambda: o.gated_scan_fwd(x.transpose(1, 2), x, x, A)),
        (ValueError, lambda: o.gated_scan_fwd(x[0], x[0], x[0], A)),
        (ValueError, lambda: o.gated_scan_fwd(*good, h0=A)),
        (ValueError, lambda: o.gated_scan_fwd(x, x.cpu(), x, A)),
        (TypeError, lambda: o.gated_scan_fwd(*good, starts=torch.zeros(1, 6, device="cuda"))),
        (ValueError, lambda: o.gated_scan_fwd(*good, starts=torch.zeros(
            6, 1, dtype=torch.bool, device="cuda"))),
        (o.SSError, lambda: o.gated_scan_fwd(*good, out=x)),
        (ValueError, lambda: o.gated_scan_bwd(*good, x, states=torch.zeros(1, 2, 8,
                                                                            device="cuda"))),
        (TypeError, lambda: o.gated_state_update(x[0].bfloat16(), x[0], x[0], x[0], A)),
        (TypeError, lambda: o.layer_norm_fwd(x, residual=x.bfloat16())),
        (ValueError, lambda: o.layer_norm_fwd(x, A[:4])),
        (o.SSError, lambda: o.layer_norm_fwd(x, eps=-1.0)),
        (o.SSError, lambda: o.layer_norm_bwd(x, x, None, x[..., 0].contiguous(),
                                             x[..., 0].contiguous(), want_dx=False)),
        (ValueError, lambda: o.layer_norm_bwd(x, x, None, A, A)),
        (ValueError, lambda: o.causal_conv_fwd(x, w[:4])),
        (ValueError, lambda: o.causal_conv_fwd(x, w, x_prev=x)),
        (TypeError, lambda: o.causal_conv_fwd(x, w.bfloat16())),
        (ValueError, lambda: o.causal_conv_update(x, x[0], w)),
    ]
    for k, (kind, f) in enumerate(cases):
        with pytest.raises(kind):
            f()
            print("not refused:", k)


def random_bf16(shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)


@pytest.fixture
def large():
    """The test's arrays go back to the device, not to the allocator's cache."""
    yield
    torch.cuda.empty_cache()


def test_recurrence_past_32_bit_offsets(large):
    """2.2e9 elements (4.5 GB) an array.  The last steps behind a start at a tile's edge equal a
    call on them alone, where every tile holds the same steps (gradients from the next tile on: the
    tile with the start takes another path, whose compiler may round a sum elsewhere)."""
    o = ops()
    B, L, d, cut = 2, 270100, 4160, 270080 - 20 * 128
    assert B * L * d > 1 << 31 and cut % 128 == 0
    x, r, i, z, dout = (random_bf16((B, L, d), s) for s in range(5))
    A = -torch.rand(d, device="cuda")
    starts = torch.zeros(B, L, dtype=torch.bool, device="cuda")
    starts[:, cut] = True
    out, states, last = o.gated_scan_fwd_states(x, r, i, A, z=z, starts=starts,
                                                return_last_state=True)
    g = o.gated_scan_bwd(x, r, i, A, dout, z=z, starts=starts, states=states)
    tail = lambda t: t[:, cut:].contiguous()  # noqa: E731
    p, s, h = o.gated_scan_fwd_states(tail(x), tail(r), tail(i), A, z=tail(z),
                                      return_last_state=True)
    q = o.gated_scan_bwd(tail(x), tail(r), tail(i), A, tail(dout), z=tail(z), states=s)
    assert torch.equal(out[:, cut:], p) and torch.equal(last, h)
    assert torch.equal(states[:, cut // 64:], s)
    for name in ("dx", "dr", "di", "dz"):
        assert torch.equal(g[name][:, cut + 64:], q[name][:, 64:]), name


def test_convolution_past_32_bit_offsets(large):
    o = ops()
    B, L, d, cut = 2, 270100, 4160, 270080 - 20 * 64
    x, dout = random_bf16((B, L, d), 1), random_bf16((B, L, d), 2)
    w = torch.randn(d, 4, device="cuda")
    out, g = o.causal_conv_fwd(x, w), o.causal_conv_bwd(x, w, dout)
    tail, prev = x[:, cut:].contiguous(), x[:, cut - 3:cut].contiguous()
    assert torch.equal(out[:, cut:], o.causal_conv_fwd(tail, w, x_prev=prev))
    q = o.causal_conv_bwd(tail, w, dout[:, cut:].contiguous(), x_prev=prev)
    assert torch.equal(g["dx"][:, cut:], q["dx"])


def test_norm_past_32_bit_offsets(large):
    o = ops()
    rows, dim, cut = 900001, 2560, 899900
    assert rows * dim > 1 << 31
    x, dout = random_bf16((rows, dim), 1), random_bf16((rows, dim), 2)
    res = torch.randn(rows, dim, device="cuda")
    out, s, mean, rstd = o.layer_norm_fwd(x, residual=res, return_stats=True)
    g = o.layer_norm_bwd(dout, s, None, mean, rstd, dsum=res, want_dresidual=True)
    p, t, m, v = o.layer_norm_fwd(x[cut:], residual=res[cut:], return_stats=True)
    q = o.layer_norm_bwd(dout[cut:], t, None, m, v, dsum=res[cut:], want_dresidual=True)
    for whole, alone in ((out, p), (s, t), (mean, m), (rstd, v), (g["dx"], q["dx"]),
                         (g["dresidual"], q["dresidual"])):
        assert torch.equal(whole[cut:], alone)


@pytest.mark.parametrize("d", [1 << 24, (1 << 24) - 27])
def test_the_widest_rows(d, large):
    """Channels do not meet in the recurrence and the convolution: the last ones of the widest rows
    equal a call on them alone.  The norm of such a row is compared with float64."""
    o = ops()
    L, lo = 35, (1 << 24) - 300
    x, r, i = (torch.randn(1, L, d, device="cuda") for _ in range(3))
    A, w = -torch.rand(d, device="cuda"), torch.randn(d, 4, device="cuda")
    c = lambda t: t[..., lo:].contiguous()  # noqa: E731
    last = (c(x), c(r), c(i), A[lo:].clone())
    assert torch.equal(c(o.gated_scan_fwd(x, r, i, A)), o.gated_scan_fwd(*last))
    g, q = o.gated_scan_bwd(x, r, i, A, x), o.gated_scan_bwd(*last, last[0])
    for name in ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dh0"):
        assert torch.equal(c(g[name]), q[name]), name
    del g
    h, hl = r[:, 0].clone(), c(r[:, 0])
    y = o.gated_state_update(h, x[:, 1].clone(), r[:, 1].clone(), i[:, 1].clone(), A)
    z = o.gated_state_update(hl, *(t[:, 1].contiguous() for t in last[:3]), last[3])
    assert torch.equal(c(y), z) and torch.equal(c(h), hl)
    # (whole numbers: sums over the steps are exact however many a wave takes)
    x, r, w = ((3 * t).clamp(-9, 9).round() for t in (x, r, w))
    last, wl = (c(x), c(r)), w[lo:].clone()
    assert torch.equal(c(o.causal_conv_fwd(x, w)), o.causal_conv_fwd(last[0], wl))
    g = o.causal_conv_bwd(x, w, r, silu=False)
    q = o.causal_conv_bwd(last[0], wl, last[1], silu=False)
    assert torch.equal(c(g["dx"]), q["dx"]) and torch.equal(g["dweight"][lo:], q["dweight"])
    assert torch.equal(g["dbias"][lo:], q["dbias"])
    del g
    win, wn = x[:, :3].clone(), last[0][:, :3].clone()
    y = o.causal_conv_update(win, x[:, 3].clone(), w)
    z = o.causal_conv_update(wn, last[0][:, 3].clone(), wl)
    assert torch.equal(c(y), z) and torch.equal(c(win), wn)
    # Small whole numbers and a power of two for rstd: sums below 2^24 are exact, so that 1 / d and
    # six more roundings of terms of at most 6 remain.
    dy, s = (torch.randint(-1, 2, (2, d), device="cuda").float() for _ in range(2))
    zero, one = torch.zeros(2, device="cuda"), torch.ones(2, device="cuda")
    g = o.layer_norm_bwd(dy, s, None, zero, one)
    xh, gy = s.double(), dy.double()
    ds = gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True)
    assert ((g["dx"].double() - ds).abs() <= 7 * 2.0 ** -24 * 3).all()
    assert torch.equal(g["dweight"].double(), (gy * xh).sum(0))
    assert torch.equal(g["dbias"].double(), gy.sum(0))
    out, mean, rstd = o.layer_norm_fwd(s, return_stats=True)
    mu = xh.mean(1)
    # at most 2^14 products a thread, each added with a rounding, then the thread sums
    assert ((mean.double() - mu).abs() <= 2.0 ** -24 * 2 * mu.abs()).all()
    v = 1 / (((xh - mu[:, None]) ** 2).mean(1) + 1e-5).sqrt()
    assert ((rstd.double() - v).abs() <= 2.0 ** -24 * (2 ** 14 + 50) * v).all()
    assert ((out.double() - (xh - mu[:, None]) * v[:, None]).abs()
            <= 2.0 ** -24 * (2 ** 14 + 60) * 2 * v.max()).all()


@pytest.mark.parametrize("L", [1, 3, 40, 700])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), torch.finfo(torch.float32).min])
def test_a_start_at_the_first_step_cuts_off_what_was_before(L, bad):
    """Whatever h0 and x_prev hold then, results, sums over tokens among them, are those of a call
    without them, and their gradients are 0."""
    o = ops()
    x, r, i, dout = (torch.randn(2, L, 70, device="cuda") for _ in range(4))
    A, w = -torch.rand(70, device="cuda"), torch.randn(70, 4, device="cuda")
    starts = torch.rand(2, L, device="cuda") < 0.05
    starts[:, 0] = True
    h0, xp = torch.full((2, 70), bad, device="cuda"), torch.full((2, 3, 70), bad, device="cuda")
    want = o.gated_scan_fwd_states(x, r, i, A, starts=starts, return_last_state=True)
    got = o.gated_scan_fwd_states(x, r, i, A, starts=starts, h0=h0, return_last_state=True)
    for p, q in zip(got, want):
        assert torch.equal(p, q) and torch.isfinite(p).all()
    g = o.gated_scan_bwd(x, r, i, A, dout, starts=starts, h0=h0)
    v = o.gated_scan_bwd(x, r, i, A, dout, starts=starts)
    for k in ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dh0"):
        assert torch.equal(g[k], v[k]) and torch.isfinite(g[k]).all(), k
    assert not g["dh0"].any()
    assert torch.equal(o.causal_conv_fwd(x, w, x_prev=xp, starts=starts),
                       o.causal_conv_fwd(x, w, starts=starts))
    g = o.causal_conv_bwd(x, w, dout, x_prev=xp, starts=starts)
    v = o.causal_conv_bwd(x, w, dout, starts=starts)
    for k in ("dx", "dweight", "dbias"):
        assert torch.equal(g[k], v[k]) and torch.isfinite(g[k]).all(), k
    assert not g["dx_prev"].any()
