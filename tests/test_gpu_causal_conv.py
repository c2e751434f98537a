"""The causal depthwise convolution on the GPU (forward, gradients, one token) against float64."""
import numpy as np
import pytest

from oracle import block_twin as bt
from oracle.rounding import Bounded
from tests.block_helpers import Guarded, check, draw_starts, gpu, starts_gpu

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


def run_case(seed, batch, L, d, k, io, silu=True, packed=False, prev=False, bias=True, offset=0):
    print(f"  case batch={batch} L={L} d={d} k={k} {io} silu={silu} packed={packed} prev={prev} "
          f"offset={offset}", flush=True)
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    x, vx = gpu(n(batch, L, d), io, offset)
    dout, vdout = gpu(n(batch, L, d), io, offset)
    w, vw = gpu(0.5 * n(d, k))
    b, vb = gpu(0.2 * n(d) if bias else None)
    xp, vxp = gpu(n(batch, k - 1, d) if prev else None, io, offset)
    st = draw_starts(rng, batch, L, 5) if packed else None
    s = starts_gpu(st)
    out = ops().causal_conv_fwd(x, w, b, x_prev=xp, starts=s, silu=silu)
    check(out, bt.conv_fwd(vx, vw, vb, vxp, st, silu)[0], io, "out")
    g = ops().causal_conv_bwd(x, w, dout, b, x_prev=xp, starts=s, silu=silu)
    ref = bt.conv_bwd(vx, vw, vdout, vb, vxp, st, silu)
    check(g["dx"], ref["dx"], io, "dx")
    check(g["dweight"], ref["dweight"], "f32", "dweight")
    check(g["dbias"], ref["dbias"], "f32", "dbias")
    if prev:
        check(g["dx_prev"], ref["dx_prev"], io, "dx_prev")
    else:
        assert g["dx_prev"] is None


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,d", [(1, 1, 1), (2, 2, 5), (1, 3, 64), (2, 4, 130), (1, 15, 66),
                                       (3, 17, 33), (2, 33, 256), (1, 64, 20), (2, 130, 68),
                                       (1, 300, 9)])
def test_forward_and_gradients(batch, L, d, io):
    run_case(L * 100 + d, batch, L, d, 4, io, packed=True, prev=True)


@pytest.mark.parametrize("k", [1, 2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("prev", [False, True])
def test_every_option(k, silu, packed, prev):
    run_case(k, 2, 70, 36, k, "bf16", silu, packed, prev, bias=prev)


@pytest.mark.parametrize("offset", [1, 2, 3, 4])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_misaligned(offset, io):
    run_case(offset, 2, 40, 64, 4, io, prev=True, offset=offset)


@pytest.mark.parametrize("prev", [False, True])
def test_matches_the_fused_front_end(prev):
    """The operator alone followed by the scan is the scan with the front end fused in: the fused
    one does not round the convolution's output, so float32 is compared."""
    from selective_state_space_36_amd import workloads as wl
    from tests.helpers import dev
    p = {k: dev(v) for k, v in wl.make_prefill(wl.WORKLOADS[0], batch=2, seqlen=90, d_inner=48,
                                               seed=2).items()}
    rng = np.random.default_rng(2)
    w, b = gpu(0.5 * rng.standard_normal((48, 4)))[0], gpu(rng.standard_normal(48))[0]
    xp = gpu(rng.standard_normal((2, 3, 48)))[0] if prev else None
    rest = (p["delta"], p["A"], p["B"], p["C"])
    fused = ops().scan_fwd_conv(p["u"], w, b, *rest, delta_bias=p["delta_bias"], x_prev=xp)
    u = ops().causal_conv_fwd(p["u"], w, b, x_prev=xp)
    apart = ops().scan_fwd(u, *rest, delta_bias=p["delta_bias"])
    torch.testing.assert_close(apart, fused, rtol=1e-4, atol=1e-4)


def test_nothing_crosses_a_start():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 40, 70))
    x[0, 9, :30], x[0, 8, 30:] = np.nan, np.inf
    starts = np.zeros((1, 40), dtype=bool)
    starts[0, 10] = True
    g, dout = gpu(x)[0], gpu(rng.standard_normal((1, 40, 70)))[0]
    w, s = gpu(rng.standard_normal((70, 4)))[0], starts_gpu(starts, torch.uint8)
    out = ops().causal_conv_fwd(g, w, starts=s)
    assert torch.equal(out[:, 10:], ops().causal_conv_fwd(g[:, 10:].contiguous(), w))
    dout[0, 10] = float("nan")
    clean = torch.randn_like(g)
    gr = ops().causal_conv_bwd(clean, w, dout, starts=s)
    assert torch.isfinite(gr["dx"][:, :10]).all()
    every = torch.ones((1, 40), dtype=torch.bool, device="cuda")
    lone = ops().causal_conv_fwd(clean, w, starts=every, silu=False)
    assert torch.equal(lone, clean * w[:, 3])


@pytest.mark.parametrize("batch,d", [(1, 1), (1, 5120), (3, 77), (128, 256), (5, 1027)])
@pytest.mark.parametrize("k", [1, 2, 3, 4])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_one_token(batch, d, k, io):
    rng = np.random.default_rng(d + k)
    x, vx = gpu(rng.standard_normal((batch, d)), io)
    w, vw = gpu(rng.standard_normal((d, k)))
    b, vb = gpu(rng.standard_normal(d))
    st, vst = gpu(rng.standard_normal((batch, k - 1, d)), io)
    out = ops().causal_conv_update(st, x, w, b, silu=k != 3)
    ref, new = bt.conv_step(vst, vx, vw, vb, k != 3)
    check(out, ref, io, "out")
    assert np.array_equal(st.double().cpu().numpy(), new)


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
def test_one_token_misaligned(offset):
    rng = np.random.default_rng(offset)
    x, vx = gpu(rng.standard_normal((3, 64)), "bf16", offset)
    st, vst = gpu(rng.standard_normal((3, 3, 64)), "bf16", offset)
    w, vw = gpu(rng.standard_normal((64, 4)), "f32", offset)
    out = ops().causal_conv_update(st, x, w)
    ref, new = bt.conv_step(vst, vx, vw)
    check(out, ref, "bf16", "out")
    assert np.array_equal(st.double().cpu().numpy(), new)


def test_prefill_then_tokens_repeat_the_whole_sequence():
    rng = np.random.default_rng(4)
    x = gpu(rng.standard_normal((2, 30, 40)), "bf16")[0]
    w, b = gpu(rng.standard_normal((40, 4)))[0], gpu(rng.standard_normal(40))[0]
    whole = ops().causal_conv_fwd(x, w, b)
    outs = [ops().causal_conv_fwd(x[:, :11].contiguous(), w, b)]
    window = x[:, 8:11].contiguous()
    for t in range(11, 30):
        outs.append(ops().causal_conv_update(window, x[:, t].contiguous(), w, b)[:, None])
    assert torch.equal(torch.cat(outs, 1), whole)


def test_two_runs_agree_and_writes_stay_inside():
    rng = np.random.default_rng(5)
    x, dout = (gpu(rng.standard_normal((3, 301, 77)), "bf16")[0] for _ in range(2))
    w = gpu(rng.standard_normal((77, 4)))[0]
    o = ops()
    out = Guarded((3, 301, 77), torch.bfloat16)
    o.causal_conv_fwd(x, w, out=out.t)
    n = o.lib().ss_causal_conv_bwd_workspace_bytes(3, 301, 77, 4, o.SS_BF16)
    ws = Guarded((max(n, 16),), torch.uint8)
    first = o.causal_conv_bwd(x, w, dout, workspace=ws.t)
    for _ in range(3):
        again = o.causal_conv_bwd(x, w, dout, workspace=ws.t)
        for k in ("dx", "dweight", "dbias"):
            assert torch.equal(first[k], again[k]), k
    assert out.intact() and ws.intact()


@pytest.mark.parametrize("io,d,k,silu", [("bf16", 8200, 4, True), ("f32", 4101, 3, False),
                                          ("bf16", 8192, 4, True), ("f32", 4096, 3, False)])
def test_a_call_that_outgrows_the_cache(io, d, k, silu):
    """Above 256 MB rows of whole cache lines are accessed non-temporally: the call equals its
    batch rows one by one, which stay below."""
    o, dt = ops(), torch.bfloat16 if io == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(d)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    x, dout, w, b = r(4, 2100, d).to(dt), r(4, 2100, d).to(dt), r(d, k), r(d)
    starts = torch.rand((4, 2100), device="cuda", generator=gen) < 0.01
    moved = x.numel() * x.element_size()
    assert 2 * moved > 256 << 20 > 3 * moved // 4
    out = o.causal_conv_fwd(x, w, b, starts=starts, silu=silu)
    g = o.causal_conv_bwd(x, w, dout, b, starts=starts, silu=silu)
    dw = torch.zeros_like(w)
    for k_ in range(4):
        c = lambda t: t[k_:k_ + 1].contiguous()  # noqa: E731
        assert torch.equal(out[k_:k_ + 1], o.causal_conv_fwd(c(x), w, b, starts=c(starts),
                                                             silu=silu))
        one = o.causal_conv_bwd(c(x), w, c(dout), b, starts=c(starts), silu=silu)
        assert torch.equal(g["dx"][k_:k_ + 1], one["dx"])
        dw += one["dweight"]
    # sums of 8400 products of unit size in another order: 2^-24 a step of at most a few hundred
    torch.testing.assert_close(g["dweight"], dw, rtol=1e-4, atol=2e-2)


def test_empty_sizes():
    o = ops()
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    w = torch.randn(8, 4, device="cuda")
    assert o.causal_conv_fwd(e(2, 0, 8), w).shape == (2, 0, 8)
    g = o.causal_conv_bwd(e(2, 0, 8), w, e(2, 0, 8), x_prev=torch.randn(2, 3, 8, device="cuda"))
    assert not g["dweight"].any() and not g["dbias"].any() and not g["dx_prev"].any()
    assert o.causal_conv_update(e(0, 3, 8), e(0, 8), w).shape == (0, 8)
    with pytest.raises(o.SSError) as err:
        o.causal_conv_fwd(e(1, 2, 8), torch.randn(8, 5, device="cuda"))
    assert err.value.status == o.SS_ERR_UNSUPPORTED


# The backward's waves walk 64 steps where that leaves 1024 of them (sequences in runs of 64, times
# groups of 128 channels), else 16.
def walks_64(batch, L, d):
    return batch * -(-L // 64) * -(-d // 128) >= 1024


@pytest.mark.parametrize("batch,L,d,k", [(350, 130, 6, 4), (350, 129, 5, 3), (520, 127, 3, 2),
                                         (520, 66, 4, 4), (260, 200, 2, 1), (120, 191, 257, 4)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_long_runs_without_silu_are_exact(batch, L, d, k, io):
    """Small whole numbers: every product and sum is exact in float32, so each gradient equals the
    definition's, whatever the runs, the starts among them and the windows between."""
    assert walks_64(batch, L, d)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    gen = torch.Generator().manual_seed(L * d + k)
    n = lambda *s: torch.randint(-3, 4, s, generator=gen).double()  # noqa: E731
    x, dout, w, xp = n(batch, L, d), n(batch, L, d), n(d, k), n(batch, k - 1, d)
    starts = torch.rand((batch, L), generator=gen) < 0.05
    up = lambda t, as_=dt: t.to(as_).cuda()  # noqa: E731
    g = ops().causal_conv_bwd(up(x), up(w, torch.float32), up(dout), x_prev=up(xp),
                              starts=starts.cuda(), silu=False)
    seq = torch.cumsum(starts.int(), 1)
    whole = torch.cat([xp, x], 1)
    dpad, dw = torch.zeros_like(whole), []
    for j in range(k):
        lag = k - 1 - j
        then = torch.cat([torch.zeros(batch, lag, dtype=seq.dtype), seq[:, :L - lag]], 1)
        m = (then == seq)[..., None] * dout
        dpad[:, j:j + L] += m * w[:, j]
        dw.append((m * whole[:, j:j + L]).sum((0, 1)))
    # (gradients of bfloat16 inputs are sums of at most four products below 9: no rounding)
    assert torch.equal(g["dx"].double().cpu(), dpad[:, k - 1:])
    assert torch.equal(g["dx_prev"].double().cpu(), dpad[:, :k - 1])
    assert torch.equal(g["dweight"].double().cpu(), torch.stack(dw, 1))
    assert torch.equal(g["dbias"].double().cpu(), dout.sum((0, 1)))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,d,k", [(350, 130, 6, 4), (345, 131, 5, 3)])
def test_long_runs(batch, L, d, k, io):
    assert walks_64(batch, L, d)
    run_case(L, batch, L, d, k, io, packed=True, prev=True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,d,k", [(2, 77, 65, 4), (1, 130, 30, 3), (2, 2, 9, 4),
                                         (350, 130, 7, 2), (3, 5, 128, 1)])
def test_gradients_stay_inside_their_arrays(batch, L, d, k, io):
    """Every array that the backward writes, between marker bytes; and the one-token form's."""
    rng = np.random.default_rng(L + d)
    n = lambda *s: gpu(rng.standard_normal(s), io)[0]  # noqa: E731
    x, dout, xp, o = n(batch, L, d), n(batch, L, d), n(batch, k - 1, d), ops()
    w, b = gpu(rng.standard_normal((d, k)))[0], gpu(rng.standard_normal(d))[0]
    s = starts_gpu(draw_starts(rng, batch, L, 7))
    want = o.causal_conv_bwd(x, w, dout, b, x_prev=xp, starts=s)
    g = dict(dx=Guarded((batch, L, d), x.dtype), dweight=Guarded((d, k), torch.float32),
             dbias=Guarded((d,), torch.float32), dx_prev=Guarded((batch, k - 1, d), x.dtype))
    code = o.SS_BF16 if io == "bf16" else o.SS_F32
    size = o.lib().ss_causal_conv_bwd_workspace_bytes(batch, L, d, k, code)
    ws = Guarded((size,), torch.uint8)
    p = lambda t: t.data_ptr()  # noqa: E731
    o._check(o.lib().ss_causal_conv_bwd(
        p(x), p(w), p(b), p(xp) or None, p(s), 1, p(dout),
        *(p(g[m].t) for m in ("dx", "dweight", "dbias", "dx_prev")), batch, L, d, k, code,
        p(ws.t), size, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    for m, buf in g.items():
        assert torch.equal(buf.t, want[m]) and buf.intact(), m
    assert ws.intact()
    state, out = Guarded((batch, k - 1, d), x.dtype), Guarded((batch, d), x.dtype)
    state.t.copy_(xp)
    ref = o.causal_conv_update(xp, x[:, 0].contiguous(), w, b)
    o.causal_conv_update(state.t, x[:, 0].contiguous(), w, b, out=out.t)
    assert torch.equal(out.t, ref) and torch.equal(state.t, xp)
    assert out.intact() and state.intact()
