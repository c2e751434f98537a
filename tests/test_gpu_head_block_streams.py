"""stream= of the operators around the multi-head scan: the call stands on that stream, behind what
stands there already.  All inputs are there before; what the last of them is made of waits on the
stream behind a long kernel, so that a call on another one would read the old values."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_36_amd import ops
    ops.lib()
    yield


def _calls(o, r):
    """name -> (call, its input that arrives late, fresh copies of what it changes)"""
    x, z, w = r(500, 640), r(500, 640), r(640)
    rng = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    B, C, dt, A = r(2, 40, 1, 16), r(2, 40, 1, 16), r(2, 40, 4), -r(4).abs()
    xs, rstd, group_rstd = r(2, 40, 4, 8), r(500).abs(), torch.ones(500, 5, device="cuda")
    x1, d1, B1, C1 = (t[:, 0].contiguous() for t in (xs, dt, B, C))
    state, xbc = r(2, 4, 16, 8), r(2, 64)
    window, taps = r(2, 3, 64), r(64, 4)
    late = lambda t: t.clone()  # noqa: E731
    return dict(
        dropout=(lambda a, **k: o.dropout(a, 0.3, rng, **k), late(x), ()),
        rms_fwd=(lambda a, **k: o.rms_norm_fwd(a, w, residual=z, scale=w, p=0.3, rng=rng, **k)[1],
                 late(x), ()),
        rms_bwd=(lambda a, **k: o.rms_norm_bwd(a, x, w, rstd, **k)["dweight"], late(x), ()),
        gated_fwd=(lambda a, **k: o.gated_norm_fwd(a, z, w, groups=5, **k), late(x), ()),
        gated_bwd=(lambda a, **k: o.gated_norm_bwd(a, x, z, w, group_rstd, groups=5,
                                                   **k)["dweight"], late(x), ()),
        scan_bwd=(lambda a, **k: o.scan2_bwd(xs, dt, A, B, C, a, **k)["dB"], late(xs), ()),
        step=(lambda a, s, **k: o.scan2_state_update(s, a, d1, A, B1, C1, **k), late(x1), (state,)),
        step_conv=(lambda a, s, v, **k: o.scan2_state_update_conv(s, v, a, taps, None, d1, A, **k),
                   late(xbc), (state, window)))


@pytest.mark.parametrize("name", ["dropout", "rms_fwd", "rms_bwd", "gated_fwd", "gated_bwd",
                                  "scan_bwd", "step", "step_conv"])
def test_the_call_stands_on_its_stream(name):
    from selective_state_space_36_amd import ops as o
    g = torch.Generator(device="cuda").manual_seed(6)
    call, late, changed = _calls(o, lambda *n: torch.randn(*n, device="cuda", generator=g))[name]
    new = late + 1
    first, second = ([t.clone() for t in changed] for _ in range(2))
    want = call(new, *first)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)       # about 10 ms
        late.copy_(new)
    got = call(late, *second, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    for a, b in zip(first, second):
        assert torch.equal(a, b)
