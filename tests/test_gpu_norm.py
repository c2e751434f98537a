"""Layer norm with the residual add on the GPU, forward and gradients, against float64."""
import numpy as np
import pytest

from oracle import block_twin as bt
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
    def __init__(self, seed, rows, dim, io, residual, params=True, shift=0.0, offset=0):
        print(f"  case rows={rows} dim={dim} {io} residual={residual} shift={shift}", flush=True)
        rng = np.random.default_rng(seed)
        n = lambda *s: rng.standard_normal(s)  # noqa: E731
        self.io, self.residual = io, residual
        self.x, self.vx = gpu(n(rows, dim) + shift, io, offset)
        self.w, self.vw = gpu(1 + 0.1 * n(dim) if params else None, "f32", offset)
        self.b, self.vb = gpu(0.1 * n(dim) if params else None)
        self.res, self.vres = gpu(3 * n(rows, dim) if residual else None, "f32", offset)
        self.dout, self.vdout = gpu(n(rows, dim), io, offset)
        self.dsum, self.vdsum = gpu(n(rows, dim) if residual else None)

    def check(self):
        o = ops()
        r = o.layer_norm_fwd(self.x, self.w, self.b, residual=self.res, return_stats=True)
        out, total, mean, rstd = r if self.residual else (r[0], None, *r[1:])
        ref, s, vm, vr, _ = bt.norm_fwd(self.vx, self.vw, self.vb, self.vres)
        check(out, ref, self.io, "out")
        check(mean, vm, "f32", "mean")
        check(rstd, vr, "f32", "rstd")
        if self.residual:
            check(total, s, "f32", "sum")
        g = o.layer_norm_bwd(self.dout, total if self.residual else self.x, self.w, mean, rstd,
                             dsum=self.dsum, want_dresidual=True)
        want = bt.norm_bwd(self.vdout, self.vx, self.vw, self.vres, self.vdsum)
        check(g["dx"], want["ds"], self.io, "dx")
        check(g["dresidual"], want["ds"], "f32", "dresidual")
        check(g["dweight"], want["dweight"], "f32", "dweight")
        check(g["dbias"], want["dbias"], "f32", "dbias")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 2560), (3, 2), (5, 63), (4, 64), (7, 100),
                                      (2, 768), (33, 130), (9, 1027), (300, 96), (3, 4096),
                                      (2, 5121), (5, 8200), (2, 20001), (3, 641), (6, 1022),
                                      (4, 1601), (5, 2049), (600, 3601), (3, 4093), (2, 4098),
                                      (3, 5126), (3, 8194), (2, 16382), (2, 8193), (2, 16386)])
def test_forward_and_gradients(rows, dim, residual, io):
    Case(rows * 10 + dim, rows, dim, io, residual).check()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_without_parameters(io):
    Case(1, 6, 200, io, True, params=False).check()
    Case(2, 6, 200, io, False, params=False).check()


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_misaligned(offset, io):
    Case(offset, 5, 256, io, True, offset=offset).check()


def test_many_rows():
    Case(3, 3001, 72, "bf16", True).check()


@pytest.mark.parametrize("dim", [100, 2560])
def test_a_mean_far_from_zero_does_not_cost_the_variance(dim):
    Case(4, 4, dim, "f32", False, shift=300.0).check()


@pytest.mark.parametrize("rows,dim", [((1 << 23) + 7, 2), ((1 << 21) + 3, 513), (4100, 8193)])
def test_more_rows_than_workgroups(rows, dim):
    """The workgroups loop over the rows: those of the second round equal a call on them alone."""
    o = ops()
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.randn(rows, dim, device="cuda", generator=g).bfloat16()
    out, mean, rstd = o.layer_norm_fwd(x, return_stats=True)
    for a, b in ((0, 9), (rows // 2, rows // 2 + 9), (rows - 9, rows)):
        alone, m, r = o.layer_norm_fwd(x[a:b].contiguous(), return_stats=True)
        assert torch.equal(out[a:b], alone)
        assert torch.equal(mean[a:b], m) and torch.equal(rstd[a:b], r)
    dx = o.layer_norm_bwd(x, x, None, mean, rstd, want_dparams=False)["dx"]
    tail = slice(rows - 9, rows)
    alone = o.layer_norm_bwd(x[tail].contiguous(), x[tail].contiguous(), None, mean[tail].clone(),
                             rstd[tail].clone(), want_dparams=False)["dx"]
    assert torch.equal(dx[tail], alone)


@pytest.mark.parametrize("io,dim", [("bf16", 2564), ("f32", 1027), ("bf16", 300),
                                    ("bf16", 2560), ("f32", 1024)])
def test_a_call_that_outgrows_the_cache(io, dim):
    """Above 256 MB rows of whole cache lines are read non-temporally: the call equals pieces of it,
    which stay below."""
    o, dt = ops(), torch.bfloat16 if io == "bf16" else torch.float32
    rows = (48 << 20) // dim
    gen = torch.Generator(device="cuda").manual_seed(dim)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    x, res, w, b, dout = r(rows, dim).to(dt), r(rows, dim), r(dim), r(dim), r(rows, dim).to(dt)
    out, s, mean, rstd = o.layer_norm_fwd(x, w, b, residual=res, return_stats=True)
    g = o.layer_norm_bwd(dout, s, w, mean, rstd, dsum=res, want_dresidual=True)
    for k in range(4):
        c = slice(k * rows // 4, (k + 1) * rows // 4)
        p, q, m, t = o.layer_norm_fwd(x[c], w, b, residual=res[c], return_stats=True)
        assert torch.equal(out[c], p) and torch.equal(s[c], q)
        assert torch.equal(mean[c], m) and torch.equal(rstd[c], t)
        h = o.layer_norm_bwd(dout[c], q, w, m, t, dsum=res[c], want_dresidual=True)
        assert torch.equal(g["dx"][c], h["dx"]) and torch.equal(g["dresidual"][c],
                                                                h["dresidual"])


def test_a_constant_row():
    o = ops()
    x = torch.full((3, 700), 2.5, device="cuda")
    b = torch.randn(700, device="cuda")
    out, mean, rstd = o.layer_norm_fwd(x, None, b, return_stats=True)
    assert torch.equal(out, b.expand(3, 700)) and torch.equal(mean, x[:, 0])
    assert torch.allclose(rstd, torch.full_like(rstd, 1e5 ** 0.5), rtol=1e-6)


def test_a_bad_row_leaves_the_others_alone():
    c = Case(5, 6, 320, "f32", True)
    c.x[2, 5] = float("nan")
    c.x[4, 0] = float("inf")
    out, s, mean, rstd = ops().layer_norm_fwd(c.x, c.w, c.b, residual=c.res, return_stats=True)
    good = [0, 1, 3, 5]
    assert torch.isfinite(out[good]).all() and torch.isnan(out[[2, 4]]).all()
    g = ops().layer_norm_bwd(c.dout, s, c.w, mean, rstd)
    assert torch.isfinite(g["dx"][good]).all() and torch.isnan(g["dx"][[2, 4]]).all()


def test_sum_without_residual_and_leading_dimensions():
    x = torch.randn(2, 3, 5, 40, device="cuda", dtype=torch.bfloat16)
    out, s, mean, rstd = ops().layer_norm_fwd(x, return_sum=True, return_stats=True)
    assert torch.equal(s, x.float()) and mean.shape == (2, 3, 5)
    flat = ops().layer_norm_fwd(x.view(30, 40))
    assert torch.equal(out.view(30, 40), flat)
    g = ops().layer_norm_bwd(torch.ones_like(x), s, None, mean, rstd, want_dparams=False)
    assert g["dx"].shape == x.shape and g["dweight"] is None and g["dresidual"] is None


def test_two_runs_agree_and_writes_stay_inside():
    c = Case(6, 777, 515, "bf16", True)
    o = ops()
    out, s = Guarded((777, 515), torch.bfloat16), Guarded((777, 515), torch.float32)
    _, _, mean, rstd = o.layer_norm_fwd(c.x, c.w, c.b, residual=c.res, out=out.t, sum_out=s.t,
                                        return_stats=True)
    ws = Guarded((max(16, o.lib().ss_layer_norm_bwd_workspace_bytes(777, 515)),), torch.uint8)
    run = lambda: o.layer_norm_bwd(c.dout, s.t, c.w, mean, rstd, dsum=c.dsum,  # noqa: E731
                                   want_dresidual=True, workspace=ws.t)
    first = run()
    for _ in range(3):
        again = run()
        for k in first:
            assert torch.equal(first[k], again[k]), k
    assert out.intact() and s.intact() and ws.intact()


def test_empty_sizes():
    o = ops()
    e = torch.empty(0, 16, device="cuda")
    out, mean, rstd = o.layer_norm_fwd(e, return_stats=True)
    assert out.shape == (0, 16)
    g = o.layer_norm_bwd(e, e, None, mean, rstd)
    assert not g["dweight"].any() and not g["dbias"].any() and g["dx"].shape == (0, 16)
    assert o.layer_norm_fwd(torch.empty(3, 0, device="cuda")).shape == (3, 0)


# Whole numbers whose sums stay below 2^24: float32 holds every sum over rows and columns exactly,
# in whatever order it is formed.
def whole(rows, dim, seed):
    """dout, s, weight, mean, rstd, dsum on the GPU, in float32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, device="cuda",  # noqa: E731
                                         generator=g).float()
    return (n(-2, 2, rows, dim), n(-4, 4, rows, dim), n(1, 2, dim), n(-1, 1, rows),
            2.0 ** n(-1, 0, rows), n(-9, 9, rows, dim))


def gradients64(dout, s, weight, mean, rstd, dsum):
    """ds with a bound on its float32 error, dweight and dbias, in float64."""
    dy, w, rs = dout.double(), weight.double(), rstd.double()[:, None]
    xh = (s.double() - mean.double()[:, None]) * rs
    g = dy * w
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    ds = rs * (g - c1 - xh * c2) + dsum.double()
    # The sums are exact; 1 / dim and its products with them round (2 U of c1 and c2), then
    # g - c1, the multiply-add with xh c2, and the last one with rstd and dsum.
    terms = rs * (g.abs() + c1.abs() + (xh * c2).abs())
    return ds, 2.0 ** -24 * (5 * terms + ds.abs()), (dy * xh).sum(0), dy.sum(0)


# Rows enough for every workgroup (512 of them, of one row or of four) to take several: groups of
# four columns with 64, 256 and 1024 threads a row, single columns likewise, and the wide rows,
# whose parameter sums 64 strands share.
@pytest.mark.parametrize("io,sdt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,dim", [(5003, 1000), (1501, 1540), (1501, 2560), (1030, 4096),
                                      (1100, 5120), (1030, 12288), (1030, 16384), (5003, 333),
                                      (1501, 2561), (1501, 3601), (1030, 4099), (1030, 8191),
                                      (300, 8193), (130, 12292), (200, 20000), (67, 20001)])
def test_gradients_where_workgroups_take_many_rows(rows, dim, io, sdt):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    dout, s, w, mean, rstd, dsum = whole(rows, dim, rows + dim)
    g = ops().layer_norm_bwd(dout.to(dt[io]), s.to(dt[sdt]), w, mean, rstd, dsum=dsum,
                             want_dresidual=True)
    ds, e, dw, db = gradients64(dout, s, w, mean, rstd, dsum)
    assert torch.equal(g["dweight"].double(), dw)
    assert torch.equal(g["dbias"].double(), db)
    assert ((g["dresidual"].double() - ds).abs() <= e).all()
    half = 2.0 ** -8 if io == "bf16" else 0.0
    assert ((g["dx"].double() - ds).abs() <= e + half * (ds.abs() + e)).all()


@pytest.mark.parametrize("io,dim", [("bf16", 2560), ("f32", 1024), ("bf16", 300), ("f32", 1027)])
def test_parameter_sums_of_a_call_that_outgrows_the_cache(io, dim):
    rows = (48 << 20) // dim
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    dout, s, w, mean, rstd, dsum = whole(rows, dim, dim)
    g = ops().layer_norm_bwd(dout.to(dt), s, w, mean, rstd, dsum=dsum)
    dw, db = torch.zeros_like(w, dtype=torch.float64), torch.zeros_like(w, dtype=torch.float64)
    for k in range(4):
        c = slice(k * rows // 4, (k + 1) * rows // 4)
        ds, e, pw, pb = gradients64(dout[c], s[c], w, mean[c], rstd[c], dsum[c])
        half = 2.0 ** -8 if io == "bf16" else 0.0
        assert ((g["dx"][c].double() - ds).abs() <= e + half * (ds.abs() + e)).all()
        dw += pw
        db += pb
    assert torch.equal(g["dweight"].double(), dw) and torch.equal(g["dbias"].double(), db)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(777, 515), (5, 4099), (3, 2), (2, 20001), (9, 260)])
def test_gradients_stay_inside_their_arrays(rows, dim, io):
    """Every array that the backward writes, between marker bytes."""
    o = ops()
    c = Case(rows + dim, rows, dim, io, True)
    _, s, mean, rstd = o.layer_norm_fwd(c.x, c.w, c.b, residual=c.res, return_stats=True)
    want = o.layer_norm_bwd(c.dout, s, c.w, mean, rstd, dsum=c.dsum, want_dresidual=True)
    g = dict(dx=Guarded((rows, dim), c.x.dtype), dresidual=Guarded((rows, dim), torch.float32),
             dweight=Guarded((dim,), torch.float32), dbias=Guarded((dim,), torch.float32))
    n = o.lib().ss_layer_norm_bwd_workspace_bytes(rows, dim)
    ws = Guarded((n,), torch.uint8)
    p = lambda t: t.data_ptr()  # noqa: E731
    o._check(o.lib().ss_layer_norm_bwd(
        p(c.dout), p(s), o.SS_F32, p(c.w), p(mean), p(rstd), p(c.dsum),
        *(p(g[k].t) for k in ("dx", "dresidual", "dweight", "dbias")), rows, dim,
        o.SS_BF16 if io == "bf16" else o.SS_F32, p(ws.t), n,
        torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    for k, buf in g.items():
        assert torch.equal(buf.t, want[k]) and buf.intact(), k
    assert ws.intact()


@pytest.mark.parametrize("shape", [(3, 0), (0,), (2, 5, 0)])
def test_statistics_of_no_columns_are_nan(shape):
    """They are allocated by the call: not what the memory held before."""
    held = [torch.full((10,), 7.0, device="cuda") for _ in range(4)]
    del held
    out, mean, rstd = ops().layer_norm_fwd(torch.empty(shape, device="cuda"), return_stats=True)
    assert out.shape == shape and mean.shape == rstd.shape == shape[:-1]
    assert torch.isnan(mean).all() and torch.isnan(rstd).all()
