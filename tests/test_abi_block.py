"""CPU checks of the recurrent block's entry points: bad arguments are refused before anything is
launched (no compute call is made here; the addresses are never dereferenced)."""
import os

import pytest
import torch

from selective_state_space_36_amd import ops

G = 1 << 34


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ops.LIB_PATH):
        from selective_state_space_36_amd import build
        build.build()
    return ops.lib()


def call(lib, name, defaults, **kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return getattr(lib, name)(*a.values())


FWD = dict(x=G, r=2 * G, i=3 * G, A=4 * G, rb=None, ib=None, z=None, starts=None, h0=None,
           hl=None, out=5 * G, states=None, batch=2, L=100, d=32, dtype=ops.SS_BF16, ws=6 * G,
           wsb=1 << 30, stream=None)
BWD = dict(x=G, r=2 * G, i=3 * G, A=4 * G, rb=None, ib=None, z=None, starts=None, h0=None,
           dout=5 * G, dhl=None, states=None, dx=6 * G, dr=7 * G, di=8 * G, dz=None, dA=9 * G,
           drb=None, dib=None, dh0=None, batch=2, L=100, d=32, dtype=ops.SS_BF16, ws=10 * G,
           wsb=1 << 30, stream=None)
STEP = dict(state=G, x=2 * G, r=3 * G, i=4 * G, A=5 * G, rb=None, ib=None, z=None, out=6 * G,
            batch=2, d=32, dtype=ops.SS_BF16, stream=None)
NFWD = dict(x=G, res=None, w=None, b=None, eps=1e-5, out=2 * G, sum=None, mean=None, rstd=None,
            rows=4, dim=32, dtype=ops.SS_BF16, stream=None)
NBWD = dict(dout=G, s=2 * G, sdt=ops.SS_BF16, w=None, mean=3 * G, rstd=4 * G, dsum=None,
            dx=5 * G, dres=None, dw=6 * G, db=7 * G, rows=4, dim=32, dtype=ops.SS_BF16, ws=8 * G,
            wsb=1 << 30, stream=None)
CFWD = dict(x=G, w=2 * G, b=None, xp=None, starts=None, silu=1, out=3 * G, batch=2, L=100, d=32,
            k=4, dtype=ops.SS_BF16, stream=None)
CBWD = dict(x=G, w=2 * G, b=None, xp=None, starts=None, silu=1, dout=3 * G, dx=4 * G, dw=5 * G,
            db=None, dxp=None, batch=2, L=100, d=32, k=4, dtype=ops.SS_BF16, ws=6 * G,
            wsb=1 << 30, stream=None)
CSTEP = dict(st=G, x=2 * G, w=3 * G, b=None, silu=1, out=4 * G, batch=2, d=32, k=4,
             dtype=ops.SS_BF16, stream=None)

BAD, UNS = ops.SS_ERR_INVALID_ARG, ops.SS_ERR_UNSUPPORTED
REFUSED = [
    ("ss_gated_scan_fwd", FWD, dict(dtype=7), UNS, b"dtype"),
    ("ss_gated_scan_fwd", FWD, dict(batch=-1), BAD, b"negative"),
    ("ss_gated_scan_fwd", FWD, dict(x=None), BAD, b"x is NULL"),
    ("ss_gated_scan_fwd", FWD, dict(r=None), BAD, b"r is NULL"),
    ("ss_gated_scan_fwd", FWD, dict(i=None), BAD, b"i is NULL"),
    ("ss_gated_scan_fwd", FWD, dict(A=None), BAD, b"A is NULL"),
    ("ss_gated_scan_fwd", FWD, dict(out=None), BAD, b"out is NULL"),
    ("ss_gated_scan_fwd", FWD, dict(x=G + 1), UNS, b"aligned"),
    ("ss_gated_scan_fwd", FWD, dict(A=4 * G + 2), UNS, b"aligned"),
    ("ss_gated_scan_fwd", FWD, dict(out=G), BAD, b"out overlaps x"),
    ("ss_gated_scan_fwd", FWD, dict(out=3 * G + 12798), BAD, b"out overlaps i"),
    ("ss_gated_scan_fwd", FWD, dict(starts=5 * G + 64), BAD, b"out overlaps starts"),
    ("ss_gated_scan_fwd", FWD, dict(h0=7 * G, hl=7 * G), BAD, b"h_last overlaps h0"),
    ("ss_gated_scan_fwd", FWD, dict(hl=5 * G), BAD, b"out overlaps h_last"),
    ("ss_gated_scan_fwd", FWD, dict(states=2 * G), BAD, b"states overlaps r"),
    ("ss_gated_scan_fwd", FWD, dict(d=(1 << 24) + 1), UNS, b"d_inner"),
    ("ss_gated_scan_fwd", FWD, dict(L=1 << 31), UNS, b"seqlen"),
    ("ss_gated_scan_fwd", FWD, dict(batch=1 << 40, L=1 << 30, d=1 << 20), BAD, b"overflow"),
    ("ss_gated_scan_fwd", FWD, dict(batch=1 << 20, L=1 << 20, d=1 << 10), BAD, b"too many"),
    ("ss_gated_scan_fwd", FWD, dict(batch=1 << 24, L=100, d=64), BAD, b"one launch"),
    ("ss_gated_scan_bwd", BWD, dict(batch=1 << 24, L=100, d=64), BAD, b"one launch"),
    ("ss_gated_state_update", STEP, dict(batch=1 << 26, d=64), BAD, b"one launch"),
    ("ss_causal_conv_fwd", CFWD, dict(batch=1 << 26, L=1, d=1), BAD, b"one launch"),
    ("ss_causal_conv_update", CSTEP, dict(batch=1 << 26, d=64), BAD, b"one launch"),
    ("ss_gated_scan_fwd", FWD, dict(L=0, h0=G, hl=G + 4), BAD, b"overlaps"),
    ("ss_gated_scan_bwd", BWD, dict(dtype=9), UNS, b"dtype"),
    ("ss_gated_scan_bwd", BWD, dict(dout=None), BAD, b"dout is NULL"),
    ("ss_gated_scan_bwd", BWD, dict(dx=None), BAD, b"dx is NULL"),
    ("ss_gated_scan_bwd", BWD, dict(dA=None), BAD, b"dA is NULL"),
    ("ss_gated_scan_bwd", BWD, dict(z=11 * G), BAD, b"dz is NULL"),
    ("ss_gated_scan_bwd", BWD, dict(dx=5 * G), BAD, b"dx overlaps dout"),
    ("ss_gated_scan_bwd", BWD, dict(dr=6 * G), BAD, b"dx overlaps dr"),
    ("ss_gated_scan_bwd", BWD, dict(dh0=9 * G), BAD, b"overlaps"),
    ("ss_gated_scan_bwd", BWD, dict(ws=None, wsb=0), BAD, b"workspace"),
    ("ss_gated_scan_bwd", BWD, dict(wsb=8), BAD, b"workspace"),
    ("ss_gated_scan_bwd", BWD, dict(ws=10 * G + 8), UNS, b"16-byte"),
    ("ss_gated_scan_bwd", BWD, dict(ws=G), BAD, b"workspace overlaps x"),
    ("ss_gated_scan_bwd", BWD, dict(states=12 * G + 2), UNS, b"aligned"),
    ("ss_gated_state_update", STEP, dict(state=None), BAD, b"state is NULL"),
    ("ss_gated_state_update", STEP, dict(out=G), BAD, b"state overlaps out"),
    ("ss_gated_state_update", STEP, dict(out=2 * G), BAD, b"out overlaps x"),
    ("ss_gated_state_update", STEP, dict(dtype=3), UNS, b"dtype"),
    ("ss_layer_norm_fwd", NFWD, dict(rows=-1), BAD, b"negative"),
    ("ss_layer_norm_fwd", NFWD, dict(eps=-1.0), BAD, b"eps"),
    ("ss_layer_norm_fwd", NFWD, dict(eps=float("nan")), BAD, b"eps"),
    ("ss_layer_norm_fwd", NFWD, dict(eps=float("inf")), BAD, b"eps"),
    ("ss_layer_norm_fwd", NFWD, dict(x=None), BAD, b"x is NULL"),
    ("ss_layer_norm_fwd", NFWD, dict(out=G), BAD, b"out overlaps x"),
    ("ss_layer_norm_fwd", NFWD, dict(res=3 * G, sum=3 * G), BAD, b"sum overlaps residual"),
    ("ss_layer_norm_fwd", NFWD, dict(mean=2 * G), BAD, b"out overlaps mean"),
    ("ss_layer_norm_fwd", NFWD, dict(w=3 * G + 1), UNS, b"aligned"),
    ("ss_layer_norm_fwd", NFWD, dict(dim=(1 << 24) + 1), UNS, b"dim"),
    ("ss_layer_norm_fwd", NFWD, dict(rows=1 << 31, dim=1), BAD, b"too many rows"),
    ("ss_layer_norm_bwd", NBWD, dict(dx=None), BAD, b"both NULL"),
    ("ss_layer_norm_bwd", NBWD, dict(sdt=5), UNS, b"dtype"),
    ("ss_layer_norm_bwd", NBWD, dict(sdt=ops.SS_BF16, dtype=ops.SS_F32), UNS, b"s is either"),
    ("ss_layer_norm_bwd", NBWD, dict(mean=None), BAD, b"mean is NULL"),
    ("ss_layer_norm_bwd", NBWD, dict(dw=G), BAD, b"dweight overlaps dout"),
    ("ss_layer_norm_bwd", NBWD, dict(dres=5 * G), BAD, b"dx overlaps dresidual"),
    ("ss_causal_conv_fwd", CFWD, dict(k=0), UNS, b"k=0"),
    ("ss_causal_conv_fwd", CFWD, dict(k=5), UNS, b"k=5"),
    ("ss_causal_conv_fwd", CFWD, dict(w=None), BAD, b"weight is NULL"),
    ("ss_causal_conv_fwd", CFWD, dict(out=G), BAD, b"out overlaps x"),
    ("ss_causal_conv_fwd", CFWD, dict(xp=3 * G), BAD, b"out overlaps x_prev"),
    ("ss_causal_conv_bwd", CBWD, dict(dxp=7 * G), BAD, b"without x_prev"),
    ("ss_causal_conv_bwd", CBWD, dict(dw=None), BAD, b"dweight is NULL"),
    ("ss_causal_conv_bwd", CBWD, dict(dx=3 * G), BAD, b"dx overlaps dout"),
    ("ss_causal_conv_bwd", CBWD, dict(xp=7 * G, dxp=7 * G), BAD, b"dx_prev overlaps x_prev"),
    ("ss_causal_conv_update", CSTEP, dict(st=None), BAD, b"conv_state is NULL"),
    ("ss_causal_conv_update", CSTEP, dict(out=G), BAD, b"conv_state overlaps out"),
    ("ss_causal_conv_update", CSTEP, dict(st=2 * G), BAD, b"conv_state overlaps x"),
    ("ss_causal_conv_update", CSTEP, dict(k=9), UNS, b"k=9"),
]


@pytest.mark.parametrize("name,defaults,kw,status,text", REFUSED,
                         ids=[f"{n[3:]}-{'-'.join(k)}-{t.decode()}" for n, _, k, _, t in REFUSED])
def test_refusals(lib, name, defaults, kw, status, text):
    assert call(lib, name, defaults, **kw) == status
    assert text in lib.ss_last_error()


def test_empty_problems_succeed_without_a_launch(lib):
    for name, defaults, kw in (("ss_gated_scan_fwd", FWD, dict(batch=0)),
                               ("ss_gated_scan_fwd", FWD, dict(d=0)),
                               ("ss_gated_scan_fwd", FWD, dict(L=0)),
                               ("ss_gated_scan_bwd", BWD, dict(d=0)),
                               ("ss_gated_state_update", STEP, dict(batch=0)),
                               ("ss_layer_norm_fwd", NFWD, dict(rows=0)),
                               ("ss_layer_norm_fwd", NFWD, dict(dim=0)),
                               ("ss_layer_norm_bwd", NBWD, dict(dim=0)),
                               ("ss_causal_conv_fwd", CFWD, dict(L=0)),
                               ("ss_causal_conv_bwd", CBWD, dict(d=0)),
                               ("ss_causal_conv_update", CSTEP, dict(batch=0))):
        assert call(lib, name, defaults, **kw) == ops.SS_OK, name
        assert lib.ss_last_error() == b""


def test_sizes_queries(lib):
    assert lib.ss_gated_scan_states_bytes(2, 130, 8) == 2 * 3 * 8 * 4
    assert lib.ss_gated_scan_states_bytes(2, 0, 8) == 0
    for q in (lambda: lib.ss_gated_scan_fwd_workspace_bytes(0, 5, 8, 1),
              lambda: lib.ss_gated_scan_fwd_workspace_bytes(-1, 5, 8, 1),
              lambda: lib.ss_gated_scan_bwd_workspace_bytes(2, 0, 8, 1, 0),
              lambda: lib.ss_gated_scan_bwd_workspace_bytes(1 << 40, 1 << 30, 8, 1, 0),
              lambda: lib.ss_layer_norm_bwd_workspace_bytes(0, 8),
              lambda: lib.ss_layer_norm_bwd_workspace_bytes(4, 1 << 25),
              lambda: lib.ss_causal_conv_bwd_workspace_bytes(2, 9, 8, 5, 1)):
        assert q() == 0
    given = lib.ss_gated_scan_bwd_workspace_bytes(2, 130, 8, 1, 1)
    assert given > 0
    assert lib.ss_gated_scan_bwd_workspace_bytes(2, 130, 8, 1, 0) >= \
        given + lib.ss_gated_scan_states_bytes(2, 130, 8)


def test_the_binding_refuses_host_tensors():
    x, A = torch.zeros(1, 2, 4), torch.zeros(4)
    for f in (lambda: ops.gated_scan_fwd(x, x, x, A),
              lambda: ops.gated_scan_fwd_states(x, x, x, A),
              lambda: ops.gated_scan_bwd(x, x, x, A, x),
              lambda: ops.gated_state_update(x[0], x[0], x[0], x[0], A),
              lambda: ops.layer_norm_fwd(x),
              lambda: ops.layer_norm_bwd(x, x, None, A, A),
              lambda: ops.causal_conv_fwd(x, A[:, None]),
              lambda: ops.causal_conv_bwd(x, A[:, None], x),
              lambda: ops.causal_conv_update(x, x[:, 0], A[:, None])):
        with pytest.raises(ValueError, match="GPU tensor"):
            f()
