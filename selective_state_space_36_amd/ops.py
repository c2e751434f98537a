"""Thin ctypes binding of libssscan.so (include/ss_scan.h) for torch tensors.

Argument marshalling only: every step of the scan runs in the library's HIP kernels.  torch
provides device memory and the stream.  There is no fallback: if the library is missing or a
call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssscan.so")

SS_OK, SS_ERR_INVALID_ARG, SS_ERR_UNSUPPORTED, SS_ERR_HIP = 0, 1, 2, 3
SS_F32, SS_BF16 = 0, 1
SS_FLAG_ZOH_EXACT = 1
SS_FLAG_STATES_GIVEN = 2
SS_GATED_CHUNK = 64

# Every symbol declared in include/ss_scan.h, with its ctypes signature.
_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_u32 = ctypes.c_uint32
SIGNATURES = {
    "ss_scan_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp,
                           _i64, _i64, _i64, _i64, _i32, _vp, _sz, _vp]),
    "ss_scan_fwd_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _i32]),
    "ss_scan_fwd_noalloc": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp,
                                   _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp]),
    "ss_scan_fwd_ex": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp,
                              _vp, _i64, _i64, _i64, _i64, _i32, _vp, _sz, _i32, _u32, _vp]),
    "ss_scan_fwd_ex_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _i32, _i32]),
    "ss_scan_fwd_states": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp,
                                  _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp, _sz, _vp]),
    "ss_scan_fwd_states_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "ss_scan_fwd_conv": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp,
                                _sz, _i32, _u32, _vp]),
    "ss_scan_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp,
                           _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                           _i32, _vp, _sz, _u32, _vp]),
    "ss_scan_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _i32]),
    "ss_scan2_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp,
                            _vp, _i64, _i64, _i64, _i64, _i64, _i64, _i32, _vp]),
    "ss_state_update_conv": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp,
                                    _vp, _vp, ctypes.c_int, _vp, _i64, _i64, _i64, _i32, _u32,
                                    _vp]),
    "ss_state_update": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp,
                               _i64, _i64, _i64, _i32, _vp]),
    "ss_state_update_ex": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int,
                                  _vp, _i64, _i64, _i64, _i32, _u32, _vp]),
    "ss_gated_scan_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _i64, _i64, _i64, _i32, _vp, _sz, _vp]),
    "ss_gated_scan_fwd_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32]),
    "ss_gated_scan_states_bytes": (_sz, [_i64, _i64, _i64]),
    "ss_gated_scan_bwd": (_i32, [_vp] * 20 + [_i64, _i64, _i64, _i32, _vp, _sz, _vp]),
    "ss_gated_scan_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32, ctypes.c_int]),
    "ss_gated_state_update": (_i32, [_vp] * 9 + [_i64, _i64, _i32, _vp]),
    "ss_layer_norm_fwd": (_i32, [_vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _i64,
                                 _i64, _i32, _vp]),
    "ss_layer_norm_bwd": (_i32, [_vp, _vp, _i32] + [_vp] * 8 + [_i64, _i64, _i32, _vp, _sz,
                                                                _vp]),
    "ss_layer_norm_bwd_workspace_bytes": (_sz, [_i64, _i64]),
    "ss_causal_conv_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _i64, _i64, _i64,
                                  _i32, _i32, _vp]),
    "ss_causal_conv_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp,
                                  _i64, _i64, _i64, _i32, _i32, _vp, _sz, _vp]),
    "ss_causal_conv_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32, _i32]),
    "ss_causal_conv_update": (_i32, [_vp, _vp, _vp, _vp, ctypes.c_int, _vp, _i64, _i64, _i32,
                                     _i32, _vp]),
    "ss_scan2_bwd": (_i32, [_vp] * 8 + [ctypes.c_int] + [_vp] * 12 + [_i64] * 6
                     + [_i32, _vp, _sz, _vp]),
    "ss_scan2_bwd_workspace_bytes": (_sz, [_i64] * 6 + [_i32]),
    "ss_scan2_state_update": (_i32, [_vp] * 9 + [ctypes.c_int, _vp] + [_i64] * 5 + [_i32, _vp]),
    "ss_scan2_state_update_conv": (_i32, [_vp, _vp, _vp, _i64, _vp, _vp, _i32, _vp, _i64, _vp,
                                          _vp, _vp, _i64, _vp, ctypes.c_int, _vp] + [_i64] * 5
                                   + [_i32, _vp, _sz, _vp]),
    "ss_scan2_state_update_conv_workspace_bytes": (_sz, [_i64] * 5),
    "ss_rms_norm_fwd": (_i32, [_vp] * 4 + [ctypes.c_int, ctypes.c_double, _vp, ctypes.c_float]
                        + [_vp] * 4 + [_i64, _i64, _i32, _vp]),
    "ss_rms_norm_bwd": (_i32, [_vp, _vp, _i32] + [_vp] * 4 + [ctypes.c_int, _vp, ctypes.c_double]
                        + [_vp] * 6 + [_i64, _i64, _i32, _vp, _sz, _vp]),
    "ss_rms_norm_bwd_workspace_bytes": (_sz, [_i64, _i64]),
    "ss_gated_norm_fwd": (_i32, [_vp, _vp, _i64, _vp, ctypes.c_int, ctypes.c_float, _vp, _vp,
                                 _i64, _i64, _i64, _i32, _vp]),
    "ss_gated_norm_bwd": (_i32, [_vp, _vp, _vp, _i64, _vp, _vp, ctypes.c_int, _vp, _vp, _vp,
                                 _i64, _i64, _i64, _i32, _vp, _sz, _vp]),
    "ss_gated_norm_bwd_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "ss_dropout": (_i32, [_vp, _vp, ctypes.c_double, _vp, _i64, _i64, _i32, _vp]),
    "ss_status_string": (ctypes.c_char_p, [_i32]),
    "ss_last_error": (ctypes.c_char_p, []),
    "ss_version": (ctypes.c_int, []),
}

_lib = None


class SSError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded library, with argument types set.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m selective_state_space_36_amd.build`"
                " (or __graft_entry__.build())")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _check(status: int) -> None:
    if status != SS_OK:
        msg = lib().ss_last_error().decode() or lib().ss_status_string(status).decode()
        raise SSError(status, msg)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SS_F32
    if t.dtype == torch.bfloat16:
        return SS_BF16
    raise TypeError(f"io tensors must be float32 or bfloat16, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dev(t: Optional[torch.Tensor], name: str, dtype=None, shape=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def workspace_bytes(batch, seqlen, d_inner, d_state, dtype=torch.bfloat16, nseg=None) -> int:
    code = SS_BF16 if dtype == torch.bfloat16 else SS_F32
    if nseg is None:
        return int(lib().ss_scan_fwd_workspace_bytes(batch, seqlen, d_inner, d_state, code))
    return int(lib().ss_scan_fwd_ex_workspace_bytes(batch, seqlen, d_inner, d_state, code, nseg))


def scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True, h0=None,
             return_last_state=False, out=None, h_last=None, workspace=None, nseg=None,
             zoh_exact=False, stream=None):
    """Prefill selective scan on the GPU (ss_scan_fwd / ss_scan_fwd_ex).

    u, delta, z: (batch, L, d_inner); B, C: (batch, L, d_state); all the same io dtype (float32 or
    bfloat16).  A: (d_inner, d_state) float32; D, delta_bias: (d_inner,) float32; h0:
    (batch, d_inner, d_state) float32.  Returns out (and h_last when return_last_state).
    nseg: None = automatic time split (workspace sized and allocated here unless given), an int
    forces that many segments (ss_scan_fwd_ex).  zoh_exact: exact zero-order-hold input term
    (SS_FLAG_ZOH_EXACT, through ss_scan_fwd_ex).
    """
    batch, L, d_inner = u.shape
    d_state = B.shape[-1]
    code = _dtype_code(u)
    for name, t in (("u", u), ("delta", delta), ("z", z)):
        _dev(t, name, u.dtype, (batch, L, d_inner))
    for name, t in (("B", B), ("C", C)):
        _dev(t, name, u.dtype, (batch, L, d_state))
    _dev(A, "A", torch.float32, (d_inner, d_state))
    _dev(D, "D", torch.float32, (d_inner,))
    _dev(delta_bias, "delta_bias", torch.float32, (d_inner,))
    _dev(h0, "h0", torch.float32, (batch, d_inner, d_state))
    if out is None:
        out = torch.empty_like(u)
    _dev(out, "out", u.dtype, (batch, L, d_inner))
    if return_last_state and h_last is None:
        h_last = torch.empty((batch, d_inner, d_state), dtype=torch.float32, device=u.device)
    _dev(h_last, "h_last", torch.float32, (batch, d_inner, d_state))
    if workspace is None:
        nbytes = workspace_bytes(batch, L, d_inner, d_state, u.dtype, nseg)
        workspace = (torch.empty(nbytes, dtype=torch.uint8, device=u.device) if nbytes
                     else None)
    ws_ptr = _ptr(workspace)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = [_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
            1 if delta_softplus else 0, _ptr(h0), _ptr(h_last), _ptr(out),
            batch, L, d_inner, d_state, code, ws_ptr, ws_len]
    if nseg is None and not zoh_exact:
        _check(lib().ss_scan_fwd(*args, _stream(stream)))
    else:
        flags = SS_FLAG_ZOH_EXACT if zoh_exact else 0
        _check(lib().ss_scan_fwd_ex(*args, int(nseg or 0), flags, _stream(stream)))
    return (out, h_last) if return_last_state else out


def scan_fwd_noalloc(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True,
                     h0=None, out=None, h_last=None, stream=None):
    """Prefill through ss_scan_fwd_noalloc: the library allocates nothing and the time split,
    when used, keeps its carries in the library's static per-GPU scratch.  out (and h_last, if
    wanted) must be given: this call allocates nothing either.  Returns out."""
    batch, L, d_inner = u.shape
    d_state = B.shape[-1]
    code = _dtype_code(u)
    for name, t in (("u", u), ("delta", delta), ("z", z)):
        _dev(t, name, u.dtype, (batch, L, d_inner))
    for name, t in (("B", B), ("C", C)):
        _dev(t, name, u.dtype, (batch, L, d_state))
    _dev(A, "A", torch.float32, (d_inner, d_state))
    _dev(D, "D", torch.float32, (d_inner,))
    _dev(delta_bias, "delta_bias", torch.float32, (d_inner,))
    _dev(h0, "h0", torch.float32, (batch, d_inner, d_state))
    if out is None:
        raise ValueError("scan_fwd_noalloc: out must be given")
    _dev(out, "out", u.dtype, (batch, L, d_inner))
    _dev(h_last, "h_last", torch.float32, (batch, d_inner, d_state))
    _check(lib().ss_scan_fwd_noalloc(
        _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
        1 if delta_softplus else 0, _ptr(h0), _ptr(h_last), _ptr(out), batch, L, d_inner,
        d_state, code, _stream(stream)))
    return out


def scan_fwd_conv(x, conv_weight, conv_bias, delta, A, B, C, D=None, z=None, delta_bias=None,
                  delta_softplus=True, x_prev=None, h0=None, return_last_state=False, out=None,
                  h_last=None, workspace=None, nseg=None, zoh_exact=False, stream=None):
    """Prefill with the fused front end (ss_scan_fwd_conv): u = silu(causal depthwise conv of x).

    x: (batch, L, d_inner) in the io dtype; conv_weight: (d_inner, k) float32, k in 1..4;
    conv_bias: (d_inner,) float32 or None; x_prev: (batch, k-1, d_inner) io dtype or None.  The
    rest as in scan_fwd.
    """
    batch, L, d_inner = x.shape
    d_state = B.shape[-1]
    code = _dtype_code(x)
    k = conv_weight.shape[-1]
    for name, t in (("x", x), ("delta", delta), ("z", z)):
        _dev(t, name, x.dtype, (batch, L, d_inner))
    for name, t in (("B", B), ("C", C)):
        _dev(t, name, x.dtype, (batch, L, d_state))
    _dev(conv_weight, "conv_weight", torch.float32, (d_inner, k))
    _dev(conv_bias, "conv_bias", torch.float32, (d_inner,))
    _dev(x_prev, "x_prev", x.dtype, (batch, k - 1, d_inner))
    _dev(A, "A", torch.float32, (d_inner, d_state))
    _dev(D, "D", torch.float32, (d_inner,))
    _dev(delta_bias, "delta_bias", torch.float32, (d_inner,))
    _dev(h0, "h0", torch.float32, (batch, d_inner, d_state))
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "out", x.dtype, (batch, L, d_inner))
    if return_last_state and h_last is None:
        h_last = torch.empty((batch, d_inner, d_state), dtype=torch.float32, device=x.device)
    _dev(h_last, "h_last", torch.float32, (batch, d_inner, d_state))
    if workspace is None:
        nbytes = workspace_bytes(batch, L, d_inner, d_state, x.dtype, nseg)
        workspace = (torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes
                     else None)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().ss_scan_fwd_conv(
        _ptr(x), _ptr(conv_weight), _ptr(conv_bias), _ptr(x_prev), int(k), _ptr(delta), _ptr(A),
        _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias), 1 if delta_softplus else 0,
        _ptr(h0), _ptr(h_last), _ptr(out), batch, L, d_inner, d_state, code, _ptr(workspace),
        ws_len, int(nseg or 0), SS_FLAG_ZOH_EXACT if zoh_exact else 0, _stream(stream)))
    return (out, h_last) if return_last_state else out


def scan_fwd_states(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True,
                    h0=None, return_last_state=False, out=None, h_last=None, states=None,
                    workspace=None, stream=None):
    """Prefill that also saves the state after every 16-step chunk (ss_scan_fwd_states), for
    scan_bwd(..., states_given=True).  Arguments as for scan_fwd; states: (batch, ceil(L / 16),
    d_inner, d_state) float32 (the states view of bwd_workspace, to hand the workspace to the
    backward) or None (allocated here).  Returns (out, states), or (out, states, h_last) with
    return_last_state."""
    batch, L, d_inner = u.shape
    d_state = B.shape[-1]
    code = _dtype_code(u)
    for name, t in (("u", u), ("delta", delta), ("z", z)):
        _dev(t, name, u.dtype, (batch, L, d_inner))
    for name, t in (("B", B), ("C", C)):
        _dev(t, name, u.dtype, (batch, L, d_state))
    _dev(A, "A", torch.float32, (d_inner, d_state))
    _dev(D, "D", torch.float32, (d_inner,))
    _dev(delta_bias, "delta_bias", torch.float32, (d_inner,))
    _dev(h0, "h0", torch.float32, (batch, d_inner, d_state))
    if out is None:
        out = torch.empty_like(u)
    _dev(out, "out", u.dtype, (batch, L, d_inner))
    if return_last_state and h_last is None:
        h_last = torch.empty((batch, d_inner, d_state), dtype=torch.float32, device=u.device)
    _dev(h_last, "h_last", torch.float32, (batch, d_inner, d_state))
    nct = (L + 15) // 16
    if states is None:
        states = torch.empty((batch, nct, d_inner, d_state), dtype=torch.float32,
                             device=u.device)
    _dev(states, "states", torch.float32, (batch, nct, d_inner, d_state))
    if workspace is None:
        nbytes = workspace_bytes(batch, L, d_inner, d_state, u.dtype, None)
        workspace = (torch.empty(nbytes, dtype=torch.uint8, device=u.device) if nbytes
                     else None)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().ss_scan_fwd_states(
        _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
        1 if delta_softplus else 0, _ptr(h0), _ptr(h_last), _ptr(out), _ptr(states), batch, L,
        d_inner, d_state, code, _ptr(workspace), ws_len, _stream(stream)))
    return (out, states, h_last) if return_last_state else (out, states)


def bwd_workspace(batch, seqlen, d_inner, d_state, dtype=torch.bfloat16, device="cuda"):
    """A workspace for scan_bwd (ss_scan_bwd_workspace_bytes bytes, or None when it needs none)
    and the float32 view of its first part that holds the chunk-end states: give the view to
    scan_fwd_states(states=...) and the workspace to scan_bwd(..., states_given=True)."""
    code = SS_BF16 if dtype == torch.bfloat16 else SS_F32
    nbytes = int(lib().ss_scan_bwd_workspace_bytes(batch, seqlen, d_inner, d_state, code))
    if nbytes == 0:
        return None, None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    nct = (seqlen + 15) // 16
    states = ws[:batch * nct * d_inner * d_state * 4].view(torch.float32).view(
        batch, nct, d_inner, d_state)
    return ws, states


def scan_bwd(u, delta, A, B, C, dout, D=None, z=None, delta_bias=None, delta_softplus=True,
             h0=None, dh_last=None, want_dD=True, want_ddelta_bias=True, want_dh0=True,
             workspace=None, states_given=False, zoh_exact=False, stream=None):
    """Gradients of scan_fwd (ss_scan_bwd) for the upstream gradient dout (same dtype and shape
    as out) and optionally dh_last.  Returns a dict: du, ddelta, dz (io dtype; dz None without
    z), dA, dB, dC (float32), dD, ddelta_bias, dh0 (float32, None when not wanted).
    workspace: uint8 device buffer of ss_scan_bwd_workspace_bytes bytes (allocated here when
    None).  states_given: the workspace already begins with the chunk-end states that
    scan_fwd_states saved for these inputs (SS_FLAG_STATES_GIVEN; see bwd_workspace), and the
    backward skips its own forward pass.  zoh_exact: gradients of the exact zero-order-hold
    input term (SS_FLAG_ZOH_EXACT; not with states_given)."""
    batch, L, d_inner = u.shape
    d_state = B.shape[-1]
    code = _dtype_code(u)
    for name, t in (("u", u), ("delta", delta), ("z", z), ("dout", dout)):
        _dev(t, name, u.dtype, (batch, L, d_inner))
    for name, t in (("B", B), ("C", C)):
        _dev(t, name, u.dtype, (batch, L, d_state))
    _dev(A, "A", torch.float32, (d_inner, d_state))
    _dev(D, "D", torch.float32, (d_inner,))
    _dev(delta_bias, "delta_bias", torch.float32, (d_inner,))
    _dev(h0, "h0", torch.float32, (batch, d_inner, d_state))
    _dev(dh_last, "dh_last", torch.float32, (batch, d_inner, d_state))
    f32 = dict(dtype=torch.float32, device=u.device)
    g = dict(du=torch.empty_like(u), ddelta=torch.empty_like(u),
             dz=torch.empty_like(u) if z is not None else None,
             dA=torch.empty((d_inner, d_state), **f32), dB=torch.empty((batch, L, d_state), **f32),
             dC=torch.empty((batch, L, d_state), **f32),
             dD=torch.empty((d_inner,), **f32) if want_dD else None,
             ddelta_bias=torch.empty((d_inner,), **f32) if want_ddelta_bias else None,
             dh0=torch.empty((batch, d_inner, d_state), **f32) if want_dh0 else None)
    flags = (SS_FLAG_STATES_GIVEN if states_given else 0) | (SS_FLAG_ZOH_EXACT if zoh_exact else 0)
    if workspace is None:
        if states_given:
            raise ValueError("states_given needs the workspace that holds the states")
        workspace, _ = bwd_workspace(batch, L, d_inner, d_state, u.dtype, u.device)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().ss_scan_bwd(
        _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
        1 if delta_softplus else 0, _ptr(h0), _ptr(dout), _ptr(dh_last), _ptr(g["du"]),
        _ptr(g["ddelta"]), _ptr(g["dz"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]),
        _ptr(g["dD"]), _ptr(g["ddelta_bias"]), _ptr(g["dh0"]), batch, L, d_inner, d_state, code,
        _ptr(workspace), ws_len, flags, _stream(stream)))
    return g


def scan2_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, h0=None,
              return_last_state=False, out=None, h_last=None, stream=None):
    """Multi-head scan with a scalar transition per head (ss_scan2_fwd).

    x, z: (batch, L, nheads, headdim); dt: (batch, L, nheads); B, C: (batch, L, ngroups,
    d_state), one io dtype.  A, D, dt_bias: (nheads,) float32.  h0: (batch, nheads, d_state,
    headdim) float32.  Returns out (and h_last when return_last_state).
    """
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(x)
    for name, t in (("x", x), ("z", z)):
        _dev(t, name, x.dtype, (batch, L, H, P))
    _dev(dt, "dt", x.dtype, (batch, L, H))
    for name, t in (("B", B), ("C", C)):
        _dev(t, name, x.dtype, (batch, L, G, N))
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias)):
        _dev(t, name, torch.float32, (H,))
    _dev(h0, "h0", torch.float32, (batch, H, N, P))
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "out", x.dtype, (batch, L, H, P))
    if return_last_state and h_last is None:
        h_last = torch.empty((batch, H, N, P), dtype=torch.float32, device=x.device)
    _dev(h_last, "h_last", torch.float32, (batch, H, N, P))
    _check(lib().ss_scan2_fwd(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                              _ptr(dt_bias), 1 if dt_softplus else 0, _ptr(h0), _ptr(h_last),
                              _ptr(out), batch, L, H, P, G, N, code, _stream(stream)))
    return (out, h_last) if return_last_state else out


def state_update(state, u, delta, A, B, C, D=None, z=None, delta_bias=None,
                 delta_softplus=True, out=None, zoh_exact=False, stream=None):
    """One decode step on the GPU (ss_state_update); `state` is updated in place.

    state: (batch, d_inner, d_state) float32; u, delta, z: (batch, d_inner); B, C:
    (batch, d_state) in the io dtype.  Returns out: (batch, d_inner).
    """
    batch, d_inner, d_state = state.shape
    code = _dtype_code(u)
    _dev(state, "state", torch.float32)
    for name, t in (("u", u), ("delta", delta), ("z", z)):
        _dev(t, name, u.dtype, (batch, d_inner))
    for name, t in (("B", B), ("C", C)):
        _dev(t, name, u.dtype, (batch, d_state))
    _dev(A, "A", torch.float32, (d_inner, d_state))
    _dev(D, "D", torch.float32, (d_inner,))
    _dev(delta_bias, "delta_bias", torch.float32, (d_inner,))
    if out is None:
        out = torch.empty_like(u)
    _dev(out, "out", u.dtype, (batch, d_inner))
    args = [_ptr(state), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
            _ptr(delta_bias), 1 if delta_softplus else 0, _ptr(out), batch, d_inner, d_state, code]
    if zoh_exact:
        _check(lib().ss_state_update_ex(*args, SS_FLAG_ZOH_EXACT, _stream(stream)))
    else:
        _check(lib().ss_state_update(*args, _stream(stream)))
    return out


def state_update_conv(state, conv_state, x, conv_weight, conv_bias, delta, A, B, C, D=None,
                      z=None, delta_bias=None, delta_softplus=True, out=None, zoh_exact=False,
                      stream=None):
    """One decode step with the fused front end (ss_state_update_conv): state (batch, d_inner,
    d_state) float32 and conv_state (batch, k-1, d_inner) io dtype are updated in place; x,
    delta, z: (batch, d_inner); conv_weight (d_inner, k) float32; conv_bias (d_inner,) or None."""
    batch, d_inner, d_state = state.shape
    code = _dtype_code(x)
    k = conv_weight.shape[-1]
    _dev(state, "state", torch.float32)
    _dev(conv_state, "conv_state", x.dtype, (batch, k - 1, d_inner))
    for name, t in (("x", x), ("delta", delta), ("z", z)):
        _dev(t, name, x.dtype, (batch, d_inner))
    for name, t in (("B", B), ("C", C)):
        _dev(t, name, x.dtype, (batch, d_state))
    _dev(conv_weight, "conv_weight", torch.float32, (d_inner, k))
    _dev(conv_bias, "conv_bias", torch.float32, (d_inner,))
    _dev(A, "A", torch.float32, (d_inner, d_state))
    _dev(D, "D", torch.float32, (d_inner,))
    _dev(delta_bias, "delta_bias", torch.float32, (d_inner,))
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "out", x.dtype, (batch, d_inner))
    _check(lib().ss_state_update_conv(
        _ptr(state), _ptr(conv_state), _ptr(x), _ptr(conv_weight), _ptr(conv_bias), int(k),
        _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
        1 if delta_softplus else 0, _ptr(out), batch, d_inner, d_state, code,
        SS_FLAG_ZOH_EXACT if zoh_exact else 0, _stream(stream)))
    return out


# ---------------------------------------------------------------------------------------------
# The recurrent block's operators.  They run on their inputs' device; `stream` (a
# torch.cuda.Stream) is as if the call stood under torch.cuda.stream(stream): outputs and
# workspaces are allocated for it, and the inputs are marked as used on it.

_IO = {torch.float32: SS_F32, torch.bfloat16: SS_BF16}


def _io_code(x) -> int:
    code = _IO.get(x.dtype)
    if code is None:
        raise TypeError(f"io tensors must be float32 or bfloat16, got {x.dtype}")
    return code


def _shape(name, t, ndim):
    if t.dim() != ndim:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {ndim} dimensions")
    return t.shape


def _expect(device, dtype, shape, *named) -> None:
    """Every (name, tensor) pair that is not None: on `device`, contiguous, of dtype and shape."""
    for name, t in named:
        if t is None:
            continue
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _expect_starts(starts, device, shape) -> None:
    if starts is not None:
        if starts.dtype is not torch.bool and starts.dtype is not torch.uint8:
            raise TypeError(f"starts must be bool or uint8, got {starts.dtype}")
        _expect(device, starts.dtype, shape, ("starts", starts))


def _elsewhere(x, stream) -> bool:
    """Whether the call has to be moved: to `stream`, or to x's device when that is not the
    current one.  Raises for a tensor that is not on a GPU."""
    if not x.is_cuda:
        raise ValueError("the tensors must be GPU tensors")
    return stream is not None or x.device.index != torch.cuda.current_device()


def _moved(fn, x, stream, args, kw):
    if stream is None:
        with torch.cuda.device(x.device):
            return fn(*args, **kw)
    if stream.device != x.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {x.device}")
    with torch.cuda.stream(stream):
        res = fn(*args, **kw)
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
    return res


def _scratch(workspace, nbytes, device):
    """(pointer, size, tensor) of the caller's workspace or of one allocated here."""
    if workspace is None:
        if nbytes == 0:
            return None, 0, None
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    else:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# The current stream's handle without a torch.cuda.Stream object around it (0.1 against 2.7 us,
# a quarter of a one-token call).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(device) -> int:
    if _current_raw_stream is not None:
        return _current_raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _gated_fwd(x, r, i, A, r_bias, i_bias, z, starts, h0, out, h_last, states, want_last,
               want_states, workspace):
    code = _io_code(x)
    batch, L, d = shape = _shape("x", x, 3)
    dev = x.device
    f32 = torch.float32
    nct = (L + SS_GATED_CHUNK - 1) // SS_GATED_CHUNK
    _expect(dev, x.dtype, shape, ("x", x), ("r", r), ("i", i), ("z", z), ("out", out))
    _expect(dev, f32, (d,), ("A", A), ("r_bias", r_bias), ("i_bias", i_bias))
    _expect(dev, f32, (batch, d), ("h0", h0), ("h_last", h_last))
    _expect(dev, f32, (batch, nct, d), ("states", states))
    _expect_starts(starts, dev, (batch, L))
    if out is None:
        out = torch.empty_like(x)
    if want_last and h_last is None:
        h_last = A.new_empty((batch, d)) if h0 is None else torch.empty_like(h0)
    if want_states and states is None:
        states = A.new_empty((batch, nct, d))
    l = lib()
    nbytes = l.ss_gated_scan_fwd_workspace_bytes(batch, L, d, code)
    ws, ws_len, keep = _scratch(workspace, nbytes, dev)
    _check(l.ss_gated_scan_fwd(
        x.data_ptr(), r.data_ptr(), i.data_ptr(), A.data_ptr(), _ptr(r_bias), _ptr(i_bias),
        _ptr(z), _ptr(starts), _ptr(h0), _ptr(h_last), out.data_ptr(), _ptr(states), batch, L, d,
        code, ws, ws_len, _raw_stream(x.device)))
    return out, states, h_last


def gated_scan_fwd(x, r, i, A, r_bias=None, i_bias=None, z=None, starts=None, h0=None,
                   return_last_state=False, out=None, h_last=None, workspace=None, stream=None):
    """Gated linear recurrence over a sequence (ss_gated_scan_fwd):

        a_t = exp(A sigmoid(r_t + r_bias)),
        h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t,   out = h (or h silu(z))

    x, r, i, z: (batch, L, d_inner), float32 or bfloat16; A (not above 0), r_bias, i_bias:
    (d_inner,) float32; starts: (batch, L) bool or uint8, true where a new sequence begins in the
    row; h0: (batch, d_inner) float32.  Returns out (and h_last when return_last_state).
    workspace: uint8 device buffer of ss_gated_scan_fwd_workspace_bytes bytes (allocated here
    when None); calls that may overlap need one each."""
    if _elsewhere(x, stream):
        return _moved(gated_scan_fwd, x, stream, (x, r, i, A),
                      dict(r_bias=r_bias, i_bias=i_bias, z=z, starts=starts, h0=h0,
                           return_last_state=return_last_state, out=out, h_last=h_last,
                           workspace=workspace))
    out, _, h_last = _gated_fwd(x, r, i, A, r_bias, i_bias, z, starts, h0, out, h_last, None,
                                return_last_state, False, workspace)
    return (out, h_last) if return_last_state else out


def gated_scan_fwd_states(x, r, i, A, r_bias=None, i_bias=None, z=None, starts=None, h0=None,
                          return_last_state=False, out=None, h_last=None, states=None,
                          workspace=None, stream=None):
    """gated_scan_fwd that also saves the state after every SS_GATED_CHUNK steps, for
    gated_scan_bwd(..., states=states).  states: (batch, ceil(L / SS_GATED_CHUNK), d_inner)
    float32, allocated here when None.  Returns (out, states), or (out, states, h_last) with
    return_last_state."""
    if _elsewhere(x, stream):
        return _moved(gated_scan_fwd_states, x, stream, (x, r, i, A),
                      dict(r_bias=r_bias, i_bias=i_bias, z=z, starts=starts, h0=h0,
                           return_last_state=return_last_state, out=out, h_last=h_last,
                           states=states, workspace=workspace))
    out, states, h_last = _gated_fwd(x, r, i, A, r_bias, i_bias, z, starts, h0, out, h_last,
                                     states, return_last_state, True, workspace)
    return (out, states, h_last) if return_last_state else (out, states)


def gated_scan_bwd(x, r, i, A, dout, r_bias=None, i_bias=None, z=None, starts=None, h0=None,
                   dh_last=None, states=None, want_dbias=True, want_dh0=True, workspace=None,
                   stream=None):
    """Gradients of gated_scan_fwd (ss_gated_scan_bwd) for the upstream gradient dout (shape and
    dtype of out) and optionally dh_last.  Returns a dict: dx, dr, di, dz (io dtype; dz None
    without z), dA, dr_bias, di_bias (float32, the biases' None when not wanted), dh0 (float32,
    None when not wanted).  states: as gated_scan_fwd_states saved them for the same inputs;
    None: recomputed here."""
    if _elsewhere(x, stream):
        return _moved(gated_scan_bwd, x, stream, (x, r, i, A, dout),
                      dict(r_bias=r_bias, i_bias=i_bias, z=z, starts=starts, h0=h0,
                           dh_last=dh_last, states=states, want_dbias=want_dbias,
                           want_dh0=want_dh0, workspace=workspace))
    code = _io_code(x)
    batch, L, d = shape = _shape("x", x, 3)
    dev = x.device
    f32 = torch.float32
    nct = (L + SS_GATED_CHUNK - 1) // SS_GATED_CHUNK
    _expect(dev, x.dtype, shape, ("x", x), ("r", r), ("i", i), ("z", z), ("dout", dout))
    _expect(dev, f32, (d,), ("A", A), ("r_bias", r_bias), ("i_bias", i_bias))
    _expect(dev, f32, (batch, d), ("h0", h0), ("dh_last", dh_last))
    _expect(dev, f32, (batch, nct, d), ("states", states))
    _expect_starts(starts, dev, (batch, L))
    like = torch.empty_like
    g = dict(dx=like(x), dr=like(x), di=like(x), dz=like(x) if z is not None else None,
             dA=like(A), dr_bias=like(A) if want_dbias else None,
             di_bias=like(A) if want_dbias else None,
             dh0=(A.new_empty((batch, d)) if h0 is None else like(h0)) if want_dh0 else None)
    l = lib()
    nbytes = l.ss_gated_scan_bwd_workspace_bytes(batch, L, d, code, states is not None)
    ws, ws_len, keep = _scratch(workspace, nbytes, dev)
    _check(l.ss_gated_scan_bwd(
        x.data_ptr(), r.data_ptr(), i.data_ptr(), A.data_ptr(), _ptr(r_bias), _ptr(i_bias),
        _ptr(z), _ptr(starts), _ptr(h0), dout.data_ptr(), _ptr(dh_last), _ptr(states),
        _ptr(g["dx"]), _ptr(g["dr"]), _ptr(g["di"]), _ptr(g["dz"]), _ptr(g["dA"]),
        _ptr(g["dr_bias"]), _ptr(g["di_bias"]), _ptr(g["dh0"]), batch, L, d, code, ws, ws_len,
        _raw_stream(x.device)))
    return g


def gated_state_update(state, x, r, i, A, r_bias=None, i_bias=None, z=None, out=None,
                       stream=None):
    """One token of the gated linear recurrence (ss_gated_state_update); `state` (batch, d_inner)
    float32 is advanced in place.  x, r, i, z: (batch, d_inner).  Returns out."""
    if _elsewhere(x, stream):
        return _moved(gated_state_update, x, stream, (state, x, r, i, A),
                      dict(r_bias=r_bias, i_bias=i_bias, z=z, out=out))
    code = _io_code(x)
    batch, d = shape = _shape("x", x, 2)
    dev = x.device
    _expect(dev, x.dtype, shape, ("x", x), ("r", r), ("i", i), ("z", z), ("out", out))
    _expect(dev, torch.float32, (d,), ("A", A), ("r_bias", r_bias), ("i_bias", i_bias))
    _expect(dev, torch.float32, shape, ("state", state))
    if out is None:
        out = torch.empty_like(x)
    _check(lib().ss_gated_state_update(
        state.data_ptr(), x.data_ptr(), r.data_ptr(), i.data_ptr(), A.data_ptr(), _ptr(r_bias),
        _ptr(i_bias), _ptr(z), out.data_ptr(), batch, d, code, _raw_stream(x.device)))
    return out


def layer_norm_fwd(x, weight=None, bias=None, residual=None, eps=1e-5, return_sum=None,
                   return_stats=False, out=None, sum_out=None, stream=None):
    """Layer norm over the last axis of x + residual (ss_layer_norm_fwd).

    x: (..., dim) float32 or bfloat16; residual: the same shape, float32 (the residual stream);
    weight, bias: (dim,) float32.  Returns out alone, or a tuple of out, then the float32 sum
    x + residual (return_sum: by default with a residual), then mean and rstd, (...) float32, with
    return_stats (layer_norm_bwd takes them; NaN, being 0 / 0, where dim is 0)."""
    if _elsewhere(x, stream):
        return _moved(layer_norm_fwd, x, stream, (x,),
                      dict(weight=weight, bias=bias, residual=residual, eps=eps,
                           return_sum=return_sum, return_stats=return_stats, out=out,
                           sum_out=sum_out))
    code = _io_code(x)
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    shape, dev, f32 = x.shape, x.device, torch.float32
    dim = shape[-1]
    rows = x.numel() // dim if dim else 0
    if return_sum is None:
        return_sum = residual is not None
    _expect(dev, x.dtype, shape, ("x", x), ("out", out))
    _expect(dev, f32, shape, ("residual", residual), ("sum_out", sum_out))
    _expect(dev, f32, (dim,), ("weight", weight), ("bias", bias))
    if out is None:
        out = torch.empty_like(x)
    if return_sum and sum_out is None:
        sum_out = (torch.empty_like(residual) if residual is not None
                   else torch.empty_like(x, dtype=f32))
    mean = rstd = None
    if return_stats:
        mean = torch.empty(shape[:-1], dtype=f32, device=dev)
        rstd = torch.empty_like(mean)
        if not dim:  # the library writes nothing then
            mean.fill_(float("nan"))
            rstd.fill_(float("nan"))
    _check(lib().ss_layer_norm_fwd(
        x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(bias), eps, out.data_ptr(),
        _ptr(sum_out), _ptr(mean), _ptr(rstd), rows, dim, code, _raw_stream(x.device)))
    res = (out, *((sum_out,) if return_sum else ()), *((mean, rstd) if return_stats else ()))
    return res if len(res) > 1 else out


def layer_norm_bwd(dout, s, weight, mean, rstd, dsum=None, want_dx=True, want_dresidual=False,
                   want_dparams=True, workspace=None, stream=None):
    """Gradients of layer_norm_fwd (ss_layer_norm_bwd) for the upstream gradient dout of out and
    optionally dsum (float32) of the sum.  s: what was normalised, x itself (dout's dtype) or the
    float32 sum; weight: (dim,) float32 or None; mean, rstd: the forward's statistics.  Returns a
    dict: dx (dout's dtype), dresidual (float32), dweight, dbias ((dim,) float32), None where not
    wanted.  dx and dresidual hold the same gradient, in the dtypes of x and of residual."""
    if _elsewhere(dout, stream):
        return _moved(layer_norm_bwd, dout, stream, (dout, s, weight, mean, rstd),
                      dict(dsum=dsum, want_dx=want_dx, want_dresidual=want_dresidual,
                           want_dparams=want_dparams, workspace=workspace))
    code = _io_code(dout)
    if dout.dim() < 1:
        raise ValueError("dout needs at least one dimension")
    shape, dev, f32 = dout.shape, dout.device, torch.float32
    dim = shape[-1]
    rows = dout.numel() // dim if dim else 0
    s_dtype = f32 if s.dtype is f32 else dout.dtype
    _expect(dev, dout.dtype, shape, ("dout", dout))
    _expect(dev, s_dtype, shape, ("s", s))
    _expect(dev, f32, shape, ("dsum", dsum))
    _expect(dev, f32, (dim,), ("weight", weight))
    _expect(dev, f32, shape[:-1], ("mean", mean), ("rstd", rstd))
    g = dict(dx=torch.empty_like(dout) if want_dx else None,
             dresidual=torch.empty_like(dout, dtype=f32) if want_dresidual else None,
             dweight=mean.new_empty((dim,)) if want_dparams else None,
             dbias=mean.new_empty((dim,)) if want_dparams else None)
    l = lib()
    nbytes = l.ss_layer_norm_bwd_workspace_bytes(rows, dim) if want_dparams else 0
    ws, ws_len, keep = _scratch(workspace, nbytes, dev)
    _check(l.ss_layer_norm_bwd(
        dout.data_ptr(), s.data_ptr(), _IO[s_dtype], _ptr(weight), mean.data_ptr(),
        rstd.data_ptr(), _ptr(dsum), _ptr(g["dx"]), _ptr(g["dresidual"]), _ptr(g["dweight"]),
        _ptr(g["dbias"]), rows, dim, code, ws, ws_len, _raw_stream(dev)))
    return g


def _conv_sizes(x, weight, x_prev, starts, bias, ndim):
    shape = _shape("x", x, ndim)
    d, dev = shape[-1], x.device
    k = _shape("weight", weight, 2)[1]
    _expect(dev, torch.float32, (d, k), ("weight", weight))
    _expect(dev, torch.float32, (d,), ("bias", bias))
    _expect(dev, x.dtype, (shape[0], max(k - 1, 0), d), ("x_prev", x_prev))
    _expect_starts(starts, dev, shape[:2])
    return shape, k


def causal_conv_fwd(x, weight, bias=None, x_prev=None, starts=None, silu=True, out=None,
                    stream=None):
    """Causal depthwise convolution (ss_causal_conv_fwd), the front end of scan_fwd_conv as an
    operator of its own: out = silu(bias + sum_j weight[:, j] x_{t-(k-1)+j}), or the bare sum with
    silu=False.  x: (batch, L, d_inner) float32 or bfloat16; weight: (d_inner, k) float32, k in
    1..4; bias: (d_inner,) float32; x_prev: (batch, k-1, d_inner) io dtype, the inputs before the
    first step; starts: (batch, L) bool or uint8, true where a new sequence begins in the row."""
    if _elsewhere(x, stream):
        return _moved(causal_conv_fwd, x, stream, (x, weight),
                      dict(bias=bias, x_prev=x_prev, starts=starts, silu=silu, out=out))
    code = _io_code(x)
    shape, k = _conv_sizes(x, weight, x_prev, starts, bias, 3)
    _expect(x.device, x.dtype, shape, ("x", x), ("out", out))
    if out is None:
        out = torch.empty_like(x)
    _check(lib().ss_causal_conv_fwd(
        x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(x_prev), _ptr(starts),
        1 if silu else 0, out.data_ptr(), *shape, k, code, _raw_stream(x.device)))
    return out


def causal_conv_bwd(x, weight, dout, bias=None, x_prev=None, starts=None, silu=True,
                    want_dbias=True, workspace=None, stream=None):
    """Gradients of causal_conv_fwd (ss_causal_conv_bwd).  Returns a dict: dx (io dtype), dweight
    ((d_inner, k) float32), dbias ((d_inner,) float32, None when not wanted), dx_prev (io dtype,
    None without x_prev)."""
    if _elsewhere(x, stream):
        return _moved(causal_conv_bwd, x, stream, (x, weight, dout),
                      dict(bias=bias, x_prev=x_prev, starts=starts, silu=silu,
                           want_dbias=want_dbias, workspace=workspace))
    code = _io_code(x)
    shape, k = _conv_sizes(x, weight, x_prev, starts, bias, 3)
    dev = x.device
    _expect(dev, x.dtype, shape, ("x", x), ("dout", dout))
    like = torch.empty_like
    g = dict(dx=like(x), dweight=like(weight),
             dbias=weight.new_empty(shape[2:]) if want_dbias else None,
             dx_prev=like(x_prev) if x_prev is not None else None)
    l = lib()
    nbytes = l.ss_causal_conv_bwd_workspace_bytes(*shape, k, code)
    ws, ws_len, keep = _scratch(workspace, nbytes, dev)
    _check(l.ss_causal_conv_bwd(
        x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(x_prev), _ptr(starts),
        1 if silu else 0, dout.data_ptr(), _ptr(g["dx"]), _ptr(g["dweight"]), _ptr(g["dbias"]),
        _ptr(g["dx_prev"]), *shape, k, code, ws, ws_len, _raw_stream(x.device)))
    return g


def causal_conv_update(conv_state, x, weight, bias=None, silu=True, out=None, stream=None):
    """One token of the convolution (ss_causal_conv_update): conv_state (batch, k-1, d_inner) io
    dtype is shifted in place, x: (batch, d_inner).  Returns out."""
    if _elsewhere(x, stream):
        return _moved(causal_conv_update, x, stream, (conv_state, x, weight),
                      dict(bias=bias, silu=silu, out=out))
    code = _io_code(x)
    shape, k = _conv_sizes(x, weight, None, None, bias, 2)
    _expect(x.device, x.dtype, shape, ("x", x), ("out", out))
    if out is None:
        out = torch.empty_like(x)
    _expect(x.device, x.dtype, (shape[0], max(k - 1, 0), shape[1]), ("conv_state", conv_state))
    _check(lib().ss_causal_conv_update(
        conv_state.data_ptr(), x.data_ptr(), weight.data_ptr(), _ptr(bias), 1 if silu else 0,
        out.data_ptr(), *shape, k, code, _raw_stream(x.device)))
    return out


# ---------------------------------------------------------------------------------------------
# The block around the multi-head scan.  Streams, devices and workspaces as above.


def _row_stride(name, t, device, dtype, shape) -> int:
    """Elements from one row of the (rows, width) tensor t to the next; its rows may be parts of
    longer ones."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    rows, width = shape
    if width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    if rows <= 1:
        return width
    if t.stride(0) < width:
        raise ValueError(f"{name} must have rows that do not overlap")
    return t.stride(0)


def _rng(p, rng, device):
    """The pointer to the generator's (seed, offset), or None where nothing is dropped."""
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p={p} is not a probability")
    if rng is None:
        if p:
            raise ValueError("dropout needs rng, the generator's seed and offset")
        return None
    _expect(device, torch.int64, (2,), ("rng", rng))
    return rng.data_ptr()


def scan2_bwd(x, dt, A, B, C, dout, D=None, z=None, dt_bias=None, dt_softplus=True, h0=None,
              dh_last=None, want_dD=True, want_ddt_bias=True, want_dh0=True, workspace=None,
              stream=None):
    """Gradients of scan2_fwd (ss_scan2_bwd) for the upstream gradient dout (shape and dtype of
    out) and optionally dh_last ((batch, nheads, d_state, headdim) float32).  Returns a dict: dx,
    ddt, dz, dB, dC (io dtype, the shapes of x, dt, z, B, C; dz None without z), dA, dD, ddt_bias
    ((nheads,) float32) and dh0 (float32), None where not wanted.  workspace: uint8 device buffer of
    ss_scan2_bwd_workspace_bytes bytes (allocated here when None); calls that may overlap need one
    each."""
    if _elsewhere(x, stream):
        return _moved(scan2_bwd, x, stream, (x, dt, A, B, C, dout),
                      dict(D=D, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus, h0=h0,
                           dh_last=dh_last, want_dD=want_dD, want_ddt_bias=want_ddt_bias,
                           want_dh0=want_dh0, workspace=workspace))
    code = _io_code(x)
    batch, L, H, P = shape = _shape("x", x, 4)
    G, N = _shape("B", B, 4)[2:]
    dev, f32 = x.device, torch.float32
    _expect(dev, x.dtype, shape, ("x", x), ("z", z), ("dout", dout))
    _expect(dev, x.dtype, (batch, L, H), ("dt", dt))
    _expect(dev, x.dtype, (batch, L, G, N), ("B", B), ("C", C))
    _expect(dev, f32, (H,), ("A", A), ("D", D), ("dt_bias", dt_bias))
    _expect(dev, f32, (batch, H, N, P), ("h0", h0), ("dh_last", dh_last))
    like = torch.empty_like
    g = dict(dx=like(x), ddt=like(dt), dz=like(x) if z is not None else None, dA=like(A),
             dB=like(B), dC=like(C), dD=like(A) if want_dD else None,
             ddt_bias=like(A) if want_ddt_bias else None,
             dh0=A.new_empty((batch, H, N, P)) if want_dh0 else None)
    if not H:  # the library writes nothing then
        g["dB"].zero_()
        g["dC"].zero_()
    l = lib()
    nbytes = l.ss_scan2_bwd_workspace_bytes(batch, L, H, P, G, N, code)
    ws, ws_len, keep = _scratch(workspace, nbytes, dev)
    _check(l.ss_scan2_bwd(
        x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z),
        _ptr(dt_bias), 1 if dt_softplus else 0, _ptr(h0), dout.data_ptr(), _ptr(dh_last),
        _ptr(g["dx"]), _ptr(g["ddt"]), _ptr(g["dz"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]),
        _ptr(g["dD"]), _ptr(g["ddt_bias"]), _ptr(g["dh0"]), batch, L, H, P, G, N, code, ws,
        ws_len, _raw_stream(dev)))
    return g


def scan2_state_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True,
                       out=None, stream=None):
    """One token of the multi-head scan (ss_scan2_state_update); `state` (batch, nheads, d_state,
    headdim) float32, scan2_fwd's h_last, is advanced in place.  x, z: (batch, nheads, headdim);
    dt: (batch, nheads); B, C: (batch, ngroups, d_state), one io dtype.  Returns out."""
    if _elsewhere(x, stream):
        return _moved(scan2_state_update, x, stream, (state, x, dt, A, B, C),
                      dict(D=D, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus, out=out))
    code = _io_code(x)
    batch, H, P = shape = _shape("x", x, 3)
    G, N = _shape("B", B, 3)[1:]
    dev, f32 = x.device, torch.float32
    _expect(dev, x.dtype, shape, ("x", x), ("z", z), ("out", out))
    _expect(dev, x.dtype, (batch, H), ("dt", dt))
    _expect(dev, x.dtype, (batch, G, N), ("B", B), ("C", C))
    _expect(dev, f32, (H,), ("A", A), ("D", D), ("dt_bias", dt_bias))
    _expect(dev, f32, (batch, H, N, P), ("state", state))
    if out is None:
        out = torch.empty_like(x)
    _check(lib().ss_scan2_state_update(
        state.data_ptr(), x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(),
        _ptr(D), _ptr(z), _ptr(dt_bias), 1 if dt_softplus else 0, out.data_ptr(), batch, H, P, G,
        N, code, _raw_stream(dev)))
    return out


def scan2_state_update_conv(state, conv_state, xbc, conv_weight, conv_bias, dt, A, ngroups=1,
                            D=None, z=None, dt_bias=None, dt_softplus=True, out=None,
                            workspace=None, stream=None):
    """One token through the convolution and the multi-head scan (ss_scan2_state_update_conv):
    state (batch, nheads, d_state, headdim) float32 and conv_state (batch, k-1, width) io dtype are
    advanced in place.  xbc: (batch, width) with width = nheads headdim + 2 ngroups d_state, the
    columns [x | B | C] before the convolution; conv_weight: (width, k) float32, k in 1..4;
    conv_bias: (width,) float32 or None; dt: (batch, nheads); z: (batch, nheads headdim) or None.
    The rows of xbc, dt and z may be parts of one projection's.  Without heads or channels
    nothing is advanced.  Returns out (batch, nheads, headdim)."""
    if _elsewhere(xbc, stream):
        return _moved(scan2_state_update_conv, xbc, stream,
                      (state, conv_state, xbc, conv_weight, conv_bias, dt, A),
                      dict(ngroups=ngroups, D=D, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus,
                           out=out, workspace=workspace))
    code = _io_code(xbc)
    batch, H, N, P = _shape("state", state, 4)
    k = _shape("conv_weight", conv_weight, 2)[1]
    width = H * P + 2 * ngroups * N
    dev, f32, io = xbc.device, torch.float32, xbc.dtype
    _expect(dev, f32, state.shape, ("state", state))
    _expect(dev, f32, (width, k), ("conv_weight", conv_weight))
    _expect(dev, f32, (width,), ("conv_bias", conv_bias))
    _expect(dev, io, (batch, max(k - 1, 0), width), ("conv_state", conv_state))
    _expect(dev, f32, (H,), ("A", A), ("D", D), ("dt_bias", dt_bias))
    _expect(dev, io, (batch, H, P), ("out", out))
    xs = _row_stride("xbc", xbc, dev, io, (batch, width))
    ds = _row_stride("dt", dt, dev, io, (batch, H))
    zs = _row_stride("z", z, dev, io, (batch, H * P)) if z is not None else 0
    if out is None:
        out = xbc.new_empty((batch, H, P))
    # (4 bytes a column: what ss_scan2_state_update_conv_workspace_bytes says, without the call)
    ws, ws_len, keep = _scratch(workspace, 4 * batch * width, dev)
    _check(lib().ss_scan2_state_update_conv(
        state.data_ptr(), _ptr(conv_state), xbc.data_ptr(), xs, conv_weight.data_ptr(),
        _ptr(conv_bias), k, dt.data_ptr(), ds, A.data_ptr(), _ptr(D), _ptr(z), zs, _ptr(dt_bias),
        1 if dt_softplus else 0, out.data_ptr(), batch, H, P, ngroups, N, code, ws, ws_len,
        _raw_stream(dev)))
    return out


def rms_norm_fwd(x, weight=None, residual=None, scale=None, norm_branch=False, p=0.0, rng=None,
                 eps=1e-5, return_sum=None, return_stats=False, out=None, sum_out=None,
                 stream=None):
    """RMS norm over the last axis of s = residual + dropout(scale * x) (ss_rms_norm_fwd); with
    norm_branch x is RMS-normalised first (the norm behind a block; scale is its weight then).

    x: (..., dim) float32 or bfloat16; residual: the same shape, float32 (the residual stream);
    weight, scale: (dim,) float32; p, rng: as in dropout.  Returns out alone, or a tuple of out,
    then the float32 sum s (return_sum: by default wherever s is not x), then with return_stats the
    statistics rstd and branch_rstd, (...) float32, that rms_norm_bwd takes (branch_rstd None
    without norm_branch; NaN, being 0 / 0, where dim is 0)."""
    if _elsewhere(x, stream):
        return _moved(rms_norm_fwd, x, stream, (x,),
                      dict(weight=weight, residual=residual, scale=scale, norm_branch=norm_branch,
                           p=p, rng=rng, eps=eps, return_sum=return_sum,
                           return_stats=return_stats, out=out, sum_out=sum_out))
    code = _io_code(x)
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    shape, dev, f32 = x.shape, x.device, torch.float32
    dim = shape[-1]
    rows = x.numel() // dim if dim else 0
    if return_sum is None:
        return_sum = residual is not None or scale is not None or norm_branch or p > 0
    _expect(dev, x.dtype, shape, ("x", x), ("out", out))
    _expect(dev, f32, shape, ("residual", residual), ("sum_out", sum_out))
    _expect(dev, f32, (dim,), ("weight", weight), ("scale", scale))
    seed = _rng(p, rng, dev)
    if out is None:
        out = torch.empty_like(x)
    if return_sum and sum_out is None:
        sum_out = torch.empty_like(x, dtype=f32)
    rstd = branch_rstd = None
    if return_stats:
        rstd = torch.empty(shape[:-1], dtype=f32, device=dev)
        branch_rstd = torch.empty_like(rstd) if norm_branch else None
        if not dim:  # the library writes nothing then
            for t in (rstd, branch_rstd):
                if t is not None:
                    t.fill_(float("nan"))
    _check(lib().ss_rms_norm_fwd(
        x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(scale), 1 if norm_branch else 0, p, seed,
        eps, out.data_ptr(), _ptr(sum_out), _ptr(rstd), _ptr(branch_rstd), rows, dim, code,
        _raw_stream(dev)))
    res = (out, *((sum_out,) if return_sum else ()),
           *((rstd, branch_rstd) if return_stats else ()))
    return res if len(res) > 1 else out


def rms_norm_bwd(dout, s, weight, rstd, x=None, scale=None, norm_branch=False, branch_rstd=None,
                 p=0.0, rng=None, dsum=None, want_dx=True, want_dresidual=False,
                 want_dparams=True, workspace=None, stream=None):
    """Gradients of rms_norm_fwd (ss_rms_norm_bwd) for the upstream gradient dout of out and
    optionally dsum (float32) of the sum.  s: what was normalised, the float32 sum or, where the
    forward had none, x itself; rstd, branch_rstd: the forward's statistics; weight, scale,
    norm_branch, p, rng: as the forward's; x: as the forward's, needed with scale or norm_branch.
    Returns a dict: dx (dout's dtype), dresidual (float32), dweight, dscale ((dim,) float32; dscale
    None without scale), None where not wanted."""
    if _elsewhere(dout, stream):
        return _moved(rms_norm_bwd, dout, stream, (dout, s, weight, rstd),
                      dict(x=x, scale=scale, norm_branch=norm_branch, branch_rstd=branch_rstd, p=p,
                           rng=rng, dsum=dsum, want_dx=want_dx, want_dresidual=want_dresidual,
                           want_dparams=want_dparams, workspace=workspace))
    code = _io_code(dout)
    if dout.dim() < 1:
        raise ValueError("dout needs at least one dimension")
    shape, dev, f32 = dout.shape, dout.device, torch.float32
    dim = shape[-1]
    rows = dout.numel() // dim if dim else 0
    s_dtype = f32 if s.dtype is f32 else dout.dtype
    _expect(dev, dout.dtype, shape, ("dout", dout), ("x", x))
    _expect(dev, s_dtype, shape, ("s", s))
    _expect(dev, f32, shape, ("dsum", dsum))
    _expect(dev, f32, (dim,), ("weight", weight), ("scale", scale))
    _expect(dev, f32, shape[:-1], ("rstd", rstd), ("branch_rstd", branch_rstd))
    want_dscale = want_dparams and scale is not None
    if x is None and (want_dscale or norm_branch):
        raise ValueError("x is needed for the gradient of scale and with norm_branch")
    if norm_branch and branch_rstd is None:
        raise ValueError("branch_rstd is needed with norm_branch")
    seed = _rng(p, rng, dev)
    g = dict(dx=torch.empty_like(dout) if want_dx else None,
             dresidual=torch.empty_like(dout, dtype=f32) if want_dresidual else None,
             dweight=rstd.new_empty((dim,)) if want_dparams else None,
             dscale=rstd.new_empty((dim,)) if want_dscale else None)
    l = lib()
    nbytes = l.ss_rms_norm_bwd_workspace_bytes(rows, dim) if want_dparams else 0
    ws, ws_len, keep = _scratch(workspace, nbytes, dev)
    _check(l.ss_rms_norm_bwd(
        dout.data_ptr(), s.data_ptr(), _IO[s_dtype], _ptr(weight), rstd.data_ptr(), _ptr(x),
        _ptr(scale), 1 if norm_branch else 0, _ptr(branch_rstd), p, seed, _ptr(dsum),
        _ptr(g["dx"]), _ptr(g["dresidual"]), _ptr(g["dweight"]), _ptr(g["dscale"]), rows, dim,
        code, ws, ws_len, _raw_stream(dev)))
    return g


def _gated_norm_z(x, z):
    """(rows, dim, z's row stride): z has x's shape, its rows may be parts of longer ones."""
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    dim = x.shape[-1]
    rows = x.numel() // dim if dim else 0
    if z is None:
        return rows, dim, 0
    if z.shape != x.shape:
        raise ValueError(f"z has shape {tuple(z.shape)}, expected {tuple(x.shape)}")
    if rows and z.dim() != 2:
        # the leading axes have to be one run of rows
        try:
            z = z.view(rows, dim)
        except RuntimeError:
            raise ValueError("z must have equally spaced rows") from None
    return rows, dim, _row_stride("z", z, x.device, x.dtype, (rows, dim)) if rows else dim


def gated_norm_fwd(x, z=None, weight=None, groups=1, gate_first=True, eps=1e-5,
                   return_stats=False, out=None, stream=None):
    """RMS norm with an output gate, over each of `groups` runs of the last axis
    (ss_gated_norm_fwd): norm(x silu(z)) * weight, or norm(x) * weight * silu(z) with
    gate_first=False; without z no gate.  x: (..., dim) float32 or bfloat16; z: the same shape (its
    rows may be parts of longer ones); weight: (dim,) float32.  Returns out, or (out, rstd) with
    return_stats: the statistics, (..., groups) float32, that gated_norm_bwd takes."""
    if _elsewhere(x, stream):
        return _moved(gated_norm_fwd, x, stream, (x,),
                      dict(z=z, weight=weight, groups=groups, gate_first=gate_first, eps=eps,
                           return_stats=return_stats, out=out))
    code = _io_code(x)
    rows, dim, zs = _gated_norm_z(x, z)
    dev = x.device
    _expect(dev, x.dtype, x.shape, ("x", x), ("out", out))
    _expect(dev, torch.float32, (dim,), ("weight", weight))
    if out is None:
        out = torch.empty_like(x)
    rstd = None
    if return_stats:
        rstd = torch.empty((*x.shape[:-1], groups), dtype=torch.float32, device=dev)
        if not dim:  # the library writes nothing then
            rstd.fill_(float("nan"))
    _check(lib().ss_gated_norm_fwd(
        x.data_ptr(), _ptr(z), zs, _ptr(weight), 1 if gate_first else 0, eps, out.data_ptr(),
        _ptr(rstd), rows, dim, groups, code, _raw_stream(dev)))
    return (out, rstd) if return_stats else out


def gated_norm_bwd(dout, x, z, weight, rstd, groups=1, gate_first=True, want_dweight=True,
                   workspace=None, stream=None):
    """Gradients of gated_norm_fwd (ss_gated_norm_bwd); x, z, weight, groups and gate_first as the
    forward's, rstd its statistics.  Returns a dict: dx, dz (io dtype; dz None without z) and
    dweight ((dim,) float32, None when not wanted)."""
    if _elsewhere(dout, stream):
        return _moved(gated_norm_bwd, dout, stream, (dout, x, z, weight, rstd),
                      dict(groups=groups, gate_first=gate_first, want_dweight=want_dweight,
                           workspace=workspace))
    code = _io_code(dout)
    rows, dim, zs = _gated_norm_z(x, z)
    dev = dout.device
    _expect(dev, dout.dtype, dout.shape, ("dout", dout), ("x", x))
    _expect(dev, torch.float32, (dim,), ("weight", weight))
    _expect(dev, torch.float32, (*dout.shape[:-1], groups), ("rstd", rstd))
    g = dict(dx=torch.empty_like(dout), dz=torch.empty_like(dout) if z is not None else None,
             dweight=rstd.new_empty((dim,)) if want_dweight else None)
    l = lib()
    nbytes = l.ss_gated_norm_bwd_workspace_bytes(rows, dim, groups) if want_dweight else 0
    ws, ws_len, keep = _scratch(workspace, nbytes, dev)
    _check(l.ss_gated_norm_bwd(
        dout.data_ptr(), x.data_ptr(), _ptr(z), zs, _ptr(weight), rstd.data_ptr(),
        1 if gate_first else 0, _ptr(g["dx"]), _ptr(g["dz"]), _ptr(g["dweight"]), rows, dim,
        groups, code, ws, ws_len, _raw_stream(dev)))
    return g


def dropout(x, p, rng, out=None, stream=None):
    """Dropout with a mask that is never stored (ss_dropout): out is x / (1 - p) where the element
    is kept and 0 where it is dropped, each with probability p (rounded to a multiple of 2^-16).
    x: (..., dim) float32 or bfloat16; rng: (2,) int64 on the device, a seed and an offset, read
    when the kernel runs.  The mask depends on rng and the element's place alone: the gradient is
    dropout(dout, p, rng), and rms_norm_fwd with the same rng drops the same elements.  Advance the
    offset between draws that are to be independent."""
    if _elsewhere(x, stream):
        return _moved(dropout, x, stream, (x, p, rng), dict(out=out))
    code = _io_code(x)
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    dim = x.shape[-1]
    rows = x.numel() // dim if dim else 0
    _expect(x.device, x.dtype, x.shape, ("x", x), ("out", out))
    if rng is None:
        raise ValueError("dropout needs rng, the generator's seed and offset")
    seed = _rng(p, rng, x.device)
    if out is None:
        out = torch.empty_like(x)
    _check(lib().ss_dropout(x.data_ptr(), out.data_ptr(), p, seed, rows, dim, code,
                            _raw_stream(x.device)))
    return out
