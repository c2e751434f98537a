"""Timed cases of the recurrent block's operators: the gated linear recurrence, the layer norm
with its residual add, and the causal depthwise convolution, each as a user's program calls it
(prefill, training step, one token).

``run`` computes either the plain torch form (``own`` false: elementary float32 operations) or the
framework's kernels (``own`` true).  ``exact`` is the definition in float64, written apart from
both.  Sizes: the layers of ``selective_state_space_36_amd.workloads`` (d_inner 1536 and 5120,
sequences of 2048 and 4096 tokens, 128 decode rows), their model width 2560, and odd generic ones.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one user's next token: nothing but latency
        dict(name="recurrence token b1", op="gated_step", batch=1, d=5120, dtype="bf16", gate=True),
        # a full serving batch's next token
        dict(name="recurrence token b128", op="gated_step", batch=128, d=5120, dtype="bf16",
             gate=True),
        # prefill of a small model's layer, output gate fused
        dict(name="recurrence prefill 8x2048x1536", op="gated_fwd", batch=8, seqlen=2048, d=1536,
             dtype="bf16", gate=True, packed=False, h0=False),
        # one very long document, resumed from a state: few channels, so time has to be split
        dict(name="recurrence prefill 1x262144", op="gated_fwd", batch=1, seqlen=1 << 18, d=1536,
             dtype="bf16", gate=False, packed=False, h0=True),
        # training step of a large layer on packed sequences
        dict(name="recurrence train 4x4096x5120", op="gated_train", batch=4, seqlen=4096, d=5120,
             dtype="bf16", gate=True, packed=True, h0=False),
        # float32 training with odd sizes, carried state in and its gradient out
        dict(name="recurrence train f32 odd", op="gated_train", batch=3, seqlen=1111, d=1027,
             dtype="f32", gate=False, packed=False, h0=True),
        # the norm before a block for one token
        dict(name="norm one row", op="norm_fwd", rows=1, dim=2560, dtype="bf16", residual=True),
        # the norm of a training step: residual stream in, gradients out
        dict(name="norm train 16384x2560", op="norm_train", rows=16384, dim=2560, dtype="bf16",
             residual=True),
        # float32, odd width, no residual
        dict(name="norm train f32 odd", op="norm_train", rows=1001, dim=1027, dtype="f32",
             residual=False),
        # the convolution's window for a serving batch's next token
        dict(name="conv token b128", op="conv_step", batch=128, d=5120, k=4, dtype="bf16",
             silu=True),
        # prefill with odd sizes in float32, resumed from a window
        dict(name="conv prefill f32 odd", op="conv_fwd", batch=3, seqlen=777, d=1537, k=3,
             dtype="f32", silu=False, packed=False, prev=True),
        # training step of a large layer on packed sequences
        dict(name="conv train 4x4096x5120", op="conv_train", batch=4, seqlen=4096, d=5120, k=4,
             dtype="bf16", silu=True, packed=True, prev=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_step", "gated_fwd", "gated_fwd", "gated_train", "gated_train",
                     "norm_fwd", "norm_train", "conv_step", "conv_fwd", "conv_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    d = _log(rng, 64, 6144)
    if rng.random() < 0.6:
        d = max(64, d // 64 * 64)
    if op == "gated_step":
        return dict(op=op, batch=_log(rng, 1, 256), d=d, dtype=dtype, gate=flip())
    if op == "conv_step":
        return dict(op=op, batch=_log(rng, 1, 256), d=d, k=rng.randint(2, 4), dtype=dtype,
                    silu=flip())
    if op in ("norm_fwd", "norm_train"):
        return dict(op=op, rows=_log(rng, 1, 16384), dim=d, dtype=dtype, residual=flip())
    batch = _log(rng, 1, 8)
    if op == "gated_fwd":
        seqlen = min(_log(rng, 1, 1 << 17), (1 << 26) // (batch * d) + 1)
        return dict(op=op, batch=batch, seqlen=seqlen, d=d, dtype=dtype, gate=flip(),
                    packed=flip(), h0=flip())
    seqlen = min(_log(rng, 1, 8192), (1 << 26) // (batch * d) + 1)
    if op == "gated_train":
        return dict(op=op, batch=batch, seqlen=seqlen, d=d, dtype=dtype, gate=flip(),
                    packed=flip(), h0=flip())
    return dict(op=op, batch=batch, seqlen=seqlen, d=d, k=rng.randint(2, 4), dtype=dtype,
                silu=flip(), packed=flip(), prev=flip())


# ---------------------------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
                .mul_(scale).to(dtype))

    def starts(batch, seqlen):
        # packed sequences of a few hundred tokens on average
        return torch.rand((batch, seqlen), generator=g, device="cuda") < 1.0 / 300.0

    op, s = case["op"], {"case": case}
    if op.startswith("gated"):
        d, batch = case["d"], case["batch"]
        # decays of 0.9 to 0.999 a step at a gate of 1/8: A = 8 log(u)
        u = torch.rand((d,), generator=g, device="cuda") * 0.099 + 0.9
        s.update(A=8.0 * torch.log(u), r_bias=normal(d, scale=0.5), i_bias=normal(d, scale=0.5))
        lead = (batch,) if op == "gated_step" else (batch, case["seqlen"])
        for n in ("x", "r", "i"):
            s[n] = normal(*lead, d, dtype=dt)
        s["z"] = normal(*lead, d, dtype=dt) if case["gate"] else None
        if op == "gated_step":
            s["state"] = normal(batch, d)
            return s
        s["starts"] = starts(*lead) if case["packed"] else None
        s["h0"] = normal(batch, d) if case["h0"] else None
        if op == "gated_train":
            s["dout"] = normal(*lead, d, dtype=dt)
            s["dh_last"] = normal(batch, d) if case["h0"] else None
    elif op.startswith("norm"):
        rows, dim = case["rows"], case["dim"]
        s.update(x=normal(rows, dim, dtype=dt), weight=1.0 + normal(dim, scale=0.1),
                 bias=normal(dim, scale=0.1),
                 residual=normal(rows, dim, scale=3.0) if case["residual"] else None)
        if op == "norm_train":
            s["dout"] = normal(rows, dim, dtype=dt)
            s["dsum"] = normal(rows, dim) if case["residual"] else None
    else:
        d, batch, k = case["d"], case["batch"], case["k"]
        s.update(weight=normal(d, k, scale=0.5), bias=normal(d, scale=0.2))
        if op == "conv_step":
            s.update(x=normal(batch, d, dtype=dt), conv_state=normal(batch, k - 1, d, dtype=dt))
            return s
        lead = (batch, case["seqlen"])
        s["x"] = normal(*lead, d, dtype=dt)
        s["x_prev"] = normal(batch, k - 1, d, dtype=dt) if case["prev"] else None
        s["starts"] = starts(*lead) if case["packed"] else None
        if op == "conv_train":
            s["dout"] = normal(*lead, d, dtype=dt)
    return s


# ---------------------------------------------------------------------------------------------
# the plain form: elementary torch operations in float32


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 by doubling the span each round; overwrites a and b."""
    span = 1
    while span < a.shape[1]:
        more = a[:, span:] * b[:, :-span]
        b[:, span:] += more
        a[:, span:] = a[:, span:] * a[:, :-span]
        span *= 2
    return b


def _gates(s):
    rg = torch.sigmoid(s["r"].float() + s["r_bias"])
    ig = torch.sigmoid(s["i"].float() + s["i_bias"])
    l = s["A"] * rg
    return rg, ig, torch.exp(l), torch.sqrt(-torch.expm1(2.0 * l))


def _gated_fwd_plain(s):
    rg, ig, a, root = _gates(s)
    x = s["x"].float()
    b = root * ig * x
    keep = a if s["starts"] is None else torch.where(s["starts"][..., None], 0.0, a)
    if s["h0"] is not None:
        b[:, 0] += keep[:, 0] * s["h0"]
    h = _scan(keep.clone(), b)
    out = h
    if s["z"] is not None:
        z = s["z"].float()
        out = h * (z * torch.sigmoid(z))
    return out.to(s["x"].dtype), h, (rg, ig, a, root, x, keep)


def _gated_bwd_plain(s, h, saved):
    rg, ig, a, root, x, keep = saved
    io = s["x"].dtype
    g = s["dout"].float()
    dz = None
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        dz = (g * h * (sg * (1.0 + z * (1.0 - sg)))).to(io)
        g = g * (z * sg)
    else:
        g = g.clone()
    if s["dh_last"] is not None:
        g[:, -1] += s["dh_last"]
    # lam_t = g_t + a_{t+1} lam_{t+1}: the same scan on the reversed sequence
    back = torch.zeros_like(keep)
    back[:, 1:] = keep[:, 1:].flip(1)
    lam = _scan(back, g.flip(1)).flip(1)
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat([first, h[:, :-1]], dim=1)
    if s["starts"] is not None:
        before = torch.where(s["starts"][..., None], 0.0, before)
    slope = torch.where(root > 0, a * a / root, 0.0)
    dl = lam * (a * before - ig * x * slope)
    dr = dl * s["A"] * rg * (1.0 - rg)
    di = lam * root * x * ig * (1.0 - ig)
    return dict(dx=(lam * root * ig).to(io), dr=dr.to(io), di=di.to(io), dz=dz,
                dA=(dl * rg).sum((0, 1)), dr_bias=dr.sum((0, 1)), di_bias=di.sum((0, 1)),
                dh0=keep[:, 0] * lam[:, 0])


def _gated_step_plain(s):
    rg, ig, a, root = _gates(s)
    s["state"].copy_(a * s["state"] + root * ig * s["x"].float())
    out = s["state"]
    if s["z"] is not None:
        z = s["z"].float()
        out = out * (z * torch.sigmoid(z))
    return out.to(s["x"].dtype), s["state"]


EPS = 1e-5


def _norm_fwd_plain(s):
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"]
    c = v - v.mean(1, keepdim=True)
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    hat = c * rstd
    return (hat * s["weight"] + s["bias"]).to(s["x"].dtype), v, hat, rstd


def _norm_bwd_plain(s, hat, rstd):
    dy = s["dout"].float()
    w = dy * s["weight"]
    ds = rstd * (w - w.mean(1, keepdim=True) - hat * (w * hat).mean(1, keepdim=True))
    if s["dsum"] is not None:
        ds = ds + s["dsum"]
    return dict(dx=ds.to(s["x"].dtype), dresidual=ds if s["residual"] is not None else None,
                dweight=(dy * hat).sum(0), dbias=dy.sum(0))


def _taps(s):
    """The k shifted copies of the padded x, zero where a tap would cross a start, and k masks."""
    x, k = s["x"].float(), s["weight"].shape[1]
    batch, seqlen, d = x.shape
    prev = x.new_zeros(batch, k - 1, d) if s["x_prev"] is None else s["x_prev"].float()
    pad = torch.cat([prev, x], dim=1)
    masks, taps = [], []
    seq = None if s["starts"] is None else torch.cumsum(s["starts"].to(torch.int32), 1)
    for j in range(k):
        lag = k - 1 - j
        tap, mask = pad[:, j:j + seqlen], None
        if seq is not None:
            then = torch.cat([seq.new_zeros(batch, lag), seq[:, :seqlen - lag]], 1)[:, :seqlen]
            mask = (then == seq)[..., None]
            tap = torch.where(mask, tap, 0.0)
        taps.append(tap)
        masks.append(mask)
    return taps, masks


def _conv_fwd_plain(s):
    taps, masks = _taps(s)
    p = s["bias"].expand_as(taps[0])
    for j, tap in enumerate(taps):
        p = p + s["weight"][:, j] * tap
    out = p * torch.sigmoid(p) if s["case"]["silu"] else p
    return out.to(s["x"].dtype), p, taps, masks


def _conv_bwd_plain(s, p, taps, masks):
    g, k, seqlen = s["dout"].float(), s["weight"].shape[1], s["x"].shape[1]
    if s["case"]["silu"]:
        sg = torch.sigmoid(p)
        g = g * (sg * (1.0 + p * (1.0 - sg)))
    dpad = torch.zeros((p.shape[0], seqlen + k - 1, p.shape[2]), device=p.device)
    for j in range(k):
        m = g if masks[j] is None else torch.where(masks[j], g, 0.0)
        dpad[:, j:j + seqlen] += m * s["weight"][:, j]
    return dict(dx=dpad[:, k - 1:].to(s["x"].dtype),
                dx_prev=dpad[:, :k - 1].to(s["x"].dtype) if s["x_prev"] is not None else None,
                dweight=torch.stack([(g * tap).sum((0, 1)) for tap in taps], 1),
                dbias=g.sum((0, 1)))


def _conv_step_plain(s):
    window = torch.cat([s["conv_state"], s["x"][:, None]], 1)
    p = s["bias"] + (window.float() * s["weight"].t()).sum(1)
    s["conv_state"].copy_(window[:, 1:])
    out = p * torch.sigmoid(p) if s["case"]["silu"] else p
    return out.to(s["x"].dtype), s["conv_state"]


def _plain(s):
    op = s["case"]["op"]
    if op == "gated_step":
        out, state = _gated_step_plain(s)
        return dict(out=out, state=state)
    if op == "gated_fwd":
        out, h, _ = _gated_fwd_plain(s)
        return dict(out=out, h_last=h[:, -1])
    if op == "gated_train":
        out, h, saved = _gated_fwd_plain(s)
        return dict(out=out, h_last=h[:, -1], **_gated_bwd_plain(s, h, saved))
    if op == "norm_fwd":
        out, v, _, _ = _norm_fwd_plain(s)
        return dict(out=out, sum=v if s["residual"] is not None else None)
    if op == "norm_train":
        out, v, hat, rstd = _norm_fwd_plain(s)
        return dict(out=out, sum=v if s["residual"] is not None else None,
                    **_norm_bwd_plain(s, hat, rstd))
    if op == "conv_step":
        out, state = _conv_step_plain(s)
        return dict(out=out, conv_state=state)
    out, p, taps, masks = _conv_fwd_plain(s)
    if op == "conv_fwd":
        return dict(out=out)
    return dict(out=out, **_conv_bwd_plain(s, p, taps, masks))


# ---------------------------------------------------------------------------------------------
# the framework's calls


def _own(s):
    from selective_state_space_36_amd import ops

    op = s["case"]["op"]
    if op == "gated_step":
        out = ops.gated_state_update(s["state"], s["x"], s["r"], s["i"], s["A"],
                                     r_bias=s["r_bias"], i_bias=s["i_bias"], z=s["z"])
        return dict(out=out, state=s["state"])
    if op.startswith("gated"):
        args = (s["x"], s["r"], s["i"], s["A"])
        kw = dict(r_bias=s["r_bias"], i_bias=s["i_bias"], z=s["z"], starts=s["starts"],
                  h0=s["h0"])
        if op == "gated_fwd":
            out, h_last = ops.gated_scan_fwd(*args, **kw, return_last_state=True)
            return dict(out=out, h_last=h_last)
        out, states, h_last = ops.gated_scan_fwd_states(*args, **kw, return_last_state=True)
        grads = ops.gated_scan_bwd(*args, s["dout"], **kw, dh_last=s["dh_last"], states=states)
        return dict(out=out, h_last=h_last, **grads)
    if op == "norm_fwd":
        r = ops.layer_norm_fwd(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
        out, total = r if s["residual"] is not None else (r, None)
        return dict(out=out, sum=total)
    if op == "norm_train":
        r = ops.layer_norm_fwd(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS,
                               return_stats=True)
        out, total, mean, rstd = r if s["residual"] is not None else (r[0], None, *r[1:])
        grads = ops.layer_norm_bwd(s["dout"], s["x"] if total is None else total, s["weight"],
                                   mean, rstd, dsum=s["dsum"],
                                   want_dresidual=s["residual"] is not None)
        return dict(out=out, sum=total, **grads)
    if op == "conv_step":
        out = ops.causal_conv_update(s["conv_state"], s["x"], s["weight"], s["bias"],
                                     silu=s["case"]["silu"])
        return dict(out=out, conv_state=s["conv_state"])
    kw = dict(x_prev=s["x_prev"], starts=s["starts"], silu=s["case"]["silu"])
    out = ops.causal_conv_fwd(s["x"], s["weight"], s["bias"], **kw)
    if op == "conv_fwd":
        return dict(out=out)
    return dict(out=out, **ops.causal_conv_bwd(s["x"], s["weight"], s["dout"], s["bias"], **kw))


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        n, res = case["rows"] * case["dim"], case["residual"]
        fwd = n * (2 * es + (8 if res else 0)) + 8 * case["dim"]
        if op == "norm_fwd":
            return dict(bytes=fwd, flops=9 * n)
        bwd = n * (es + (4 if res else es) + (4 if res else 0) + es + (4 if res else 0))
        return dict(bytes=fwd + bwd + 12 * case["dim"], flops=24 * n)
    n = case["batch"] * case["d"] * case.get("seqlen", 1)
    if op == "gated_step":
        return dict(bytes=n * (es * (5 if case["gate"] else 4) + 8) + 12 * case["d"],
                    flops=25 * n)
    if op == "conv_step":
        k = case["k"]
        return dict(bytes=n * es * (2 + 2 * (k - 1)) + 4 * (k + 1) * case["d"],
                    flops=(2 * k + 6) * n)
    if op.startswith("conv"):
        taps = 2 * case["k"] + 6
        if op == "conv_fwd":
            return dict(bytes=n * es * 2, flops=taps * n)
        return dict(bytes=n * es * 5, flops=4 * taps * n)
    fwd = n * es * (5 if case["gate"] else 4)
    if op == "gated_fwd":
        return dict(bytes=fwd, flops=25 * n)
    return dict(bytes=fwd + n * es * (9 if case["gate"] else 7), flops=90 * n)


# ---------------------------------------------------------------------------------------------
# the definition in float64


def _sig64(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _conv64(s, case):
    """(out, pre-activation) step by step: a ring of the last k inputs, emptied at a start."""
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    batch, seqlen, d = x.shape
    k = w.shape[1]
    window = [x.new_zeros(batch, d)] * (k - 1)
    if s["x_prev"] is not None:
        window = list(s["x_prev"].double().unbind(1))
    pre = torch.empty_like(x)
    for t in range(seqlen):
        if s["starts"] is not None:
            fresh = s["starts"][:, t, None]
            window = [v.masked_fill(fresh, 0.0) for v in window]
        window = window + [x[:, t]]
        p = b
        for j in range(k):
            p = p + w[:, j] * window[j]
        pre[:, t] = p
        window = window[1:]
    return pre


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = {n: v.double() for n, v in s.items()
           if isinstance(v, torch.Tensor) and v.is_floating_point()}

    if op.startswith("norm"):
        v = f64["x"] + (f64["residual"] if case["residual"] else 0.0)
        n = v.shape[1]
        mu = v.sum(1) / n
        var = ((v - mu[:, None]) ** 2).sum(1) / n
        xh = (v - mu[:, None]) / torch.sqrt(var + EPS)[:, None]
        r = dict(out=xh * f64["weight"] + f64["bias"], sum=v if case["residual"] else None)
        if op == "norm_train":
            dy = f64["dout"]
            dxh = dy * f64["weight"]
            # through the two row sums: the centre and the scale
            ds = (n * dxh - dxh.sum(1)[:, None] - xh * (dxh * xh).sum(1)[:, None]) \
                / (n * torch.sqrt(var + EPS)[:, None])
            if case["residual"]:
                ds = ds + f64["dsum"]
            r.update(dx=ds, dresidual=ds if case["residual"] else None,
                     dweight=(dy * xh).sum(0), dbias=dy.sum(0))
        return r

    if op == "conv_step":
        w, window = f64["weight"], torch.cat([f64["conv_state"], f64["x"][:, None]], 1)
        p = f64["bias"] + sum(w[:, j] * window[:, j] for j in range(w.shape[1]))
        return dict(out=p * _sig64(p) if case["silu"] else p, conv_state=window[:, 1:])

    if op.startswith("conv"):
        pre = _conv64(s, case)
        r = dict(out=pre * _sig64(pre) if case["silu"] else pre)
        if op == "conv_train":
            g = f64["dout"]
            if case["silu"]:
                q = _sig64(pre)
                g = g * q * (1.0 + pre * (1.0 - q))
            x, w = f64["x"], f64["weight"]
            batch, seqlen, d = x.shape
            k = w.shape[1]
            prev = f64["x_prev"] if case["prev"] else x.new_zeros(batch, k - 1, d)
            dx, dprev = torch.zeros_like(x), torch.zeros_like(prev)
            dw, idx = torch.zeros_like(w), torch.arange(seqlen, device=x.device)
            last = torch.full((batch, seqlen), -(1 << 30), device=x.device)
            if s["starts"] is not None:   # the latest start at or before each step
                last = torch.where(s["starts"], idx, last).cummax(1).values
            for j in range(k):
                lag = k - 1 - j
                reach = ((idx - lag) >= last)[..., None].double()   # tap in the same sequence
                gm = g * reach
                n = min(lag, seqlen)
                if seqlen > lag:
                    dx[:, :seqlen - lag] += w[:, j] * gm[:, lag:]
                    dw[:, j] += (gm[:, lag:] * x[:, :seqlen - lag]).sum((0, 1))
                if n:
                    dprev[:, j:j + n] += w[:, j] * gm[:, :n]
                    dw[:, j] += (gm[:, :n] * prev[:, j:j + n]).sum((0, 1))
            r.update(dx=dx, dx_prev=dprev if case["prev"] else None, dweight=dw,
                     dbias=g.sum((0, 1)))
        return r

    rg, ig = _sig64(f64["r"] + f64["r_bias"]), _sig64(f64["i"] + f64["i_bias"])
    a = torch.exp(f64["A"] * rg)
    root = torch.sqrt(torch.clamp(1.0 - a * a, min=0.0))
    silu = lambda z: z * _sig64(z)  # noqa: E731
    if op == "gated_step":
        h = a * f64["state"] + root * ig * f64["x"]
        return dict(out=h * silu(f64["z"]) if case["gate"] else h, state=h)

    keep = a if s["starts"] is None else a * (~s["starts"])[..., None].double()
    b = root * ig * f64["x"]
    seqlen = a.shape[1]
    first = f64["h0"] if case["h0"] else torch.zeros_like(b[:, 0])
    h = torch.empty_like(b)
    state, rows = first, list(zip(keep.unbind(1), b.unbind(1), h.unbind(1)))
    for at, bt, ht in rows:      # one step of the definition after the other
        torch.addcmul(bt, at, state, out=ht)
        state = ht
    r = dict(out=h * silu(f64["z"]) if case["gate"] else h, h_last=h[:, -1])
    if op == "gated_fwd":
        return r
    g, dz = f64["dout"], None
    if case["gate"]:
        z, q = f64["z"], _sig64(f64["z"])
        dz = g * h * (q + z * q * (1.0 - q))
        g = g * z * q
    lam = torch.empty_like(g)
    carry = f64["dh_last"] if case["h0"] else torch.zeros_like(g[:, 0])
    for t in range(seqlen - 1, -1, -1):
        lam[:, t] = g[:, t] + carry
        carry = keep[:, t] * lam[:, t]
    dl = torch.empty_like(g)
    dl[:, 0] = lam[:, 0] * keep[:, 0] * first
    dl[:, 1:] = lam[:, 1:] * keep[:, 1:] * h[:, :-1]
    dl -= lam * ig * f64["x"] * a * a / root
    dr = dl * f64["A"] * rg * (1.0 - rg)
    di = lam * root * f64["x"] * ig * (1.0 - ig)
    r.update(dx=lam * root * ig, dr=dr, di=di, dz=dz, dA=(dl * rg).sum((0, 1)),
             dr_bias=dr.sum((0, 1)), di_bias=di.sum((0, 1)), dh0=carry)
    return r
