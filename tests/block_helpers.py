"""Helpers of the recurrent block's GPU tests: inputs as torch tensors with their exact float64
values, and the comparison with a Bounded reference."""
from __future__ import annotations

import numpy as np
import torch

from oracle.rounding import half_step

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def gpu(x, io="f32", offset=0):
    """numpy -> (GPU tensor in io dtype, its exact float64 values).  offset > 0: the tensor is
    contiguous but starts that many elements into its allocation."""
    if x is None:
        return None, None
    t = torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(DTYPES[io])
    back = t.double().numpy()
    if not offset:
        return t.cuda(), back
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    view = buf[offset:].view(t.shape)
    view.copy_(t)
    return view, back


def starts_gpu(starts, dtype=torch.bool):
    return None if starts is None else torch.from_numpy(starts).to(dtype).cuda()


def draw_starts(rng, batch, L, mean=9):
    s = rng.random((batch, L)) < 1.0 / mean
    s[0, 0] = True
    return s


def check(got, want, io, what, factor=1.0):
    """got (GPU tensor) against a Bounded: its float32 bound times `factor` (the kernel's order of
    operations rounds at most that many times as often), then half a step of the io dtype."""
    assert got is not None, what
    g = got.detach().double().cpu().numpy()
    assert g.shape == want.v.shape, (what, g.shape, want.v.shape)
    e = factor * want.e
    e = e + half_step(io) * (np.abs(want.v) + e)
    err = np.abs(g - want.v)
    bad = ~(err <= e)
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(bad, err / (e + 1e-300), -1)), err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; worst at "
                             f"{tuple(int(v) for v in k)}: got {g[k]!r}, want {want.v[k]!r} "
                             f"+- {e[k]:.3e}")


class Guarded:
    """An output buffer between two runs of marker bytes that the kernel has to leave alone."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.pad = 512
        self.raw = torch.full((n + 2 * self.pad,), 0xA5, dtype=torch.uint8, device="cuda")
        self.n = n
        self.t = self.raw[self.pad:self.pad + n].view(dtype).view(shape)

    def intact(self):
        return bool((self.raw[:self.pad] == 0xA5).all()) and \
            bool((self.raw[self.pad + self.n:] == 0xA5).all())
