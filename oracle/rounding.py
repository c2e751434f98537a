"""float64 values that carry a bound on what a float32 evaluation of the same formula may be off.

TEST INFRASTRUCTURE ONLY.  ``Bounded(v, e)`` holds the exact value v (float64) and e >= 0, a first
order a-priori bound on the error of the value that float32 arithmetic computes: every operation
adds its own rounding (U = 2^-24 relative for +, -, *, fma; two U for a one-ulp hardware exp2, log2,
rcp, sqrt) to the errors that its operands bring.  Reordering a sum or splitting a product changes
the order of the roundings but not their number by more than the factor the caller states.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -126      # results below the smallest normal number may be flushed to zero


class Bounded:
    __array_ufunc__ = None

    def __init__(self, v, e=None):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.zeros_like(self.v) if e is None else np.broadcast_to(e, self.v.shape)

    @staticmethod
    def of(x):
        return x if isinstance(x, Bounded) else Bounded(x)

    def _round(self, v, e):
        return Bounded(v, e + U * (np.abs(v) + e) + TINY)

    def __add__(self, o):
        o = Bounded.of(o)
        return self._round(self.v + o.v, self.e + o.e)

    __radd__ = __add__

    def __neg__(self):
        return Bounded(-self.v, self.e)

    def __sub__(self, o):
        return self + (-Bounded.of(o))

    def __rsub__(self, o):
        return Bounded.of(o) + (-self)

    def __mul__(self, o):
        o = Bounded.of(o)
        return self._round(self.v * o.v,
                           np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e)

    __rmul__ = __mul__

    def __getitem__(self, k):
        return Bounded(self.v[k], self.e[k])

    @property
    def shape(self):
        return self.v.shape

    def sum(self, axis, depth):
        """Sum with at most `depth` roundings on the way of any term."""
        return Bounded(self.v.sum(axis), self.e.sum(axis)
                       + depth * U * (np.abs(self.v) + self.e).sum(axis))


def stack(items, axis):
    return Bounded(np.stack([i.v for i in items], axis), np.stack([i.e for i in items], axis))


def where(cond, a, b):
    a, b = Bounded.of(a), Bounded.of(b)
    return Bounded(np.where(cond, a.v, b.v), np.where(cond, a.e, b.e))


def exp(x):
    """exp2(x log2 e): the product rounds (and the constant is rounded), exp2 is off by one ulp."""
    v = np.exp(x.v)
    return Bounded(v, v * np.expm1(x.e + 2 * U * np.abs(x.v)) + 2 * U * v + TINY)


def rcp(x):
    v = 1.0 / x.v
    return Bounded(v, np.abs(v) * (x.e / np.maximum(np.abs(x.v) - x.e, TINY) + 2 * U) + TINY)


def sqrt(x):
    v = np.sqrt(np.maximum(x.v, 0.0))
    return Bounded(v, np.sqrt(np.maximum(x.v, 0.0) + x.e) - v + 2 * U * v + TINY ** 0.5)


def sigmoid(x):
    with np.errstate(over="ignore"):
        e = exp(-x)
        big = e.v > 1e37                      # exp2 overflows: 1 / inf = 0
        s = rcp(Bounded(1.0) + where(big, 1.0, e))
        v = 1.0 / (1.0 + e.v)
    return where(big, Bounded(v, v + TINY), Bounded(v, s.e))


def one_minus_square(w, a):
    """-expm1(w) = 1 - a^2 for a = e^(w/2): a series for w > -1/4 (six roundings, all of terms
    that keep their sign at most 1/8 of the sum apart), elsewhere fma(-a, a, 1)."""
    v = -np.expm1(w.v)
    series = w.e * np.exp(w.v) + 6 * U * v + TINY
    square = 2 * a.v * a.e + a.e ** 2 + U * v
    near = np.abs(w.v + 0.25) < 1e-4          # either branch
    return Bounded(v, np.where(near, np.maximum(series, square),
                               np.where(w.v > -0.25, series, square)))


def half_step(dtype):
    """Relative rounding of a float32 value to the io dtype: half a step."""
    return {"f32": 0.0, "bf16": 2.0 ** -8}[dtype]
