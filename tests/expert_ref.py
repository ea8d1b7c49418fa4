"""The experts' operators in 64 bits (numpy), and bounds on how far an fp32
computation rounded once may be from them.

Products of 16-bit (and 8-bit) numbers are exact in fp32 or rounded once, and
every addition of a partial sum is off by at most one unit in its last place
(2^-23 of it: a matrix unit may cut instead of rounding), so a sum of K terms
is within (K + 1) 2^-23 of the sum of the terms' magnitudes.  The store adds
half a step of its type."""
from __future__ import annotations

import numpy as np

from .layer_ref import store_bound

ULP = 2.0 ** -23


def experts(offsets, cap):
    """(rank, expert, first row, end) of every expert, offsets taken into the buffer."""
    for d, ends in enumerate(np.asarray(offsets)):
        for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
            lo = min(max(int(lo), 0), cap)
            yield d, i, lo, min(max(int(hi), lo), cap)


def product(rows, weight, offsets, out, transposed, dt):
    """-> the outputs and their bounds (0 where out keeps what it holds)."""
    want, bound = out.copy(), np.zeros_like(out)
    for d, i, lo, hi in experts(offsets, rows.shape[1]):
        x, w = rows[d, lo:hi], weight[d, i].T if transposed else weight[d, i]
        want[d, lo:hi] = x @ w
        bound[d, lo:hi] = (x.shape[1] + 1) * ULP * (np.abs(x) @ np.abs(w)) + store_bound(want[d, lo:hi], dt)
    return want, bound


def weight_grad(dout, rows, offsets, shape, transposed, dt):
    want, bound = np.zeros(shape), np.zeros(shape)
    for d, i, lo, hi in experts(offsets, rows.shape[1]):
        a, b = (dout[d, lo:hi], rows[d, lo:hi]) if transposed else (rows[d, lo:hi], dout[d, lo:hi])
        want[d, i] = a.T @ b
        bound[d, i] = (hi - lo + 1) * ULP * (np.abs(a).T @ np.abs(b))
    return want, bound + store_bound(want, dt)
