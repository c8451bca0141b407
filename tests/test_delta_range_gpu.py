"""gated_delta_rule on numbers of very different size within one call: no token loses to one that it does not depend
on, and a state keeps its precision through what has decayed.

Bounds, relative to what the recurrence itself adds up (delta_ref.delta's size m: for each column |q| times the lengths
of what S's column consists of, each part as far as it has decayed): an output is off by u |o| for its rounding and
2^-10 m, as for calls of like numbers (test_delta_gpu); a state's column, in the norm, by 2^-18 of its length."""

from __future__ import annotations

import random

import pytest

import delta_ref as ref
import tree_ref as tr
from test_delta_gpu import BF16, F16, Delta, dev, torch  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = {F16: 2.0 ** -7, BF16: 1.0}      # of values and states that are not made large


def made(ns, heads, dtype, g, seed=0, trees=None):
    """Values and states of one size; the state forgets by g a token."""
    d = Delta(ns, *heads, dtype, seed=seed, raw=True, trees=trees)
    d.v, d.state = (d.v.float() * SIZES[dtype]).to(dtype), d.state * SIZES[dtype]
    d.a[:] = g
    d.b[:] = 0.1 + 0.9 * d.b
    return d


def check(d, out, state, columns=slice(None)):
    out, state = out.cpu().double(), state.cpu()
    hk, hv, dk, dv = d.shape
    at = 0
    for b, n in enumerate(d.ns):
        rows = slice(at, at + n)
        at += n
        g, beta = ref.gates(d.a[rows], d.b[rows], d.a_log, d.dt_bias)
        o, size, last = ref.delta(d.q[rows], d.k[rows], d.v[rows], g, beta, d.state[d.index[b]], dk ** -0.5, d.unit,
                                  d.eps, d.trees[b] if d.trees else None)
        off = (out[rows] - o).abs()
        least = 2.0 ** -24 if d.dtype == F16 else 2.0 ** -126
        bound = 1.01 * ref.U[d.dtype] * o.abs() + 2.0 ** -10 * size + least
        bad = ~(off <= bound)
        assert not bad.any(), (b, bad.nonzero()[:4].tolist(), int(bad.sum()), float((off / bound).max()))
        if d.trees:
            assert torch.equal(state[d.index[b]], d.state[d.index[b]])
        else:
            off = (state[d.index[b]].double() - last).norm(dim=1)
            assert (off <= 2.0 ** -18 * last.norm(dim=1)).all(), (b, float((off / last.norm(dim=1)).max()))


def run(d, dev):  # noqa: F811
    check(d, *d.call(dev))


HEADS = [(1, 2, 128, 128), (1, 3, 64, 64)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("power", [10, 13, 17])
@pytest.mark.parametrize("n", [64, 165])
def test_a_state_keeps_its_precision_when_large_parts_have_gone(dev, n, power, heads, dtype):  # noqa: F811
    """One token's values, or the state before the call, 2^power times the rest; gone by the end of the first
    chunk, through decay or in one step."""
    for gone in ("decay", "reset"):
        for large in ("token", "state"):
            d = made([n], heads, dtype, -0.5 if gone == "decay" else -0.01, seed=power)
            if gone == "reset":
                d.a[40] = -60.0
            if large == "token":
                d.v[3] = (d.v[3].float() * 2.0 ** power).to(dtype)
            else:
                d.state *= 2.0 ** power
            run(d, dev)
