"""gated_delta_rule in the forms that calls of many sequences and heads take: value heads of one key head prepared
together (two, three or four, from 512 workgroups on), and 64 columns of a head a workgroup (where 32 would be more
than 256).  Bounds as in test_delta_gpu; for 9 to 16 tokens, which go token by token as fewer do, twice its 2^-19."""

from __future__ import annotations

import random

import pytest

import delta_ref as ref
import tree_ref as tr
from test_delta_gpu import BF16, F16, Delta, dev, torch  # noqa: F401
from test_delta_range_gpu import check, made

pytestmark = pytest.mark.gpu

# together: 4, 2, 3 value heads (by value heads / key heads); with 64 sequences of up to eight chunks
MANY = [(1, 4, 128, 64), (1, 2, 64, 128), (1, 3, 64, 64), (1, 3, 128, 128), (2, 4, 64, 64), (1, 4, 64, 192)]


def lengths(rng):
    """64 sequences: one of eight chunks, most shorter than one, around a chunk's end, and none."""
    ns = [500] + [rng.choice([1, 2, 7, 15, 16, 17, 30, 63, 64, 65]) for _ in range(61)] + [130, 0]
    rng.shuffle(ns)
    return ns


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", MANY)
def test_many_sequences(dev, dtype, heads):  # noqa: F811
    ns = lengths(random.Random(heads[3]))
    fresh = {b for b in range(0, 64, 5) if ns[b]}
    d = Delta(ns, *heads, dtype, seed=heads[1], fresh=tuple(fresh))
    d.check(*d.call(dev))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", [(1, 4, 128, 64), (1, 2, 64, 128)])
def test_many_sequences_with_large_values(dev, dtype, heads):  # noqa: F811
    """Several chunks, at any place of a workgroup's columns, go token by token beside others that do not."""
    rng = random.Random(1)
    ns = lengths(rng)
    d = made(ns, heads, dtype, -0.05, seed=2)
    for _ in range(12):
        i, h, c = rng.randrange(sum(ns)), rng.randrange(heads[1]), rng.randrange(heads[3])
        d.v[i, h, c] = (d.v[i, h, c].float() * 2.0 ** (20 if dtype == F16 else 40)).to(dtype)
    d.a[sum(ns) // 2] = -90.0
    keep = [b for b, n in enumerate(ns) if n]
    out, state = d.call(dev)
    d.ns, d.index = [ns[b] for b in keep], [d.index[b] for b in keep]
    check(d, out, state)


def test_many_sequences_nan_stays_where_it_is(dev):  # noqa: F811
    ns = lengths(random.Random(3))
    d = Delta(ns, 1, 4, 128, 64, BF16, seed=4)
    want, state_want = d.call(dev)
    b = ns.index(500)
    at = sum(ns[:b])
    d.v[at + 100, 2, 33] = float("nan")
    out, state = d.call(dev)
    hit, lost = torch.zeros_like(want, dtype=torch.bool), torch.zeros_like(state, dtype=torch.bool)
    hit[at + 100:at + 500, 2, 33] = True
    lost[d.index[b], 2, :, 33] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.isnan(out[hit]).all()
    assert torch.equal(state[~lost], state_want[~lost]) and torch.isnan(state[lost]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n", [9, 13, 16])
def test_up_to_16_tokens_are_fp32(dev, n, dtype):  # noqa: F811
    heads = (2, 4, 128, 128)
    d = Delta([n, 1, n - 1], *heads, dtype, seed=n)
    out, _ = d.call(dev)
    at = 0
    for b, c in enumerate(d.ns):
        rows = slice(at, at + c)
        at += c
        g, beta = ref.gates(d.a[rows], d.b[rows], d.a_log, d.dt_bias)
        o, size, _ = ref.delta(d.q[rows], d.k[rows], d.v[rows], g, beta, d.state[d.index[b]], 128 ** -0.5, True, d.eps)
        off = (out[rows].cpu().double() - o).abs()
        assert (off <= 1.01 * ref.U[dtype] * o.abs() + 2.0 ** -18 * size + 2.0 ** -24).all()


@pytest.mark.parametrize("heads", [(2, 4, 128, 128), (1, 3, 64, 64)])
@pytest.mark.parametrize("n", [333, 64])
def test_bf16_outputs_are_hardly_further_off_than_their_rounding(dev, n, heads):  # noqa: F811
    """As a whole, against the exact outputs rounded: what the state, the new rows and the products with queries lose
    for outputs, each an eighth of bfloat16's own rounding, makes the root of 1 + 3/64 of it: less than 1.1."""
    for trees in (None, [tr.random_tree(n, random.Random(n), 2)] if n <= 64 else None):
        d = Delta([n], *heads, BF16, seed=n, trees=trees)
        out, _ = d.call(dev)
        g, beta = ref.gates(d.a, d.b, d.a_log, d.dt_bias)
        o, _, _ = ref.delta(d.q, d.k, d.v, g, beta, d.state[d.index[0]], heads[2] ** -0.5, True, d.eps,
                            trees[0] if trees else None)
        rounding = (o.to(BF16).double() - o).norm()
        assert (out.cpu().double() - o).norm() <= 1.1 * rounding
