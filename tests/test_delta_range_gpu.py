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


def check(d, out, state, steps=0.0):
    out, state = out.cpu().double(), state.cpu()
    hk, hv, dk, dv = d.shape
    at = 0
    for b, n in enumerate(d.ns):
        rows = slice(at, at + n)
        at += n
        g, beta = ref.gates(d.a[rows], d.b[rows], d.a_log, d.dt_bias)
        o, size, last = ref.delta(d.q[rows], d.k[rows], d.v[rows], g, beta, d.state[d.index[b]], dk ** -0.5, d.unit,
                                  d.eps, d.trees[b] if d.trees else None)
        most = torch.finfo(d.dtype).max                # (what lies beyond is infinite there)
        off = (out[rows].clamp(-most, most) - o.clamp(-most, most)).abs()
        least = 2.0 ** -24 if d.dtype == F16 else 2.0 ** -126
        bound = 1.01 * ref.U[d.dtype] * o.abs() + 2.0 ** -10 * size + least
        bad = ~(off <= bound)
        assert not bad.any(), (b, bad.nonzero()[:4].tolist(), int(bad.sum()), float((off / bound).max()))
        if d.trees:
            assert torch.equal(state[d.index[b]], d.state[d.index[b]])
        else:
            off = (state[d.index[b]].double() - last).norm(dim=1)
            assert (off <= 2.0 ** -18 * last.norm(dim=1) + steps).all(), (b, float((off / last.norm(dim=1)).max()))


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


def grow(d, rows, columns, ratio):
    """Values `ratio` times the rest; fp16's as far as it goes, against smaller others."""
    if d.dtype == F16:
        ratio = min(ratio, 2.0 ** 20)
    d.v[rows, :, columns] = (d.v[rows, :, columns].float() * ratio).to(d.dtype)
    assert torch.isfinite(d.v).all()


FEW, EVERY = slice(5, 6), slice(None)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("power", [16, 21, 24, 26, 30, 40])
@pytest.mark.parametrize("columns", [FEW, EVERY], ids=["column", "row"])
def test_no_token_loses_to_a_later_one(dev, columns, power, heads, dtype):  # noqa: F811
    """Large values late in a chunk, early in it, after its first token, before and after a token alone."""
    for rows in (slice(60, 61), slice(10, 40), slice(1, 64), slice(64 + 50, 64 + 52)):
        d = made([64, 150, 17], heads, dtype, -0.02, seed=power)
        grow(d, rows, columns, 2.0 ** power)
        run(d, dev)
    d = made([130], heads, dtype, -0.02, seed=power)
    grow(d, slice(0, 30), columns, 2.0 ** power)
    grow(d, slice(31, 64), columns, 2.0 ** power)
    d.a[30] = d.a[31] = -80.0
    run(d, dev)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("power", [13, 17, 20, 24, 30, 40])
def test_tokens_after_large_ones_that_have_gone(dev, power, heads, dtype):  # noqa: F811
    for columns in (FEW, EVERY):
        for last in (40, 62, 63):
            d = made([64, 90], heads, dtype, -0.02, seed=power)
            grow(d, slice(3, 30), columns, 2.0 ** power)
            d.a[last] = -90.0
            run(d, dev)
        # a token that writes nothing, as large as it may be
        d = made([64, 90], heads, dtype, -0.3, seed=power)
        grow(d, slice(20, 21), columns, 2.0 ** power)
        d.b[20] = 0.0
        run(d, dev)
    d = made([64, 90], heads, dtype, -0.02, seed=power)
    d.state *= 2.0 ** power
    d.a[40] = -90.0
    run(d, dev)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("g", [-0.01, -0.3, -0.7])
def test_what_decays_over_values_of_zero(dev, g, dtype):  # noqa: F811
    """Nothing new is written but what the keys take back of a state that fades: no part of it is lost."""
    for index in (None, [-1]):
        d = made([64], (1, 2, 128, 64), dtype, g, seed=3)
        d.v[3:] = 0
        if index:
            d.v[:3] *= 64
            d.state[:] = 0
        run(d, dev)


@pytest.mark.parametrize("size", [2.0 ** 123, 2.0 ** 99, 2.0 ** -100])
def test_sizes_at_the_ends_of_the_type(dev, size):  # noqa: F811
    d = made([100, 20], (1, 2, 64, 64), BF16, -0.1, seed=1)
    d.v, d.state = (d.v.float() * size).to(BF16), d.state * size
    run(d, dev)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("power", [13, 20, 24, 30, 40])
@pytest.mark.parametrize("columns", [FEW, EVERY], ids=["column", "row"])
def test_no_branch_of_a_tree_loses_to_another(dev, columns, power, heads, dtype):  # noqa: F811
    """Large values on one branch, at the roots, and before drafts that have forgotten them."""
    rng = random.Random(power)
    # two roots side by side; one root with two branches; drafts anyhow; a chain
    trees = [[-1, -1], [-1] + [0 if i < 3 else i - 2 for i in range(1, 40)], tr.random_tree(64, rng, 3), tr.chain(20)]
    ns = [len(t) for t in trees]
    for g, large in ((-0.02, (0, 3, 45, 125)), (-0.02, (1, 2 + 38, 42 + 63)), (-0.5, (2, 42, 106))):
        d = made(ns, heads, dtype, g, seed=power, trees=trees)
        for i in large:
            grow(d, slice(i, i + 1), columns, 2.0 ** power)
        d.a[106 + 10] = -90.0
        run(d, dev)
    d = made(ns, heads, dtype, -0.3, seed=power, trees=trees)
    d.state *= 2.0 ** power
    d.a[2] = d.a[42] = -90.0
    run(d, dev)


@pytest.mark.parametrize("size", [2.0 ** 123, 2.0 ** 99, 2.0 ** -100])
def test_sizes_at_the_ends_of_the_type_in_a_tree(dev, size):  # noqa: F811
    trees = [tr.random_tree(30, random.Random(2), 2), tr.chain(5)]
    d = made([30, 5], (1, 2, 64, 64), BF16, -0.1, seed=1, trees=trees)
    d.v, d.state = (d.v.float() * size).to(BF16), d.state * size
    run(d, dev)


def far(n, heads, dtype, power, trees=None):
    """Raw keys and queries, most of less than unit length; those of tokens 9 and 20 (of one value head's key head)
    2^power times as long, and little written between."""
    d = Delta([n], *heads, dtype, seed=power, raw=True, unit=False, trees=trees)
    d.a[:] = -0.02
    d.b[:] = 0.1 + 0.9 * d.b
    for i in (9, 20):
        d.k[i] = (d.k[i].float() * 2.0 ** power).to(dtype)
        d.q[i] = (d.q[i].float() * 2.0 ** power).to(dtype)
    return d


@pytest.mark.parametrize("n,tree", [(22, False), (40, False), (100, False), (22, True), (40, True)])
@pytest.mark.parametrize("of_state", [0.0, 1.0])
def test_keys_whose_products_leave_fp32(dev, of_state, n, tree):  # noqa: F811
    """Infinite products of keys or queries stay with the tokens that see both: what comes before them, or lies on
    another branch, is right; what the definition makes infinite is not finite here."""
    # token 9 on one branch and 20 on another, if there are branches
    trees = [[-1, -1] + [i - 2 for i in range(2, n)]] if tree else None
    for power in (40, 70, 100):
        d = far(n, (1, 2, 64, 64), BF16, power, trees=trees)
        d.state *= of_state
        out, state = d.call(dev)
        out = out.cpu().double()
        g, beta = ref.gates(d.a, d.b, None, None)
        o, size, last = ref.delta(d.q, d.k, d.v, g, beta, d.state[d.index[0]], 0.125, False, 0.0,
                                  d.trees[0] if d.trees else None)
        off, bound = (out - o).abs(), 1.01 * ref.U[BF16] * o.abs() + 2.0 ** -10 * size
        sees = [any(j in (9, 20) for j in (tr.path(d.trees[0], i) if d.trees else range(i + 1))) for i in range(len(o))]
        free = ~torch.tensor(sees)
        assert free.any() and (off[free] <= bound[free]).all(), power
        small = o.abs().amax((1, 2)) < 1e30
        assert (off[small] <= bound[small]).all(), power
        if d.trees:
            assert torch.equal(state.cpu(), d.state)


@pytest.mark.parametrize("n", [30, 64])
def test_a_key_at_the_end_of_the_type(dev, n):  # noqa: F811
    """Keys with an element of 2^127 are numbers like others."""
    for trees in (None, [tr.chain(n)]):
        d = Delta([n], 1, 2, 64, 64, BF16, seed=1, raw=True, unit=False, trees=trees)
        d.state *= 2.0 ** -130
        d.v = (d.v.float() * 2.0 ** -120).to(BF16)
        d.a[:] = -0.02
        d.b[:] = 2.0 ** -100
        d.k[7] = 0
        d.k[7, :, 3] = 2.0 ** 127
        d.k[8:, :, 3] = 0
        d.q = (d.q.float() * 2.0 ** 60).to(BF16)
        # (fp32 has steps of 2^-149 for this state: eight roundings by half of one, through the key to u, 2^127 beta, and
        # back, 2^127: 2^7)
        check(d, *d.call(dev), steps=2.0 ** 7)


@pytest.mark.parametrize("n", [5, 70])
@pytest.mark.parametrize("tree", [False, True])
def test_unit_length_of_rows_far_below_the_epsilon(dev, tree, n):  # noqa: F811
    """x / sqrt(sum x^2 + eps) of rows so small that eps in their measure leaves fp32: 1000 x, not zero."""
    n = min(n, 64) if tree else n
    d = Delta([n], 1, 2, 64, 64, BF16, seed=3, trees=[tr.chain(n)] if tree else None)
    for x, power in ((d.q, -70), (d.k, -75)):
        x[1::3] = (x[1::3].float() * 2.0 ** power).to(BF16)
        x[2::3] = (x[2::3].float() * 2.0 ** -8).to(BF16)
    run(d, dev)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", HEADS)
def test_keys_of_zeros_count_for_nothing(dev, heads, dtype):  # noqa: F811
    """Such a token writes nothing, whatever its value; sqrt(eps) does not make it the chunk's heaviest row."""
    for ratio in (1.0, 2.0 ** 9):
        d = made([64, 40, 130], heads, dtype, -0.05, seed=2)
        d.k[::7] = 0
        grow(d, slice(0, None, 7), EVERY, ratio)
        run(d, dev)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("power", [10, 20, 30])
def test_tokens_that_write_nothing_beside_large_ones(dev, power, dtype):  # noqa: F811
    """beta 0, or values and states of zero: what their outputs add up is of the tokens before, as far as it is there."""
    rng = random.Random(power)
    trees = [[-1] + [max(0, i - rng.randint(1, 3)) for i in range(1, 60)], tr.random_tree(40, rng, 2)]
    for of_tree in (trees, None):
        for g in (-0.05, -0.6, -2.0):
            d = made([60, 40] if of_tree else [130, 65], (1, 2, 128, 64), dtype, g, seed=power, trees=of_tree)
            grow(d, slice(11, 14), EVERY, 2.0 ** power)
            grow(d, slice(75, 77), FEW, 2.0 ** power)
            d.b[::2] = 0.0
            d.a[20::9] = -20.0
            d.a[5::13] = -5.0
            run(d, dev)
            d.v[1::5] = 0
            d.v[2::5] = 0
            run(d, dev)


@pytest.mark.parametrize("n", [40, 64, 130])
@pytest.mark.parametrize("tree", [False, True])
def test_raw_keys_of_very_different_lengths(dev, tree, n):  # noqa: F811
    """Long keys whose tokens write nothing, and short ones whose tokens do."""
    n = min(n, 64) if tree else n
    for power in (12, 24, 40):
        d = Delta([n], 1, 2, 64, 64, BF16, seed=power, raw=True, unit=False, trees=[tr.chain(n)] if tree else None)
        d.a[:] = -0.02
        d.state[:] = 0
        d.v[::2] = 0
        d.k[1::2] = (d.k[1::2].float() * 2.0 ** -power).to(BF16)
        d.k[::2, :, ::2], d.k[1::2, :, 1::2] = 0, 0        # (of no common channel: nothing is taken back)
        check(d, *d.call(dev))


@pytest.mark.parametrize("tree", [False, True])
def test_replayed_from_a_graph_with_large_values_and_without(dev, tree):  # noqa: F811
    """What goes token by token is decided on the device, at each replay anew."""
    import int4_weight_only_w4a16_amd as w4
    rng = random.Random(4)
    trees = [tr.random_tree(n, rng, 2) for n in (50, 64)] if tree else None
    every = []
    for large in (False, True):
        d = made([50, 64] if tree else [70, 130], (1, 2, 64, 64), BF16, -0.05, seed=3, trees=trees)
        if large:
            grow(d, slice(7, 9), FEW, 2.0 ** 35)
            grow(d, slice(100, 101), EVERY, 2.0 ** 35)
        args = d.args(dev)
        out = w4.gated_delta_rule(**{**args, "state": args["state"].clone()})
        after = args["state"].clone()
        w4.gated_delta_rule(**{**args, "state": after})
        every.append((args, out, after))
    live = {k: v.clone() if torch.is_tensor(v) else v for k, v in every[0][0].items()}
    out = torch.zeros_like(every[0][1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        w4.gated_delta_rule(**live, out=out)
    for i in (0, 1, 1, 0, 1):
        for k, v in every[i][0].items():
            if torch.is_tensor(v):
                live[k].copy_(v)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, every[i][1]) and torch.equal(live["state"], every[i][2]), i
        w4.gated_delta_rule(**{**every[0][0], "state": every[0][0]["state"].clone()})
