"""A served batch with drafted tokens, through its layers: all of them together against the same tokens one
at a time.  A layer that attends appends the drafts to its cache (positions by depth) and attends along the
tree; a layer with a state goes through short_conv and gated_delta_rule with the tree.  Then the accepted
path of each sequence is made its own: appended where the drafts were, and the states moved on.

Both ways are within the operators' bounds of the exact result (tests/test_kv4_tree_gpu.py,
tests/test_delta_gpu.py), so within twice those of each other; the convolution, the rotated queries and
the cache hold the same bits."""

from __future__ import annotations

import random

import pytest

import delta_ref as ref
import tree_ref as tr

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import int4_weight_only_w4a16_amd as w4  # noqa: E402
import kv4_ref  # noqa: E402
from test_kv4_tree_gpu import dev, ints, reference, starts  # noqa: E402,F401

HK, HV, DK, DV, WIDTH = 2, 4, 64, 64, 4                # the layer with a state
QH, KH, D, GROUP, PAGE = 8, 2, 64, 32, 32              # the layer that attends
CHANNELS = 2 * HK * DK + HV * DV


class Layers:
    def __init__(self, dev, lens, room, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        self.dev, self.dtype, self.lens = dev, dtype, list(lens)
        B = len(lens)
        self.cache = kv4_ref.Cache(lens, KH, D, GROUP, PAGE, dtype, seed=seed, room=room)
        self.cache.fill()
        self.pages, self.table = self.cache.pages(dev), ints(self.cache.table, dev)
        angle = torch.arange(max(lens) + room)[:, None] / 100.0 ** (torch.arange(D // 2) / (D // 2))
        self.cos, self.sin = angle.cos().to(dev), angle.sin().to(dev)
        self.weight = torch.randn(CHANNELS, WIDTH, generator=g).to(dev)
        self.a_log, self.dt_bias = torch.rand(HV, generator=g).to(dev), -3 * torch.rand(HV, generator=g).to(dev)
        self.rows = torch.randn(B, WIDTH - 1, CHANNELS, generator=g).to(dtype).to(dev)
        self.state = (0.3 * torch.randn(B, HV, DK, DV, generator=g)).to(dev)
        self.index = ints(range(B), dev)

    def step(self, x, ns, depths, trees=None):
        """Outputs of both layers for new tokens x (a dict of rows), with what went into them."""
        dev, cu, most = self.dev, starts(ns, self.dev), max(ns)
        tree = None
        if trees:
            tree = torch.tensor(tr.signed([w for t in trees for w in tr.words_of(t)]), dtype=torch.int64, device=dev)
        mixed = w4.short_conv(x["mix"], self.weight, self.rows, self.index, cu, most, tree=tree)
        q, k, v = mixed.split([HK * DK, HK * DK, HV * DV], 1)
        q, k, v = q.unflatten(1, (HK, DK)), k.unflatten(1, (HK, DK)), v.unflatten(1, (HV, DV))
        held = w4.gated_delta_rule(q, k, v, x["a"], x["b"], self.state, self.index, cu, most, a_log=self.a_log,
                                   dt_bias=self.dt_bias, tree=tree, unit_qk=True)
        after = [l + n for l, n in zip(self.lens, ns)]
        kv_len = ints(after, dev)
        positions = ints([l + d for l, ds in zip(self.lens, depths) for d in ds], dev)
        turned = w4.kv4_append(self.pages, x["k"], x["v"], self.table, cu, kv_len, most, q=x["q"], cos=self.cos,
                               sin=self.sin, positions=positions)
        args = (turned, self.pages, self.table, cu, kv_len)
        seen = (w4.kv4_tree_attention(*args, tree, most, max(after)) if trees else
                w4.kv4_attention(*args, most, max(after)))
        if not trees:
            self.lens = after
        return dict(mixed=mixed, held=held, turned=turned, seen=seen)


def tokens(g, T, dtype, dev):
    r = lambda *shape: torch.randn(T, *shape, generator=g).to(dtype).to(dev)
    return dict(mix=r(CHANNELS), a=r(HV), b=r(HV), q=r(QH, D), k=r(KH, D), v=r(KH, D))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_drafts_then_the_accepted_ones(dev, dtype):  # noqa: F811
    rng, g = random.Random(3), torch.Generator().manual_seed(3)
    lens = [70, 33, 5, 128]
    drafted, single = (Layers(dev, lens, 90, dtype, 7) for _ in range(2))
    for turn in range(3):
        sizes = [[12, 1, 24, 7], [3, 30, 1, 9], [64, 5, 2, 16]][turn]
        trees = [tr.random_tree(n, rng, roots=min(n, 2), back=4) for n in sizes]
        x = tokens(g, sum(sizes), dtype, dev)
        paths = [tr.path(t, len(t) - 1) for t in trees]
        first = [sum(sizes[:b]) for b in range(len(sizes))]
        accepted = [[at + i for i in p] for at, p in zip(first, paths)]
        before = list(drafted.lens)
        states, rows = drafted.state.clone(), drafted.rows.clone()
        got = drafted.step(x, sizes, [[len(tr.path(t, i)) - 1 for i in range(len(t))] for t in trees], trees)
        assert torch.equal(drafted.state, states) and torch.equal(drafted.rows, rows)

        # what each output may be off by
        host = kv4_ref.Cache([l + n for l, n in zip(before, sizes)], KH, D, GROUP, PAGE, dtype, seed=0)
        host.table, host.num_pages = drafted.cache.table, drafted.cache.num_pages
        host.back(drafted.pages)
        o, _, rough, mag, size = reference(host, got["turned"].cpu(), trees)
        u, e = ref.U[dtype], (2.0 ** -15 * size.clamp(min=1.0))[..., None]
        may_see = 1.01 * u * o.abs() + 1.1 * u * rough + 2.2 * e * mag + 2.0 ** -24
        gates = ref.gates(x["a"].cpu(), x["b"].cpu(), drafted.a_log.cpu(), drafted.dt_bias.cpu())
        may_hold = torch.zeros(sum(sizes), HV, DV, dtype=torch.float64)
        for b, (at, n) in enumerate(zip(first, sizes)):
            part = slice(at, at + n)
            q, k, v = (t.unflatten(1, (-1, 64)) for t in got["mixed"][part].cpu().split([HK * DK, HK * DK, HV * DV], 1))
            held, most, _ = ref.delta(q, k, v, gates[0][part], gates[1][part], states[b].cpu(), DK ** -0.5,
                                      parents=trees[b])
            may_hold[part] = 1.01 * u * held.abs() + 2.0 ** -10 * most + 2.0 ** -24

        # one at a time: the sequences' accepted tokens, those of the shorter ones' paths without a turn
        for i in range(max(map(len, paths))):
            there = [len(p) > i for p in paths]
            at = [p[i] for p, t in zip(accepted, there) if t]
            out = single.step({k: v[at] for k, v in x.items()}, [int(t) for t in there],
                              [[0] if t else [] for t in there])
            assert torch.equal(out["mixed"], got["mixed"][at]) and torch.equal(out["turned"], got["turned"][at])
            for name, may in (("seen", may_see), ("held", may_hold)):
                off = (out[name].double() - got[name][at].double()).abs().cpu()
                assert (off <= 2 * may[at]).all(), (turn, i, name, float((off / may[at]).max()))

        # and the accepted ones of all at once, where the drafts were
        every = [i for p in accepted for i in p]
        out = drafted.step({k: v[every] for k, v in x.items()}, [len(p) for p in paths],
                           [list(range(len(p))) for p in paths])
        assert torch.equal(out["mixed"], got["mixed"][every])
        assert torch.equal(drafted.rows, single.rows) and drafted.lens == single.lens
        off = (drafted.state.double() - single.state.double()).pow(2).mean((2, 3)).sqrt()
        assert (off <= 2.0 ** -17 * single.state.double().pow(2).mean((2, 3)).sqrt()).all()
        used = [kv4_ref.Cache(single.lens, KH, D, GROUP, PAGE, dtype, seed=0) for _ in range(2)]
        for c, layers in zip(used, (drafted, single)):
            c.table, c.num_pages = layers.cache.table, layers.cache.num_pages
            c.back(layers.pages)
        for b in range(len(lens)):
            for mine, theirs in zip(used[0].sequence(b), used[1].sequence(b)):
                assert torch.equal(mine, theirs)
        single.state.copy_(drafted.state)              # (the next turn starts alike)
