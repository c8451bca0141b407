"""short_conv and gated_delta_rule against the definitions in 64 bits on the CPU.

Bounds, u the unit roundoff of the 16-bit type (2^-11 or 2^-8):
  convolution  u |y| for the output's rounding, and 2^-20 (sum |w x| + |bias|): at most five fp32 roundings of
               the sum, and SiLU (whose slope is below 1.1) with a few more; the state holds inputs, exactly
  delta rule   With keys of at most unit length and beta in [0, 1] a token's step does not lengthen S's columns, so
               that errors do not grow but by what is added.  Output: u |o|, and of the size m of what an output
               sums up as if nothing cancelled (delta_ref.delta): a few tokens work in fp32 throughout (sums of
               Dk <= 128 terms in trees: 2^-19 m); longer calls round the state, the new rows and the products of
               queries and keys to 11 bits (2^-12 each, relative) for the output alone: 2^-10 m.
               State: fp32 and products of 22 bits, errors of random sign that add up in quadrature as the
               state's own terms do: the norm of the error is at most 2^-18 of the state's, an element's 2^-13 of
               the rms (or of itself)."""

from __future__ import annotations

import random

import pytest

import delta_ref as ref
import tree_ref as tr

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import int4_weight_only_w4a16_amd as w4  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16
FEW = 8            # tokens of the tighter bound


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    w4.load_library()
    return torch.device("cuda:0")


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def starts(ns, dev):
    at = [0]
    for n in ns:
        at.append(at[-1] + n)
    return ints(at, dev)


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def words(trees, dev):
    return torch.tensor(tr.signed([w for t in trees for w in tr.words_of(t)]), dtype=torch.int64, device=dev)


# ---- convolution ----

class Conv:
    """A call's inputs, on the CPU; indices name states in a pool with more than enough of them."""

    def __init__(self, ns, C, W, dtype, seed=0, bias=True, silu=True, fresh=(), trees=None, index=None):
        g = torch.Generator().manual_seed(seed)
        self.ns, self.C, self.W, self.dtype, self.silu, self.trees = ns, C, W, dtype, silu, trees
        self.x = randn(g, sum(ns), C).to(dtype)
        self.weight, self.bias = randn(g, C, W), randn(g, C) if bias else None
        self.states = len(ns) + 2
        self.state = randn(g, self.states, W - 1, C).to(dtype)
        self.index = index or torch.randperm(self.states, generator=g)[:len(ns)].tolist()
        self.seen = [0 if b in fresh else 7 + b for b in range(len(ns))]
        for b in fresh:        # what a fresh sequence's state holds does not matter
            self.state[self.index[b]] = float("nan")

    def call(self, dev, **kw):
        state = self.state.to(dev)
        tree = words(self.trees, dev) if self.trees else None
        out = w4.short_conv(kw.pop("x", self.x.to(dev)), self.weight.to(dev), state, ints(self.index, dev),
                            starts(self.ns, dev), kw.pop("max_q", max(self.ns)),
                            bias=None if self.bias is None else self.bias.to(dev), seen=ints(self.seen, dev),
                            tree=tree, silu=self.silu, **kw)
        return out, state

    def check(self, out, state, stored=True):
        out, state = out.cpu().double(), state.cpu()
        at, moved = 0, set()
        for b, n in enumerate(self.ns):
            i = self.index[b]
            there = 0 <= i < self.states
            before = (self.state[i].double() if there and self.seen[b] else
                      torch.zeros(self.W - 1, self.C, dtype=torch.float64))
            y, mag, last = ref.conv(self.x[at:at + n].double(), self.weight.double(),
                                    None if self.bias is None else self.bias.double(), self.silu, before,
                                    self.trees[b] if self.trees else None)
            bound = 1.01 * ref.U[self.dtype] * y.abs() + 2.0 ** -20 * mag + 2.0 ** -24
            off = (out[at:at + n] - y).abs()
            assert (off <= bound).all(), (b, float((off / bound).max()))
            if n and there and not self.trees:
                moved.add(i)
                assert torch.equal(state[i].double(), last), b
            at += n
        for i in set(range(self.states)) - moved:
            assert torch.equal(state[i].view(torch.int16), self.state[i].view(torch.int16))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [8, 520, 1032])
def test_conv_lengths(dev, dtype, W, C):
    ns = [1, 0, 2, 3, 4, 5, 9, 63, 1]
    c = Conv(ns, C, W, dtype, seed=W, fresh=(2, 4, 8))
    c.check(*c.call(dev))
    c = Conv([64, 1, 2, 200, 0, 65, 7], C, W, dtype, seed=C, fresh=(1, 3), bias=W != 3, silu=W != 2)
    c.check(*c.call(dev))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_of_a_tree(dev, dtype, W):
    rng = random.Random(W)
    trees = [tr.random_tree(n, rng, roots) for n, roots in ((1, 1), (64, 3), (17, 1), (5, 5))]
    c = Conv([len(t) for t in trees], 264, W, dtype, fresh=(2,), trees=trees)
    c.check(*c.call(dev))
    chain = Conv([40], 264, W, dtype, seed=1, trees=[tr.chain(40)])
    row = Conv([40], 264, W, dtype, seed=1)
    assert torch.equal(chain.call(dev)[0], row.call(dev)[0])


def test_conv_states_that_are_not_there(dev):
    """An index outside the pool: zeros before the sequence, and nothing kept."""
    c = Conv([3, 70, 2, 5], 64, 4, BF16, index=[-1, 6, 1, 1000000])
    c.check(*c.call(dev))


def test_conv_of_views_and_rows_behind_the_last_sequence(dev):
    c = Conv([70, 1, 33], 64, 4, F16)
    wide = torch.full((108, 160), 5.0, dtype=F16, device=dev)
    wide[:104, 80:144] = c.x.to(dev)
    out = torch.full((108, 72), 3.0, dtype=F16, device=dev)
    got, state = c.call(dev, x=wide[:, 80:144], out=out[:, :64])
    c.check(got[:104], state)
    assert (out[104:] == 3).all() and (out[:, 64:] == 3).all()
    # of a sequence with more tokens than max_q the first ones count
    out.fill_(3)
    got, state = c.call(dev, max_q=40, out=out[:104, :64])
    assert (got[40:70] == 3).all()
    full, _ = c.call(dev)
    assert torch.equal(got[:40], full[:40]) and torch.equal(got[70:], full[70:])
    assert torch.equal(state[c.index[0]].cpu(), c.x[37:40])


def test_conv_in_pieces_is_the_same(dev):
    c = Conv([150], 72, 4, BF16)
    want, state_want = c.call(dev)
    state, outs, at = c.state.to(dev), [], 0
    for n in (1, 2, 3, 70, 1, 73):
        outs.append(w4.short_conv(c.x[at:at + n].to(dev), c.weight.to(dev), state, ints(c.index, dev), starts([n], dev),
                                  n, bias=c.bias.to(dev)))
        at += n
    assert torch.equal(torch.cat(outs), want) and torch.equal(state, state_want)


def test_conv_extremes(dev):
    c = Conv([5], 8, 4, BF16, bias=False)
    c.x[:] = torch.tensor([3e38, -3e38, 1e-38, 0.0, float("inf"), -1e4, 80.0, -80.0])
    c.weight[:] = torch.tensor([0.0, 0.0, 0.0, 1.0])
    out, _ = c.call(dev)
    got = out.cpu().double()
    assert (got[:, 0] > 3e38).all() and got[0, 4] == float("inf")       # (then 0 times infinity)
    assert (got[:, [1, 3, 5]] == 0).all() and torch.equal(out[:, 6].cpu(), c.x[:, 6])
    assert (got[:, 7].abs() < 1e-30).all()


@pytest.mark.parametrize("tree", [False, True])
def test_conv_on_another_stream_and_replayed_from_a_graph(dev, tree):
    """Rows, lengths, indices, states and words are read on the device: a captured call follows them."""
    rng = random.Random(9)
    made = [Conv([9, 30, 2], 72, 4, BF16, seed=s, fresh=f, trees=[tr.random_tree(n, rng, 2) for n in (9, 30, 2)])
            for s, f in ((1, ()), (2, (1,)), (3, (0, 2)))]
    def args(c):
        return dict(x=c.x.to(dev), weight=c.weight.to(dev), state=c.state.to(dev), state_index=ints(c.index, dev),
                    cu_seqlens=starts(c.ns, dev), max_q=30, bias=c.bias.to(dev), seen=ints(c.seen, dev),
                    tree=words(c.trees, dev) if tree else None)
    every = []
    for c in made:
        eager = args(c)
        every.append((args(c), w4.short_conv(**eager), eager["state"]))
    live = {k: v.clone() if torch.is_tensor(v) else v for k, v in every[0][0].items()}
    out = torch.zeros_like(every[0][1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        w4.short_conv(**live, out=out)
    for i in (0, 1, 2, 0, 2, 1):
        for k, v in every[i][0].items():
            if torch.is_tensor(v):
                live[k].copy_(v)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, every[i][1]), i
        assert torch.equal(live["state"].view(torch.int16), every[i][2].view(torch.int16)), i
        w4.short_conv(**{**every[0][0], "state": every[0][0]["state"].clone()})


# ---- delta rule ----

class Delta:
    def __init__(self, ns, hk, hv, dk, dv, dtype, seed=0, raw=False, unit=True, fresh=(), trees=None, index=None,
                 slow=False):
        g = torch.Generator().manual_seed(seed)
        self.ns, self.dtype, self.unit, self.trees = ns, dtype, unit, trees
        self.shape = (hk, hv, dk, dv)
        T = sum(ns)
        self.q, self.k = ((randn(g, T, hk, dk) + 0.3).to(dtype) for _ in range(2))
        if not unit:           # at most unit length
            self.q, self.k = ((x.float() / 2 / dk ** 0.5).to(dtype) for x in (self.q, self.k))
        self.v = (randn(g, T, hv, dv) + 0.2).to(dtype)
        if raw:
            self.a = -torch.rand(T, hv, generator=g) * torch.rand(hv, generator=g)
            self.b = torch.rand(T, hv, generator=g)
            self.a_log = self.dt_bias = None
        else:
            self.a, self.b = (randn(g, T, hv).to(dtype) for _ in range(2))
            self.a_log = 2 * torch.rand(hv, generator=g)
            self.dt_bias = -6 * torch.rand(hv, generator=g) - (6 if slow else 0)
        self.states = len(ns) + 2
        self.state = 0.5 * randn(g, self.states, hv, dk, dv)
        self.index = index or torch.randperm(self.states, generator=g)[:len(ns)].tolist()
        self.seen = [0 if b in fresh else 7 + b for b in range(len(ns))]
        for b in fresh:
            self.state[self.index[b]] = float("nan")
        self.eps = 1e-6

    def args(self, dev):
        d = lambda t: None if t is None else t.to(dev)
        return dict(q=d(self.q), k=d(self.k), v=d(self.v), a=d(self.a), b=d(self.b), state=self.state.to(dev),
                    state_index=ints(self.index, dev), cu_seqlens=starts(self.ns, dev), max_q=max(self.ns),
                    a_log=d(self.a_log), dt_bias=d(self.dt_bias), seen=ints(self.seen, dev),
                    tree=words(self.trees, dev) if self.trees else None, unit_qk=self.unit, eps=self.eps)

    def call(self, dev, **kw):
        args = {**self.args(dev), **kw}
        return w4.gated_delta_rule(**args), args["state"]

    def check(self, out, state, scale=None, tight=None):
        out, state = out.cpu().double(), state.cpu()
        hk, hv, dk, dv = self.shape
        scale = scale or dk ** -0.5
        if tight is None:
            tight = not self.trees and max(self.ns) <= FEW
        rough = 2.0 ** -19 if tight else 2.0 ** -10
        at, moved = 0, set()
        for b, n in enumerate(self.ns):
            i, rows = self.index[b], slice(at, at + n)
            at += n
            there = 0 <= i < self.states
            S = self.state[i] if there and self.seen[b] else torch.zeros(hv, dk, dv)
            g, beta = ref.gates(self.a[rows], self.b[rows], self.a_log, self.dt_bias)
            o, size, last = ref.delta(self.q[rows], self.k[rows], self.v[rows], g, beta, S, scale, self.unit, self.eps,
                                      self.trees[b] if self.trees else None)
            off, bound = (out[rows] - o).abs(), 1.01 * ref.U[self.dtype] * o.abs() + rough * size + 2.0 ** -24
            assert (off <= bound).all(), (b, float((off / bound).max()))
            if n and there and not self.trees:
                moved.add(i)
                off, rms = (state[i].double() - last).abs(), last.pow(2).mean((1, 2), keepdim=True).sqrt()
                assert torch.isfinite(state[i]).all()
                assert (off.pow(2).mean((1, 2), keepdim=True).sqrt() <= 2.0 ** -18 * rms).all(), \
                    (b, float((off.pow(2).mean((1, 2), keepdim=True).sqrt() / rms).max()))
                assert (off <= 2.0 ** -13 * torch.maximum(rms, last.abs())).all()
        for i in set(range(self.states)) - moved:
            assert torch.equal(state[i].view(torch.int32), self.state[i].view(torch.int32))


HEADS = [(1, 1, 64, 64), (2, 4, 128, 128), (1, 3, 128, 64), (2, 2, 64, 128), (1, 2, 128, 192), (1, 1, 64, 256)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", HEADS)
def test_delta_tokens(dev, dtype, heads):
    d = Delta([1, 3, 0, 8, 2], *heads, dtype, seed=heads[3], fresh=(1, 2))
    d.check(*d.call(dev))
    d = Delta([1, 1], *heads, dtype, seed=1, raw=True, unit=False)
    d.check(*d.call(dev))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", HEADS)
def test_delta_prompts(dev, dtype, heads):
    """Whole chunks of 64 tokens, parts of one, one token more, sequences without tokens."""
    d = Delta([64, 1, 0, 65, 130, 17, 200], *heads, dtype, seed=heads[2], fresh=(0, 4))
    d.check(*d.call(dev))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", HEADS)
def test_delta_raw_gates_and_keys(dev, dtype, heads):
    d = Delta([70, 128, 3], *heads, dtype, seed=3, raw=True, unit=False, fresh=(1,))
    d.check(*d.call(dev, scale=0.7), scale=0.7)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heads", HEADS)
def test_delta_of_a_tree(dev, dtype, heads):
    rng = random.Random(heads[3])
    trees = [tr.random_tree(n, rng, roots) for n, roots in ((1, 1), (64, 3), (17, 1), (0, 0), (5, 5), (33, 1))]
    d = Delta([len(t) for t in trees], *heads, dtype, fresh=(2,), trees=trees)
    d.check(*d.call(dev))
    chain = Delta([40], *heads, dtype, seed=1, trees=[tr.chain(40)])
    chain.check(*chain.call(dev))


@pytest.mark.parametrize("n", [5, 700])
def test_delta_slow_decay_keeps_its_precision(dev, n):
    d = Delta([n], 1, 2, 128, 128, BF16, seed=5, slow=True)
    d.check(*d.call(dev))


def test_delta_states_that_are_not_there(dev):
    for ns in ([3, 7, 2, 5], [3, 70, 2, 65]):
        d = Delta(ns, 1, 2, 64, 64, BF16, index=[-1, 6, 1, 1000000])
        d.check(*d.call(dev))


@pytest.mark.parametrize("ns", [[5, 3], [100, 3]])
def test_delta_of_views_and_rows_behind_the_last_sequence(dev, ns):
    d = Delta(ns, 2, 4, 64, 64, F16)
    T, hk, hv = sum(ns), 2, 4
    wide = torch.full((T + 4, 704), 5.0, dtype=F16, device=dev)
    q, k, v = wide[:, 8:136], wide[:, 136:264], wide[:, 264:520]
    a, b = wide[:, 521:525], wide[:, 530:534]
    for view, x in ((q, d.q), (k, d.k), (v, d.v), (a, d.a), (b, d.b)):
        view[:T] = x.reshape(T, -1).to(dev)
    out = torch.full((T + 4, 5 * 64), 3.0, dtype=F16, device=dev)
    heads = lambda t, h: t.unflatten(1, (h, 64))
    got, state = d.call(dev, q=heads(q, hk), k=heads(k, hk), v=heads(v, hv), a=a, b=b, out=heads(out[:, :256], hv))
    d.check(got[:T], state)
    assert (out[T:] == 3).all() and (out[:, 256:] == 3).all()
    # of a sequence with more tokens than max_q the first ones count
    out.fill_(3)
    cut, state = d.call(dev, max_q=ns[0] - 2, out=heads(out[:T, :256], hv))
    assert (cut[ns[0] - 2:ns[0]] == 3).all() and (cut[ns[0]:] != 3).any()
    short = Delta(ns, 2, 4, 64, 64, F16)
    keep = torch.cat([torch.arange(ns[0] - 2), torch.arange(ns[0], T)])
    for x in ("q", "k", "v", "a", "b"):
        setattr(short, x, getattr(short, x)[keep])
    short.ns = [ns[0] - 2, ns[1]]
    short.check(cut[keep], state)


@pytest.mark.parametrize("pieces", [[1, 1, 2, 3], [64, 64, 22], [1, 63, 5, 130]])
def test_delta_in_pieces(dev, pieces):
    """A sequence in pieces, prompts and tokens, against the definition at its end."""
    n = sum(pieces)
    d = Delta([n], 1, 2, 128, 64, BF16, seed=2)
    state, outs, at = d.state.to(dev), [], 0
    for c in pieces:
        rows = slice(at, at + c)
        outs.append(w4.gated_delta_rule(d.q[rows].to(dev), d.k[rows].to(dev), d.v[rows].to(dev), d.a[rows].to(dev),
                                        d.b[rows].to(dev), state, ints(d.index, dev), starts([c], dev), c,
                                        a_log=d.a_log.to(dev), dt_bias=d.dt_bias.to(dev), unit_qk=True))
        at += c
    d.check(torch.cat(outs), state, tight=False)


@pytest.mark.parametrize("n", [4, 90])
def test_delta_gates_at_their_ends(dev, n):
    """Forgetting all (g = -inf, and far below what fp32 holds), nothing, writing nothing: exact limits, no NaN."""
    d = Delta([n], 1, 4, 64, 64, F16, raw=True)
    d.a[:, 0] = -float("inf")
    d.a[:, 1] = 0.0
    d.a[:, 2] = -1e30
    d.a[1::3, 3] = -500.0
    d.b[:, 1] = 0.0
    d.b[:, 2] = 1.0
    out, state = d.call(dev)
    d.check(out, state)
    # head 1: nothing kept less, nothing written
    assert torch.equal(state[d.index[0], 1].cpu(), d.state[d.index[0], 1])


@pytest.mark.parametrize("n", [3, 80])
def test_delta_sizes_far_from_one(dev, n):
    """Keys, queries and values whose squares leave fp32, and small ones."""
    for kq, vs in ((1e25, 1e20), (1e-12, 1e-15), (1e30, 1e-20), (1.0, 1e30)):
        d = Delta([n], 1, 2, 64, 64, BF16, seed=4)
        d.q, d.k, d.v = (d.q.float() * kq).to(BF16), (d.k.float() * kq).to(BF16), (d.v.float() * vs).to(BF16)
        d.state *= vs
        d.eps = 0.0
        out, state = d.call(dev)
        hk, hv, dk, dv = d.shape
        g, beta = ref.gates(d.a, d.b, d.a_log, d.dt_bias)
        o, size, last = ref.delta(d.q, d.k, d.v, g, beta, d.state[d.index[0]], dk ** -0.5, True, 0.0)
        off = (out.cpu().double() - o).abs()
        assert (off <= 1.01 * 2.0 ** -8 * o.abs() + 2.0 ** -10 * size).all(), (kq, vs)
        off = (state[d.index[0]].cpu().double() - last).abs()
        assert off.pow(2).mean().sqrt() <= 2.0 ** -18 * last.pow(2).mean().sqrt(), (kq, vs)


@pytest.mark.parametrize("ns", [[4, 3], [90, 70]])
def test_delta_nan_stays_in_its_sequence_and_head(dev, ns):
    d = Delta(ns, 2, 4, 64, 64, BF16)
    want, state_want = d.call(dev)
    d.v[1, 1, 5] = float("nan")              # one column of one head
    d.k[ns[0] + 2, 1, 0] = float("inf")      # a key head, with both its value heads, from there on
    out, state = d.call(dev)
    hit = torch.zeros_like(want, dtype=torch.bool)
    hit[1:ns[0], 1, 5] = True
    hit[ns[0] + 2:, 2:] = True
    assert torch.equal(out[~hit], want[~hit])
    assert torch.isnan(out[1:ns[0], 1, 5]).all() and torch.isnan(out[ns[0] + 2:, 2:]).all()
    lost = torch.zeros_like(state, dtype=torch.bool)
    lost[d.index[0], 1, :, 5] = True
    lost[d.index[1], 2:] = True
    assert torch.equal(state[~lost], state_want[~lost]) and torch.isnan(state[d.index[0], 1, :, 5]).all()


@pytest.mark.parametrize("ns", [[1, 2, 1], [100, 20, 70]])
def test_delta_on_another_stream_and_replayed_from_a_graph(dev, ns):
    """Inputs, lengths, state indices and states are read on the device: a captured call follows them."""
    made = [Delta(n, 2, 4, 128, 64, BF16, seed=s, fresh=f) for s, n, f in
            ((1, ns, ()), (2, [n for n in ns[1:] + ns[:1]], (1,)), (3, [0] + ns[1:], (2,)))]
    T, most = sum(ns), max(ns)
    def padded(x):
        return torch.cat([x, x.new_zeros(T - x.shape[0], *x.shape[1:])])
    every = []
    for d in made:
        for name in ("q", "k", "v", "a", "b"):
            setattr(d, name, padded(getattr(d, name)))
        args = d.args(dev)
        args["max_q"] = most
        out = w4.gated_delta_rule(**{**args, "state": args["state"].clone()},
                                  out=torch.zeros(T, 4, 64, dtype=BF16, device=dev))
        args2 = d.args(dev)
        args2["max_q"] = most
        w4.gated_delta_rule(**args2)
        every.append((args, out, args2["state"]))
    live = {k: v.clone() if torch.is_tensor(v) else v for k, v in every[0][0].items()}
    out = torch.zeros(T, 4, 64, dtype=BF16, device=dev)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        w4.gated_delta_rule(**live, out=out)
    for i in (0, 1, 2, 0, 2, 1):
        for k, v in every[i][0].items():
            if torch.is_tensor(v):
                live[k].copy_(v)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, every[i][1]), i
        assert torch.equal(live["state"].view(torch.int32), every[i][2].view(torch.int32)), i
        w4.gated_delta_rule(**{**every[0][0], "state": every[0][0]["state"].clone()})


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n", [9, 15, 16, 17, 18])
def test_delta_around_the_longest_call_token_by_token(dev, n, dtype):
    d = Delta([n, 1, n - 1, 0, n], 2, 4, 128, 128, dtype, seed=n, fresh=(2,), index=[3, 0, 1, 2, -1])
    d.check(*d.call(dev), tight=False)
    chain = Delta([n], 1, 2, 64, 64, dtype, seed=n, trees=[tr.chain(n)])
    chain.check(*chain.call(dev), tight=False)


@pytest.mark.parametrize("heads", [(2, 4, 128, 128), (1, 3, 64, 64)])
@pytest.mark.parametrize("n", [333, 64])
def test_delta_fp16_outputs_are_little_further_off_than_their_rounding(dev, n, heads):
    """As a whole, against the exact outputs rounded: one more rounding to eleven bits, of the state, enters the
    outputs, and its share is at most as large as theirs: together less than 1.5 times (the root of two)."""
    for trees in (None, [tr.random_tree(n, random.Random(n), 2)] if n <= 64 else None):
        d = Delta([n], *heads, F16, seed=n, trees=trees)
        out, _ = d.call(dev)
        g, beta = ref.gates(d.a, d.b, d.a_log, d.dt_bias)
        o, _, _ = ref.delta(d.q, d.k, d.v, g, beta, d.state[d.index[0]], heads[2] ** -0.5, True, d.eps,
                            trees[0] if trees else None)
        rounding = (o.to(F16).double() - o).norm()
        assert (out.cpu().double() - o).norm() <= 1.5 * rounding


@pytest.mark.parametrize("ns,index", [([9500, 130, 9500], [1, 0, -1]), ([640] * 20 + [3] + [640] * 19, None)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_delta_cut_into_several_launches(dev, dtype, ns, index):
    """More chunks than the workspace holds, against a few heads at a time, which it holds.  Cut between sequences:
    the same bits.  Within one: up to the cut.  There the state goes through memory, exactly but for the power of
    two that its 16-bit parts are made with, so what follows differs by those parts' 2^-22: states by less than the
    2^-18 that each may be off, and an output, if that takes it over a border, by one step of its type, twice its u."""
    T, hk, hv, d = sum(ns), 16, 64, 128
    g = torch.Generator(device=dev).manual_seed(1)
    r = lambda *shape: torch.randn(*shape, generator=g, device=dev)
    q, k, v = r(T, hk, d).to(dtype), r(T, hk, d).to(dtype), r(T, hv, d).to(dtype)
    a, b = r(T, hv).to(dtype), r(T, hv).to(dtype)
    a_log, dt_bias = torch.rand(hv, generator=g, device=dev), -4 * torch.rand(hv, generator=g, device=dev)
    start = r(len(ns) + 1, hv, d, d)
    call = lambda hks, hvs, state: w4.gated_delta_rule(
        q[:, hks], k[:, hks], v[:, hvs], a[:, hvs], b[:, hvs], state, ints(index or list(range(len(ns))), dev),
        starts(ns, dev), max(ns), a_log=a_log[hvs].contiguous(), dt_bias=dt_bias[hvs].contiguous(), unit_qk=True)
    state = start.clone()
    out = call(slice(0, hk), slice(0, hv), state)
    assert torch.isfinite(out).all()
    for i in (0, 7, 15):
        hvs = slice(4 * i, 4 * i + 4)
        few = start[:, hvs].contiguous()
        want = call(slice(i, i + 1), hvs, few)
        at = 0
        for b_, n in enumerate(ns):
            part = slice(at, at + min(n, 64 * 128))        # (at least 132 chunks fit)
            at += n
            assert torch.equal(out[part, hvs], want[part])
        if index is None:
            assert torch.equal(out[:, hvs], want) and torch.equal(state[:, hvs], few)
        u = ref.U[dtype]
        off, size = (out[:, hvs].double() - want.double()).norm(dim=2), want.double().norm(dim=2)
        assert (off <= (2 * u + 2.0 ** -18) * size + 2.0 ** -24).all()
        off, size = (state[:, hvs].double() - few.double()).norm(dim=(2, 3)), few.double().norm(dim=(2, 3))
        assert (off <= 2.0 ** -18 * size).all()


def test_delta_nan_stays_on_its_branch(dev):
    rng = random.Random(5)
    trees = [tr.random_tree(n, rng, 2) for n in (20, 64, 9)]
    d = Delta([len(t) for t in trees], 2, 4, 64, 64, BF16, trees=trees)
    want, _ = d.call(dev)
    d.v[3, 1, 5] = float("nan")              # a column of a head, in the first tree
    d.k[20 + 4, 1, 0] = float("inf")         # a key head, in the second
    d.q[84 + 2, 0, 0] = float("nan")         # a query head, in the third: its own row alone
    out, state = d.call(dev)
    hit = torch.zeros_like(want, dtype=torch.bool)
    for j in range(20):
        hit[j, 1, 5] = 3 in tr.path(trees[0], j)
    for j in range(64):
        hit[20 + j, 2:] = 4 in tr.path(trees[1], j)
    hit[84 + 2, :2] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.isnan(out[hit]).all()
    assert torch.equal(state.cpu(), d.state)


def test_two_sequences_of_one_call_on_two_streams(dev):
    """Calls under way at the same time, each with a workspace of its own."""
    made = [Delta([300, 41], 2, 4, 128, 64, BF16, seed=s) for s in range(2)]
    want = [d.call(dev) for d in made]
    args = [d.args(dev) for d in made]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    got = [w4.gated_delta_rule(**a, stream=s.cuda_stream, workspace=torch.empty(1 << 24, dtype=torch.uint8, device=dev))
           for a, s in zip(args, streams)]
    torch.cuda.synchronize()
    for (out, state), o, a in zip(want, got, args):
        assert torch.equal(o, out) and torch.equal(a["state"], state)


def test_binding_refusals(dev):
    d = Delta([3], 1, 2, 64, 64, F16)
    good = d.args(dev)
    for bad in (dict(k=good["k"].float()), dict(k=good["k"][:2]), dict(v=good["v"].cpu()), dict(a=good["a"].float()),
                dict(a=good["a"][:, :1]), dict(a_log=None), dict(state=good["state"].half()),
                dict(state=good["state"][:, :1]), dict(state_index=good["state_index"].long()),
                dict(cu_seqlens=good["cu_seqlens"][:1]), dict(seen=good["seen"].float()),
                dict(tree=torch.zeros(2, dtype=torch.int64, device=dev)),
                dict(out=torch.zeros(3, 2, 64, device=dev)), dict(q=good["q"].float())):
        with pytest.raises(ValueError):
            w4.gated_delta_rule(**{**good, **bad})
    tree = torch.zeros(3, dtype=torch.int64, device=dev)
    for bad in (dict(tree=tree, max_q=65), dict(scale=0.0), dict(eps=-1.0), dict(max_q=-1)):
        with pytest.raises(w4.W4A16Error) as e:
            w4.gated_delta_rule(**{**good, **bad})
        assert e.value.status == w4.W4A16_ERR_SHAPE
    c = Conv([3], 16, 4, F16)
    x, w, s, i, cu = c.x.to(dev), c.weight.to(dev), c.state.to(dev), ints(c.index, dev), starts([3], dev)
    for args in ((x.float(), w, s, i, cu), (x, w.half(), s, i, cu), (x, w[:8], s, i, cu), (x, w, s.float(), i, cu),
                 (x, w, s[:, :2], i, cu), (x, w, s, i.long(), cu), (x, w, s, i, cu[:1]), (x.T, w, s, i, cu)):
        with pytest.raises(ValueError):
            w4.short_conv(*args, 3)
    with pytest.raises(w4.W4A16Error):
        w4.short_conv(x[:, :12].contiguous(), w[:12].contiguous(), s[:, :, :12].contiguous(), i, cu, 3)
