"""kv4_tree_attention against 64-bit attention along every token's path, with the bounds of
kv4_attention (tests/test_kv4_gpu.py): u |o| for the output's rounding, 1.1 u sum p s |c - 8| for the
rounded products of weight and step, and the logits' fp32 error e = 2^-15 max(1, scale sum |q| |k|) as a
relative error of the weights, 2.2 e sum p (|v| + 24 s); e for the lse."""

from __future__ import annotations

import math
import random

import pytest

import kv4_ref as ref
import tree_ref as tr

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import int4_weight_only_w4a16_amd as w4  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16


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


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def tree_words(trees, dev, noise=0):
    """The words of all trees' tokens; with `noise` the bits that mean nothing are set at random."""
    rng = random.Random(noise)
    words = []
    for parents in trees:
        for i, w in enumerate(tr.words_of(parents)):
            words.append(w | (rng.getrandbits(64) >> i << i if noise else 0))
    return torch.tensor(tr.signed(words), dtype=torch.int64, device=dev)


def reference(cache, q, trees, window=0):
    """out, lse, sum p s |c - 8|, sum p (|v| + 24 s) and max scale sum |q| |k| of every token and head."""
    T, hq, D = q.shape
    G, scale = hq // cache.heads, D ** -0.5
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    rough, mag = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    size = torch.zeros(T, hq, dtype=torch.float64)
    at = 0
    for b, parents in enumerate(trees):
        k, c8, s, v = cache.sequence(b)
        n, length = len(parents), cache.lens[b]
        for i in range(n):
            way = tr.path(parents, i)
            first = max(0, length - n + len(way) - window) if window else 0
            slots = [t for t in range(first, length - n)] + [length - n + j for j in way if length - n + j >= 0]
            if not slots:
                continue
            for h in range(cache.heads):
                rows = slice(h * G, (h + 1) * G)
                qq = q[at + i, rows].double()
                z = scale * (qq @ k[h, slots].T)
                p = torch.softmax(z, -1)
                out[at + i, rows] = p @ v[h, slots]
                rough[at + i, rows] = p @ (s[h, slots] * c8[h, slots].abs())
                mag[at + i, rows] = p @ (v[h, slots].abs() + 24 * s[h, slots])
                lse[at + i, rows] = torch.logsumexp(z, -1)
                size[at + i, rows] = scale * (qq.abs() @ k[h, slots].abs().T).amax(-1)
        at += n
    return out, lse, rough, mag, size


def check(out, lse, q, cache, trees, window=0):
    o, l, rough, mag, size = reference(cache, q, trees, window)
    u = ref.U[q.dtype]
    e = (2.0 ** -15 * size.clamp(min=1.0))[..., None]
    got, glse = out.cpu().double(), lse.cpu().double()
    bound = 1.01 * u * o.abs() + 1.1 * u * rough + 2.2 * e * mag + 2.0 ** -24
    assert torch.isfinite(got).all()
    assert ((got - o).abs() <= bound).all(), float(((got - o).abs() / bound).max())
    seen = torch.isfinite(l)
    assert torch.equal(torch.isfinite(glse), seen) and (glse[~seen] == -math.inf).all()
    assert ((glse - l).abs()[seen] <= e[..., 0][seen]).all()
    assert (got[~seen] == 0).all()


def attend(dev, cache, q, trees, noise=0, **kw):
    ns = [len(t) for t in trees]
    return w4.kv4_tree_attention(q.to(dev), cache.pages(dev), ints(cache.table, dev), starts(ns, dev),
                                 ints(cache.lens, dev), tree_words(trees, dev, noise), max(ns), max(cache.lens),
                                 return_lse=True, **kw)


def make(seed, sizes, lens, hk, D, group, page, dtype, hq, roots=1):
    rng = random.Random(seed)
    trees = [tr.random_tree(n, rng, roots) for n in sizes]
    cache = ref.Cache(lens, hk, D, group, page, dtype, seed=seed)
    cache.fill()
    return trees, cache, (1.5 * randn(seed, sum(sizes), hq, D)).to(dtype)


SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group", SHAPES)
@pytest.mark.parametrize("hq", [2, 6, 14])
def test_every_shape(dev, dtype, D, group, hq):
    """16 rows and 32 a workgroup and the kernel for many rows (29 tokens x 7); sequences with no
    tokens, one, only drafts, drafts over the border of a tile and of a page."""
    sizes, lens = [1, 0, 7, 29], [40, 9, 7, 110]
    trees, cache, q = make(D + group, sizes, lens, 2, D, group, 64, dtype, hq)
    out, lse = attend(dev, cache, q, trees, noise=1)
    check(out, lse, q, cache, trees)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hk,sizes,lens,page,window,roots", [
    (1, 1, [1], [1], 32, 0, 1),
    (4, 4, [64], [64], 64, 0, 3),                 # nothing but drafts, several first tokens
    (8, 1, [64, 63], [65, 300], 32, 0, 2),        # 512 rows
    (5, 1, [33], [32 * 5 + 1], 96, 0, 1),         # drafts over two tiles
    (4, 2, [9, 12], [4, 12], 32, 0, 1),           # more tokens than slots
    (4, 2, [64, 5], [400, 70], 64, 64, 4),        # the least window
    (16, 1, [31, 2], [500, 130], 32, 100, 1),
    (40, 8, [3, 16, 1], [700, 33, 2000], 64, 0, 1),
])
def test_masks_and_lengths(dev, dtype, hq, hk, sizes, lens, page, window, roots):
    trees, cache, q = make(hq + page, sizes, lens, hk, 128, 64, page, dtype, hq, roots)
    out, lse = attend(dev, cache, q, trees, window=window, noise=2)
    check(out, lse, q, cache, trees, window)


@pytest.mark.parametrize("dtype,hq,sizes,lens", [(BF16, 5, [8], [7001]), (F16, 8, [40, 12], [5000, 2049]),
                                                 (BF16, 7, [64], [4100]), (F16, 2, [64], [9000])])
def test_sequences_split_over_workgroups(dev, dtype, hq, sizes, lens):
    trees, cache, q = make(3, sizes, lens, 1, 64, 32, 64, dtype, hq)
    out, lse = attend(dev, cache, q, trees)
    check(out, lse, q, cache, trees)
    assert torch.equal(out, attend(dev, cache, q, trees)[0])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,n", [(4, 6), (8, 30), (8, 64)])
def test_a_chain_is_plain_attention(dev, dtype, hq, n):
    trees, cache, q = make(5, [n], [300], 2, 128, 64, 64, dtype, hq)
    trees = [tr.chain(n)]
    out, lse = attend(dev, cache, q, trees)
    want, lse_want = w4.kv4_attention(q.to(dev), cache.pages(dev), ints(cache.table, dev), starts([n], dev),
                                      ints([300], dev), n, 300, return_lse=True)
    # fp16, few rows: kv4_attention's reference may also move for a value step in a slot that no row sees
    # (pages are full of NaN past the sequence), which rounds the weights at other places; both lie
    # within the bound of the same exact value
    check(out, lse, q, cache, trees)
    check(want, lse_want, q, cache, trees)
    if dtype is BF16 or hq * n // 2 > 192:
        assert torch.equal(out, want) and torch.equal(lse, lse_want)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq", [4, 16])
def test_what_a_token_does_not_descend_from_does_not_reach_it(dev, dtype, hq):
    """NaN in one draft's slot reaches that draft and those that descend from it, and no other."""
    n = 40
    trees, cache, q = make(7, [n], [160], 2, 128, 64, 32, dtype, hq)
    want, lse_want = attend(dev, cache, q, trees)
    cache.poison(0, 160 - n + 11)
    out, lse = attend(dev, cache, q, trees)
    hit = torch.tensor([11 in tr.path(trees[0], i) for i in range(n)])
    assert 1 <= hit.sum() < n - 12
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], lse_want[~hit])
    assert torch.isnan(out[hit]).all()


def test_limits_cut_rows_and_slots_and_move_none(dev):
    """max_q below a sequence's tokens, max_kv below its slots, rows behind the last sequence and page ids
    outside the pages: what is not there is not seen, what is not computed is left as it was."""
    trees, cache, q = make(9, [20, 6], [100, 90], 1, 128, 64, 32, BF16, 5)
    full, lse_full = attend(dev, cache, q, trees)
    T = 26
    more = torch.cat([q, q[:3]])
    words = torch.cat([tree_words(trees, dev), torch.zeros(3, dtype=torch.int64, device=dev)])
    out = torch.full((T + 3, 5, 128), 7.0, dtype=BF16, device=dev)
    lse = torch.full((T + 3, 5), 7.0, device=dev)
    got, _ = w4.kv4_tree_attention(more.to(dev), cache.pages(dev), ints(cache.table, dev), starts([20, 6], dev),
                                   ints([100, 90], dev), words, 13, 100, out=out, lse=lse, return_lse=True)
    keep = list(range(13)) + list(range(20, 26))
    # (chunks of slots may differ with max_q: two results, each within 2^-8 (|o| + 1.1 spread) of the
    # same value, |o| and the spread of values s |c - 8| below 2 and 4)
    assert (got[keep].float() - full[keep].float()).abs().max() < 0.05
    assert (got[13:20] == 7).all() and (got[T:] == 7).all() and (lse[13:20] == 7).all()
    # of 100 slots 85 are there: the first five drafts' among them
    cut, _ = w4.kv4_tree_attention(q.to(dev), cache.pages(dev), ints(cache.table, dev), starts([20, 6], dev),
                                   ints([100, 90], dev), tree_words(trees, dev), 20, 85, return_lse=True)
    k, c8, s, v = cache.sequence(0)
    for i in (0, 3, 19):
        slots = list(range(80)) + [80 + j for j in tr.path(trees[0], i) if 80 + j < 85]
        z = q[i].double() @ k[0, slots].T * 128 ** -0.5
        want = torch.softmax(z, -1) @ v[0, slots]
        assert (cut[i].cpu().double() - want).abs().max() < 0.05
    table = cache.table.copy()
    table[1, :] = -1
    gone, lse_gone = w4.kv4_tree_attention(q.to(dev), cache.pages(dev), ints(table, dev), starts([20, 6], dev),
                                           ints([100, 90], dev), tree_words(trees, dev), 20, 100, return_lse=True)
    assert torch.equal(gone[:20], full[:20]) and (gone[20:] == 0).all() and (lse_gone[20:] == -math.inf).all()


def test_on_another_stream_and_replayed_from_a_graph(dev):
    """The tree, lengths and queries are read on the device: a captured call follows them."""
    made = [make(s, [12, 9], [500, 333], 2, 128, 64, 64, BF16, 8) for s in (1, 2, 3)]
    cache = made[0][1]
    pages, table, cu = cache.pages(dev), ints(cache.table, dev), starts([12, 9], dev)
    kv = ints([500, 333], dev)
    inputs = [(q.to(dev), tree_words(trees, dev)) for trees, _, q in made]
    eager = [w4.kv4_tree_attention(q, pages, table, cu, kv, t, 12, 500, return_lse=True) for q, t in inputs]
    q, tree = (x.clone() for x in inputs[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        w4.kv4_tree_attention(q, pages, table, cu, kv, tree, 12, 500)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        out, lse = w4.kv4_tree_attention(q, pages, table, cu, kv, tree, 12, 500, return_lse=True)
    for i in (0, 1, 2, 1, 0):
        q.copy_(inputs[i][0])
        tree.copy_(inputs[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i][0]) and torch.equal(lse, eager[i][1])
        w4.kv4_tree_attention(*inputs[2][:1], pages, table, cu, kv, inputs[2][1], 12, 500)


def test_binding_refusals(dev):
    trees, cache, q = make(1, [3], [40], 1, 64, 32, 32, F16, 2)
    args = lambda tree, **kw: dict(dict(q=q.to(dev), pages=cache.pages(dev), block_table=ints(cache.table, dev),
                                        cu_seqlens=starts([3], dev), kv_len=ints([40], dev), tree=tree, max_q=3,
                                        max_kv=40), **kw)
    words = tree_words(trees, dev)
    for bad in (words.int(), words[:2], words.cpu(), words.double()):
        with pytest.raises(ValueError):
            w4.kv4_tree_attention(**args(bad))
    for kw in (dict(max_q=65), dict(window=63), dict(window=-1)):
        with pytest.raises(w4.W4A16Error) as e:
            w4.kv4_tree_attention(**args(words, **kw))
        assert e.value.status == w4.W4A16_ERR_SHAPE


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group,hq", [(64, 64, 8), (128, 32, 8), (128, 64, 40), (256, 128, 16)])
def test_many_trees_split_over_workgroups(dev, D, group, hq, dtype):
    """Enough rows, and slots, that several rows are joined by a workgroup."""
    sizes = 4 * [20, 9, 24, 1, 0, 17]
    lens = [700, 2600, 1300, 30, 5, 1025] + 18 * [900]
    trees, cache, q = make(21, sizes, lens, 8, D, group, 32, dtype, hq)
    out, lse = attend(dev, cache, q, trees)
    check(out, lse, q, cache, trees)
    assert torch.equal(out, attend(dev, cache, q, trees)[0])
