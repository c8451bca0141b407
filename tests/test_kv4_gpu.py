"""The attention block on the 4-bit key/value cache (qk_norm_rope, kv4_append, kv4_read,
kv4_attention, kv4_attention_mass, kv4_evict) against 64-bit references on the CPU.

Bounds, u the unit roundoff of the 16-bit type (2^-11 or 2^-8):
  norm and rotation   u |y| for the one rounding, and 2^-18 of |a| + |b| of the pair for fp32
                      (a sum of at most 256 squares and a few products)
  stored values       codes of unrounded 16-bit inputs are equal to the reference's, whose fp32
                      steps are the same; after the norm, |m + s c - y| <= s / 2 (nearest code)
                      + 15 u s + u |m| (rounded parameters) + 2^-18 max |y|
  attention           u |o| for the output's rounding, 1.1 u sum p s |c - 8| for the rounded
                      products of weight and step, and the logits' fp32 error e as a relative
                      error of the weights: 2.2 e sum p (|v| + 24 s), with
                      e = 2^-24 (D + 16) sum |q| (|k| + ...) <= 2^-15 max(1, scale sum |q| |k|)
  lse                 e as above
  mass                the rows' weights sum up with relative error 2 e, and 2^-22 of the result
"""

from __future__ import annotations

import math

import numpy as np
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import int4_weight_only_w4a16_amd as w4  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16
E_LOGIT = 2.0 ** -15


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    w4.load_library()
    return torch.device("cuda:0")


def starts(ns, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device=dev)


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def randn(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)).float()


def tables(rot, length=200, base=1e4):
    a = np.arange(length)[:, None] * base ** (-np.arange(0, rot, 2) / rot)[None]
    return torch.from_numpy(np.cos(a)).float(), torch.from_numpy(np.sin(a)).float()


# ---- norm and rotation ----

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm,in_place", [
    (1, 40, 8, 128, 128, False, True, False),
    (3, 5, 1, 64, 64, True, True, True),
    (17, 4, 4, 128, 32, False, True, True),
    (5, 2, 1, 256, 64, False, True, False),
    (4, 3, 3, 256, 256, True, True, False),
    (9, 7, 1, 64, 16, False, True, False),
    (6, 2, 1, 128, 128, False, False, False),       # rotation only
    (6, 2, 1, 128, 0, False, True, False),          # norm only
    (2, 1, 0, 128, 64, True, True, False),          # no keys
    (33, 1, 3, 64, 48, False, True, True),
])
def test_norm_rope(dev, dtype, T, hq, hk, D, rot, inter, norm, in_place):
    eps = 1e-6
    qkv = randn(T + D, T, (hq + 2 * hk) * D + 8).to(dtype)
    qkv[0, :D] = 0                                      # a head of zeros: only eps under the root
    qw, kw = 1 + 0.1 * randn(1, D), 1 + 0.1 * randn(2, D)
    cos, sin = tables(rot) if rot else (None, None)
    pos = torch.from_numpy(np.random.default_rng(3).integers(0, 200, T)).int()
    pos[0] = 199
    d_qkv = qkv.to(dev)
    q, k = d_qkv[:, :hq * D].view(T, hq, D), d_qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
    args = dict(q_weight=qw.to(dev), k_weight=kw.to(dev)) if norm else {}
    if rot:
        args.update(cos=cos.to(dev), sin=sin.to(dev), positions=pos.to(dev), interleaved=inter)
    if in_place:
        args.update(q_out=q, k_out=k)
    qo, ko = w4.qk_norm_rope(q, k, eps=eps, **args)
    for got, lo, n, w in ((qo, 0, hq, qw), (ko, hq * D, hk, kw)):
        x = qkv[:, lo:lo + n * D].reshape(T, n, D)
        want = ref.norm_rope(x, w if norm else None, cos, sin, pos.long(), inter, eps)
        plain = ref.norm_rope(x, w if norm else None, None, None, None, inter, eps)
        size = plain.abs().amax(-1, keepdim=True) if n else plain
        assert got.dtype == dtype and got.shape == x.shape
        err = (got.cpu().double() - want).abs()
        assert (err <= ref.U[dtype] * want.abs() + 2.0 ** -17 * size + 2.0 ** -24).all()
    # what lies beside the heads is untouched
    assert torch.equal(d_qkv[:, (hq + hk) * D:].cpu(), qkv[:, (hq + hk) * D:])


def test_norm_rope_position_outside_the_tables_gives_nan(dev):
    q = randn(1, 3, 2, 64).to(BF16).to(dev)
    cos, sin = (t.to(dev) for t in tables(32, 50))
    qo, ko = w4.qk_norm_rope(q, q.clone(), cos=cos, sin=sin, positions=ints([0, 50, -1], dev))
    for y in (qo, ko):
        assert torch.isfinite(y[0]).all() and torch.isnan(y[1:]).all()


# ---- into the cache and back ----

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group", SHAPES)
def test_append_stores_the_reference_codes_and_read_gives_them_back(dev, dtype, D, group):
    heads, page = 3, 96
    # new tokens and slots: none at all, one into an empty cache, one after others, a run that
    # straddles tiles and pages, a full tile, a token without room left over
    ns, lens = [0, 1, 1, 70, 32, 3, 0], [0, 1, 34, 120, 64, 96, 40]
    cache = ref.Cache(lens, heads, D, group, page, dtype, seed=D + group)
    cache.fill()
    T = sum(ns)
    x = randn(D, T, 2 * heads * D).to(dtype)
    x[1, :group] = 0.25                                  # a constant group
    x[2, :group] = 0
    x[5, heads * D] = float("inf")                       # values: one group of token 5
    k, v = x[:, :heads * D].view(T, heads, D), x[:, heads * D:].view(T, heads, D)
    d_x = x.to(dev)
    dk, dv = d_x[:, :heads * D].view(T, heads, D), d_x[:, heads * D:].view(T, heads, D)
    pages = cache.pages(dev)
    table, cu, kv = ints(cache.table, dev), starts(ns, dev), ints(lens, dev)
    assert w4.kv4_append(pages, dk, dv, table, cu, kv, max(ns)) is None
    at = 0
    for b, n in enumerate(ns):
        for i in range(n):
            t = lens[b] - n + i
            cache.put(b, t, k[at + i], torch.nan_to_num(v[at + i].float(), posinf=0.0) if at + i == 5 else v[at + i])
            if at + i == 5:                              # the group with the infinity: NaN
                words = cache.tile(b, t)
                words[0, cache.param_at(True, 0, t % 32)] = 0
        at += n
    got = ref.Cache(lens, heads, D, group, page, dtype, seed=D + group)
    got.back(pages)
    bad = [(b, t) for b in range(len(ns)) for t in range(lens[b] - ns[b], lens[b])]
    token5 = bad[5]
    w = got.tile(*token5)
    at5 = got.param_at(True, 0, token5[1] % 32)
    assert torch.isnan(got.get(*token5)[1][3][0, :group]).all()
    # codes of that group mean nothing; take the reference's
    for j in range(group):
        a, s = got.value_at(token5[1] % 32, j)
        keep = np.uint32(0xF << int(s))
        w[0, a] = (w[0, a] & ~keep) | (cache.tile(*token5)[0, a] & keep)
    w[0, at5] = cache.tile(*token5)[0, at5]
    np.testing.assert_array_equal(got.words, cache.words)    # every bit, older slots and spare pages too
    # back: the new slots, and all slots
    for counts in (ns, lens):
        cu2 = starts(counts, dev)
        rk, rv = w4.kv4_read(pages, table, cu2, kv, sum(counts), D, dtype)
        want = [cache.get(b, t) for b in range(len(ns)) for t in range(lens[b] - counts[b], lens[b])]
        where = [(b, t) for b in range(len(ns)) for t in range(lens[b] - counts[b], lens[b])]
        wk, wv = (torch.stack([g[i][3] for g in want]).float().to(dtype) for i in (0, 1))
        row = where.index(token5)
        assert torch.isnan(rv[row, 0, :group]).all()
        rv[row, 0, :group] = 0
        wv[row, 0, :group] = 0
        assert torch.equal(rk.cpu(), wk) and torch.equal(rv.cpu(), wv)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hk,D,group,rot,inter", [
    (10, 2, 128, 64, 128, False), (3, 3, 64, 32, 32, True), (4, 1, 256, 128, 64, False), (7, 1, 128, 128, 64, True)])
def test_append_with_norm_and_rotation(dev, dtype, hq, hk, D, group, rot, inter):
    ns, lens = [1, 40, 0, 5], [70, 40, 9, 37]
    cache = ref.Cache(lens, hk, D, group, 64, dtype, seed=5)
    T = sum(ns)
    x = (3 * randn(D, T, (hq + 2 * hk) * D)).to(dtype)
    d_x = x.to(dev)
    cut = [hq * D, (hq + hk) * D]
    view = lambda t: (t[:, :cut[0]].view(T, hq, D), t[:, cut[0]:cut[1]].view(T, hk, D), t[:, cut[1]:].view(T, hk, D))
    q, k, v = view(d_x)
    qw, kw = 1 + 0.1 * randn(1, D), 1 + 0.1 * randn(2, D)
    cos, sin = tables(rot)
    pos = torch.from_numpy(np.random.default_rng(3).integers(0, 200, T)).int()
    pages = cache.pages(dev)
    args = (ints(cache.table, dev), starts(ns, dev), ints(lens, dev))
    qo = w4.kv4_append(pages, k, v, *args, 40, q=q, q_weight=qw.to(dev), k_weight=kw.to(dev), cos=cos.to(dev),
                       sin=sin.to(dev), positions=pos.to(dev), interleaved=inter)
    hq_, hk_, hv_ = view(x)
    want_q = ref.norm_rope(hq_, qw, cos, sin, pos.long(), inter, 1e-6)
    err = (qo.cpu().double() - want_q).abs()
    assert (err <= ref.U[dtype] * want_q.abs() + 2.0 ** -17 * want_q.abs().amax(-1, keepdim=True)).all()
    want_k = ref.norm_rope(hk_, kw, cos, sin, pos.long(), inter, 1e-6)
    cache.back(pages)
    u, at = ref.U[dtype], 0
    for b, n in enumerate(ns):
        for i in range(n):
            for (c, s, m, y), x64 in zip(cache.get(b, lens[b] - n + i), (want_k[at], hv_[at].double())):
                bound = s / 2 + 15 * u * s + u * m.abs() + 2.0 ** -17 * x64.abs().amax(-1, keepdim=True)
                assert ((y - x64).abs() <= bound).all()
                # the step is the group's range over 15, and the codes use it
                g = x64.reshape(hk, -1, group)
                rng = ((g.amax(-1) - g.amin(-1)) / 15)[..., None].expand(g.shape).reshape(hk, D)
                assert ((s - rng).abs() <= 1.01 * u * rng + 2.0 ** -16 * g.abs().amax()).all()
            at += 1


def test_append_skips_slots_past_the_table_and_unknown_pages(dev):
    D, group = 64, 32
    cache = ref.Cache([40, 40], 1, D, group, 32, F16, seed=1)
    cache.fill()
    before = cache.words.copy()
    table = cache.table.copy()
    table[0, 1] = cache.num_pages          # past the pages
    table[1, 1] = -5
    k = randn(1, 20, 1, D).to(F16).to(dev)
    pages = cache.pages(dev)
    # sequence 0: slots 32.. lie on an unknown page; sequence 1: slots past its table's two pages too
    w4.kv4_append(pages, k, k, ints(table, dev), starts([8, 12], dev), ints([40, 70], dev), 12)
    cache.back(pages)
    np.testing.assert_array_equal(cache.words, before)
    k, v = w4.kv4_read(pages, ints(table, dev), starts([10, 0], dev), ints([40, 70], dev), 10, D, F16)
    assert torch.isfinite(k[:2]).all() and torch.isnan(k[2:]).all() and torch.isnan(v[2:]).all()


# ---- attention ----

def attend(dev, cache, q, ns, **kw):
    pages = cache.pages(dev)
    return w4.kv4_attention(q.to(dev), pages, ints(cache.table, dev), starts(ns, dev), ints(cache.lens, dev),
                            kw.pop("max_q", max(ns)), kw.pop("max_kv", max(cache.lens)), return_lse=True, **kw)


def check_attention(out, lse, q, cache, ns, scale=None, causal=True, window=0):
    scale = scale or q.shape[2] ** -0.5
    o, l, rough, mag, size, _ = ref.attention(cache, q, ns, scale, causal, window)
    u = ref.U[q.dtype]
    e = (E_LOGIT * size.clamp(min=1.0))[..., None]
    got = out.cpu().double()
    bound = 1.01 * u * o.abs() + 1.1 * u * rough + 2.2 * e * mag + 2.0 ** -24
    assert torch.isfinite(got).all()
    assert ((got - o).abs() <= bound).all(), float(((got - o).abs() / bound).max())
    seen = torch.isfinite(l)
    glse = lse.cpu().double()
    assert torch.equal(torch.isfinite(glse), seen) and (glse[~seen] == -math.inf).all()
    assert ((glse - l).abs()[seen] <= e[..., 0][seen]).all()
    assert (got[~seen] == 0).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group", SHAPES)
def test_attention_every_shape(dev, dtype, D, group):
    # sequences with no tokens, no slots, one slot, a partial tile, whole tiles, several pages
    ns, lens = [1, 0, 1, 2, 1, 1], [1, 20, 31, 64, 65, 200]
    cache = ref.Cache(lens, 2, D, group, 64, dtype, seed=D)
    cache.fill()
    q = (1.5 * randn(7, sum(ns), 6, D)).to(dtype)
    out, lse = attend(dev, cache, q, ns)
    check_attention(out, lse, q, cache, ns)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hk,ns,lens,page,window,causal", [
    (1, 1, [1], [1], 32, 0, True),
    (5, 5, [3, 1], [40, 3], 32, 0, True),
    (16, 1, [1, 2], [100, 33], 96, 0, True),               # 16 and 32 rows
    (17, 1, [1], [70], 32, 0, True),                       # 17 rows
    (8, 1, [5, 1, 3], [130, 64, 3], 64, 0, True),          # 40 rows; a sequence that is all new
    (10, 2, [37, 20], [64, 20], 64, 0, True),              # prompts
    (4, 2, [6, 1], [3, 0], 32, 0, True),                   # more tokens than slots: empty rows
    (4, 2, [9, 1], [150, 90], 32, 17, True),               # window inside a tile
    (4, 1, [50], [100], 32, 1, True),                      # a window of one
    (4, 2, [3, 7], [100, 5], 64, 0, False),                # every slot, from any token
])
def test_attention_masks_and_lengths(dev, dtype, hq, hk, ns, lens, page, window, causal):
    cache = ref.Cache(lens, hk, 128, 64, page, dtype, seed=hq + page)
    cache.fill()
    T = sum(ns)
    wide = (1.5 * randn(11, T, (hq + 3) * 128)).to(dtype)
    q = wide[:, 128:(hq + 1) * 128].view(T, hq, 128) if T > 1 else wide[:, :hq * 128].reshape(T, hq, 128)
    d_q = wide.to(dev)[:, 128:(hq + 1) * 128].view(T, hq, 128) if T > 1 else q.to(dev)    # strided, as a view of qkv
    pages = cache.pages(dev)
    out, lse = w4.kv4_attention(d_q, pages, ints(cache.table, dev), starts(ns, dev), ints(lens, dev), max(ns),
                                max(lens), window=window, causal=causal, return_lse=True)
    check_attention(out, lse, q, cache, ns, window=window, causal=causal)


@pytest.mark.parametrize("dtype,hq,ns,lens,page", [
    (BF16, 5, [1], [7001], 256), (F16, 8, [1, 1, 1], [5000, 1, 2049], 64), (BF16, 2, [9], [4100], 96),
    (F16, 1, [600], [700], 128), (BF16, 3, [257, 130], [300, 900], 32)])
def test_attention_long(dev, dtype, hq, ns, lens, page):
    """Sequences split over workgroups, and many rows."""
    cache = ref.Cache(lens, 1, 64, 64, page, dtype, seed=3)
    cache.fill()
    q = (2.5 * randn(5, sum(ns), hq, 64)).to(dtype)
    out, lse = attend(dev, cache, q, ns)
    check_attention(out, lse, q, cache, ns)
    again, _ = attend(dev, cache, q, ns)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("ns", [[4], [40]])
def test_attention_what_a_row_does_not_see_does_not_reach_it(dev, dtype, ns):
    """NaN in slots that the mask hides from a row (later tokens' own, and before the window) leave
    it as it is; the row that sees one gets NaN."""
    n = ns[0]
    cache = ref.Cache([100], 2, 128, 64, 32, dtype, seed=9)
    cache.fill()
    q = randn(5, n, 4, 128).to(dtype)
    want, lse_want = attend(dev, cache, q, ns, window=60)
    cache.poison(0, 99)                    # the last token's own slot
    cache.poison(0, 100 - n + 1 - 60 - 1)  # just before the first token's window, where there is one
    out, lse = attend(dev, cache, q, ns, window=60)
    assert torch.equal(out[:-1], want[:-1]) and torch.equal(lse[:-1], lse_want[:-1])
    assert torch.isnan(out[-1]).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group", SHAPES)
def test_attention_many_rows_every_shape(dev, dtype, D, group):
    ns, lens = [70, 0, 3], [130, 20, 40]                  # 210 rows and 9
    cache = ref.Cache(lens, 2, D, group, 64, dtype, seed=D)
    cache.fill()
    q = (1.5 * randn(7, sum(ns), 6, D)).to(dtype)
    out, lse = attend(dev, cache, q, ns)
    check_attention(out, lse, q, cache, ns)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hk,ns,lens,page,window,causal", [
    (10, 2, [39, 20], [64, 20], 64, 0, True),
    (8, 1, [25, 30], [3, 0], 32, 0, True),                 # more tokens than slots: empty rows
    (8, 2, [50, 1], [150, 90], 32, 17, True),              # window inside a tile
    (4, 1, [50], [100], 96, 1, True),                      # a window of one
    (8, 2, [60, 49], [100, 5], 64, 0, False),              # every slot, from any token
    (6, 1, [32], [4100], 32, 0, True),                     # 192 rows: the last that go a few at a time
    (1, 1, [193], [193], 32, 0, True),
])
def test_attention_many_rows_masks_and_lengths(dev, dtype, hq, hk, ns, lens, page, window, causal):
    cache = ref.Cache(lens, hk, 128, 64, page, dtype, seed=hq + page)
    cache.fill()
    q = (1.5 * randn(11, sum(ns), hq, 128)).to(dtype)
    out, lse = attend(dev, cache, q, ns, window=window, causal=causal)
    check_attention(out, lse, q, cache, ns, window=window, causal=causal)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_many_rows_what_a_row_does_not_see_does_not_reach_it(dev, dtype):
    n, big = 110, torch.finfo(F16).max
    cache = ref.Cache([200], 2, 128, 64, 32, dtype, seed=9)
    cache.fill()
    q = randn(5, n, 4, 128).to(dtype)
    want, lse_want = attend(dev, cache, q, [n], window=60)
    wide = randn(2, 2, 128)
    wide[:, 70], wide[:, 71] = -big, big                   # (its m + 15 s lies past fp16's end)
    cache.put(0, 199, randn(1, 2, 128), wide)
    out, lse = attend(dev, cache, q, [n], window=60)
    assert torch.equal(out[:-1], want[:-1])
    check_attention(out, lse, q, cache, [n], window=60)
    cache.poison(0, 199)                   # the last token's own slot
    cache.poison(0, 200 - n + 1 - 60 - 1)  # just before the first token's window
    out, lse = attend(dev, cache, q, [n], window=60)
    assert torch.equal(out[:-1], want[:-1]) and torch.equal(lse[:-1], lse_want[:-1])
    assert torch.isnan(out[-1]).all()


def test_attention_scale_extremes_and_equal_logits(dev):
    cache = ref.Cache([77], 1, 128, 128, 32, F16, seed=2)
    cache.fill(scale_k=20.0)
    q = (20 * randn(1, 1, 3, 128)).to(F16)
    out, lse = attend(dev, cache, q, [1])              # logits of hundreds: one slot takes all
    check_attention(out, lse, q, cache, [1])
    zero = torch.zeros_like(q)
    out, lse = attend(dev, cache, zero, [1])           # equal logits: the mean
    check_attention(out, lse, zero, cache, [1])
    assert abs(float(lse[0, 0]) - math.log(77)) < 1e-5
    out, lse = attend(dev, cache, q, [1], scale=0.01)
    check_attention(out, lse, q, cache, [1], scale=0.01)


def test_attention_rising_logits_move_the_reference(dev):
    """Later tiles hold larger logits, so that the running reference moves in every tile."""
    lens = [1000]
    cache = ref.Cache(lens, 1, 64, 64, 64, BF16, seed=4)
    cache.fill()
    d = torch.ones(1, 64)
    for t in range(0, 1000, 7):
        cache.put(0, t, d * (t / 250.0), torch.full((1, 64), float(t % 5)))
    q = torch.ones(1, 2, 64).to(BF16)
    out, lse = attend(dev, cache, q, [1])
    check_attention(out, lse, q, cache, [1])


def test_attention_unknown_pages_and_lengths_past_the_table_are_not_seen(dev):
    cache = ref.Cache([64, 64], 1, 64, 32, 32, F16, seed=1)
    cache.fill()
    q = randn(1, 2, 2, 64).to(F16)
    table = cache.table.copy()
    table[0, 1] = cache.num_pages + 3
    pages = cache.pages(dev)
    out, lse = w4.kv4_attention(q.to(dev), pages, ints(table, dev), starts([1, 1], dev), ints([64, 500], dev), 1, 500,
                                return_lse=True)
    # sequence 0 sees slots 0..31 only; sequence 1's length counts its table's 64 slots
    short = ref.Cache([32, 64], 1, 64, 32, 32, F16, seed=1)
    short.words, short.table = cache.words, cache.table
    o, l, *_ = ref.attention(short, q, [1, 1], 64 ** -0.5)
    assert (out.cpu().double() - o).abs().max() < 2e-2 and (lse.cpu().double() - l).abs().max() < 1e-3


def test_attention_on_another_stream_and_replayed_from_a_graph(dev):
    cache = ref.Cache([900, 50], 2, 128, 64, 64, BF16, seed=6)
    cache.fill()
    q = randn(3, 2, 8, 128).to(BF16).to(dev)
    pages, table, cu = cache.pages(dev), ints(cache.table, dev), starts([1, 1], dev)
    kv = ints([900, 50], dev)
    eager = {}
    for lens in ((900, 50), (640, 33), (1, 0)):
        kv.copy_(ints(lens, dev))
        eager[lens] = [t.clone() for t in w4.kv4_attention(q, pages, table, cu, kv, 1, 900, return_lse=True)]
    kv.copy_(ints((900, 50), dev))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out, lse = w4.kv4_attention(q, pages, table, cu, kv, 1, 900, return_lse=True, stream=st)
    st.synchronize()
    assert torch.equal(out, eager[(900, 50)][0]) and torch.equal(lse, eager[(900, 50)][1])
    graph = torch.cuda.CUDAGraph()
    acc = torch.zeros(2, 2, 900, device=dev)
    with torch.cuda.graph(graph, stream=st):
        out, lse = w4.kv4_attention(q, pages, table, cu, kv, 1, 900, return_lse=True, stream=st)
        w4.kv4_attention_mass(q, pages, table, cu, kv, lse, acc, 1, 900, stream=st)
    for lens in ((900, 50), (640, 33), (1, 0), (900, 50)):
        kv.copy_(ints(lens, dev))
        acc.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[lens][0]) and torch.equal(lse, eager[lens][1]), lens
        # all weight of 8 query heads over 2 heads arrives, where anything is seen
        for b, n in enumerate(lens):
            total = acc[b].sum(-1).cpu()
            assert torch.allclose(total, torch.full((2,), 4.0 if n else 0.0), atol=1e-4), lens


# ---- the weight of every slot ----

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hk,D,group,ns,lens,window,causal", [
    (5, 1, 128, 64, [1, 0, 1], [33, 7, 1], 0, True),
    (8, 2, 64, 32, [3, 1], [100, 200], 0, True),
    (6, 3, 128, 128, [40, 70], [64, 70], 0, True),
    (4, 1, 256, 64, [5], [90], 20, True),
    (3, 1, 256, 32, [4, 5], [2, 70], 0, True),          # empty rows
    (4, 2, 128, 32, [33], [65], 0, False),
    (2, 2, 64, 64, [130], [300], 50, True),
    (8, 8, 64, 64, [66, 70], [1100, 1200], 0, True),    # more slots: four and eight tiles together
    (4, 4, 128, 64, [70], [4500], 0, True),
    (2, 2, 256, 128, [70], [2100], 900, True),
    (16, 16, 64, 32, [66, 66], [1400, 1300], 0, True),
])
def test_attention_mass(dev, dtype, hq, hk, D, group, ns, lens, window, causal):
    cache = ref.Cache(lens, hk, D, group, 32, dtype, seed=8)
    cache.fill()
    q = (1.5 * randn(4, sum(ns), hq, D)).to(dtype)
    room = max(lens) + 5
    acc = torch.rand(len(ns), hk, room)
    _, lse, _, _, size, weights = ref.attention(cache, q, ns, D ** -0.5, causal, window)
    got = w4.kv4_attention_mass(q.to(dev), cache.pages(dev), ints(cache.table, dev), starts(ns, dev), ints(lens, dev),
                                lse.float().to(dev), acc.clone().to(dev), max(ns), max(lens), causal=causal,
                                window=window).cpu().double()
    e = 2 * E_LOGIT * max(1.0, float(size.max()))
    for b, w in enumerate(weights):
        add = torch.zeros(hk, room, dtype=torch.float64)
        add[:, :lens[b]] = w.sum((1, 2))
        want = acc[b].double() + add
        assert ((got[b] - want).abs() <= e * add + 2.0 ** -22 * want).all()
        assert torch.equal(got[b, :, lens[b]:], acc[b, :, lens[b]:].double())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("ns", [[4], [40]])
def test_attention_and_mass_of_values_at_the_type_s_end(dev, dtype, ns):
    """A group from the type's lowest to its highest number, whose m + 15 s lies past it: rows
    that do not see it, or to which it adds nothing, are as they are without it."""
    n, big = ns[0], torch.finfo(F16).max                 # (bfloat16: wide as well, without an overflow)
    cache = ref.Cache([100], 2, 128, 64, 32, dtype, seed=9)
    cache.fill()
    k, v = randn(1, 2, 128), randn(2, 2, 128)
    k[:, 0], k[:, 1], v[:, 70], v[:, 71] = -big, big, -big, big
    cache.put(0, 99, k, v)                               # the last token's own slot
    cache.put(0, 50, k, randn(3, 2, 128))
    q = randn(5, n, 4, 128).to(dtype)
    q[..., :64] = 0                                      # the keys' wide group
    out, lse = attend(dev, cache, q, ns)
    check_attention(out, lse, q, cache, ns)
    acc = w4.kv4_attention_mass(q.to(dev), cache.pages(dev), ints(cache.table, dev), starts(ns, dev), ints([100], dev),
                                lse, torch.zeros(1, 2, 100, device=dev), n, 100).cpu().double()
    _, _, _, _, size, weights = ref.attention(cache, q, ns, 128 ** -0.5)
    want = weights[0].sum((1, 2))
    assert ((acc[0] - want).abs() <= (4 * E_LOGIT * max(1.0, float(size.max())) + 2.0 ** -22) * want).all()


# ---- eviction ----

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group,lens,budget,recent", [
    (128, 64, [200, 64, 0, 65, 1], 64, 16),
    (64, 32, [333, 100], 50, 0),             # no recent ones
    (64, 64, [333, 31], 33, 33),             # recent ones only
    (256, 128, [130], 129, 7),               # one slot goes
    (256, 32, [90, 300], 1, 0),
    (128, 128, [3000], 1000, 100),
    (128, 32, [70], 96, 10),                 # nothing to cut
])
def test_evict(dev, dtype, D, group, lens, budget, recent):
    heads, page = 2, 32
    per = -(-budget // page)
    cache = ref.Cache(lens, heads, D, group, page, dtype, seed=D + budget, spare=per * len(lens) + 1)
    cache.fill()
    rng = np.random.default_rng(budget)
    room = max(lens) + 3
    # many equal weights, both zeros, negatives, infinities and a NaN
    acc = rng.integers(0, 6, (len(lens), heads, room)).astype(np.float32) / 4
    acc[rng.random(acc.shape) < 0.1] = -0.0
    acc[rng.random(acc.shape) < 0.1] *= -1
    acc[..., 5:6] = np.inf
    acc[..., 9:10] = np.nan
    acc[..., 11:12] = -np.inf
    dst = cache.free[:per * len(lens)].reshape(len(lens), per).astype(np.int32)
    pages = cache.pages(dev)
    kept, new, out = w4.kv4_evict(pages, ints(cache.table, dev), ints(lens, dev), torch.from_numpy(acc).to(dev),
                                  budget, recent, ints(dst, dev), D, max(lens))
    after = ref.Cache(lens, heads, D, group, page, dtype, seed=D + budget, spare=per * len(lens) + 1)
    after.back(pages)
    assert new.cpu().tolist() == [min(n, budget) for n in lens]
    touched = np.zeros(cache.num_pages, dtype=bool)
    for b, n in enumerate(lens):
        keep = min(n, budget)
        touched[dst[b, :-(-keep // page)]] = True
        for h in range(heads):
            want = ref.evict_slots(acc[b, h].tolist(), n, budget, recent)
            assert kept[b, h].cpu().tolist() == want + [-1] * (budget - keep)
            np.testing.assert_array_equal(out[b, h].cpu().numpy(),
                                          np.concatenate([acc[b, h][want], np.zeros(budget - keep, np.float32)]))
        step = max(1, keep // 40)                          # (a sample of the slots, first and last ones among them)
        for t in sorted(set(range(0, keep, step)) | set(range(max(0, keep - 3), keep))):
            now = after.get(b, t, dst)
            for h in range(heads):
                src = cache.get(b, int(kept[b, h, t]))
                for x, y in zip(now, src):
                    for got, old in zip(x, y):
                        np.testing.assert_array_equal(got[h].numpy(), old[h].numpy())
    np.testing.assert_array_equal(after.words[~touched], cache.words[~touched])


@pytest.mark.parametrize("lens,budget,recent", [([8200, 5000], 2048, 9), ([8193, 1], 100, 0), ([32768, 9001], 4000, 100),
                                                ([33100, 32900], 1000, 50)])
def test_evict_selects_of_long_sequences(dev, lens, budget, recent):
    """Different weights, with runs of equal ones: what is kept and its weights."""
    page, per = 128, -(-budget // 128)
    rng = np.random.default_rng(budget)
    acc = rng.random((len(lens), 1, max(lens) + 1)).astype(np.float32)
    acc[:, :, 1000:1400] = acc[:, :, 2000:2400] = np.float32(0.9)
    pages = w4.kv4_new_pages(len(lens) * per, 1, 64, 64, page, device=dev)
    table = torch.full((len(lens), -(-max(lens) // page)), -1, dtype=torch.int32, device=dev)
    dst = torch.arange(len(lens) * per, dtype=torch.int32, device=dev).view(len(lens), per)
    kept, new, out = w4.kv4_evict(pages, table, ints(lens, dev), torch.from_numpy(acc).to(dev), budget, recent, dst, 64,
                                  max(lens))
    assert new.cpu().tolist() == [min(n, budget) for n in lens]
    for b, n in enumerate(lens):
        want = ref.evict_slots(acc[b, 0].tolist(), n, budget, recent)
        assert kept[b, 0].cpu().tolist() == want + [-1] * (budget - len(want))
        np.testing.assert_array_equal(out[b, 0].cpu().numpy()[:len(want)], acc[b, 0][want])


def test_evicted_cache_attends_like_the_kept_slots(dev):
    """Attention and further appends go on from an evicted cache."""
    D, group, page, lens, budget = 128, 64, 32, [150], 70
    cache = ref.Cache(lens, 1, D, group, page, BF16, seed=1, spare=4)
    cache.fill()
    pages = cache.pages(dev)
    acc = torch.rand(1, 1, 150, device=dev)
    dst = ints(cache.free[:4].reshape(1, 4), dev)
    kept, new, _ = w4.kv4_evict(pages, ints(cache.table, dev), ints(lens, dev), acc, budget, 8, dst, D, 150)
    new += 1
    k = randn(2, 1, 1, D).to(BF16).to(dev)
    w4.kv4_append(pages, k, k, dst, starts([1], dev), new, 1)
    q = randn(3, 1, 4, D).to(BF16)
    out, lse = w4.kv4_attention(q.to(dev), pages, dst, starts([1], dev), new, 1, budget + 1, return_lse=True)
    cut = ref.Cache([budget + 1], 1, D, group, page, BF16, seed=1, spare=4)
    cut.num_pages, cut.table = cache.num_pages, dst.cpu().numpy()
    cut.back(pages)
    check_attention(out, lse, q, cut, [1])
    assert sorted(kept[0, 0].tolist()) == kept[0, 0].tolist()
