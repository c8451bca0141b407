"""The 4-bit cache's operators where a call leaves the ordinary: buffers that do not fit, slots
that nobody sees and that hold anything, weights and values far below the largest,
lengths past the tables and the given maxima, prompts of very many rows, pages that
are not there, numbers near the types' ends; and the paths that only long sequences
take."""

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


def slots_of(cache, b):
    """As cache.get for every slot of sequence b at once: (codes, s, m, value) of keys and of values,
    each [heads, slots, D] in 64 bits."""
    t, d = np.arange(cache.lens[b]), np.arange(cache.D)
    words, r32 = cache.words[cache.table[b, t // cache.page], :, (t % cache.page) // 32], (t % 32)[:, None]
    out = []
    for value, place in ((False, cache.key_at), (True, cache.value_at)):
        at, shift = (np.broadcast_to(x, (len(t), cache.D)) for x in place(r32, d[None, :]))
        take = lambda index: np.take_along_axis(words, np.broadcast_to(index[:, None], (*words.shape[:2], cache.D)), 2)
        par = take(cache.param_at(value, np.broadcast_to(d // cache.group, at.shape), r32))
        s, m = (torch.from_numpy(((par >> np.uint32(i)) & np.uint32(0xFFFF)).astype(np.uint16).view(np.int16))
                .view(cache.dtype).double().transpose(0, 1) for i in (0, 16))
        c = torch.from_numpy(((take(at) >> shift[:, None].astype(np.uint32)) & 15).astype(np.int64)).double().transpose(0, 1)
        out.append((c, s, m, m + s * c))
    return out


# ---- buffers that do not fit ----

def test_workspace_that_is_not_the_cache_s_is_refused(dev):
    """Of any type, but contiguous memory on the cache's device, of which there is enough."""
    cache = ref.Cache([2000], 1, 64, 32, 32, F16, seed=1)
    cache.fill()
    q = randn(1, 1, 2, 64).to(F16).to(dev)
    args = (q, cache.pages(dev), ints(cache.table, dev), starts([1], dev), ints([2000], dev), 1, 2000)
    want = w4.kv4_attention(*args)
    need = w4.kv4_attention_workspace_bytes(1, 2, 1, 64, 1, 2000)
    assert need > 0
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(2 * need, dtype=torch.uint8, device=dev)[::2],
                torch.empty(need, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError):
            w4.kv4_attention(*args, workspace=bad)
    with pytest.raises(w4.W4A16Error):
        w4.kv4_attention(*args, workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev))
    for good in (torch.empty(need, dtype=torch.uint8, device=dev), torch.empty(need // 4, dtype=torch.float32, device=dev)):
        assert torch.equal(w4.kv4_attention(*args, workspace=good), want)
    short = (q, *args[1:4], ints([20], dev), 1, 20)             # none needed: still refused
    with pytest.raises(ValueError):
        w4.kv4_attention(*short, workspace=torch.empty(64, dtype=torch.uint8))


# ---- slots that no row sees ----

def put_words(cache, b, t, code, step, offset, rng):
    """Parameters `step` and `offset` (16-bit patterns, None: random) and random codes in slot t."""
    words, r32, d = cache.tile(b, t), t % 32, np.arange(cache.D)
    for value, place in ((False, cache.key_at), (True, cache.value_at)):
        at, shift = place(r32, d)
        shift = np.broadcast_to(shift, d.shape).astype(np.uint32)
        for j in range(cache.D):
            keep = np.uint32(0xFFFFFFFF ^ (0xF << int(shift[j])))
            words[:, at[j]] = (words[:, at[j]] & keep) | np.uint32((code if code is not None else rng.integers(16)) << int(shift[j]))
        for g in range(cache.ng):
            s, m = (int(rng.integers(1 << 16)) if p is None else p for p in (step, offset))
            words[:, cache.param_at(value, g, r32)] = np.uint32(s | m << 16)


PATTERNS = {F16: dict(inf=0x7C00, low=0xFC00, big=0x7BFF, end=0xFBFF), BF16: dict(inf=0x7F80, low=0xFF80, big=0x7F7F, end=0xFF7F)}


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group,hq", [(64, 64, 4), (128, 128, 6), (128, 64, 2), (256, 32, 2), (64, 32, 40)])
@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("what", ["infinite", "wide", "wide down", "low", "random"])
def test_slots_that_no_row_sees_may_hold_anything(dev, dtype, D, group, hq, n, what):
    """Past the sequence's end and before the window: the results are bit for bit those with plain
    slots there (2 to 240 rows)."""
    lens, window, heads = [45, 70, 33], 20, 2
    p = PATTERNS[dtype]
    pair = {"infinite": (p["inf"], p["inf"]), "wide": (p["big"], 0), "wide down": (p["big"], p["end"]),
            "low": (p["inf"], p["low"]), "random": (None, None)}[what]
    q = randn(5, 3 * n, hq, D).to(dtype).to(dev)
    got = []
    for garbage in (False, True):
        cache = ref.Cache(lens, heads, D, group, 64, dtype, seed=3)
        cache.fill()
        rng = np.random.default_rng(6)
        for b, length in enumerate(lens):
            unseen = list(range(max(0, length - n + 1 - window))) + list(range(length, -(-length // 64) * 64))
            for t in unseen:
                if garbage:
                    put_words(cache, b, t, None if what == "random" else 9, *pair, rng)
                else:
                    put_words(cache, b, t, 0, 0, 0, rng)
        args = (cache.pages(dev), ints(cache.table, dev), starts([n] * 3, dev), ints(lens, dev))
        out, lse = w4.kv4_attention(q, *args, n, max(lens), window=window, return_lse=True)
        acc = w4.kv4_attention_mass(q, *args, lse, torch.zeros(3, heads, max(lens), device=dev), n, max(lens),
                                    window=window)
        got.append((out, lse, acc))
    for plain, other in zip(*got):
        assert torch.isfinite(plain).all()
        assert torch.equal(plain, other)


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("G", [1, 200])
def test_attention_of_constant_groups_at_bfloat16_s_end(dev, group, G):
    """One slot whose groups are all -3.3e38 or all 3.3e38: its value comes out as it is."""
    cache = ref.Cache([1], 1, 128, group, 32, BF16, seed=3)
    v = torch.full((1, 128), -3.3e38)
    v[:, 64:] *= -1 if group == 64 else 1
    cache.put(0, 0, randn(1, 1, 128), v)
    out = w4.kv4_attention(torch.ones(1, G, 128, dtype=BF16, device=dev), cache.pages(dev), ints(cache.table, dev),
                           starts([1], dev), ints([1], dev), 1, 1)
    assert torch.equal(out.cpu(), v.to(BF16).expand(1, G, 128))


# ---- weights and values far below the largest ----

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 64), (128, 32), (256, 64)])
@pytest.mark.parametrize("G", [1, 20, 200])
@pytest.mark.parametrize("gap,size,sink", [(12.5, 0.02, 0.001), (10.5, 0.001, 0.001), (17.0, 0.02, 1.0), (9.0, 1e-4, 0.0), (17.0, 0.02, 0.0)])
def test_attention_small_values_behind_a_dominant_slot(dev, dtype, D, group, G, gap, size, sink):
    """The first slot's logit lies `gap` above the rest, whose values are small: their share of the
    output still has the type's precision.  512 sequences on the same pages, so that one workgroup
    walks over all slots.

    Only channel 0 of q is not zero, which leaves of the logits' error a few roundings of one
    product: e = 2^-20 scale |q_0| max (s (2B + 15) + |m|), and 2^-20 for the exponent.  The weights'
    products are summed as P (B + c): 2^-18 (B + 16) sum p s for that sum.  The rest is the header's
    bound, u |o| + 1.1 u sum p (s |c - 8| + |m + 8 s|), and half a step of the output type's smallest
    numbers."""
    copies, heads, n_slots = 512, 2, 5001
    cache = ref.Cache([n_slots], heads, D, group, 256, dtype, seed=D + group)
    cache.rng = np.random.default_rng(11)
    # values: a mean of each channel and as much around it
    mean = torch.from_numpy(cache.rng.standard_normal((heads, 1, D))).float() * size
    cache.fill(scale_k=0.7, scale_v=size)
    for b, t0 in ((0, t) for t in range(0, n_slots, 32)):       # the means go onto the offsets
        words, count = cache.tile(b, t0), min(32, n_slots - t0)
        for g in range(cache.ng):
            at = cache.param_at(True, g, np.arange(count))
            m = torch.from_numpy((words[:, at] >> np.uint32(16)).astype(np.uint16).view(np.int16)).view(dtype).float()
            m = (m + mean[:, 0, g * group].unsqueeze(1)).to(dtype)
            m16 = m.view(torch.int16).numpy().astype(np.uint16).astype(np.uint32)
            words[:, at] = (words[:, at] & np.uint32(0xFFFF)) | (m16 << np.uint32(16))
    scale = D ** -0.5
    q0 = 1.0 / scale / 0.7
    first_k = randn(8, heads, D)
    first_k[:, 0] = (gap + 2.0) * 0.7                           # the other logits: deviation 1
    cache.put(0, 0, first_k, sink * randn(9, heads, D))
    q = torch.zeros(1, G * heads, D)
    q[0, :, 0] = q0 * torch.linspace(0.9, 1.0, G * heads)
    q = q.to(dtype)
    (_, ks, km, k), (vc, s, m, v) = slots_of(cache, 0)
    ks0 = float(ks[..., 0].max()) * (2 * (128 if dtype == BF16 else 64) + 15) + float(km[..., 0].abs().max())
    e = 2.0 ** -20 * (1 + scale * float(q[..., 0].abs().max()) * ks0)
    u, base = ref.U[dtype], (128 if dtype == BF16 else 64) + 16
    args = (ints(np.repeat(cache.table, copies, 0), dev), starts([1] * copies, dev), ints([n_slots] * copies, dev))
    out, lse = w4.kv4_attention(q.expand(copies, -1, -1).contiguous().to(dev), cache.pages(dev), *args, 1, n_slots,
                                return_lse=True)
    assert torch.equal(out, out[:1].expand_as(out))
    got, worst = out[0].cpu().double(), 0.0
    for h in range(heads):
        rows = slice(h * G, (h + 1) * G)
        z = scale * (q[0, rows].double() @ k[h].T)
        p = torch.softmax(z, -1)
        want = p @ v[h]
        bound = (1.01 * u * want.abs() + 1.1 * u * (p @ (s[h] * (vc[h] - 8).abs() + (m[h] + 8 * s[h]).abs()))
                 + 2.2 * e * (p @ v[h].abs()) + 2.0 ** -18 * base * (p @ s[h]) + (2.0 ** -25 if dtype == F16 else 0))
        ratio = ((got[rows] - want).abs() / bound).max()
        worst = max(worst, float(ratio))
        assert ((lse[0, rows].cpu().double() - torch.logsumexp(z, -1)).abs() <= e).all()
    assert worst <= 1, worst


# ---- lengths past the tables and the given maxima ----

def by_definition(cache, q, ns, lens, visible, scale, causal, window, rows):
    """Attention of the first `rows` tokens of each sequence: token i of n sits in slot len - n + i, and
    slots at or past visible[b] are not seen.  Returns out, lse, the bound's magnitudes and the weights."""
    T, hq, D = q.shape
    G = hq // cache.heads
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    rough, mag = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    size = torch.zeros(T, hq, dtype=torch.float64)
    acc, at = [], 0
    for b, n in enumerate(ns):
        (_, _, _, k), (vc, s, _, v) = slots_of(cache, b)
        c8 = vc - 8
        total = torch.zeros(cache.heads, cache.lens[b], dtype=torch.float64)
        for i in range(min(n, rows)):
            lo, hi = ref.sees(i, n, lens[b], causal, window)
            hi = min(hi, visible[b])
            if hi <= lo:
                continue
            for h in range(cache.heads):
                r = slice(h * G, (h + 1) * G)
                qq = q[at + i, r].double()
                z = scale * (qq @ k[h, lo:hi].T)
                p = torch.softmax(z, -1)
                out[at + i, r] = p @ v[h, lo:hi]
                rough[at + i, r] = p @ (s[h, lo:hi] * c8[h, lo:hi].abs())
                mag[at + i, r] = p @ (v[h, lo:hi].abs() + 24 * s[h, lo:hi])
                lse[at + i, r] = torch.logsumexp(z, -1)
                size[at + i, r] = scale * (qq.abs() @ k[h, lo:hi].abs().T).amax(-1)
                total[h, lo:hi] += p.sum(0)
        acc.append(total)
        at += n
    return out, lse, rough, mag, size, acc


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,window,causal", [(4, 0, True), (4, 30, True), (4, 0, False), (48, 0, True), (48, 30, True)])
@pytest.mark.parametrize("ns,lens,max_q,max_kv", [
    ([3, 9, 4], [66, 100, 40], 9, 200),            # past the tables' 64 slots
    ([7, 5, 12], [60, 64, 33], 5, 64),             # more tokens than max_q
    ([6, 9, 2], [50, 64, 20], 9, 47),              # more slots than max_kv
    ([6, 12, 1], [70, 200, 64], 4, 40),            # all of it; one whose tokens lie past the end
])
def test_positions_do_not_move_with_the_limits(dev, dtype, hq, window, causal, ns, lens, max_q, max_kv):
    cache = ref.Cache([64, 64, 64], 2, 128, 64, 32, dtype, seed=4)
    cache.fill()
    q = (1.5 * randn(6, sum(ns), hq, 128)).to(dtype)
    args = (cache.pages(dev), ints(cache.table, dev), starts(ns, dev), ints(lens, dev))
    out = torch.full_like(q, 7.0, device=dev)
    lse = torch.full(q.shape[:2], 7.0, device=dev)
    w4.kv4_attention(q.to(dev), *args, max_q, max_kv, window=window, causal=causal, out=out, lse=lse)
    visible = [min(n, 64, max_kv) for n in lens]
    o, l, rough, mag, size, acc = by_definition(cache, q, ns, lens, visible, 128 ** -0.5, causal, window, max_q)
    done = torch.cat([torch.arange(n) < max_q for n in ns])
    assert (out.cpu()[~done] == 7).all() and (lse.cpu()[~done] == 7).all()      # further tokens are left alone
    e = E_LOGIT * size.clamp(min=1.0)
    bound = 1.01 * ref.U[dtype] * o.abs() + 1.1 * ref.U[dtype] * rough + 2.2 * e[..., None] * mag + 2.0 ** -24
    assert ((out.cpu().double() - o).abs() <= bound)[done].all()
    seen = torch.isfinite(l) & done[:, None]
    got = lse.cpu().double()
    assert ((got - l).abs()[seen] <= e[seen]).all() and (got[done[:, None] & ~seen] == -math.inf).all()
    weights = w4.kv4_attention_mass(q.to(dev), *args, lse, torch.zeros(3, 2, max(64, max_kv), device=dev), max_q, max_kv,
                                    window=window, causal=causal).cpu().double()
    assert (weights[:, :, 64:] == 0).all()
    weights = weights[:, :, :64]
    e = 4 * E_LOGIT * max(1.0, float(size.max()))
    for b, want in enumerate(acc):
        assert ((weights[b] - want).abs() <= e * want + 2.0 ** -22 * want).all()


def test_append_of_more_tokens_than_max_q_stores_the_first_ones(dev):
    """... in their own slots; the others' slots stay as they are."""
    D, ns, lens, max_q = 64, [7, 3, 40], [50, 20, 41], 4
    cache = ref.Cache(lens, 2, D, 32, 32, F16, seed=2)
    cache.fill()
    x = randn(3, sum(ns), 2, D).to(F16)
    pages = cache.pages(dev)
    w4.kv4_append(pages, x.to(dev), x.to(dev), ints(cache.table, dev), starts(ns, dev), ints(lens, dev), max_q)
    at = 0
    for b, n in enumerate(ns):
        for i in range(min(n, max_q)):
            cache.put(b, lens[b] - n + i, x[at + i], x[at + i])
        at += n
    got = ref.Cache(lens, 2, D, 32, 32, F16, seed=2)
    got.back(pages)
    np.testing.assert_array_equal(got.words, cache.words)


# ---- prompts of very many rows ----

@pytest.mark.parametrize("dtype,hq,D,n", [(F16, 2048, 64, 515), (BF16, 4096, 128, 260)])
def test_attention_and_mass_of_a_million_rows(dev, dtype, hq, D, n):
    """Every row against 64-bit products (on the GPU, a token at a time)."""
    cache = ref.Cache([n + 5], 1, D, 64, 64, dtype, seed=7)
    cache.fill()
    gen = torch.Generator(device=dev)
    gen.manual_seed(3)
    q = (1.5 * torch.randn(n, hq, D, generator=gen, device=dev)).to(dtype)
    args = (cache.pages(dev), ints(cache.table, dev), starts([n], dev), ints([n + 5], dev))
    out, lse = w4.kv4_attention(q, *args, n, n + 5, return_lse=True)
    acc = w4.kv4_attention_mass(q, *args, lse, torch.zeros(1, 1, n + 5, device=dev), n, n + 5)[0, 0].double()
    (_, _, _, k), (c, s, _, v) = ([t[0].to(dev) for t in part] for part in slots_of(cache, 0))
    kt, rough, mag = k.T.contiguous(), s * (c - 8).abs(), v.abs() + 24 * s
    u, total, worst = ref.U[dtype], torch.zeros_like(acc), 0.0
    for i in range(n):
        seen, qq = n + 5 - n + i + 1, q[i].double()
        z = (qq @ kt)[:, :seen] * D ** -0.5
        p = torch.softmax(z, -1)
        total[:seen] += p.sum(0)
        size = (qq.abs() @ kt.abs())[:, :seen].amax(-1, keepdim=True) * D ** -0.5
        e = E_LOGIT * size.clamp(min=1.0)
        want = p @ v[:seen]
        bound = 1.01 * u * want.abs() + 1.1 * u * (p @ rough[:seen]) + 2.2 * e * (p @ mag[:seen]) + 2.0 ** -24
        worst = max(worst, float(((out[i].double() - want).abs() / bound).max()))
        assert ((lse[i].double() - torch.logsumexp(z, -1)).abs() <= e[:, 0]).all(), i
    assert worst <= 1, worst
    # (the sizes of the logits here are below 60; sums of up to a million weights in fp32)
    assert ((acc - total).abs() <= 4 * E_LOGIT * 60 * total).all()


# ---- pages that are not there ----

@pytest.mark.parametrize("dtype", [F16, BF16])
def test_evict_gives_nan_for_kept_slots_that_are_not_there(dev, dtype):
    """As kv4_read does for such slots: what the destination held before does not show."""
    D, lens, budget = 128, [96, 40], 70
    cache = ref.Cache(lens, 2, D, 64, 32, dtype, seed=1, spare=6)
    cache.fill()
    dst = cache.free[:6].reshape(2, 3).astype(np.int32)
    for page in dst.ravel():                               # old, valid contents
        cache.words[page] = cache.words[cache.table[0, 0]]
    table = cache.table.copy()
    table[0, 1], table[1, 0] = cache.num_pages, -1         # slots 32..63 of the first, 0..31 of the second
    pages = cache.pages(dev)
    acc = torch.rand(2, 2, 96, device=dev)
    kept, new, _ = w4.kv4_evict(pages, ints(table, dev), ints(lens, dev), acc, budget, 8, ints(dst, dev), D, 96)
    k, v = (t.cpu() for t in w4.kv4_read(pages, ints(dst, dev), starts([70, 40], dev), new, 110, D, dtype))
    for b, (first, count) in enumerate(((0, 70), (70, 40))):
        for h in range(2):
            for t in range(count):
                slot = int(kept[b, h, t])
                gone = 32 <= slot < 64 if b == 0 else slot < 32
                if gone:
                    assert torch.isnan(k[first + t, h]).all() and torch.isnan(v[first + t, h]).all()
                else:
                    want = cache.get(b, slot)
                    assert torch.equal(k[first + t, h].double(), want[0][3][h].float().to(dtype).double())
                    assert torch.equal(v[first + t, h].double(), want[1][3][h].float().to(dtype).double())


# ---- numbers near the types' ends ----

def test_norm_of_heads_whose_squares_leave_fp32(dev):
    """bfloat16 numbers from 1e-30 to 3e38: the norm is as good as that of ordinary ones."""
    x = randn(4, 6, 3, 128)
    x *= torch.tensor([1.0, 1e19, 1e25, 1e38, 1e-22, 1e-30])[:, None, None] / x.abs().amax(-1, keepdim=True)
    x = x.to(BF16)
    w = 1 + 0.1 * randn(1, 128)
    for eps in (0.0, 1e-6):
        qo, ko = w4.qk_norm_rope(x.to(dev), x.to(dev), w.to(dev), w.to(dev), eps=eps)
        want = ref.norm_rope(x, w, None, None, None, False, eps)
        for y in (qo, ko):
            assert ((y.cpu().double() - want).abs() <= ref.U[BF16] * want.abs() + 2.0 ** -17 * want.abs().amax(-1, keepdim=True)).all()


def test_keys_past_the_type_s_end_are_stored_as_nan(dev):
    """fp16 keys that the norm's weight takes past 65504, and bfloat16 groups wider than fp32 holds:
    their parameters would be infinite.  Every reader gives NaN for them, and for them alone."""
    for dtype in (F16, BF16):
        cache = ref.Cache([40], 1, 64, 32, 32, dtype, seed=1)
        cache.fill()
        pages, args = cache.pages(dev), (ints(cache.table, dev), starts([1], dev), ints([40], dev))
        k = randn(3, 1, 1, 64)
        weight = torch.ones(64)
        if dtype == F16:
            weight[:32] = 1e5
        else:
            k[0, 0, 0], k[0, 0, 1] = 3.3e38, -3.3e38
        v = randn(4, 1, 1, 64).to(dtype).to(dev)
        w4.kv4_append(pages, k.to(dtype).to(dev), v, *args, 1, k_weight=weight.to(dev) if dtype == F16 else None)
        rk, rv = w4.kv4_read(pages, *args, 1, 64, dtype)
        assert torch.isnan(rk[0, 0, :32]).all() and torch.isfinite(rk[0, 0, 32:]).all() and torch.isfinite(rv).all()
        for G in (1, 200):
            out = w4.kv4_attention(torch.ones(1, G, 64, dtype=dtype, device=dev), pages, *args, 1, 40)
            assert torch.isnan(out).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,n", [(1, 1), (5, 6), (20, 1), (50, 6)])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32)])
def test_attention_of_values_that_grow(dev, dtype, hq, n, D, group):
    """Values from 1 to thousands, slot after slot, the new tokens' own the largest: steps beyond 2 in
    every tile, and rows that do not see the last ones."""
    lens = [190]
    cache = ref.Cache(lens, 1, D, group, 64, dtype, seed=2)
    k, v = randn(3, 190, 1, D), randn(4, 190, 1, D) * 2.0 ** (torch.arange(190) / 15.0)[:, None, None]
    for t in range(190):
        cache.put(0, t, k[t], v[t])
    q = (1.5 * randn(5, n, hq, D)).to(dtype)
    args = (cache.pages(dev), ints(cache.table, dev), starts([n], dev), ints(lens, dev))
    out, lse = w4.kv4_attention(q.to(dev), *args, n, 190, return_lse=True)
    o, l, rough, mag, size, _ = by_definition(cache, q, [n], lens, lens, D ** -0.5, True, 0, n)
    e, u = E_LOGIT * size.clamp(min=1.0), ref.U[dtype]
    assert ((out.cpu().double() - o).abs() <= 1.01 * u * o.abs() + 1.1 * u * rough + 2.2 * e[..., None] * mag).all()
    assert ((lse.cpu().double() - l).abs() <= e).all()


# ---- slots split over workgroups, windows over several of them, many pages ----

@pytest.mark.parametrize("dtype,D,group,hq,hk,ns,lens,page,window", [
    # few rows: several chunks with 256 channels, and windows that begin inside one
    (F16, 256, 32, 2, 1, [1], [3001], 32, 0),
    (BF16, 256, 128, 3, 1, [2, 1], [2777, 1500], 96, 0),
    (BF16, 128, 64, 5, 1, [3], [4099], 64, 1001),
    (F16, 128, 32, 10, 2, [1, 4], [5000, 2345], 32, 1500),
    (F16, 256, 64, 1, 1, [1], [4001], 64, 999),
    (BF16, 64, 32, 30, 1, [4], [3333], 32, 1111),
    # many rows: parts with 128 and 256 channels, and windows over several
    (BF16, 128, 64, 2, 1, [110], [3210], 64, 0),
    (F16, 128, 32, 4, 1, [60, 7], [2500, 2100], 32, 0),
    (BF16, 128, 128, 2, 1, [130], [4000], 128, 1700),
    (F16, 256, 32, 2, 1, [120], [2600], 64, 0),
    (BF16, 256, 64, 1, 1, [200, 100], [2222, 1999], 32, 1400),
    (F16, 64, 64, 3, 1, [150], [5000], 32, 2500),
])
def test_split_slots_and_windows(dev, dtype, D, group, hq, hk, ns, lens, page, window):
    cache = ref.Cache(lens, hk, D, group, page, dtype, seed=D + hq)
    cache.fill()
    q = (1.5 * randn(8, sum(ns), hq, D)).to(dtype)
    args = (cache.pages(dev), ints(cache.table, dev), starts(ns, dev), ints(lens, dev))
    out, lse = w4.kv4_attention(q.to(dev), *args, max(ns), max(lens), window=window, return_lse=True)
    o, l, rough, mag, size, acc = by_definition(cache, q, ns, lens, lens, D ** -0.5, True, window, max(ns))
    e, u = E_LOGIT * size.clamp(min=1.0), ref.U[dtype]
    assert ((out.cpu().double() - o).abs() <= 1.01 * u * o.abs() + 1.1 * u * rough + 2.2 * e[..., None] * mag + 2.0 ** -24).all()
    assert ((lse.cpu().double() - l).abs() <= e).all()
    before = torch.rand(len(ns), hk, max(lens))
    got = w4.kv4_attention_mass(q.to(dev), *args, lse, before.to(dev), max(ns), max(lens), window=window).cpu().double()
    e = 4 * E_LOGIT * max(1.0, float(size.max()))
    for b, add in enumerate(acc):
        want = before[b, :, :lens[b]].double() + add
        assert ((got[b, :, :lens[b]] - want).abs() <= e * add + 2.0 ** -22 * want).all()
        assert torch.equal(got[b, :, lens[b]:], before[b, :, lens[b]:].double())


@pytest.mark.parametrize("dtype,D,group,page", [(BF16, 128, 64, 32), (F16, 64, 32, 32), (F16, 256, 128, 64)])
def test_many_rows_in_one_part_over_more_than_64_pages(dev, dtype, D, group, page):
    """512 sequences on the same pages, so that one workgroup walks over all of them: the page ids
    that a wave holds are loaded again on the way, twice for the longest."""
    lens, copies, G = [page * 140 + 5], 512, 200
    cache = ref.Cache(lens, 1, D, group, page, dtype, seed=5)
    cache.fill()
    q = (1.5 * randn(6, 1, G, D)).to(dtype)
    out, lse = w4.kv4_attention(q.expand(copies, -1, -1).contiguous().to(dev), cache.pages(dev),
                                ints(np.repeat(cache.table, copies, 0), dev), starts([1] * copies, dev),
                                ints(lens * copies, dev), 1, lens[0], return_lse=True)
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    o, l, rough, mag, size, _ = by_definition(cache, q, [1], lens, lens, D ** -0.5, True, 0, 1)
    e, u = E_LOGIT * size.clamp(min=1.0), ref.U[dtype]
    assert ((out[:1].cpu().double() - o).abs() <= 1.01 * u * o.abs() + 1.1 * u * rough + 2.2 * e[..., None] * mag + 2.0 ** -24).all()
    assert ((lse[:1].cpu().double() - l).abs() <= e).all()
