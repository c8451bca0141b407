"""The 4-bit cache's operators where a call leaves the ordinary: buffers that do not fit, slots
that nobody sees and that hold anything."""

from __future__ import annotations

import numpy as np
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import int4_weight_only_w4a16_amd as w4  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16


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
