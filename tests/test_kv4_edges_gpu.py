"""The 4-bit cache's operators where a call leaves the ordinary: buffers that do not fit."""

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
