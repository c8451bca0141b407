"""The attention block of examples/attention_block.py: linears, norm, rotation, 4-bit cache,
attention, weights and eviction together, against 64-bit attention over the values that the
cache holds (read back), for prompts, single tokens and after an eviction.

The bound for the block's attention output is that of the operator: one rounding of the
output (2^-8), one of the products of weight and step (1.1 * 2^-8 of at most the values'
spread), and 2.2 * 2^-15 of the logits' size; with values of at most a few units that is
below 3e-2 absolute.  A wrong slot, head or position would be off by the values' spread."""

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import int4_weight_only_w4a16_amd as w4  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def check(block, counts):
    D, G = block.head_dim, block.q_heads // block.kv_heads
    total = sum(block.lengths)
    starts = torch.tensor([0] + block.lengths, dtype=torch.int32, device="cuda").cumsum(0).int()
    k, v = w4.kv4_read(block.pages, block.table, starts, block.kv_len, total, D, torch.bfloat16)
    q, out = block.last["q"].double().cpu(), block.last["out"].double().cpu()
    lse = block.last["lse"].double().cpu()
    k, v = k.double().cpu(), v.double().cpu()
    row = at = 0
    for n, c in zip(block.lengths, counts):
        kb, vb = k[at:at + n], v[at:at + n]
        for i in range(c):
            seen = n - c + i + 1
            for h in range(block.kv_heads):
                z = q[row + i, h * G:(h + 1) * G] @ kb[:seen, h].T / math.sqrt(D)
                want = torch.softmax(z, -1) @ vb[:seen, h]
                # (the read values are rounded, the stored ones are not)
                assert (out[row + i, h * G:(h + 1) * G] - want).abs().max() < 3e-2 * max(1.0, vb[:, h].abs().max())
                assert (lse[row + i, h * G:(h + 1) * G] - torch.logsumexp(z, -1)).abs().max() < 3e-2
        row += c
        at += n


def test_block_prompts_tokens_and_eviction(example):
    torch.manual_seed(1)
    block = example.AttentionBlock(hidden=512, q_heads=6, kv_heads=2, head_dim=64, group=32, page=32, batch=3,
                                   budget=64, recent=16, room=64)
    x = lambda n: torch.randn(n, 512, device="cuda", dtype=torch.bfloat16)
    y = block(x(100), [70, 29, 1])
    assert y.shape == (100, 512) and torch.isfinite(y).all()
    check(block, [70, 29, 1])
    # every query's weight is somewhere: 3 query heads a key/value head
    assert torch.allclose(block.weight.sum(-1).cpu(), torch.tensor([[210.0] * 2, [87.0] * 2, [3.0] * 2]), rtol=1e-3)
    kept = block.evict()
    assert block.lengths == [64, 29, 1] and block.kv_len.tolist() == [64, 29, 1]
    assert kept[0, :, -16:].tolist() == [list(range(54, 70))] * 2
    for _ in range(3):
        block(x(3), [1, 1, 1])
        check(block, [1, 1, 1])
    assert block.lengths == [67, 32, 4] and block.positions == [73, 32, 4]
    with pytest.raises(ValueError):
        block(x(70), [62, 4, 4])
