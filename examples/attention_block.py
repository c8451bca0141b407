"""An attention block of a decoder layer on INT4 weights and a 4-bit key/value cache.

  hidden -> merged QKV projection (W4A16)
         -> norm and rotation of queries and keys, keys and values into the cache (one launch)
         -> attention over the cache
         -> output projection (W4A16)

A prompt goes through in one call, then tokens one at a time.  The attention weight
that every cached slot gets is added up along the way, and a cache that outgrows its
budget is cut to the slots with most weight and the recent ones.

    python examples/attention_block.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int4_weight_only_w4a16_amd as w4  # noqa: E402


def random_weights(K: int, N: int, group: int, seed: int, device):
    """A seeded stand-in for a checkpoint's linear: qweight and scales."""
    import numpy as np
    rng = np.random.default_rng(seed)
    q = w4.pack_gptq_v2(rng.integers(0, 16, size=(K, N), dtype=np.uint8))
    scales = rng.uniform(0.5, 1.5, size=(K // group, N)) * 0.2 / K ** 0.5
    return torch.from_numpy(q).to(device), torch.from_numpy(scales.astype(np.float16)).to(device)


class AttentionBlock:
    """One block with the caches of a batch of sequences; `budget` slots a sequence at most
    (and room for a chunk of new ones), of which the `recent` last are always kept."""

    def __init__(self, hidden=5120, q_heads=40, kv_heads=8, head_dim=128, group=64, page=64, batch=2,
                 budget=1024, recent=128, room=1024, rope_base=1e6, weight_group=128, device="cuda"):
        self.q_heads, self.kv_heads, self.head_dim, self.weight_group = q_heads, kv_heads, head_dim, weight_group
        self.budget, self.recent, self.room = budget, recent, room
        width = (q_heads + 2 * kv_heads) * head_dim
        self.qkv = random_weights(hidden, width, weight_group, 1, device)
        self.out = random_weights(q_heads * head_dim, hidden, weight_group, 2, device)
        self.q_norm = torch.ones(head_dim, device=device)
        self.k_norm = torch.ones(head_dim, device=device)
        rate = rope_base ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
        angle = torch.arange(1 << 14, dtype=torch.float64)[:, None] * rate
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)
        # two sets of pages: the cache, and where an eviction puts what it keeps
        per = -(-(budget + room) // page)
        self.pages = w4.kv4_new_pages(2 * batch * per, kv_heads, head_dim, group, page, device)
        tables = torch.arange(2 * batch * per, dtype=torch.int32, device=device).view(2, batch, per)
        self.table, self.spare = tables[0].contiguous(), tables[1].contiguous()
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device=device)
        self.lengths = [0] * batch              # the same on the host, for the plan of a launch
        self.positions = [0] * batch            # tokens seen; an eviction does not change them
        self.weight = torch.zeros(batch, kv_heads, budget + room, device=device)

    def __call__(self, x, counts):
        """x [sum(counts), hidden]: counts[b] new tokens of each sequence, in order."""
        if max(n + c for n, c in zip(self.lengths, counts)) > self.budget + self.room:
            raise ValueError("more tokens than the cache has room for: call evict() in between")
        if max(p + c for p, c in zip(self.positions, counts)) > self.cos.shape[0]:
            raise ValueError("a sequence is longer than the rotation's tables")
        dev, D = x.device, self.head_dim
        new = torch.tensor(counts, dtype=torch.int32, device=dev)
        cu = torch.zeros(len(counts) + 1, dtype=torch.int32, device=dev)
        cu[1:] = torch.cumsum(new, 0)
        pos = torch.cat([torch.arange(p, p + c, dtype=torch.int32) for p, c in zip(self.positions, counts)]).to(dev)
        self.kv_len += new
        self.lengths = [n + c for n, c in zip(self.lengths, counts)]
        self.positions = [p + c for p, c in zip(self.positions, counts)]
        most, longest = max(counts), max(self.lengths)

        qkv = w4.linear(x, *self.qkv, self.weight_group)
        q, k, v = (t.view(x.shape[0], -1, D) for t in qkv.split(
            [self.q_heads * D, self.kv_heads * D, self.kv_heads * D], 1))
        q = w4.kv4_append(self.pages, k, v, self.table, cu, self.kv_len, most, q=q, q_weight=self.q_norm,
                          k_weight=self.k_norm, cos=self.cos, sin=self.sin, positions=pos)
        out, lse = w4.kv4_attention(q, self.pages, self.table, cu, self.kv_len, most, longest, return_lse=True)
        w4.kv4_attention_mass(q, self.pages, self.table, cu, self.kv_len, lse, self.weight, most, longest)
        self.last = dict(q=q, cu=cu, out=out, lse=lse)
        return w4.linear(out.view(x.shape[0], -1), *self.out, self.weight_group)

    def evict(self):
        """Cut the caches that hold more than the budget; the others move as they are."""
        kept, self.kv_len, weight = w4.kv4_evict(self.pages, self.table, self.kv_len, self.weight, self.budget,
                                                 self.recent, self.spare, self.head_dim, max(self.lengths))
        self.table, self.spare = self.spare, self.table
        self.lengths = [min(n, self.budget) for n in self.lengths]
        self.weight.zero_()
        self.weight[:, :, :self.budget] = weight
        return kept


def main():
    torch.manual_seed(0)
    block = AttentionBlock()
    x = torch.randn(1500, 5120, device="cuda", dtype=torch.bfloat16)
    y = block(x, [900, 600])
    print(f"prompts of 900 and 600 tokens: out {tuple(y.shape)}, rms {y.float().square().mean().sqrt():.3f}")
    for step in range(200):
        y = block(torch.randn(2, 5120, device="cuda", dtype=torch.bfloat16), [1, 1])
        if max(block.lengths) >= block.budget + 64:      # (not for every token)
            before = list(block.lengths)
            block.evict()
            print(f"step {step}: slots {before} -> {block.lengths}")
    torch.cuda.synchronize()
    total = block.weight.sum(-1)
    print(f"after 200 tokens: slots {block.lengths}, positions {block.positions}, "
          f"attention weight kept per head {total.mean(1).tolist()}")
    assert torch.isfinite(y).all()


if __name__ == "__main__":
    main()
