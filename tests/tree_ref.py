"""Trees of drafted tokens: their words, and what a token descends from, written plainly."""

from __future__ import annotations

import random


def words_of(parents):
    """The word of each token from its parent's index (-1: none): bit j for every j that it descends from."""
    words = []
    for i, p in enumerate(parents):
        assert -1 <= p < i
        words.append(0 if p < 0 else words[p] | 1 << p)
    return words


def random_tree(n, rng: random.Random, roots=1, back=8):
    """Parents of n tokens, the first `roots` of them without one."""
    return [-1 if i < roots else rng.randint(max(0, i - back), i - 1) for i in range(n)]


def chain(n):
    return list(range(-1, n - 1))


def path(parents, i):
    """The tokens from the root to i."""
    found = [i]
    while parents[found[0]] >= 0:
        found.insert(0, parents[found[0]])
    return found


def signed(words):
    """Words as int64 values (bit 63 is the sign)."""
    return [w - (1 << 64) if w >> 63 & 1 else w for w in words]
