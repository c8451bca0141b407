"""Layers that mix tokens through a state of fixed size instead of a cache.

Names match the C ABI in ``include/w4a16.h`` but for its prefix:
  short_conv        causal convolution of each channel with SiLU, on a rolling state
  gated_delta_rule  w4a16_delta_rule: the gated delta rule, for tokens, prompts and
                    trees of drafted tokens
plus ``delta_rule_workspace_bytes``.  The two operators are bound in C++
(``csrc/delta_binding.cpp``, in ``_kv4.so``; see their docstrings).

A sequence's tokens are rows ``cu_seqlens[b]`` .. of the inputs, its state
``state[state_index[b]]`` of a pool; the call moves it on in place.  With a
``tree`` (int64 [tokens], as for ``kv4_tree_attention``) the tokens are drafts and
the states stay: call again with the accepted ones.
"""

from __future__ import annotations

import ctypes

from . import load_library

W4A16_SILU = 0x40
W4A16_UNIT_QK = 0x80

OPERATORS = ("short_conv", "gated_delta_rule")


def __getattr__(name: str):
    if name not in OPERATORS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from . import kv4
    globals()[name] = kv4.operator(name)
    return globals()[name]


def declare(lib: ctypes.CDLL) -> None:
    """Argument and result types of the entry points."""
    p, i64, i32, f32, u32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                 ctypes.c_uint, ctypes.c_size_t)
    lib.w4a16_short_conv.argtypes = [p, i64, p, p, p, p, p, p, p, p, i64] + [i64] * 6 + [u32, p]
    lib.w4a16_short_conv.restype = i32
    lib.w4a16_delta_rule.argtypes = ([p, i64] * 5 + [p] * 8 + [i64] + [i64] * 8 + [f32, f32, u32, p, sz, p])
    lib.w4a16_delta_rule.restype = i32
    lib.w4a16_delta_rule_workspace_bytes.argtypes = [i64] * 7 + [i32]
    lib.w4a16_delta_rule_workspace_bytes.restype = sz


def delta_rule_workspace_bytes(batch: int, tokens: int, key_heads: int, value_heads: int, key_dim: int,
                               value_dim: int, max_q: int, tree: bool = False) -> int:
    """Workspace bytes gated_delta_rule needs (0: none)."""
    return int(load_library().w4a16_delta_rule_workspace_bytes(batch, tokens, key_heads, value_heads, key_dim,
                                                               value_dim, max_q, int(tree)))
