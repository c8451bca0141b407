"""The attention block around the linear on a 4-bit key/value cache.

Names match the C ABI in ``include/w4a16.h`` without its prefix:
  qk_norm_rope        norm of each query and key head and the rotation, one pass
  kv4_append          the same, and keys and values quantised into the cache
  kv4_read            the values a cache holds
  kv4_attention       softmax attention over the cache
  kv4_attention_mass  the attention weight every cached slot got, accumulated
  kv4_evict           the slots with most weight and the recent ones kept
plus ``kv4_new_pages``, ``kv4_page_bytes`` and ``kv4_attention_workspace_bytes``.
The six operators are bound in C++ (``csrc/kv4_binding.cpp``, built to
``_kv4.so``; see their docstrings): they run once for each layer and token,
where a decode step waits for launches.

A cache is a uint8 device tensor ``pages`` [num_pages, kv_heads, page_size / 32,
32 * (D + 8 * D / group_size)] whose shape carries the geometry; a block table
int32 [batch, pages of a sequence] says which pages hold a sequence's slots,
``kv_len`` int32 [batch] how many slots it uses (the tokens of this call among
them), ``cu_seqlens`` int32 [batch + 1] which rows of q, k and v are its tokens.
"""

from __future__ import annotations

import ctypes
import os

from . import load_library

W4A16_ROPE_INTERLEAVED = 0x10
W4A16_NONCAUSAL = 0x20

OPERATORS = ("qk_norm_rope", "kv4_append", "kv4_read", "kv4_attention", "kv4_attention_mass", "kv4_evict")
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_kv4.so")


def operator(name: str):
    """One of OPERATORS, from the built binding."""
    load_library()                      # torch first, then the library that the binding calls
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is not built; run __graft_entry__.build() first")
    from . import _kv4
    return getattr(_kv4, name)


def __getattr__(name: str):
    if name not in OPERATORS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    globals()[name] = operator(name)
    return globals()[name]


def declare(lib: ctypes.CDLL) -> None:
    """Argument and result types of the cache's entry points."""
    p, i64, i32, f32, u32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                 ctypes.c_uint, ctypes.c_size_t)
    for name, args in (
            ("w4a16_qk_norm_rope", [p, i64, p, i64, p, p, f32, p, p, p, p, i64, p] + [i64] * 7 + [u32, p]),
            ("w4a16_kv4_append", [p, i64, p, i64, p, i64, p, p, f32, p, p, p, p, i64, p, p, p, p]
             + [i64] * 12 + [u32, p]),
            ("w4a16_kv4_read", [p] * 6 + [i64] * 8 + [u32, p]),
            ("w4a16_kv4_attention", [p, i64, p, p, p, p, p, i64, p] + [i64] * 11
             + [f32, i64, u32, p, sz, p]),
            ("w4a16_kv4_attention_mass", [p, i64, p, p, p, p, p, p, i64] + [i64] * 11 + [f32, i64, u32, p]),
            ("w4a16_kv4_evict", [p, p, p, p, i64, i64, i64, p, i64, p, p, p] + [i64] * 8 + [u32, p])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i32
    lib.w4a16_kv4_page_bytes.argtypes = [i64] * 4
    lib.w4a16_kv4_page_bytes.restype = sz
    lib.w4a16_kv4_attention_workspace_bytes.argtypes = [i64] * 7
    lib.w4a16_kv4_attention_workspace_bytes.restype = sz


def kv4_page_bytes(kv_heads: int, head_dim: int, group_size: int, page_size: int) -> int:
    """Bytes of one page (0 for a geometry the cache does not take)."""
    return int(load_library().w4a16_kv4_page_bytes(kv_heads, head_dim, group_size, page_size))


def kv4_new_pages(num_pages: int, kv_heads: int, head_dim: int, group_size: int, page_size: int,
                  device="cuda"):
    """Zero-filled pages of a cache (their contents need not be set before use)."""
    import torch
    if kv4_page_bytes(kv_heads, head_dim, group_size, page_size) == 0:
        raise ValueError("the cache takes head_dim 64, 128 or 256, group_size 32, 64 or 128 (at most "
                         "head_dim) and a page_size that is a multiple of 32")
    return torch.zeros((num_pages, kv_heads, page_size // 32, 32 * (head_dim + 8 * (head_dim // group_size))),
                       dtype=torch.uint8, device=device)


def kv4_attention_workspace_bytes(batch: int, q_heads: int, kv_heads: int, head_dim: int, max_q: int,
                                  max_kv: int, window: int = 0) -> int:
    """Workspace bytes kv4_attention needs (0: none)."""
    return int(load_library().w4a16_kv4_attention_workspace_bytes(batch, q_heads, kv_heads, head_dim, max_q,
                                                                  max_kv, window))
