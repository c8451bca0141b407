"""The attention block around the linear on a 4-bit key/value cache.

Names match the C ABI in ``include/w4a16.h`` without its prefix:
  qk_norm_rope        norm of each query and key head and the rotation, one pass
  kv4_append          the same, and keys and values quantised into the cache
  kv4_read            the values a cache holds
  kv4_attention       softmax attention over the cache
  kv4_attention_mass  the attention weight every cached slot got, accumulated
  kv4_evict           the slots with most weight and the recent ones kept
plus ``kv4_new_pages`` and ``kv4_page_bytes``.

A cache is a uint8 device tensor ``pages`` [num_pages, kv_heads, page_size / 32,
32 * (D + 8 * D / group_size)] whose shape carries the geometry; a block table
int32 [batch, pages of a sequence] says which pages hold a sequence's slots,
``kv_len`` int32 [batch] how many slots it uses (the tokens of this call among
them), ``cu_seqlens`` int32 [batch + 1] which rows of q, k and v are its tokens.
"""

from __future__ import annotations

import ctypes
from typing import Optional

from . import (W4A16_OK, W4A16_X_BF16, W4A16Error, _stream_handle, load_library)

W4A16_ROPE_INTERLEAVED = 0x10
W4A16_NONCAUSAL = 0x20


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


def _raise(status: int, what: str) -> None:
    if status != W4A16_OK:
        raise W4A16Error(status, what)


def _flag(dtype) -> int:
    import torch
    if dtype == torch.bfloat16:
        return W4A16_X_BF16
    if dtype != torch.float16:
        raise ValueError("q, k and v must be float16 or bfloat16")
    return 0


def _heads(name: str, t, like=None):
    """Token stride of a [T, heads, D] tensor whose heads and channels are contiguous."""
    if t.dim() != 3 or not t.is_cuda or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
        raise ValueError(f"{name} must be a device tensor [tokens, heads, channels], contiguous but for "
                         "the stride between tokens")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must have the type and device of the other inputs")
    # a single token may carry any stride
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _plain(name: str, t, dtype, device, shape=None):
    if t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr()


def _geometry(pages, head_dim: int):
    """(kv_heads, group_size, page_size, num_pages) of a cache of that head_dim."""
    import torch
    if pages.dim() != 4 or pages.dtype != torch.uint8 or not pages.is_cuda or not pages.is_contiguous():
        raise ValueError("pages must be a contiguous uint8 device tensor "
                         "[pages, kv_heads, page_size / 32, tile bytes]")
    num_pages, kv_heads, tiles, tile = pages.shape
    groups = (tile // 32 - head_dim) // 8
    if groups < 1 or head_dim % groups or tile != 32 * (head_dim + 8 * groups):
        raise ValueError(f"pages with tiles of {tile} bytes do not hold heads of {head_dim} channels")
    return kv_heads, head_dim // groups, 32 * tiles, num_pages


def _sequences(pages, table, cu_seqlens, kv_len):
    """(batch, table stride) after the checks of the arrays that describe the sequences."""
    import torch
    if table.dim() != 2:
        raise ValueError("block_table must be [batch, pages]")
    batch = table.shape[0]
    i32 = torch.int32
    _plain("block_table", table, i32, pages.device)
    _plain("kv_len", kv_len, i32, pages.device, (batch,))
    if cu_seqlens is not None:
        _plain("cu_seqlens", cu_seqlens, i32, pages.device, (batch + 1,))
    return batch, table.shape[1]


def _rope(cos, sin, positions, q_weight, k_weight, D: int, T: int, device):
    """Addresses of the rotation's tables and the norms' weights, rot_dim and max_pos."""
    import torch
    f32 = torch.float32
    weights = [None if w is None else _plain("norm weight", w, f32, device, (D,)) for w in (q_weight, k_weight)]
    if (cos is None) != (sin is None) or (cos is None) != (positions is None):
        raise ValueError("cos, sin and positions go together")
    if cos is None:
        return weights, None, None, None, 0, 0
    if cos.dim() != 2:
        raise ValueError("cos and sin must be [positions, rot_dim / 2]")
    return (weights, _plain("cos", cos, f32, device), _plain("sin", sin, f32, device, cos.shape),
            _plain("positions", positions, torch.int32, device, (T,)), 2 * cos.shape[1], cos.shape[0])


def _empty(shape, dtype, device, stream):
    """An uninitialised tensor whose memory belongs to the stream the call runs on."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _out(t, like, shape, stream):
    if t is None:
        return _empty(shape, like.dtype, like.device, stream)
    if t.shape != shape:
        raise ValueError(f"an output must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t


class _on:
    """The device of a tensor as the current one, where it is another."""
    __slots__ = ("guard",)

    def __init__(self, device):
        import torch
        self.guard = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of each head of q [T, q_heads, D] and k [T, kv_heads, D] (weights fp32
    [D], None: no norm), then the rotation of the first rot_dim channels by cos and sin
    (fp32 [positions, rot_dim / 2], None: no rotation) at positions (int32 [T]); pairs
    are (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved.  Returns q_out and k_out
    (allocated unless given; they may be q and k themselves)."""
    qs, ks = _heads("q", q), _heads("k", k, q)
    T, hq, D = q.shape
    hk = k.shape[1]
    if k.shape[0] != T or k.shape[2] != D:
        raise ValueError("q and k must have the same tokens and channels")
    flags = _flag(q.dtype) | (W4A16_ROPE_INTERLEAVED if interleaved else 0)
    (qw, kw), c, s, pos, rot, max_pos = _rope(cos, sin, positions, q_weight, k_weight, D, T, q.device)
    q_out, k_out = _out(q_out, q, q.shape, stream), _out(k_out, k, k.shape, stream)
    qos, kos = _heads("q_out", q_out, q), _heads("k_out", k_out, q)
    with _on(q.device):
        _raise(load_library().w4a16_qk_norm_rope(
            q.data_ptr(), qs, k.data_ptr(), ks, qw, kw, eps, c, s, pos, q_out.data_ptr(), qos, k_out.data_ptr(),
            kos, T, hq, hk, D, rot, max_pos, flags, _stream_handle(stream)), "w4a16_qk_norm_rope")
    return q_out, k_out


def kv4_append(pages, k, v, block_table, cu_seqlens, kv_len, max_q: int, q=None, q_weight=None, k_weight=None,
               cos=None, sin=None, positions=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
               stream=None):
    """Quantise this call's keys and values [T, kv_heads, D] into the cache's last slots
    (kv_len counts them already); keys, and queries q [T, q_heads, D] if given, go through
    the norm and rotation of qk_norm_rope first, in the same launch.  max_q: at least the
    most tokens of any sequence.  Returns q_out (None without q)."""
    ks, vs = _heads("k", k), _heads("v", v, k)
    T, hk, D = k.shape
    heads, group, page, num_pages = _geometry(pages, D)
    if v.shape != k.shape or hk != heads or k.device != pages.device:
        raise ValueError("k and v must be [tokens, kv_heads, channels] of the cache, on its device")
    batch, stride = _sequences(pages, block_table, cu_seqlens, kv_len)
    flags = _flag(k.dtype) | (W4A16_ROPE_INTERLEAVED if interleaved else 0)
    (qw, kw), c, s, pos, rot, max_pos = _rope(cos, sin, positions, q_weight, k_weight, D, T, k.device)
    hq = qs = qos = 0
    qp = qo = None
    if q is not None:
        qs, hq = _heads("q", q, k), q.shape[1]
        if q.shape[0] != T or q.shape[2] != D:
            raise ValueError("q must have the tokens and channels of k")
        q_out = _out(q_out, q, q.shape, stream)
        qos = _heads("q_out", q_out, k)
        qp, qo = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    with _on(k.device):
        _raise(load_library().w4a16_kv4_append(
            qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, qw, kw, eps, c, s, pos, qo, qos, pages.data_ptr(),
            block_table.data_ptr(), cu_seqlens.data_ptr(), kv_len.data_ptr(), T, hq, hk, D, rot, max_pos, group,
            page, num_pages, batch, stride, max_q, flags, _stream_handle(stream)), "w4a16_kv4_append")
    return q_out


def kv4_read(pages, block_table, cu_seqlens, kv_len, rows: int, head_dim: int, dtype, k_out=None, v_out=None,
             stream=None):
    """The values (k, v), each [rows, kv_heads, head_dim] of dtype, of the last
    cu_seqlens[b + 1] - cu_seqlens[b] slots of every sequence; rows = cu_seqlens[batch]."""
    import torch
    heads, group, page, num_pages = _geometry(pages, head_dim)
    batch, table_stride = _sequences(pages, block_table, cu_seqlens, kv_len)
    flags = _flag(dtype)
    shape = torch.Size((rows, heads, head_dim))
    outs = [_empty(shape, dtype, pages.device, stream) if t is None else t for t in (k_out, v_out)]
    ptr = [_plain("an output", t, dtype, pages.device, shape) for t in outs]
    with _on(pages.device):
        _raise(load_library().w4a16_kv4_read(
            pages.data_ptr(), block_table.data_ptr(), cu_seqlens.data_ptr(), kv_len.data_ptr(), ptr[0], ptr[1],
            rows, heads, head_dim, group, page, num_pages, batch, table_stride, flags, _stream_handle(stream)),
            "w4a16_kv4_read")
    return outs[0], outs[1]


def kv4_attention_workspace_bytes(batch: int, q_heads: int, kv_heads: int, head_dim: int, max_q: int,
                                  max_kv: int, window: int = 0) -> int:
    """Workspace bytes kv4_attention needs (0: none)."""
    return int(load_library().w4a16_kv4_attention_workspace_bytes(batch, q_heads, kv_heads, head_dim, max_q,
                                                                  max_kv, window))


def _attention_inputs(q, pages, block_table, cu_seqlens, kv_len):
    qs = _heads("q", q)
    T, hq, D = q.shape
    heads, group, page, num_pages = _geometry(pages, D)
    if hq % heads or q.device != pages.device:
        raise ValueError("q must be on the cache's device with a multiple of its heads")
    batch, stride = _sequences(pages, block_table, cu_seqlens, kv_len)
    return qs, T, hq, D, heads, group, page, num_pages, batch, stride


def kv4_attention(q, pages, block_table, cu_seqlens, kv_len, max_q: int, max_kv: int,
                  scale: Optional[float] = None, causal: bool = True, window: int = 0, out=None,
                  return_lse: bool = False, lse=None, workspace=None, stream=None):
    """softmax(scale q . k) v over the cache for q [T, q_heads, D] (scale: 1 / sqrt(D)
    unless given).  A token sees the slots up to its own (with causal=False all of its
    sequence's; with a window only that many last ones); one that sees none gets zeros.
    max_q, max_kv: at least the most new tokens and slots of any sequence.  Returns out,
    or (out, lse) with return_lse (lse fp32 [T, q_heads], -inf where nothing is seen)."""
    import torch
    qs, T, hq, D, heads, group, page, num_pages, batch, stride = _attention_inputs(q, pages, block_table,
                                                                                   cu_seqlens, kv_len)
    flags = _flag(q.dtype) | (0 if causal else W4A16_NONCAUSAL)
    out = _out(out, q, q.shape, stream)
    outs = _heads("out", out, q)
    if lse is None and return_lse:
        lse = _empty((T, hq), torch.float32, q.device, stream)
    lse_ptr = None if lse is None else _plain("lse", lse, torch.float32, q.device, (T, hq))
    lib = load_library()
    need = lib.w4a16_kv4_attention_workspace_bytes(batch, hq, heads, D, max_q, max_kv, window)
    if workspace is None and need:
        workspace = _empty((need,), torch.uint8, q.device, stream)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _on(q.device):
        _raise(lib.w4a16_kv4_attention(
            q.data_ptr(), qs, pages.data_ptr(), block_table.data_ptr(), cu_seqlens.data_ptr(), kv_len.data_ptr(),
            out.data_ptr(), outs, lse_ptr, T, hq, heads, D, group, page, num_pages, batch, stride, max_q, max_kv,
            D ** -0.5 if scale is None else scale, window, flags,
            None if workspace is None else workspace.data_ptr(), nbytes, _stream_handle(stream)),
            "w4a16_kv4_attention")
    return (out, lse) if return_lse else out


def kv4_attention_mass(q, pages, block_table, cu_seqlens, kv_len, lse, acc, max_q: int, max_kv: int,
                       scale: Optional[float] = None, causal: bool = True, window: int = 0, stream=None):
    """Add to acc (fp32 [batch, kv_heads, slots], slots >= max_kv) the attention weight that
    every cached slot got from this call's queries: the sum of exp(scale q . k - lse) over
    the tokens that see it and the query heads of its head.  The other arguments as
    kv4_attention had and gave them.  Returns acc."""
    import torch
    qs, T, hq, D, heads, group, page, num_pages, batch, stride = _attention_inputs(q, pages, block_table,
                                                                                   cu_seqlens, kv_len)
    flags = _flag(q.dtype) | (0 if causal else W4A16_NONCAUSAL)
    lse_ptr = _plain("lse", lse, torch.float32, q.device, (T, hq))
    acc_ptr = _plain("acc", acc, torch.float32, q.device)
    if acc.dim() != 3 or acc.shape[0] != batch or acc.shape[1] != heads:
        raise ValueError("acc must be [batch, kv_heads, slots]")
    with _on(q.device):
        _raise(load_library().w4a16_kv4_attention_mass(
            q.data_ptr(), qs, pages.data_ptr(), block_table.data_ptr(), cu_seqlens.data_ptr(), kv_len.data_ptr(),
            lse_ptr, acc_ptr, acc.shape[2], T, hq, heads, D, group, page, num_pages, batch, stride, max_q, max_kv,
            D ** -0.5 if scale is None else scale, window, flags, _stream_handle(stream)),
            "w4a16_kv4_attention_mass")
    return acc


def kv4_evict(pages, block_table, kv_len, acc, budget: int, recent: int, dst_table, head_dim: int, max_kv: int,
              stream=None):
    """Cut every sequence and head to at most budget slots: the last `recent` and, of the
    others, those with the largest acc (fp32 [batch, kv_heads, slots >= max_kv]; equal ones:
    the lowest slots).  What is kept is copied, in its order, into the pages of dst_table
    (int32 [batch, pages]; in the same tensor, none of them in use by block_table).  Returns
    (kept int32 [batch, kv_heads, budget], new_len int32 [batch], acc of the kept slots
    fp32 [batch, kv_heads, budget]); -1 and 0 beyond new_len."""
    import torch
    heads, group, page, num_pages = _geometry(pages, head_dim)
    batch, stride = _sequences(pages, block_table, None, kv_len)
    acc_ptr = _plain("acc", acc, torch.float32, pages.device)
    if acc.dim() != 3 or acc.shape[0] != batch or acc.shape[1] != heads:
        raise ValueError("acc must be [batch, kv_heads, slots]")
    dst = _plain("dst_table", dst_table, torch.int32, pages.device)
    if dst_table.dim() != 2 or dst_table.shape[0] != batch:
        raise ValueError("dst_table must be [batch, pages]")
    if budget < 1:
        raise ValueError("budget must be positive")
    kept = _empty((batch, heads, budget), torch.int32, pages.device, stream)
    new_len = _empty((batch,), torch.int32, pages.device, stream)
    acc_out = _empty((batch, heads, budget), torch.float32, pages.device, stream)
    with _on(pages.device):
        _raise(load_library().w4a16_kv4_evict(
            pages.data_ptr(), block_table.data_ptr(), kv_len.data_ptr(), acc_ptr, acc.shape[2], budget, recent, dst,
            dst_table.shape[1], kept.data_ptr(), new_len.data_ptr(), acc_out.data_ptr(), heads, head_dim, group,
            page, num_pages, batch, stride, max_kv, 0, _stream_handle(stream)), "w4a16_kv4_evict")
    return kept, new_len, acc_out
