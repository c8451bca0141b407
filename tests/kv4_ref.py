"""A plain 4-bit key/value cache and its operators in 64 bits on the CPU, written
from the layout and the formulas of include/w4a16.h, element by element where the
library works word by word."""

from __future__ import annotations

import math

import numpy as np
import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}      # unit roundoff


def rounded(x: torch.Tensor, dtype) -> torch.Tensor:
    """float64 -> fp32 -> dtype, as float64 (the inputs are fp32 values)."""
    return x.float().to(dtype).double()


def quantise(x: torch.Tensor, group: int, dtype):
    """Codes, s and m of x [..., D] (fp32 values held in any float type)."""
    y = x.float().reshape(*x.shape[:-1], -1, group)
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = ((hi - lo) * torch.tensor(1 / 15, dtype=torch.float32)).to(dtype).float()
    m = lo.to(dtype).float()
    c = torch.where(s > 0, (y - m) * (1 / s), torch.zeros_like(y)).round().clamp(0, 15)
    return c.reshape(x.shape).to(torch.int64), s[..., 0], m[..., 0]


class Cache:
    """Pages in a shuffled order with every byte set to 0xFF (parameters: NaN) before
    the sequences' slots are written."""

    def __init__(self, lens, heads, D, group, page, dtype, seed, spare=2, room=0):
        self.lens, self.heads, self.D, self.group, self.page, self.dtype = list(lens), heads, D, group, page, dtype
        self.ng = D // group
        self.tile_words = 8 * (D + 8 * self.ng)
        rng = np.random.default_rng(seed)
        need = [max(1, -(-(n + room) // page)) for n in lens]
        self.num_pages = sum(need) + spare
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), max(need, default=1)), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.words = np.full((self.num_pages, heads, page // 32, self.tile_words), 0xFFFFFFFF, dtype=np.uint32)
        self.rng = rng

    # -- the layout --
    def key_at(self, r32, d):
        w = (r32 // 16) * (self.D // 32) + d // 32
        lane = 16 * ((d % 32) // 8) + r32 % 16
        return (w // 4) * 256 + 4 * lane + w % 4, 4 * ((d % 8) // 2 + 4 * (d % 2))

    def value_at(self, r32, d):
        w = d // 16
        lane = 16 * ((r32 % 16) // 4) + d % 16
        return 4 * self.D + (w // 4) * 256 + 4 * lane + w % 4, 4 * (r32 % 4 + 4 * (r32 // 16))

    def param_at(self, value, g, r32):
        return 8 * self.D + (32 * self.ng if value else 0) + 32 * g + r32

    def tile(self, b, t, table=None):
        """Words [heads, tile words] of the tile that holds slot t."""
        page = (self.table if table is None else table)[b, t // self.page]
        return self.words[page, :, (t % self.page) // 32]

    def _bits(self, s, m):
        s16 = s.to(self.dtype).view(torch.int16).numpy().astype(np.uint16).astype(np.uint32)
        m16 = m.to(self.dtype).view(torch.int16).numpy().astype(np.uint16).astype(np.uint32)
        return s16 | (m16 << np.uint32(16))

    def put(self, b, t, k, v):
        """Quantise k, v [heads, D] into slot t of sequence b."""
        words, r32 = self.tile(b, t), t % 32
        d = np.arange(self.D)
        for value, x, place in ((False, k, self.key_at), (True, v, self.value_at)):
            c, s, m = quantise(x, self.group, self.dtype)
            at, shift = place(r32, d)
            shift = np.broadcast_to(shift, d.shape).astype(np.uint32)
            for h in range(self.heads):
                for j in range(self.D):
                    w = int(words[h, at[j]]) & ~(0xF << int(shift[j])) & 0xFFFFFFFF
                    words[h, at[j]] = w | (int(c[h, j]) << int(shift[j]))
            par = self._bits(s, m)
            for g in range(self.ng):
                words[:, self.param_at(value, g, r32)] = par[:, g]

    def get(self, b, t, table=None):
        """(codes, s, m, value) of keys and of values in slot t, each [heads, D] in 64 bits."""
        words, r32 = self.tile(b, t, table), t % 32
        d = np.arange(self.D)
        out = []
        for value, place in ((False, self.key_at), (True, self.value_at)):
            at, shift = place(r32, d)
            c = (words[:, at] >> np.broadcast_to(shift, d.shape).astype(np.uint32)) & 15
            par = words[:, self.param_at(value, d // self.group, r32)]
            half = [torch.from_numpy(((par >> np.uint32(16 * i)) & np.uint32(0xFFFF)).astype(np.uint16).view(np.int16))
                    .view(self.dtype).double() for i in (0, 1)]
            c = torch.from_numpy(c.astype(np.int64)).double()
            out.append((c, half[0], half[1], half[1] + half[0] * c))
        return out

    def fill(self, scale_k=1.0, scale_v=1.0):
        """Random keys and values in every slot in use, whole tiles at a time (the tiles' slots
        beyond the sequence's keep 0xFF parameters)."""
        d = np.arange(self.D)
        for b, n in enumerate(self.lens):
            for t0 in range(0, n, 32):
                words, count = self.tile(b, t0), min(32, n - t0)
                r32 = np.arange(32)
                for value, place, scale in ((False, self.key_at, scale_k), (True, self.value_at, scale_v)):
                    x = torch.from_numpy(self.rng.standard_normal((self.heads, 32, self.D)) * scale).float()
                    c, s, m = quantise(x, self.group, self.dtype)
                    at, shift = place(r32[:, None], d[None, :])
                    at, shift = np.broadcast_arrays(at, shift)
                    c = c.numpy().astype(np.uint32) << shift.astype(np.uint32)
                    for h in range(self.heads):
                        lo = 4 * self.D if value else 0
                        words[h, lo:lo + 4 * self.D] = 0
                        np.bitwise_or.at(words[h], at.ravel(), c[h].ravel())
                    par = self._bits(s, m)
                    for g in range(self.ng):
                        words[:, self.param_at(value, g, r32[:count])] = par[:, :count, g]

    def poison(self, b, t):
        """NaN parameters in slot t of sequence b."""
        for value in (False, True):
            for g in range(self.ng):
                self.tile(b, t)[:, self.param_at(value, g, t % 32)] = 0xFFFFFFFF

    def sequence(self, b):
        """(key values, value codes - 8, value s, values) of sequence b: [heads, slots, D]."""
        n = self.lens[b]
        if n == 0:
            z = torch.zeros(self.heads, 0, self.D, dtype=torch.float64)
            return z, z, z, z
        got = [self.get(b, t) for t in range(n)]
        return (torch.stack([g[0][3] for g in got], 1), torch.stack([g[1][0] - 8 for g in got], 1),
                torch.stack([g[1][1] for g in got], 1), torch.stack([g[1][3] for g in got], 1))

    def pages(self, dev):
        w = torch.from_numpy(self.words.view(np.uint8).copy())
        return w.reshape(self.num_pages, self.heads, self.page // 32, 4 * self.tile_words).to(dev)

    def back(self, pages):
        """Take over what a device tensor of pages holds."""
        self.words = pages.cpu().numpy().reshape(self.num_pages, self.heads, self.page // 32, -1).copy().view(np.uint32)


def sees(i, n, length, causal=True, window=0):
    """[lo, hi) of the slots that new token i of n sees."""
    hi = min(length, length - n + i + 1) if causal else length
    lo = max(0, length - n + i + 1 - window) if window else 0
    return lo, max(lo, hi)


def attention(cache: Cache, q, ns, scale, causal=True, window=0):
    """q [T, q_heads, D] of sequences with ns[b] new tokens.  Returns out, lse, the
    magnitudes sum p s |c - 8| and sum p |v|, the logits' magnitude max sum |q| |k|, and
    the weights per sequence [heads, group, n, slots]."""
    T, hq, D = q.shape
    G = hq // cache.heads
    out = torch.zeros(T, hq, D, dtype=torch.float64)
    rough, mag = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    size = torch.zeros(T, hq, dtype=torch.float64)
    weights, at = [], 0
    for b, n in enumerate(ns):
        k, c8, s, v = cache.sequence(b)
        length = cache.lens[b]
        p_all = torch.zeros(cache.heads, G, n, length, dtype=torch.float64)
        for i in range(n):
            lo, hi = sees(i, n, length, causal, window)
            if hi <= lo:
                continue
            for h in range(cache.heads):
                qq = q[at + i, h * G:(h + 1) * G].double()
                z = scale * (qq @ k[h, lo:hi].T)
                p = torch.softmax(z, -1)
                rows = slice(h * G, (h + 1) * G)
                out[at + i, rows] = p @ v[h, lo:hi]
                rough[at + i, rows] = p @ (s[h, lo:hi] * c8[h, lo:hi].abs())
                mag[at + i, rows] = p @ (v[h, lo:hi].abs() + 24 * s[h, lo:hi])
                lse[at + i, rows] = torch.logsumexp(z, -1)
                size[at + i, rows] = scale * (qq.abs() @ (k[h, lo:hi].abs()).T).amax(-1)
                p_all[h, :, i, lo:hi] = p
        weights.append(p_all)
        at += n
    return out, lse, rough, mag, size, weights


def norm_rope(x, weight, cos, sin, pos, interleaved, eps):
    """x [T, heads, D] in 64 bits; weight, cos may be None."""
    x = x.double().clone()
    if weight is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * weight.double()
    if cos is not None:
        half = cos.shape[1]
        c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
        i = torch.arange(half)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        xa, xb = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
    return x


def evict_slots(acc, length, budget, recent):
    """The kept slots of one head, in order."""
    if length <= budget:
        return list(range(length))
    old = length - recent
    key = [(0 if math.isnan(a) else 1, -a if not math.isnan(a) else 0.0, t) for t, a in enumerate(acc[:old])]
    return sorted(t for _, _, t in sorted(key)[:budget - recent]) + list(range(old, length))
