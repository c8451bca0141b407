"""The operators around a 4-bit key/value cache, as cases to measure.

Between the merged QKV linear and the output linear an attention block prepares queries and keys
(a norm for each head and the position rotation), stores keys and values in 4 bits, attends over
that cache, adds up how much weight every cached slot got, and drops the slots with the least.
Each case is one pass through one of these five operators:

  norm_rope  qk_norm_rope: RMS norm of each query and key head and the rotation, 16-bit results
  append     kv4_append: the same norm and rotation, keys and values quantised into the cache, and
             the stored values read back (kv4_read)
  attention  kv4_attention: softmax attention of a few or many queries over the cache
  mass       kv4_attention_mass: the attention weight of every cached slot, added over the queries
  evict      kv4_evict: the slots with most weight and the recent ones kept, compacted into other
             pages, and what was kept read back (kv4_read)

The cache.  A page holds page_size slots (tokens) of every key/value head; `pages` is uint8
[pages, kv_heads, page_size / 32, tile bytes], a tile being 32 slots of one head.  A group of
`group` neighbouring channels of one slot has a step s and an offset m in the activation type, and
4-bit codes c: the value is m + s c, with m = round(min), s = round((max - min) / 15) and c the
nearest code.  With word = int32, lane = 16 b + r (b < 4, r < 16), w < head_dim / 16:
  words [head_dim/64][64 lanes][4]   key codes, w = 4 chunk + i: slot 16 (w / (head_dim/32)) + r,
                                     channels 32 (w mod (head_dim/32)) + 8 b + 2 (n mod 4) + n / 4
                                     in nibble n
  words [head_dim/64][64 lanes][4]   value codes: channel 16 w + r, slot 4 b + n mod 4 + 16 (n / 4)
                                     in nibble n
  words [head_dim/group][32 slots]   key parameters, s in the low half and m in the high half
  words [head_dim/group][32 slots]   value parameters
"""

import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


# ---- the cases ----

def listed():
    return [
        # one new token of one sequence: the smallest call of a decode step
        dict(name="norm_rope_token", op="norm_rope", dtype="bf16", T=1, hq=40, hk=8, d=128, rot=128,
             interleaved=False),
        # a prompt of several thousand tokens, interleaved pairs, half of each head rotated
        dict(name="norm_rope_prompt", op="norm_rope", dtype="f16", T=8192, hq=32, hk=8, d=128, rot=64,
             interleaved=True),
        # one decode step of a served batch: one token for each sequence
        dict(name="append_batch", op="append", dtype="bf16", B=64, n_min=1, n_max=1, kv_min=300,
             kv_max=6000, hq=40, hk=8, d=128, rot=128, interleaved=False, group=64, page=64),
        # ragged chunks of prompts, wide heads, a partial rotation
        dict(name="append_prompts", op="append", dtype="f16", B=3, n_min=901, n_max=2500, kv_min=901,
             kv_max=7000, hq=16, hk=4, d=256, rot=64, interleaved=False, group=128, page=256),
        # decode of one short sequence: latency counts
        dict(name="attend_short", op="attention", dtype="bf16", B=1, n_min=1, n_max=1, kv_min=700,
             kv_max=700, hq=40, hk=8, d=128, group=64, page=64, window=0),
        # decode of one very long context
        dict(name="attend_long", op="attention", dtype="bf16", B=1, n_min=1, n_max=1, kv_min=131071,
             kv_max=131071, hq=40, hk=8, d=128, group=128, page=256, window=0),
        # decode of a ragged batch, finest groups
        dict(name="attend_batch", op="attention", dtype="f16", B=32, n_min=1, n_max=1, kv_min=1000,
             kv_max=24000, hq=32, hk=8, d=128, group=32, page=32, window=0),
        # chunked prefill of two prompts over what their caches hold
        dict(name="attend_prompts", op="attention", dtype="bf16", B=2, n_min=1500, n_max=2500,
             kv_min=6000, kv_max=12000, hq=40, hk=8, d=128, group=64, page=128, window=0),
        # weights of a decode step of a batch whose caches will be cut
        dict(name="mass_batch", op="mass", dtype="bf16", B=8, n_min=1, n_max=1, kv_min=2000,
             kv_max=16000, hq=40, hk=8, d=128, group=64, page=64, window=0),
        # weights of a prompt's last chunk
        dict(name="mass_prompt", op="mass", dtype="f16", B=1, n_min=2048, n_max=2048, kv_min=8191,
             kv_max=8191, hq=32, hk=8, d=128, group=128, page=128, window=0),
        # one sequence cut to a quarter
        dict(name="evict_one", op="evict", dtype="bf16", B=1, kv_min=8192, kv_max=8192, hk=8, d=128,
             group=64, page=64, budget=2048, recent=256),
        # a ragged batch cut to one budget; the shortest sequences fit and keep all
        dict(name="evict_batch", op="evict", dtype="f16", B=16, kv_min=3000, kv_max=33001, hk=8, d=128,
             group=64, page=128, budget=4096, recent=1024),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attention", "attention", "mass", "evict"])
    d = rng.choice([64, 128, 128, 256])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 4, 5, 7, 8])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]))
    rope = dict(hq=hq, hk=hk, d=d, rot=rng.choice([d, d // 2, d // 4]), interleaved=rng.random() < 0.5)
    if op == "norm_rope":
        return dict(c, T=_log(rng, 1, 6000), **rope)
    cache = dict(hk=hk, d=d, group=rng.choice([32, 64] if d == 64 else [32, 64, 128]),
                 page=rng.choice([32, 64, 96, 256]))
    if op == "append":
        B = _log(rng, 1, 64)
        n = _log(rng, 1, 4000 // B)
        kv = n + _log(rng, 1, 4000)
        return dict(c, B=B, n_min=rng.randint(1, n), n_max=n, kv_min=n, kv_max=kv, **{**rope, **cache})
    if op == "evict":
        B = _log(rng, 1, 12)
        kv = _log(rng, 500, 30000)
        budget = rng.randint(kv // 8, kv // 2)
        return dict(c, B=B, kv_min=rng.randint(kv // 8, kv), kv_max=kv, budget=budget,
                    recent=rng.randint(0, budget // 2), **cache)
    few = rng.random() < 0.6
    if few:         # decode: one token, or a few drafted ones
        B = _log(rng, 1, 32)
        n = rng.choice([1, 1, 1, 2, 3, 5])
        kv = n + _log(rng, 100, 300000 // B)
    else:           # prompts and chunks of them
        B = _log(rng, 1, 4)
        n = _log(rng, 60, 4000 // B)
        kv = n + _log(rng, 1, 6000)
    return dict(c, B=B, n_min=rng.randint(1, n), n_max=n, kv_min=rng.randint(n, kv), kv_max=kv, hq=hq,
                window=rng.choice([0, 0, 0, 1000]), **cache)


def _spread(lo, hi, B):
    """B whole numbers from hi down to lo."""
    return [hi] if B == 1 else [hi - (hi - lo) * b // (B - 1) for b in range(B)]


def _lengths(case):
    """New tokens and slots in use (the new ones among them) of every sequence."""
    kv = _spread(case["kv_min"], case["kv_max"], case["B"])
    return [min(n, k) for n, k in zip(_spread(case["n_min"], case["n_max"], case["B"])[::-1], kv)], kv


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def _seen(n, kv, window):
    """Pairs of a query and a slot it sees: query i of n sits in slot kv - n + i."""
    if not window:
        return n * kv - n * (n - 1) // 2
    return sum(min(kv - n + i + 1, window) for i in range(n))


def work(case):
    op = case["op"]
    if op == "norm_rope":
        T, heads = case["T"], case["hq"] + case["hk"]
        return {"bytes": 4 * T * heads * case["d"] + 4 * T * case["rot"] + 4 * T, "flops": 10 * T * heads * case["d"]}
    d, hk = case["d"], case["hk"]
    slot = hk * (d + 8 * (d // case["group"]))      # bytes of one slot of all heads
    if op == "append":
        T = sum(_lengths(case)[0])
        # queries in and out, keys and values in, the cache written and read, values out
        return {"bytes": T * (4 * case["hq"] * d + 4 * hk * d + 4 * case["rot"] + 2 * slot + 4 * hk * d),
                "flops": T * (10 * case["hq"] + 20 * hk) * d}
    if op == "evict":
        kv = _spread(case["kv_min"], case["kv_max"], case["B"])
        new = [min(k, case["budget"]) for k in kv]
        # weights in; the kept slots read and written, read again and given out as values
        return {"bytes": 4 * hk * sum(kv) + sum(new) * (3 * slot + 4 * hk * d + 8 * hk), "flops": hk * sum(kv)}
    ns, kvs = _lengths(case)
    T, hq, w = sum(ns), case["hq"], case["window"]
    slots = sum(min(k, w + n) if w else k for n, k in zip(ns, kvs))
    pairs = sum(_seen(n, k, w) for n, k in zip(ns, kvs))
    if op == "mass":
        return {"bytes": slots * (slot // 2 + 8 * hk) + T * hq * (2 * d + 4), "flops": 2 * d * hq * pairs}
    return {"bytes": slots * slot + T * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}


# ---- the inputs ----

def _groups(x, group):
    return x.reshape(*x.shape[:-1], x.shape[-1] // group, group)


def _quantise(x, group, dtype):
    """Codes (0..15), s and m of x [..., d] in 32 bits; s and m hold values of `dtype`."""
    y = _groups(x, group)
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s, m = ((hi - lo) / 15).to(dtype).float(), lo.to(dtype).float()
    c = torch.where(s > 0, (y - m) * (1 / s), torch.zeros_like(y)).round().clamp(0, 15)
    return c, s, m


def _words(c):
    """Codes [..., 8], nibble n last, as int32 words."""
    return (c.to(torch.int64) << (4 * torch.arange(8, device=DEV))).sum(-1).to(torch.int32)


def _tiles(k, v, group, dtype):
    """k, v [heads, tiles, 32, d] (32 bits) as tiles, uint8 [heads, tiles, tile bytes]."""
    H, N, _, d = k.shape
    ck, sk, mk = _quantise(k, group, dtype)
    cv, sv, mv = _quantise(v, group, dtype)
    # slots (sub, r), channels (j, b, half, odd): words in the order (sub, j), lanes (b, r)
    ck = ck.reshape(H, N, 2, 16, d // 32, 4, 4, 2).permute(0, 1, 2, 4, 5, 3, 7, 6)
    wk = _words(ck.reshape(H, N, d // 64, 4, 64, 8)).transpose(-1, -2)
    # slots (half, b, i), channels (w, r)
    cv = cv.reshape(H, N, 2, 4, 4, d // 16, 16).permute(0, 1, 5, 3, 6, 2, 4)
    wv = _words(cv.reshape(H, N, d // 64, 4, 64, 8)).transpose(-1, -2)
    parts = [wk, wv]
    for s, m in ((sk, mk), (sv, mv)):
        sm = torch.cat([s, m], -1).to(dtype).transpose(2, 3).contiguous()      # [H, N, groups, 32, 2]
        parts.append(sm.view(torch.int32))
    return torch.cat([p.reshape(H, N, -1) for p in parts], -1).contiguous().view(torch.uint8)


def _inputs(g, case, T):
    """Keys and values as the linear gives them: channels differ in size."""
    d, hk, dt = case["d"], case["hk"], TYPES[case["dtype"]]
    size = torch.exp(0.2 * torch.randn(hk, d, generator=g, device=DEV))
    return (torch.randn(T, hk, d, generator=g, device=DEV) * size).to(dt)


def _cache(g, case, kvs, extra=0):
    """Pages with the sequences' slots filled, in an order that says nothing, and their table; `extra`
    more pages for each sequence in a second table."""
    page, hk, d = case["page"], case["hk"], case["d"]
    need = [-(-k // page) for k in kvs]
    wide = max(need)
    count = sum(need) + extra * len(kvs)
    order = torch.randperm(count, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(kvs), wide, dtype=torch.int32, device=DEV)
    at = 0
    per = page // 32
    tile = 32 * (d + 8 * (d // case["group"]))
    pages = torch.empty(count, hk, per, tile, dtype=torch.uint8, device=DEV)
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        k, v = (_inputs(g, case, n * page).float().reshape(n * per, 32, hk, d).permute(2, 0, 1, 3)
                for _ in range(2))
        t = _tiles(k, v, case["group"], TYPES[case["dtype"]])
        pages[order[at:at + n].long()] = t.reshape(hk, n, per, tile).transpose(0, 1)
        at += n
    more = order[at:].reshape(len(kvs), extra).contiguous() if extra else None
    return pages, table, more


def _rope_inputs(g, case, T, first):
    """The QKV linear's output, split as views, norm weights, the tables and the tokens' positions."""
    d, hq, hk, dt = case["d"], case["hq"], case["hk"], TYPES[case["dtype"]]
    qkv = (2 * torch.randn(T, (hq + 2 * hk) * d, generator=g, device=DEV)).to(dt)
    q, k, v = qkv.split([hq * d, hk * d, hk * d], 1)
    weight = [1 + 0.1 * torch.randn(d, generator=g, device=DEV) for _ in range(2)]
    length = 16384
    rate = 1e6 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / case["rot"])
    angle = torch.arange(length, dtype=torch.float64, device=DEV)[:, None] * rate
    return dict(q=q.view(T, hq, d), k=k.view(T, hk, d), v=v.view(T, hk, d), qw=weight[0], kw=weight[1],
                cos=angle.cos().float(), sin=angle.sin().float(), pos=first)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op == "norm_rope":
        first = torch.randint(0, 16384 - case["T"], (1,), generator=g, device=DEV, dtype=torch.int32)
        pos = first + torch.arange(case["T"], dtype=torch.int32, device=DEV)
        return dict(case=case, **_rope_inputs(g, case, case["T"], pos))
    if op == "evict":
        kvs = _spread(case["kv_min"], case["kv_max"], case["B"])
        new = [min(k, case["budget"]) for k in kvs]
        pages, table, dst = _cache(g, case, kvs, -(-case["budget"] // case["page"]))
        # weights after many steps: a few large, most small, some never attended to and equal
        acc = torch.exp(2 * torch.randn(case["B"], case["hk"], max(kvs), generator=g, device=DEV) - 4)
        acc = torch.where(torch.rand(acc.shape, generator=g, device=DEV) < 0.05, torch.zeros_like(acc), acc)
        return dict(case=case, pages=pages, table=table, dst=dst, acc=acc, cu=_starts(new), rows=sum(new),
                    kv=torch.tensor(kvs, dtype=torch.int32, device=DEV), max_kv=max(kvs))
    ns, kvs = _lengths(case)
    pages, table, _ = _cache(g, case, kvs)
    T = sum(ns)
    s = dict(case=case, pages=pages, table=table, cu=_starts(ns), rows=T, max_n=max(ns), max_kv=max(kvs),
             kv=torch.tensor(kvs, dtype=torch.int32, device=DEV))
    if op == "append":
        pos = torch.cat([torch.arange(k - n, k, dtype=torch.int32) for n, k in zip(ns, kvs)]).to(DEV)
        return dict(s, **_rope_inputs(g, case, T, pos))
    # queries that prefer some slots: logits of a standard deviation of about 2
    s["q"] = (2 * torch.randn(T, case["hq"], case["d"], generator=g, device=DEV)).to(TYPES[case["dtype"]])
    if op == "mass":
        s["lse"] = _attention(s, need_out=False)["lse"]
        s["acc"] = torch.rand(case["B"], case["hk"], max(kvs), generator=g, device=DEV)
    return s


# ---- the operators, in elementary operations and 32 bits ----

def _norm_rope(x, weight, s):
    """x [T, heads, d] in 32 bits: RMS norm over d, then the rotation of the first `rot` channels."""
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    at = s["pos"].long()
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    y = x[..., :rot]
    a, b = (y[..., ::2], y[..., 1::2]) if inter else (y[..., :rot // 2], y[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _values(s, table):
    """Every slot of the table's pages in 32 bits: k, v [B, heads, slots, d]."""
    case = s["case"]
    d, hk, group, dt = case["d"], case["hk"], case["group"], TYPES[case["dtype"]]
    B, n = table.shape
    t = s["pages"][table.reshape(-1).long()].view(torch.int32)       # [B n, heads, tiles, words]
    t = t.reshape(B, n, hk, t.shape[2], -1).transpose(1, 2).reshape(B, hk, -1, t.shape[-1])
    N, half, par = t.shape[2], 16 * d // 4, 32 * (d // group)
    shift = 4 * torch.arange(8, device=DEV, dtype=torch.int32)

    def codes(w):       # [B, heads, tiles, d/16 words, 64 lanes, 8 nibbles]
        w = w.reshape(B, hk, N, d // 64, 64, 4).transpose(-1, -2).reshape(B, hk, N, d // 16, 64)
        return ((w[..., None] >> shift) & 15).float()

    def values(c, p):   # codes [B, heads, tiles, 32, d] and parameters
        p = p.contiguous().view(dt).reshape(B, hk, N, d // group, 32, 2).transpose(3, 4).float()
        x = _groups(c, group) * p[..., :1] + p[..., 1:]
        return x.reshape(B, hk, N * 32, d)

    ck = codes(t[..., :half]).reshape(B, hk, N, 2, d // 32, 4, 16, 2, 4)     # sub, j, b, r, odd, half
    ck = ck.permute(0, 1, 2, 3, 6, 4, 5, 8, 7).reshape(B, hk, N, 32, d)
    cv = codes(t[..., half:2 * half]).reshape(B, hk, N, d // 16, 4, 16, 2, 4)    # w, b, r, half, i
    cv = cv.permute(0, 1, 2, 6, 4, 7, 3, 5).reshape(B, hk, N, 32, d)
    return values(ck, t[..., 2 * half:2 * half + par]), values(cv, t[..., 2 * half + par:])


def _padded(x, s):
    """Rows [T, heads, d] as [B, heads, most new tokens, d], and which of those are there."""
    i = torch.arange(s["max_n"], device=DEV)
    start = s["cu"][:-1, None].long()
    there = i < s["cu"][1:, None] - start
    at = torch.where(there, start + i, torch.zeros_like(start))
    return x[at].transpose(1, 2), there, at


def _logits(s, k):
    """Scaled and masked logits [B, heads, group of query heads, new tokens, slots]."""
    case = s["case"]
    q, there, at = _padded(s["q"].float(), s)
    B, hk, S, d = k.shape
    G = case["hq"] // hk
    z = (q.reshape(B, hk, G * s["max_n"], d) @ k.transpose(-1, -2)) / math.sqrt(d)
    slot = torch.arange(S, device=DEV)
    last = (s["kv"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + torch.arange(s["max_n"], device=DEV)
    see = (slot <= last[..., None]) & there[..., None]
    if case["window"]:
        see = see & (slot > last[..., None] - case["window"])
    see = see[:, None, None]
    return z.reshape(B, hk, G, s["max_n"], S).masked_fill_(~see, -math.inf), there, at


def _attention(s, need_out=True):
    case = s["case"]
    k, v = _values(s, s["table"])
    z, there, at = _logits(s, k)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0].flatten(1, 2).transpose(1, 2)[there]
    if not need_out:
        return {"lse": lse.contiguous()}
    B, hk, G, n, S = p.shape
    o = (p / torch.where(total > 0, total, torch.ones_like(total))).reshape(B, hk, G * n, S) @ v
    o = o.reshape(B, hk * G, n, -1).transpose(1, 2)[there]
    return {"out": o.to(TYPES[case["dtype"]]), "lse": lse.contiguous()}


def _mass(s):
    k, _ = _values(s, s["table"])
    z, there, at = _logits(s, k)
    lse, _, _ = _padded(s["lse"][..., None], s)             # [B, query heads, n, 1]
    p = torch.exp(z - lse.reshape(*z.shape[:4], 1))
    add = p.sum((2, 3))[..., :s["max_kv"]]
    s["acc"] += add
    return {"acc": s["acc"]}


def _evict(s):
    case = s["case"]
    slot = torch.arange(s["max_kv"], device=DEV)
    kv = s["kv"][:, None, None]
    key = torch.where(slot >= kv - case["recent"], torch.full_like(s["acc"], math.inf), s["acc"])
    key = torch.where(slot >= kv, torch.full_like(key, -math.inf), key)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :case["budget"]]
    kept = torch.sort(order, dim=-1).values
    new = torch.minimum(s["kv"], torch.full_like(s["kv"], case["budget"]))
    there = torch.arange(kept.shape[-1], device=DEV) < new[:, None, None]
    acc = torch.where(there, torch.gather(s["acc"], 2, kept), torch.zeros_like(kept, dtype=torch.float32))
    k, v = _values(s, s["table"])
    rows = there[:, 0]
    at = kept[..., None].expand(*kept.shape, case["d"])
    k, v = (torch.gather(x, 2, at).transpose(1, 2)[rows].to(TYPES[case["dtype"]]) for x in (k, v))
    return {"kept": torch.where(there, kept, torch.full_like(kept, -1)).to(torch.int32), "len": new,
            "acc": acc, "k": k, "v": v}


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    dt = TYPES[case["dtype"]]
    if case["op"] == "norm_rope":
        return {"q": _norm_rope(s["q"], s["qw"], s).to(dt), "k": _norm_rope(s["k"], s["kw"], s).to(dt)}
    if case["op"] == "append":
        q = _norm_rope(s["q"], s["qw"], s).to(dt)
        stored = []
        for x in (_norm_rope(s["k"], s["kw"], s), s["v"].float()):
            c, step, m = _quantise(x, case["group"], dt)
            stored.append((c * step + m).reshape(x.shape).to(dt))
        return {"q": q, "k": stored[0], "v": stored[1]}
    return {"attention": _attention, "mass": _mass, "evict": _evict}[case["op"]](s)


def _run_own(s):
    import int4_weight_only_w4a16_amd as w4
    case = s["case"]
    op = case["op"]
    if op == "norm_rope":
        q, k = w4.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["pos"], eps=EPS,
                               interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if op == "append":
        q = w4.kv4_append(s["pages"], s["k"], s["v"], s["table"], s["cu"], s["kv"], s["max_n"], q=s["q"],
                          q_weight=s["qw"], k_weight=s["kw"], cos=s["cos"], sin=s["sin"],
                          positions=s["pos"], eps=EPS, interleaved=case["interleaved"])
        k, v = w4.kv4_read(s["pages"], s["table"], s["cu"], s["kv"], s["rows"], case["d"], q.dtype)
        return {"q": q, "k": k, "v": v}
    if op == "attention":
        out, lse = w4.kv4_attention(s["q"], s["pages"], s["table"], s["cu"], s["kv"], s["max_n"], s["max_kv"],
                                    window=case["window"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "mass":
        return {"acc": w4.kv4_attention_mass(s["q"], s["pages"], s["table"], s["cu"], s["kv"], s["lse"],
                                             s["acc"], s["max_n"], s["max_kv"], window=case["window"])}
    kept, new, acc = w4.kv4_evict(s["pages"], s["table"], s["kv"], s["acc"], case["budget"], case["recent"],
                                  s["dst"], case["d"], s["max_kv"])
    k, v = w4.kv4_read(s["pages"], s["dst"], s["cu"], new, s["rows"], case["d"], TYPES[case["dtype"]])
    return {"kept": kept, "len": new, "acc": acc, "k": k, "v": v}


# ---- the operators from their definition, in 64 bits ----

def _exact_slots(s, b, count):
    """Slots 0 .. count - 1 of sequence b: k, v [heads, count, d], word by word from the layout."""
    case = s["case"]
    d, group, dt, page = case["d"], case["group"], TYPES[case["dtype"]], case["page"]
    t = torch.arange(count, device=DEV)
    words = s["pages"].view(torch.int32)[s["table"][b, t // page].long(), :, (t % page) // 32]   # [count, heads, words]
    words = words.transpose(0, 1)
    r = (t % 32)[:, None]
    c = torch.arange(d, device=DEV)[None]
    key_w = (r // 16) * (d // 32) + c // 32
    key_at = (key_w // 4) * 256 + 4 * (16 * ((c % 32) // 8) + r % 16) + key_w % 4
    key_n = (c % 8) // 2 + 4 * (c % 2)
    val_at = 4 * d + (c // 64) * 256 + 4 * (16 * ((r % 16) // 4) + c % 16) + (c // 16) % 4
    val_n = r % 4 + 4 * (r // 16) + 0 * c
    found = []
    for at, n, base in ((key_at, key_n, 8 * d), (val_at, val_n, 8 * d + 32 * (d // group))):
        code = torch.gather(words, 2, at.expand(words.shape[0], count, d))
        code = torch.bitwise_and(code >> (4 * n).to(torch.int32), 15).double()
        par = torch.gather(words, 2, (base + 32 * (c // group) + r).expand(words.shape[0], count, d))
        par = par.contiguous().view(dt).reshape(*par.shape, 2).double()
        found.append(par[..., 1] + par[..., 0] * code)
    return found


def _exact_rope(x, weight, s):
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    i = torch.arange(rot // 2, device=DEV)
    first, second = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    turn = torch.complex(s["cos"].double()[s["pos"].long()], s["sin"].double()[s["pos"].long()])[:, None]
    z = torch.complex(x[..., first], x[..., second]) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_stored(x, group, dtype):
    y = _groups(x, group)
    m = y.min(-1, keepdim=True).values
    s = ((y.max(-1, keepdim=True).values - m) / 15).to(dtype).double()
    m = m.to(dtype).double()
    return (m + s * ((y - m) / s).round().clamp(0, 15)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    if op == "norm_rope":
        return {"q": _exact_rope(s["q"], s["qw"], s), "k": _exact_rope(s["k"], s["kw"], s)}
    if op == "append":
        return {"q": _exact_rope(s["q"], s["qw"], s),
                "k": _exact_stored(_exact_rope(s["k"], s["kw"], s), case["group"], dt),
                "v": _exact_stored(s["v"].double(), case["group"], dt)}
    hk, d = case["hk"], case["d"]
    if op == "evict":
        kept = torch.full((case["B"], hk, case["budget"]), -1, dtype=torch.int32, device=DEV)
        acc = torch.zeros(kept.shape, dtype=torch.float64, device=DEV)
        new, rows = [], [[], []]
        for b, n in enumerate(s["kv"].tolist()):
            new.append(min(n, case["budget"]))
            old = max(0, n - case["recent"])
            for h in range(hk):
                at = torch.arange(n, device=DEV)
                if n > case["budget"]:
                    best = torch.argsort(-s["acc"][b, h, :old].double(), stable=True)[:new[-1] - (n - old)]
                    at = torch.cat([best.sort().values, at[old:]])
                kept[b, h, :new[-1]] = at.to(torch.int32)
            full = _exact_slots(s, b, n)
            at = kept[b, :, :new[-1]].long()
            acc[b, :, :new[-1]] = torch.gather(s["acc"][b].double(), 1, at)
            for rs, x in zip(rows, full):
                rs.append(torch.gather(x, 1, at[..., None].expand(hk, new[-1], d)).transpose(0, 1))
        return {"kept": kept, "len": torch.tensor(new, dtype=torch.int32, device=DEV), "acc": acc,
                "k": torch.cat(rows[0]), "v": torch.cat(rows[1])}
    G = case["hq"] // hk
    outs, lses = [], []
    acc = s["acc"].double() if op == "mass" else None
    cu = s["cu"].tolist()
    for b, kv in enumerate(s["kv"].tolist()):
        n = cu[b + 1] - cu[b]
        k, v = _exact_slots(s, b, kv)
        q = s["q"][cu[b]:cu[b + 1]].double().reshape(n, hk, G, d)
        at = torch.arange(kv - n, kv, device=DEV)[:, None]
        slot = torch.arange(kv, device=DEV)
        hide = (slot > at) | (slot <= at - case["window"] if case["window"] else slot < 0)
        for h in range(hk):
            z = (q[:, h].reshape(n * G, d) @ k[h].T).reshape(n, G, kv) * d ** -0.5
            z = z.masked_fill(hide[:, None], -math.inf)
            if op == "mass":
                lse = s["lse"][cu[b]:cu[b + 1]].double().reshape(n, hk, G)[:, h]
                acc[b, h, :kv] += torch.exp(z - lse[..., None]).sum((0, 1))
                continue
            lses.append(torch.logsumexp(z, -1))
            outs.append((torch.softmax(z, -1).reshape(n * G, kv) @ v[h]).reshape(n, G, d))
        if op == "attention":
            outs[b:] = [torch.stack(outs[b:], 1).reshape(n, hk * G, d)]
            lses[b:] = [torch.stack(lses[b:], 1).reshape(n, hk * G)]
    if op == "mass":
        return {"acc": acc}
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
