"""Token mixing by the gated delta rule, and trees of drafted tokens, as cases to measure.

Beside attention layers a decoder may have layers that mix tokens through a state of fixed size: a
short causal convolution of the merged projection's channels, then the gated delta rule.  And a
decode step may check several candidate continuations at once, a tree of drafted tokens, through
either kind of layer.  Each case is one pass through one of these operators:

  conv       short_conv: depthwise causal convolution and SiLU over [state, tokens], the state moved on
  delta      gated_delta_rule: for each value head, from S (Dk x Dv) of the sequence's state
               S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = S^T q / sqrt(Dk)
             with k and q of unit length, g = -exp(a_log) softplus(a + dt_bias), beta = sigmoid(b)
  attention  kv4_tree_attention: softmax attention of drafted tokens over the 4-bit cache

A tree is an int64 for each token: bit j says that it descends from its sequence's new token j.  A
token sees what came before the new tokens, its ancestors and itself; states stay as they are.

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
import random

import torch

own = False

EPS = 1e-6
CHUNK = 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


# ---- the cases ----

def listed():
    return [
        # one new token of one sequence: the smallest call of a decode step
        dict(name="conv_token", op="conv", dtype="bf16", B=1, n_min=1, n_max=1, channels=10240, width=4,
             fresh=0, tree=False),
        # prompts of several lengths, half of them continued from an earlier chunk
        dict(name="conv_prompts", op="conv", dtype="bf16", B=3, n_min=1700, n_max=5001, channels=10240, width=4,
             fresh=1, tree=False),
        # drafted tokens of a served batch
        dict(name="conv_drafts", op="conv", dtype="f16", B=16, n_min=9, n_max=40, channels=8192, width=4,
             fresh=0, tree=True),
        # one new token of one sequence
        dict(name="delta_token", op="delta", dtype="bf16", B=1, n_min=1, n_max=1, hk=16, hv=48, dk=128, dv=128,
             fresh=0, tree=False),
        # a decode step of a served batch: the states are what has to be moved
        dict(name="delta_batch", op="delta", dtype="bf16", B=64, n_min=1, n_max=1, hk=16, hv=48, dk=128, dv=128,
             fresh=0, tree=False),
        # a chain of a few accepted tokens for each sequence
        dict(name="delta_accepted", op="delta", dtype="f16", B=12, n_min=1, n_max=5, hk=16, hv=32, dk=128, dv=128,
             fresh=0, tree=False),
        # one long prompt
        dict(name="delta_prompt", op="delta", dtype="bf16", B=1, n_min=8191, n_max=8191, hk=16, hv=48, dk=128, dv=128,
             fresh=1, tree=False),
        # ragged prompts, some of them continued, narrower keys
        dict(name="delta_prompts", op="delta", dtype="f16", B=5, n_min=333, n_max=2500, hk=8, hv=32, dk=64, dv=128,
             fresh=3, tree=False),
        # drafted tokens of a served batch
        dict(name="delta_drafts", op="delta", dtype="bf16", B=8, n_min=12, n_max=47, hk=16, hv=48, dk=128, dv=128,
             fresh=0, tree=True),
        # a few drafted tokens over a short cache: latency counts
        dict(name="attend_drafts_short", op="attention", dtype="bf16", B=1, n_min=7, n_max=7, kv_min=1000, kv_max=1000,
             hq=40, hk=8, d=128, group=64, page=64, window=0),
        # a served batch with trees of several sizes
        dict(name="attend_drafts_batch", op="attention", dtype="bf16", B=12, n_min=5, n_max=37, kv_min=900,
             kv_max=12000, hq=40, hk=8, d=128, group=64, page=64, window=0),
        # the largest tree over one long context, finest groups
        dict(name="attend_drafts_long", op="attention", dtype="f16", B=1, n_min=64, n_max=64, kv_min=65000,
             kv_max=65000, hq=32, hk=8, d=128, group=32, page=128, window=0),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "delta", "delta", "attention"])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]))
    if op == "attention":
        d = rng.choice([64, 128, 128, 256])
        hk = rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 16)
        n = _log(rng, 1, 64)
        kv = n + _log(rng, 50, 60000 // B)
        return dict(c, B=B, n_min=rng.randint(1, n), n_max=n, kv_min=rng.randint(n, kv), kv_max=kv, hk=hk,
                    hq=hk * rng.choice([1, 2, 4, 5, 8]), d=d, group=rng.choice([32, 64] if d == 64 else [32, 64, 128]),
                    page=rng.choice([32, 64, 96, 256]), window=rng.choice([0, 0, 0, 1000]))
    form = rng.choice(["tokens", "prompts", "drafts"])
    if form == "tokens":
        B = _log(rng, 1, 64)
        n = rng.choice([1, 1, 1, 2, 3, 6])
    elif form == "drafts":
        B = _log(rng, 1, 8)
        n = _log(rng, 1, 64)
    else:
        B = _log(rng, 1, 6)
        n = _log(rng, 10, 6000 // B)
    c.update(B=B, n_min=rng.randint(1, n), n_max=n, fresh=0 if form == "drafts" else rng.randint(0, B),
             tree=form == "drafts")
    if op == "conv":
        return dict(c, channels=8 * _log(rng, 8, 1280), width=rng.choice([2, 3, 4, 4]))
    hk = rng.choice([1, 2, 4, 8, 16])
    return dict(c, hk=hk, hv=hk * rng.choice([1, 2, 3]), dk=rng.choice([64, 128, 128]), dv=rng.choice([64, 128, 128]))


def _spread(lo, hi, B):
    """B whole numbers from hi down to lo."""
    return [hi] if B == 1 else [hi - (hi - lo) * b // (B - 1) for b in range(B)]


def _counts(case):
    """New tokens of every sequence."""
    ns = _spread(case["n_min"], case["n_max"], case["B"])
    if case["op"] == "attention":
        return [min(n, k) for n, k in zip(ns[::-1], _spread(case["kv_min"], case["kv_max"], case["B"]))]
    return ns


def work(case):
    ns = _counts(case)
    T, B = sum(ns), case["B"]
    if case["op"] == "conv":
        C, w = case["channels"], case["width"]
        states = 2 * C * (w - 1) * (B - case["fresh"] + (0 if case["tree"] else B))
        return {"bytes": 4 * T * C + states + 4 * C * w, "flops": T * C * (2 * w + 4)}
    if case["op"] == "delta":
        hk, hv, dk, dv = (case[x] for x in ("hk", "hv", "dk", "dv"))
        tokens = 2 * T * (2 * hk * dk + 2 * hv * dv + 2 * hv)
        states = 4 * hv * dk * dv * (B - case["fresh"] + (0 if case["tree"] else B))
        # the fewer of: token by token, and whole chunks (the state's three products, half of five within a chunk)
        flops = 0
        for n in ns:
            m = n if case["tree"] else min(n, CHUNK)
            flops += hv * n * min(8 * dk * dv, 6 * dk * dv + m * (2 * dk + 3 * dv))
        return {"bytes": tokens + states, "flops": flops}
    kvs = _spread(case["kv_min"], case["kv_max"], B)
    d, hk, hq, w = case["d"], case["hk"], case["hq"], case["window"]
    seen = [min(k, w + n) if w else k for n, k in zip(ns, kvs)]
    slot = hk * (d + 8 * (d // case["group"]))      # bytes of one slot of all heads
    # (of the new tokens, about as many ancestors as half of them)
    pairs = sum(n * min(k - n // 2, w or k) for n, k in zip(ns, kvs))
    return {"bytes": sum(seen) * slot + T * (hq * (4 * d + 4) + 8), "flops": 4 * d * hq * pairs}


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


def _cache(g, case, kvs):
    """Pages with the sequences' slots filled, in an order that says nothing, and their table."""
    page, hk, d = case["page"], case["hk"], case["d"]
    need = [-(-k // page) for k in kvs]
    order = torch.randperm(sum(need), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(kvs), max(need), dtype=torch.int32, device=DEV)
    per = page // 32
    tile = 32 * (d + 8 * (d // case["group"]))
    pages = torch.empty(sum(need), hk, per, tile, dtype=torch.uint8, device=DEV)
    size = torch.exp(0.2 * torch.randn(hk, 1, 1, d, generator=g, device=DEV))      # channels differ in size
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        k, v = (torch.randn(hk, n * per, 32, d, generator=g, device=DEV) * size for _ in range(2))
        t = _tiles(k, v, case["group"], TYPES[case["dtype"]])
        pages[order[at:at + n].long()] = t.reshape(hk, n, per, tile).transpose(0, 1)
        at += n
    return pages, table


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def _trees(ns, seed):
    """A tree for each sequence, its first token the root: the ancestors of every token, as bits."""
    rng = random.Random(seed)
    words = []
    for n in ns:
        seq = [0]
        for i in range(1, n):
            parent = rng.randint(max(0, i - 6), i - 1)
            seq.append(seq[parent] | 1 << parent)
        words += seq
    return torch.tensor([w - (w >> 63 << 64) for w in words], dtype=torch.int64, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ns = _counts(case)
    T, B, dt = sum(ns), case["B"], TYPES[case["dtype"]]
    randn = lambda *shape: torch.randn(*shape, generator=g, device=DEV)
    s = dict(case=case, cu=_starts(ns), max_n=max(ns), tree=None)
    if case["op"] == "attention" or case["tree"]:
        s["tree"] = _trees(ns, seed)
    if case["op"] == "attention":
        kvs = _spread(case["kv_min"], case["kv_max"], B)
        s["pages"], s["table"] = _cache(g, case, kvs)
        s.update(kv=torch.tensor(kvs, dtype=torch.int32, device=DEV), max_kv=max(kvs))
        # queries that prefer some slots: logits of a standard deviation of about 2
        s["q"] = (2 * randn(T, case["hq"], case["d"])).to(dt)
        return s
    # a pool of states, two of them not in use; sequences that start have seen nothing
    s["index"] = torch.randperm(B + 2, generator=g, device=DEV)[:B].to(torch.int32)
    s["seen"] = torch.tensor([0 if b < case["fresh"] else 100 + b for b in range(B)], dtype=torch.int32, device=DEV)
    if case["op"] == "conv":
        C, w = case["channels"], case["width"]
        # the channels are a part of the merged projection's
        s["x"] = randn(T, C + 128).to(dt)[:, :C]
        s["weight"] = randn(C, w) / math.sqrt(w)
        s["bias"] = 0.1 * randn(C)
        s["state"] = randn(B + 2, w - 1, C).to(dt)
        return s
    hk, hv, dk, dv = (case[x] for x in ("hk", "hv", "dk", "dv"))
    # what the convolution and SiLU give, keys that have something in common
    x = torch.nn.functional.silu(randn(T, 2 * hk * dk + hv * dv) + 0.3).to(dt)
    q, k, v = x.split([hk * dk, hk * dk, hv * dv], 1)
    gates = (0.5 * randn(T, 2 * hv)).to(dt)
    # decay rates and times between slow and fast heads
    rate = 1 + 15 * torch.rand(hv, generator=g, device=DEV)
    time = torch.exp(math.log(1e-3) + math.log(100) * torch.rand(hv, generator=g, device=DEV))
    s.update(q=q.view(T, hk, dk), k=k.view(T, hk, dk), v=v.view(T, hv, dv), a=gates[:, :hv], b=gates[:, hv:],
             a_log=torch.log(rate), dt_bias=time + torch.log(-torch.expm1(-time)))
    s["state"] = 0.3 * randn(B + 2, hv, dk, dv)
    return s


# ---- the operators, in elementary operations and 32 bits ----

def _ancestors(s):
    """[B, max_n, max_n] truth values: token i comes after token j (its own among them) in its sequence or tree."""
    i = torch.arange(s["max_n"], device=DEV)
    before = i[:, None] > i
    if s["tree"] is not None:
        words, there = _padded(s["tree"][:, None], s)
        before = before & ((words >> i) & 1).bool()
    else:
        there = i < (s["cu"][1:] - s["cu"][:-1])[:, None]
    return (before | (i[:, None] == i)) & there[..., None], there


def _padded(x, s):
    """Rows [T, ...] as [B, most new tokens, ...], zeros where there are none, and which are there."""
    i = torch.arange(s["max_n"], device=DEV)
    start = s["cu"][:-1, None].long()
    there = i < s["cu"][1:, None] - start
    at = torch.where(there, start + i, torch.zeros_like(start))
    return x[at] * there.reshape(*there.shape, *[1] * (x.dim() - 1)).to(x.dtype), there


def _state_rows(s):
    """The sequences' states in 32 bits, zeros where a sequence has seen nothing."""
    rows = s["state"][s["index"].long()].float()
    return torch.where((s["seen"] > 0).reshape(-1, *[1] * (rows.dim() - 1)), rows, torch.zeros_like(rows))


def _conv(s):
    case, w = s["case"], s["case"]["width"]
    x, there = _padded(s["x"].float(), s)
    rows = torch.cat([_state_rows(s), x], 1)        # [B, width - 1 + max_n, C]
    i = torch.arange(s["max_n"], device=DEV)
    at = i.expand(case["B"], -1)
    y = x * s["weight"][:, w - 1] + s["bias"]
    if s["tree"] is not None:
        words = _padded(s["tree"][:, None], s)[0]
        bits = ((words >> i) & 1).bool() & (i < i[:, None])
        parent = torch.where(bits, i, torch.full_like(i, -1)).amax(-1)          # the latest ancestor
    else:
        parent = at - 1
    for j in range(1, w):
        # one row back; before the first new token, back through the state
        at = torch.where(at >= 0, torch.gather(parent, 1, at.clamp(min=0)), at - 1)
        y = y + torch.gather(rows, 1, (at + w - 1)[..., None].expand_as(x)) * s["weight"][:, w - 1 - j]
    out = (y / (1 + torch.exp(-y)))[there].to(s["x"].dtype)
    if s["tree"] is None:
        n = (s["cu"][1:] - s["cu"][:-1]).long()
        last = n[:, None] + torch.arange(w - 1, device=DEV)
        s["state"][s["index"].long()] = torch.gather(
            rows, 1, last[..., None].expand(-1, -1, rows.shape[-1])).to(s["x"].dtype)
    return {"out": out, "state": s["state"]}


def _unit(x):
    x = x.float()
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS)


def _delta_inputs(s):
    """q, k, v [B, value heads, tokens, channels], g and beta [B, value heads, tokens], for all padded rows."""
    case = s["case"]
    r = case["hv"] // case["hk"]
    q, k = (_padded(_unit(s[x]), s)[0].repeat_interleave(r, 2).transpose(1, 2) for x in ("q", "k"))
    v, there = _padded(s["v"].float(), s)
    z = s["a"].float() + s["dt_bias"]
    soft = torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))
    g = _padded(-torch.exp(s["a_log"]) * soft, s)[0].transpose(1, 2)
    beta = _padded(1 / (1 + torch.exp(-s["b"].float())), s)[0].transpose(1, 2)
    return q / math.sqrt(case["dk"]), k, v.transpose(1, 2), g, beta, there


def _delta_tokens(s):
    """Token by token, for calls of a few."""
    q, k, v, g, beta, there = _delta_inputs(s)
    S = _state_rows(s)
    outs = []
    for t in range(s["max_n"]):
        S = S * torch.exp(g[:, :, t])[..., None, None]
        u = beta[:, :, t, None] * (v[:, :, t] - (S * k[:, :, t, :, None]).sum(2))
        S = S + k[:, :, t, :, None] * u[:, :, None]
        outs.append((S * q[:, :, t, :, None]).sum(2))
    return torch.stack(outs, 2), S, there


def _delta_chunks(s):
    """Chunks of 64 tokens, or a tree as one: within a chunk a triangular system, between chunks the state."""
    q, k, v, g, beta, there = _delta_inputs(s)
    S = _state_rows(s)
    B, H, n, _ = q.shape
    whole = s["tree"] is not None
    C = n if whole else CHUNK
    fill = -n % C
    cut = lambda x: torch.nn.functional.pad(x, (0, 0, 0, fill)).reshape(B, H, -1, C, x.shape[-1])
    q, k, v, g, beta = cut(q), cut(k), cut(v), cut(g[..., None])[..., 0].double(), cut(beta[..., None])
    if whole:
        after = _ancestors(s)[0][:, None, None]
        G = (after.double() @ g[..., None])[..., 0]
    else:
        i = torch.arange(C, device=DEV)
        after = i[:, None] >= i
        G = torch.cumsum(g, -1)
    own_row = torch.eye(C, device=DEV)
    gap = torch.where(after, G[..., :, None] - G[..., None, :], torch.full_like(G[..., None], -math.inf))
    decay = torch.exp(gap).float()
    A = beta * (k @ k.transpose(-1, -2)) * decay * (1 - own_row)
    inv = own_row.expand_as(A).clone()
    for r in range(1, C):
        inv[..., r, :] -= (A[..., r, None, :r] @ inv[..., :r, :])[..., 0, :]
    inv = inv * beta.transpose(-1, -2)
    within = (q @ k.transpose(-1, -2)) * decay
    grow = torch.exp(G).float()[..., None]
    left = torch.exp(G[..., -1:] - G).float()[..., None]
    outs = []
    for c in range(q.shape[2]):
        u = inv[:, :, c] @ (v[:, :, c] - grow[:, :, c] * (k[:, :, c] @ S))
        outs.append(grow[:, :, c] * (q[:, :, c] @ S) + within[:, :, c] @ u)
        if not whole:
            S = grow[:, :, c, -1:] * S + (left[:, :, c] * k[:, :, c]).transpose(-1, -2) @ u
    return torch.cat(outs, 2)[:, :, :n], S, there


def _delta(s):
    few = s["tree"] is None and s["max_n"] <= 8
    o, S, there = _delta_tokens(s) if few else _delta_chunks(s)
    if s["tree"] is None:
        s["state"][s["index"].long()] = S
    return {"out": o.transpose(1, 2)[there].to(s["v"].dtype), "state": s["state"]}


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


def _attention(s):
    case = s["case"]
    k, v = _values(s, s["table"])
    B, hk, S, d = k.shape
    G, n = case["hq"] // hk, s["max_n"]
    q, there = _padded(s["q"].float(), s)
    z = q.transpose(1, 2).reshape(B, hk, G * n, d) @ k.transpose(-1, -2) / math.sqrt(d)
    after = _ancestors(s)[0]
    first = (s["kv"] - (s["cu"][1:] - s["cu"][:-1])).long()[:, None]       # slot of the first new token
    new = torch.arange(S, device=DEV) - first                              # slots as new tokens
    among = torch.gather(after, 2, new.clamp(0, n - 1)[:, None].expand(B, n, S))
    see = torch.where((new < 0)[:, None], there[..., None], among & (new < n)[:, None])
    if case["window"]:
        depth = after.sum(-1)                                              # its own token counted
        see = see & ((new >= 0)[:, None] | (new[:, None] >= depth[..., None] - case["window"]))
    z = z.reshape(B, hk, G, n, S).masked_fill_(~see[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0].flatten(1, 2).transpose(1, 2)[there]
    o = (p / torch.where(total > 0, total, torch.ones_like(total))).reshape(B, hk, G * n, S) @ v
    o = o.reshape(B, hk * G, n, -1).transpose(1, 2)[there]
    return {"out": o.to(TYPES[case["dtype"]]), "lse": lse.contiguous()}


def run(s):
    if own:
        return _run_own(s)
    return {"conv": _conv, "delta": _delta, "attention": _attention}[s["case"]["op"]](s)


def _run_own(s):
    import int4_weight_only_w4a16_amd as w4
    case = s["case"]
    if case["op"] == "conv":
        out = w4.short_conv(s["x"], s["weight"], s["state"], s["index"], s["cu"], s["max_n"], bias=s["bias"],
                            seen=s["seen"], tree=s["tree"])
        return {"out": out, "state": s["state"]}
    if case["op"] == "delta":
        out = w4.gated_delta_rule(s["q"], s["k"], s["v"], s["a"], s["b"], s["state"], s["index"], s["cu"], s["max_n"],
                                  a_log=s["a_log"], dt_bias=s["dt_bias"], seen=s["seen"], tree=s["tree"],
                                  unit_qk=True, eps=EPS)
        return {"out": out, "state": s["state"]}
    out, lse = w4.kv4_tree_attention(s["q"], s["pages"], s["table"], s["cu"], s["kv"], s["tree"], s["max_n"],
                                     s["max_kv"], window=case["window"], return_lse=True)
    return {"out": out, "lse": lse}


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


def _paths(s):
    """For each sequence, the indices of every new token's ancestors in order, its own last."""
    cu = s["cu"].tolist()
    words = s["tree"].tolist() if s["tree"] is not None else None
    found = []
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        if words is None:
            found.append([None] * n)
        else:
            found.append([[j for j in range(i) if words[cu[b] + i] >> j & 1] + [i] for i in range(n)])
    return cu, found


def _exact_conv(s):
    w = s["case"]["width"]
    cu, paths = _paths(s)
    out = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
    state = s["state"].double()
    weight, bias = s["weight"].double(), s["bias"].double()
    for b, slot in enumerate(s["index"].tolist()):
        x = s["x"][cu[b]:cu[b + 1]].double()
        old = state[slot].clone() if int(s["seen"][b]) > 0 else torch.zeros_like(state[slot])
        rows = torch.cat([old, x])
        if s["tree"] is None:
            windows = rows.unfold(0, w, 1)                                  # [n, C, w]
        else:
            took = [(list(range(w - 1)) + [w - 1 + j for j in path])[-w:] for path in paths[b]]
            windows = rows[torch.tensor(took, device=DEV)].transpose(1, 2)
        y = (windows * weight).sum(-1) + bias
        out[cu[b]:cu[b + 1]] = y * torch.sigmoid(y)
        if s["tree"] is None:
            state[slot] = rows[-(w - 1):]
    return {"out": out, "state": state}


def _exact_delta(s):
    case = s["case"]
    hv, dk = case["hv"], case["dk"]
    cu, paths = _paths(s)
    state = s["state"].double()
    unit = lambda x: x.double() / (x.double().pow(2).sum(-1, keepdim=True) + EPS).sqrt()
    head = torch.arange(hv, device=DEV) // (hv // case["hk"])
    q, k = unit(s["q"])[:, head] * dk ** -0.5, unit(s["k"])[:, head]
    v, beta = s["v"].double(), torch.sigmoid(s["b"].double())
    keep = torch.exp(-torch.exp(s["a_log"].double()) * torch.nn.functional.softplus(s["a"].double() + s["dt_bias"].double()))

    def token(S, t):
        S = S * keep[t][..., None, None]
        u = beta[t][..., None] * (v[t] - torch.einsum("bhkv,bhk->bhv", S, k[t]))
        S = S + k[t][..., None] * u[:, :, None]
        return S, torch.einsum("bhkv,bhk->bhv", S, q[t])

    out = torch.empty(v.shape, dtype=torch.float64, device=DEV)
    slots = s["index"].long()
    S = state[slots] * (s["seen"] > 0).double()[:, None, None, None]
    if s["tree"] is not None:
        for b, of_tokens in enumerate(paths):
            after = {}
            for i, path in enumerate(of_tokens):
                begin = after[path[-2]] if len(path) > 1 else S[b:b + 1]
                after[i], out[cu[b] + i:cu[b] + i + 1] = token(begin, torch.tensor([cu[b] + i], device=DEV))
        return {"out": out, "state": state}
    ns = [cu[b + 1] - cu[b] for b in range(len(cu) - 1)]
    for i in range(max(ns)):
        still = [b for b, n in enumerate(ns) if n > i]
        t = torch.tensor([cu[b] + i for b in still], device=DEV)
        if len(still) == len(ns):
            S, out[t] = token(S, t)
        else:
            on = torch.tensor(still, device=DEV)
            S[on], out[t] = token(S[on], t)
    state[slots] = S
    return {"out": out, "state": state}


def _exact_attention(s):
    case = s["case"]
    hk, d, window = case["hk"], case["d"], case["window"]
    G = case["hq"] // hk
    cu, paths = _paths(s)
    outs, lses = [], []
    for b, kv in enumerate(s["kv"].tolist()):
        n = cu[b + 1] - cu[b]
        k, v = _exact_slots(s, b, kv)
        hide = torch.ones(n, kv, dtype=torch.bool)
        for i, path in enumerate(paths[b]):
            hide[i, :kv - n] = False
            if window:      # the path is what it would be as a sequence of its own
                hide[i, :max(0, kv - n + len(path) - window)] = True
            hide[i, [kv - n + j for j in path]] = False
        hide = hide.to(DEV)[:, None]
        q = s["q"][cu[b]:cu[b + 1]].double().reshape(n, hk, G, d)
        per_head = [[], []]
        for h in range(hk):
            z = (q[:, h].reshape(n * G, d) @ k[h].T).reshape(n, G, kv) * d ** -0.5
            z = z.masked_fill(hide, -math.inf)
            per_head[0].append((torch.softmax(z, -1).reshape(n * G, kv) @ v[h]).reshape(n, G, d))
            per_head[1].append(torch.logsumexp(z, -1))
        outs.append(torch.stack(per_head[0], 1).reshape(n, hk * G, d))
        lses.append(torch.stack(per_head[1], 1).reshape(n, hk * G))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "delta": _exact_delta, "attention": _exact_attention}[case["op"]](s)
