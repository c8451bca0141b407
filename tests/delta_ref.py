"""The short convolution and the gated delta rule in 64 bits on the CPU, token by token as defined,
with what bounds the kernels' errors."""

from __future__ import annotations

import torch

import tree_ref as tr

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}      # unit roundoff


def conv(x, weight, bias, silu, before, parents=None):
    """x [n, C] of one sequence, before [width - 1, C] (the rows in front of it), all in 64 bits.  Returns
    out, sum |w x| + |bias| and the rows that the next call finds before it."""
    W = weight.shape[1]
    parents = tr.chain(x.shape[0]) if parents is None else parents
    out, mag = torch.zeros_like(x), torch.zeros_like(x)
    for i in range(x.shape[0]):
        rows = torch.cat([before, x[tr.path(parents, i)]])[-W:]
        y = (weight.T * rows).sum(0) + (0 if bias is None else bias)
        mag[i] = (weight.T * rows).abs().sum(0) + (0 if bias is None else bias.abs())
        out[i] = y * torch.sigmoid(y) if silu else y
    return out, mag, torch.cat([before, x])[-(W - 1):]


def gates(a, b, a_log, dt_bias):
    """g and beta [n, heads] in 64 bits."""
    if a_log is None:
        return a.double(), b.double()
    g = -torch.exp(a_log.double()) * torch.nn.functional.softplus(a.double() + dt_bias.double(), threshold=1e9)
    return g, torch.sigmoid(b.double())


def delta(q, k, v, g, beta, S, scale, unit=True, eps=1e-6, parents=None):
    """q, k [n, key heads, Dk], v [n, heads, Dv] of one sequence, g and beta [n, heads], S [heads, Dk, Dv].
    Returns out, the size of what each output sums up (|q| times the lengths of S's columns as if nothing
    cancelled), and the last state."""
    q, k, v, S = q.double(), k.double(), v.double(), S.double()
    r = v.shape[1] // k.shape[1]
    if unit:
        q, k = (x / (x.pow(2).sum(-1, keepdim=True) + eps).sqrt() for x in (q, k))
    q, k = (x.repeat_interleave(r, 1) for x in (q, k))
    out, size = torch.zeros_like(v), torch.zeros_like(v)
    after = {}
    in_a_row = parents is None
    parents = tr.chain(v.shape[0]) if in_a_row else parents
    last = S
    for t, p in enumerate(parents):
        S0, m0 = after[p] if p >= 0 else (S, S.pow(2).sum(1).sqrt())
        keep = torch.exp(g[t])[:, None]
        S1 = keep[..., None] * S0
        u = beta[t][:, None] * (v[t] - (S1 * k[t][..., None]).sum(1))
        S1 = S1 + k[t][..., None] * u[:, None]
        m1 = keep * m0 + k[t].pow(2).sum(-1, keepdim=True).sqrt() * u.abs()
        out[t] = scale * (S1 * q[t][..., None]).sum(1)
        size[t] = scale * q[t].pow(2).sum(-1, keepdim=True).sqrt() * m1
        after[t] = (S1, m1)
        last = S1
        if in_a_row:
            after.pop(t - 1, None)
    return out, size, last
