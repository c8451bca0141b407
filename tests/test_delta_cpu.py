"""What short_conv and delta_rule refuse, through the C ABI on the CPU: every check runs before
any HIP call, so the made-up addresses below are never touched.  And the references' own forms."""

import ctypes

import pytest

import int4_weight_only_w4a16_amd as w4
from test_kv4_boundary_cpu import call, lib  # noqa: F401


def conv(lib, **kw):  # noqa: F811
    d = dict(x=0x1000, xs=512, weight=0x2000, bias=0x3000, state=0x4000, index=0x5000, seen=0x6000, cu=0x7000,
             tree=None, out=0x8000, os=512, T=4, C=512, W=4, states=9, batch=2, max_q=3, flags=0, stream=None)
    return call(lib.w4a16_short_conv, d, kw)


def delta(lib, **kw):  # noqa: F811
    d = dict(q=0x1000, qs=256, k=0x2000, ks=256, v=0x3000, vs=512, a=0x4000, as_=4, b=0x5000, bs=4, a_log=0x6000,
             dt=0x7000, state=0x8000, index=0x9000, seen=0xa000, cu=0xb000, tree=None, out=0xc000, os=512, T=4, hk=2,
             hv=4, dk=128, dv=128, states=9, batch=2, max_q=3, scale=ctypes.c_float(0.1), eps=ctypes.c_float(1e-6),
             flags=0, ws=0xd0000, wsb=1 << 40, stream=None)
    return call(lib.w4a16_delta_rule, d, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), w4.W4A16_ERR_NULL), (dict(weight=None), w4.W4A16_ERR_NULL), (dict(state=None), w4.W4A16_ERR_NULL),
    (dict(out=None), w4.W4A16_ERR_NULL), (dict(index=None), w4.W4A16_ERR_NULL), (dict(cu=None), w4.W4A16_ERR_NULL),
    (dict(x=0x1008), w4.W4A16_ERR_ALIGN), (dict(weight=0x2004), w4.W4A16_ERR_ALIGN),
    (dict(bias=0x3004), w4.W4A16_ERR_ALIGN), (dict(state=0x4002), w4.W4A16_ERR_ALIGN),
    (dict(out=0x8004), w4.W4A16_ERR_ALIGN), (dict(index=0x5002), w4.W4A16_ERR_ALIGN),
    (dict(seen=0x6001), w4.W4A16_ERR_ALIGN), (dict(tree=0x9004), w4.W4A16_ERR_ALIGN),
    (dict(C=0), w4.W4A16_ERR_SHAPE), (dict(C=12, xs=16, os=16), w4.W4A16_ERR_SHAPE), (dict(xs=504), w4.W4A16_ERR_SHAPE),
    (dict(os=516), w4.W4A16_ERR_SHAPE), (dict(W=1), w4.W4A16_ERR_SHAPE), (dict(W=5), w4.W4A16_ERR_SHAPE),
    (dict(T=-1), w4.W4A16_ERR_SHAPE), (dict(T=(1 << 28) + 1), w4.W4A16_ERR_SHAPE), (dict(batch=65536), w4.W4A16_ERR_SHAPE),
    (dict(max_q=-1), w4.W4A16_ERR_SHAPE), (dict(tree=0x9000, max_q=65), w4.W4A16_ERR_SHAPE),
    (dict(states=-1), w4.W4A16_ERR_SHAPE), (dict(C=1 << 24, xs=1 << 24, os=1 << 24, T=1 << 28, max_q=1 << 28), w4.W4A16_ERR_SHAPE),
    (dict(flags=0x2), w4.W4A16_ERR_FLAGS), (dict(flags=w4.W4A16_UNIT_QK), w4.W4A16_ERR_FLAGS),
    (dict(T=0, x=None), w4.W4A16_OK), (dict(batch=0, cu=None), w4.W4A16_OK), (dict(max_q=0), w4.W4A16_OK)])
def test_conv_refusals(lib, kw, status):  # noqa: F811
    assert conv(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    *[(dict([(n, None)]), w4.W4A16_ERR_NULL) for n in ("q", "k", "v", "a", "b", "state", "index", "cu", "out", "dt")],
    (dict(a_log=None), w4.W4A16_ERR_NULL),
    *[(dict([(n, 0x1008)]), w4.W4A16_ERR_ALIGN) for n in ("q", "k", "v", "state", "out")],
    (dict(a=0x4001), w4.W4A16_ERR_ALIGN), (dict(a_log=None, dt=None, a=0x4002), w4.W4A16_ERR_ALIGN),
    (dict(b=0x5001), w4.W4A16_ERR_ALIGN), (dict(dt=0x7002), w4.W4A16_ERR_ALIGN), (dict(tree=0x1004), w4.W4A16_ERR_ALIGN),
    (dict(index=0x9002), w4.W4A16_ERR_ALIGN),
    (dict(dk=96), w4.W4A16_ERR_SHAPE), (dict(dk=256, qs=512, ks=512), w4.W4A16_ERR_SHAPE), (dict(dv=32), w4.W4A16_ERR_SHAPE),
    (dict(dv=320, vs=1280, os=1280), w4.W4A16_ERR_SHAPE), (dict(hk=3), w4.W4A16_ERR_SHAPE), (dict(hk=0), w4.W4A16_ERR_SHAPE),
    (dict(hv=0), w4.W4A16_ERR_SHAPE), (dict(qs=248), w4.W4A16_ERR_SHAPE), (dict(ks=260), w4.W4A16_ERR_SHAPE),
    (dict(vs=504), w4.W4A16_ERR_SHAPE), (dict(os=0), w4.W4A16_ERR_SHAPE), (dict(as_=3), w4.W4A16_ERR_SHAPE),
    (dict(bs=0), w4.W4A16_ERR_SHAPE), (dict(T=-1), w4.W4A16_ERR_SHAPE), (dict(batch=70000), w4.W4A16_ERR_SHAPE),
    (dict(max_q=-2), w4.W4A16_ERR_SHAPE), (dict(tree=0x1000, max_q=65), w4.W4A16_ERR_SHAPE),
    (dict(scale=ctypes.c_float(0)), w4.W4A16_ERR_SHAPE), (dict(scale=ctypes.c_float(float("nan"))), w4.W4A16_ERR_SHAPE),
    (dict(eps=ctypes.c_float(-1)), w4.W4A16_ERR_SHAPE), (dict(eps=ctypes.c_float(float("inf"))), w4.W4A16_ERR_SHAPE),
    (dict(flags=w4.W4A16_SILU), w4.W4A16_ERR_FLAGS), (dict(flags=0x100), w4.W4A16_ERR_FLAGS),
    (dict(T=0, q=None), w4.W4A16_OK), (dict(batch=0), w4.W4A16_OK), (dict(max_q=0, cu=None), w4.W4A16_OK)])
def test_delta_refusals(lib, kw, status):  # noqa: F811
    assert delta(lib, **kw) == status


def test_valid_calls_reach_the_device_check(lib):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    for kw in (dict(), dict(bias=None, seen=None), dict(tree=0xe000, max_q=64), dict(flags=w4.W4A16_X_BF16 | w4.W4A16_SILU)):
        assert conv(lib, **kw) == w4.W4A16_ERR_DEVICE
    for kw in (dict(), dict(a_log=None, dt=None, seen=None), dict(tree=0xe000, max_q=64), dict(T=900, max_q=700),
               dict(flags=w4.W4A16_X_BF16 | w4.W4A16_UNIT_QK), dict(dv=192, vs=768, os=768)):
        assert delta(lib, **kw) == w4.W4A16_ERR_DEVICE


@pytest.mark.parametrize("hk,hv,dk,batch,max_q", [(2, 4, 128, 3, 17), (16, 48, 128, 1, 8191), (16, 64, 128, 2, 4480),
                                                  (16, 64, 128, 2, 20000), (1, 1, 64, 1, 100), (4, 32, 64, 40, 640)])
def test_workspace_of_both_types(lib, hk, hv, dk, batch, max_q):  # noqa: F811
    """What the size function says is enough for a call of either type, and for one of them no more than that."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    T = batch * max_q
    need = w4.delta_rule_workspace_bytes(batch, T, hk, hv, dk, 128, max_q)
    assert need > 0 and w4.delta_rule_workspace_bytes(batch, T, hk, hv, dk, 128, max_q) == need
    sizes = dict(T=T, hk=hk, hv=hv, dk=dk, dv=128, qs=hk * dk, ks=hk * dk, vs=hv * 128, os=hv * 128, as_=hv, bs=hv,
                 batch=batch, max_q=max_q)
    short = []
    for flags in (0, w4.W4A16_X_BF16):
        sizes["flags"] = flags
        assert delta(lib, **sizes, wsb=need) == w4.W4A16_ERR_DEVICE
        assert delta(lib, **sizes, ws=None, wsb=0) == w4.W4A16_ERR_NULL
        assert delta(lib, **sizes, ws=0xd0008, wsb=need) == w4.W4A16_ERR_ALIGN
        assert delta(lib, **sizes, wsb=1024) == w4.W4A16_ERR_WORKSPACE
        short.append(delta(lib, **sizes, wsb=need - 1))
    assert w4.W4A16_ERR_WORKSPACE in short
    for n in (1, 16):                      # token by token: none
        assert w4.delta_rule_workspace_bytes(batch, batch * n, hk, hv, dk, 128, n) == 0
    assert w4.delta_rule_workspace_bytes(batch, 64 * batch, hk, hv, dk, 128, 64, tree=True) == 0


def test_a_chunk_s_triangular_form_is_the_recurrence():
    """The form that long calls are computed in, against the definition: U = T (V - e^G K S)."""
    import torch

    import delta_ref as ref
    import tree_ref as tr
    g = torch.Generator().manual_seed(0)
    n, d = 30, 16
    for parents in (tr.chain(n), tr.random_tree(n, __import__("random").Random(1), 2)):
        q, k = (torch.randn(n, 1, d, generator=g, dtype=torch.float64) for _ in range(2))
        v, S = torch.randn(n, 1, 8, generator=g, dtype=torch.float64), torch.randn(1, d, 8, generator=g, dtype=torch.float64)
        lg, beta = -torch.rand(n, 1, generator=g, dtype=torch.float64), torch.rand(n, 1, generator=g, dtype=torch.float64)
        out, size, last = ref.delta(q, k, v, lg, beta, S, 0.3, True, 0.0, parents)
        kin = torch.zeros(n, n, dtype=torch.float64)
        for i in range(n):
            kin[i, tr.path(parents, i)] = 1
        G = kin @ lg[:, 0]
        decay = torch.where(kin > 0, torch.exp(G[:, None] - G[None]), torch.zeros_like(kin))
        qn, kn = (x[:, 0] / x[:, 0].norm(dim=-1, keepdim=True) for x in (q, k))
        A = torch.tril(beta * (kn @ kn.T) * decay, -1)
        U = torch.linalg.solve(torch.eye(n, dtype=torch.float64) + A, beta * (v[:, 0] - torch.exp(G)[:, None] * (kn @ S[0])))
        o = 0.3 * (torch.exp(G)[:, None] * (qn @ S[0]) + (decay * (qn @ kn.T)) @ U)
        assert (o - out[:, 0]).abs().max() < 1e-12 and (out.abs() <= size + 1e-12).all()
        if parents == tr.chain(n):
            end = torch.exp(G[-1]) * S[0] + (torch.exp(G[-1] - G)[:, None] * kn).T @ U
            assert (end - last[0]).abs().max() < 1e-12


def test_short_conv_names_its_own_argument(lib):  # noqa: F811
    import torch
    x, weight, state = torch.zeros(3, 16), torch.zeros(16, 4), torch.zeros(1, 3, 16)
    index = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="^x must be float16 or bfloat16"):
        w4.short_conv(x, weight, state, index, torch.tensor([0, 3], dtype=torch.int32), 3)


def test_a_workspace_for_the_largest_call_does_for_smaller_ones(lib):  # noqa: F811
    """A program keeps one workspace, of the size for its most sequences and longest prompt."""
    for hk, hv, dk, dv in ((16, 48, 128, 128), (16, 64, 128, 256), (1, 2, 64, 64)):
        size = lambda batch, max_q, T: w4.delta_rule_workspace_bytes(batch, T, hk, hv, dk, dv, max_q)
        for batch, max_q in ((64, 8192), (3, 20000), (7, 3000), (200, 700), (2, 11000)):
            most = size(batch, max_q, batch * max_q)
            for b in {1, 2, 3, batch // 2, batch - 1, batch}:
                for q in {1, 17, 64, 65, max_q // 3, max_q // 2, max_q - 64, max_q}:
                    if 1 <= b <= batch and 1 <= q:
                        assert size(b, q, b * q) <= most, (batch, max_q, b, q)
                        assert size(b, q, q) <= most
