"""What kv4_tree_attention refuses, through the C ABI on the CPU: every check runs before any
HIP call, so the made-up addresses below are never touched."""

import pytest

import int4_weight_only_w4a16_amd as w4
from test_kv4_boundary_cpu import GEO, call, lib  # noqa: F401


def tree(lib, **kw):  # noqa: F811
    d = dict(q=0x1000, qs=5120, pages=0x9000, table=0xa000, cu=0xb000, kv=0xc000, tree=0xe000, out=0x2000, os=5120,
             lse=0x3000, T=4, hq=40, **GEO, max_q=4, max_kv=640, scale=0.1, window=0, flags=0, ws=0xd000,
             wsb=1 << 30, stream=None)
    return call(lib.w4a16_kv4_tree_attention, d, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(tree=None), w4.W4A16_ERR_NULL),
    (dict(tree=0xe004), w4.W4A16_ERR_ALIGN),
    (dict(max_q=65), w4.W4A16_ERR_SHAPE),
    (dict(window=1), w4.W4A16_ERR_SHAPE),
    (dict(window=63), w4.W4A16_ERR_SHAPE),
    (dict(window=-1), w4.W4A16_ERR_SHAPE),
    (dict(flags=w4.W4A16_NONCAUSAL), w4.W4A16_ERR_FLAGS),
    (dict(flags=0x40), w4.W4A16_ERR_FLAGS),
    (dict(q=None), w4.W4A16_ERR_NULL),
    (dict(out=0x2004), w4.W4A16_ERR_ALIGN),
    (dict(pages=None), w4.W4A16_ERR_NULL),
    (dict(hq=41), w4.W4A16_ERR_SHAPE),
    (dict(D=96), w4.W4A16_ERR_SHAPE),
    (dict(group=16), w4.W4A16_ERR_GROUP),
    (dict(scale=0.0), w4.W4A16_ERR_SHAPE),
    # more workgroups than a launch has
    (dict(hq=60000, hk=60000, D=64, group=64, page=32, qs=60000 * 64, os=60000 * 64, max_q=1, max_kv=1 << 20),
     w4.W4A16_ERR_SHAPE),
    (dict(max_kv=100000, wsb=0), w4.W4A16_ERR_WORKSPACE),
    (dict(max_kv=100000, ws=None), w4.W4A16_ERR_NULL),
    (dict(T=0, tree=None), w4.W4A16_OK),
    (dict(max_q=0), w4.W4A16_OK),
    (dict(batch=0), w4.W4A16_OK),
])
def test_refusals(lib, kw, status):  # noqa: F811
    assert tree(lib, **kw) == status


def test_a_valid_call_reaches_the_device_check(lib):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    for kw in (dict(), dict(window=64), dict(max_q=64)):
        assert tree(lib, **kw) == w4.W4A16_ERR_DEVICE
