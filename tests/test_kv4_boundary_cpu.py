"""What the 4-bit cache's entry points refuse, through the C ABI on the CPU: every check
runs before any HIP call, so the made-up addresses below are never touched."""

import ctypes
import math
import os

import pytest

import int4_weight_only_w4a16_amd as w4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4.LIB_PATH):
        from int4_weight_only_w4a16_amd import _build
        _build.build()
    return w4.load_library()


def call(f, defaults, kw):
    assert set(kw) <= set(defaults)
    return f(*{**defaults, **kw}.values())


GEO = dict(hk=8, D=128, group=64, page=64, num_pages=100, batch=4, stride=10)


def norm_rope(lib, **kw):
    d = dict(q=0x1000, qs=5120, k=0x2000, ks=1024, qw=0x3000, kw=0x4000, eps=1e-6, cos=0x5000, sin=0x6000,
             pos=0x7000, qo=0x8000, qos=5120, ko=0x9000, kos=1024, T=4, hq=40, hk=8, D=128, rot=128, max_pos=100,
             flags=0, stream=None)
    return call(lib.w4a16_qk_norm_rope, d, kw)


def append(lib, **kw):
    d = dict(q=0x1000, qs=5120, k=0x2000, ks=1024, v=0x2800, vs=1024, qw=0x3000, kw=0x4000, eps=1e-6, cos=0x5000,
             sin=0x6000, pos=0x7000, qo=0x8000, qos=5120, pages=0x9000, table=0xa000, cu=0xb000, kv=0xc000, T=4,
             hq=40, hk=8, D=128, rot=128, max_pos=100, group=64, page=64, num_pages=100, batch=4, stride=10,
             max_q=1, flags=0, stream=None)
    return call(lib.w4a16_kv4_append, d, kw)


def read(lib, **kw):
    d = dict(pages=0x9000, table=0xa000, cu=0xb000, kv=0xc000, k=0x1000, v=0x2000, rows=4, **GEO, flags=0,
             stream=None)
    return call(lib.w4a16_kv4_read, d, kw)


def attention(lib, **kw):
    d = dict(q=0x1000, qs=5120, pages=0x9000, table=0xa000, cu=0xb000, kv=0xc000, out=0x2000, os=5120, lse=0x3000,
             T=4, hq=40, **GEO, max_q=1, max_kv=640, scale=0.1, window=0, flags=0, ws=0xd000, wsb=1 << 30,
             stream=None)
    return call(lib.w4a16_kv4_attention, d, kw)


def mass(lib, **kw):
    d = dict(q=0x1000, qs=5120, pages=0x9000, table=0xa000, cu=0xb000, kv=0xc000, lse=0x3000, acc=0x4000,
             acc_stride=640, T=4, hq=40, **GEO, max_q=1, max_kv=640, scale=0.1, window=0, flags=0, stream=None)
    return call(lib.w4a16_kv4_attention_mass, d, kw)


def evict(lib, **kw):
    d = dict(pages=0x9000, table=0xa000, kv=0xc000, acc=0x4000, acc_stride=640, budget=320, recent=32, dst=0x5000,
             dst_stride=5, kept=0x6000, new=0x7000, acc_out=0x8000, **GEO, max_kv=640, flags=0, stream=None)
    return call(lib.w4a16_kv4_evict, d, kw)


S, N, A, G, F = (w4.W4A16_ERR_SHAPE, w4.W4A16_ERR_NULL, w4.W4A16_ERR_ALIGN, w4.W4A16_ERR_GROUP, w4.W4A16_ERR_FLAGS)
CACHED = [append, read, attention, mass, evict]


@pytest.mark.parametrize("f", CACHED)
@pytest.mark.parametrize("kw,status", [
    (dict(D=96), S), (dict(D=512), S), (dict(hk=0), S), (dict(page=48), S), (dict(page=0), S), (dict(page=16), S),
    (dict(group=16), G), (dict(group=256), G), (dict(group=0), G), (dict(batch=-1), S), (dict(batch=65536), S),
    (dict(num_pages=-1), S), (dict(stride=-1), S), (dict(stride=1 << 26), S), (dict(page=1 << 24), S),
    (dict(pages=0), N), (dict(table=0), N), (dict(kv=0), N), (dict(pages=0x9008), A), (dict(table=0xa002), A),
    (dict(flags=0x100), F), (dict(flags=w4.W4A16_GATE_UP_SILU), F),
])
def test_cache_arguments_refused(lib, f, kw, status):
    if f is not read and f is not evict and kw.get("D") in (96, 512):
        kw = dict(kw, qs=1 << 20, **({"os": 1 << 20} if f is attention else {}))
    assert f(lib, **kw) == status


@pytest.mark.parametrize("f,kw,status", [
    (norm_rope, dict(D=100), S), (norm_rope, dict(T=-1), S), (norm_rope, dict(qs=5112), S),
    (norm_rope, dict(qs=5124), S), (norm_rope, dict(kos=1000), S), (norm_rope, dict(rot=24), S),
    (norm_rope, dict(rot=144), S), (norm_rope, dict(rot=0), S), (norm_rope, dict(max_pos=0), S),
    (norm_rope, dict(eps=-1.0), S), (norm_rope, dict(eps=math.nan), S), (norm_rope, dict(q=0), N),
    (norm_rope, dict(ko=0), N), (norm_rope, dict(sin=0), N), (norm_rope, dict(pos=0), N),
    (norm_rope, dict(q=0x1004), A), (norm_rope, dict(kw=0x4004), A), (norm_rope, dict(cos=0x5008), A),
    (norm_rope, dict(pos=0x7001), A), (norm_rope, dict(flags=w4.W4A16_NONCAUSAL), F),
    (norm_rope, dict(hq=-1), S), (norm_rope, dict(T=1 << 28, hq=1 << 15, qs=1 << 22, qos=1 << 22), S),
    (append, dict(hq=36), S), (append, dict(ks=1016), S), (append, dict(vs=1028), S), (append, dict(max_q=-1), S),
    (append, dict(k=0), N), (append, dict(v=0), N), (append, dict(q=0), N), (append, dict(qo=0), N),
    (append, dict(cu=0), N), (append, dict(v=0x2804), A), (append, dict(cu=0xb001), A), (append, dict(rot=8), S),
    (append, dict(flags=w4.W4A16_NONCAUSAL), F),
    (read, dict(rows=-1), S), (read, dict(k=0), N), (read, dict(v=0x2008), A),
    (attention, dict(hq=36), S), (attention, dict(hq=0), S), (attention, dict(qs=5112), S),
    (attention, dict(os=100), S), (attention, dict(max_q=-1), S), (attention, dict(max_kv=-1), S),
    (attention, dict(window=-1), S), (attention, dict(scale=0.0), S), (attention, dict(scale=-1.0), S),
    (attention, dict(scale=math.inf), S), (attention, dict(scale=math.nan), S), (attention, dict(q=0), N),
    (attention, dict(out=0), N), (attention, dict(out=0x2004), A), (attention, dict(lse=0x3001), A),
    (attention, dict(cu=0), N), (attention, dict(max_q=1 << 24), S),
    (attention, dict(flags=w4.W4A16_NONCAUSAL, window=5), F),
    (attention, dict(batch=1, max_kv=100000, ws=0), N), (attention, dict(batch=1, max_kv=100000, ws=0xd008), A),
    (attention, dict(batch=1, max_kv=100000, wsb=64), w4.W4A16_ERR_WORKSPACE),
    (mass, dict(lse=0), N), (mass, dict(acc=0), N), (mass, dict(acc_stride=639), S), (mass, dict(acc=0x4002), A),
    (mass, dict(scale=0.0), S), (mass, dict(hq=41), S),
    (evict, dict(budget=0), S), (evict, dict(recent=-1), S), (evict, dict(recent=321), S),
    (evict, dict(dst_stride=4), S), (evict, dict(acc_stride=600), S), (evict, dict(max_kv=-1), S),
    (evict, dict(acc=0), N), (evict, dict(dst=0), N), (evict, dict(kept=0), N), (evict, dict(new=0), N),
    (evict, dict(acc_out=0), N), (evict, dict(kept=0x6002), A),
])
def test_arguments_refused(lib, f, kw, status):
    assert f(lib, **kw) == status


def test_nothing_to_do_is_ok_whatever_the_pointers(lib):
    assert norm_rope(lib, T=0, q=0, k=0, qo=0, ko=0) == w4.W4A16_OK
    assert append(lib, T=0, q=0, k=0, v=0, qo=0, pages=0) == w4.W4A16_OK
    assert read(lib, rows=0, k=0, v=0, pages=0) == w4.W4A16_OK
    for kw in (dict(T=0), dict(batch=0), dict(max_q=0)):
        assert attention(lib, pages=0, ws=0, **kw) == w4.W4A16_OK
        assert mass(lib, pages=0, **kw) == w4.W4A16_OK
    assert evict(lib, batch=0, pages=0) == w4.W4A16_OK
    # ... but wrong shapes are still wrong
    assert norm_rope(lib, T=0, D=100) == S and attention(lib, T=0, hq=41) == S


def test_page_and_workspace_bytes(lib):
    assert w4.kv4_page_bytes(8, 128, 64, 64) == 8 * 64 * (128 + 16)
    assert w4.kv4_page_bytes(1, 256, 32, 32) == 32 * (256 + 64)
    for bad in ((0, 128, 64, 64), (8, 96, 32, 64), (8, 128, 16, 64), (8, 64, 128, 64), (8, 128, 64, 40)):
        assert w4.kv4_page_bytes(*bad) == 0
    size = w4.kv4_attention_workspace_bytes
    assert size(1, 40, 8, 128, 1, 100000) > 0
    for none in (size(0, 40, 8, 128, 1, 1000), size(1, 41, 8, 128, 1, 1000), size(1, 40, 0, 128, 1, 1000),
                 size(1, 40, 8, 100, 1, 1000), size(1, 40, 8, 128, 0, 1000), size(1, 40, 8, 128, 1, -1)):
        assert none == 0


def test_binding_refuses_tensors_that_do_not_fit(lib):
    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        w4.qk_norm_rope(q, q)                          # not on a device
    with pytest.raises(ValueError):
        w4.kv4_new_pages(4, 2, 96, 32, 64, device="cpu")
    pages = w4.kv4_new_pages(4, 2, 64, 32, 64, device="cpu")
    assert pages.shape == (4, 2, 2, 32 * (64 + 16))
    table, cu, kv = (torch.zeros(s, dtype=torch.int32) for s in ((1, 4), (2,), (1,)))
    with pytest.raises(ValueError):
        w4.kv4_attention(q, pages, table, cu, kv, 1, 64)
    with pytest.raises(ValueError):
        w4.kv4_read(pages, table, cu, kv, 1, 64, torch.float16)
    with pytest.raises(ValueError):
        w4.kv4_evict(pages, table, kv, torch.zeros(1, 2, 64), 32, 0, table, 64, 64)
