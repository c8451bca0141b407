"""What the 4-bit cache's entry points take and refuse at the edges, through the C ABI on the
CPU: every check runs before any HIP call, and a call that passes them all ends here with
W4A16_ERR_DEVICE, so the made-up addresses below are never touched."""

import pytest

import int4_weight_only_w4a16_amd as w4
from test_kv4_boundary_cpu import append, attention, evict, lib, mass, norm_rope, read  # noqa: F401

S = w4.W4A16_ERR_SHAPE


@pytest.fixture(autouse=True)
def no_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")


# ---- prompts of very many rows ----

@pytest.mark.parametrize("hq,hk,D", [(40, 8, 128), (32, 8, 64), (128, 8, 128), (64, 64, 128), (16, 4, 256)])
def test_attention_of_long_prompts(lib, hq, hk, D):  # noqa: F811
    """Up to 65535 tiles of 256 rows (128 with 256 channels) over all heads; the weights have no such limit."""
    kw = dict(hq=hq, hk=hk, D=D, qs=hq * D, os=hq * D, max_kv=1 << 20)
    most = 65535 // hk * (256 if D <= 128 else 128) // (hq // hk)
    assert most > 100000
    for tokens in (4096, 8192, 16384, 32768, 100000, most):
        assert attention(lib, **kw, max_q=tokens) == w4.W4A16_ERR_DEVICE
        assert mass(lib, hq=hq, hk=hk, D=D, qs=hq * D, max_q=tokens) == w4.W4A16_ERR_DEVICE
    assert attention(lib, **kw, max_q=most + 1) == S
    assert attention(lib, **kw, max_q=most + 1, T=0) == S
    assert mass(lib, hq=hq, hk=hk, D=D, qs=hq * D, max_q=most + 1) == w4.W4A16_ERR_DEVICE
    assert w4.kv4_attention_workspace_bytes(1, hq, hk, D, most + 1, 1 << 20) == 0


def test_rows_of_a_head_are_32_bits(lib):  # noqa: F811
    assert mass(lib, hq=256, hk=1, qs=256 * 128, max_q=1 << 22) == S
    assert mass(lib, hq=255, hk=1, qs=255 * 128, max_q=1 << 22) == w4.W4A16_ERR_DEVICE
    for f in (attention, mass):
        assert f(lib, hq=1 << 40) == S and f(lib, hq=-8) == S


# ---- launches count threads in 32 bits ----

def test_launches_of_more_threads_are_refused_before_them(lib):  # noqa: F811
    taken = w4.W4A16_ERR_DEVICE
    rope = dict(hq=32, hk=0, qs=4096, qos=4096)
    assert norm_rope(lib, T=(1 << 23) - 1, **rope) == taken and norm_rope(lib, T=1 << 23, **rope) == S
    wide = dict(hq=16, hk=0, D=256, rot=64, qs=4096, qos=4096)
    assert norm_rope(lib, T=(1 << 23) - 1, **wide) == taken and norm_rope(lib, T=1 << 23, **wide) == S
    # (eight more workgroups for the tiles)
    assert append(lib, T=(1 << 23) - 5, batch=1, max_q=1, hq=32, qs=4096, qos=4096) == taken
    assert append(lib, T=1 << 23, batch=1, max_q=1, hq=32, qs=4096, qos=4096) == S
    assert read(lib, rows=(1 << 29) - 32) == taken and read(lib, rows=1 << 29) == S
    long = dict(acc_stride=1 << 31)
    assert mass(lib, max_kv=(1 << 30) - 256, **long) == taken and mass(lib, max_kv=1 << 30, **long) == S
    pages = dict(dst_stride=1 << 24, recent=0)
    assert evict(lib, budget=(1 << 29) - 32, **pages) == taken and evict(lib, budget=1 << 29, **pages) == S


def test_append_takes_any_bound_on_the_tokens_of_a_sequence(lib):  # noqa: F811
    """max_q beyond the tokens that there are costs no workgroups: 512 sequences, a bound of 2^28."""
    assert append(lib, batch=512, max_q=1 << 28) == w4.W4A16_ERR_DEVICE
    assert append(lib, batch=512, max_q=(1 << 28) + 1) == S


# ---- the example ----

def test_example_refuses_positions_past_its_tables():
    """Evictions keep a cache small for any number of tokens; the rotation's tables end."""
    import importlib.util
    import os

    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    block = example.AttentionBlock(hidden=128, q_heads=2, kv_heads=1, head_dim=64, group=32, page=32, batch=2, budget=64,
                                   recent=16, room=64, device="cpu")
    block.positions, block.lengths = [100, (1 << 14) - 2], [64, 64]
    with pytest.raises(ValueError, match="tables"):
        block(torch.zeros(4, 128, dtype=torch.bfloat16), [1, 3])
    assert block.positions == [100, (1 << 14) - 2] and block.kv_len.tolist() == [0, 0]
