"""CPU checks of the paged operators' Python handles: sizes that a 32-bit field cannot hold."""
from types import SimpleNamespace

import pytest
import torch

import continuous_batching_transformer_gb300 as cbt
from continuous_batching_transformer_gb300 import binding as B
from continuous_batching_transformer_gb300 import model, paged


@pytest.fixture(scope="module", autouse=True)
def built():
    cbt.build()


def cache_stub(index=-1):
    """What the handles read of a PagedKV, on the CPU."""
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    return SimpleNamespace(block_table=i32(2, 3), kv_lens=i32(2), rows=2, head_dim=64, n_kv_heads=2, index=index,
                           device=torch.device("cpu"), err=i32(2),
                           layers=[B.PagedKvDesc(None, 0, 0, 0, 0, 4, 64, 2, 64)])


@pytest.mark.parametrize("past", [2 ** 31, 2 ** 32, 2 ** 32 + 64, -2 ** 32 + 64, 2 ** 63])
def test_sizes_past_32_bits_are_refused(past):
    """Cut to 32 bits, most of these would pass for small sizes."""
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    pool = torch.zeros(1 << 16, dtype=torch.bfloat16)
    attn = dict(n_heads=4, max_kv=128, max_q=4, max_tokens=8, window=5, sinks=1)
    kv = dict(page_tokens=64, n_kv_heads=2, head_dim=64, n_layers=1)
    pm = dict(page_tokens=64, max_tokens=8, n_pages=8)
    calls = [(lambda **k: paged.Attention(cache_stub(), **k), attn),
             (lambda **k: paged.PagedKV(pool, None, None, **k), kv),
             (lambda **k: paged.PageMap(i32(2, 3), i32(2), None, None, **k), pm),
             (lambda **k: paged.RopeAppend(cache_stub(), None, **k), dict(n_heads=4)),
             (lambda head_dim, **k: paged.Rope(head_dim, **k), dict(head_dim=64, rot_dim=32, original_len=4096))]
    for call, ok in calls:
        for name in ok:
            with pytest.raises(ValueError, match=name):
                call(**{**ok, name: past})
    engine = SimpleNamespace(shape=SimpleNamespace(n_layers=1, head_dim=64), arena=pool, handle=None)
    for name in ("window", "sinks"):
        with pytest.raises(ValueError, match=name):
            model.Engine.set_attention(engine, **{name: past})


def test_sizes_are_whole_numbers():
    for bad in (4.0, "4", None):
        with pytest.raises(TypeError):
            paged.RopeAppend(cache_stub(), None, n_heads=bad)


def test_an_engine_refuses_the_rope_of_another_head_size():
    engine = SimpleNamespace(shape=SimpleNamespace(n_layers=1, head_dim=128), arena=torch.zeros(1), handle=None)
    with pytest.raises(ValueError, match="head_dim"):
        model.Engine.set_attention(engine, paged.Rope(64))
    with pytest.raises(B.CbtError):  # taken, but for the missing engine
        model.Engine.set_attention(engine, paged.Rope(128, rot_dim=64))
