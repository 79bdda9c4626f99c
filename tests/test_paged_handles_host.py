"""CPU checks of the paged operators' Python handles: sizes that a 32-bit field cannot hold, handles that
threads share."""
import ctypes
import threading
import time
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


class SlowCall:
    """In place of the launch: sees the arguments, lets other threads run, and sees them again."""

    def __init__(self, *args):
        self.torn = []
        self.seen = set()

    def join(self, raw):
        pass

    def __call__(self, fn, a):
        look = lambda: tuple(getattr(a, n) for n, t in a._fields_ if t in (ctypes.c_void_p, ctypes.c_int32))
        before = look()
        time.sleep(0.001)
        self.seen.add(before)
        if look() != before:
            self.torn.append(before)


@pytest.mark.parametrize("kind", ["append", "attention", "map"])
def test_threads_that_share_a_handle(kind, monkeypatch):
    """A call's arguments are its own until it has been queued."""
    monkeypatch.setattr(paged, "_Device", SlowCall)
    monkeypatch.setattr(paged, "_tensor", lambda t, *a, **k: t)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    bf = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)
    cache = cache_stub()
    cache.call = SlowCall()
    if kind == "append":
        h = paged.RopeAppend(cache, None, n_heads=4)
        make = lambda n: (0, bf(n, 8 * 64), i32(n), i32(n), bf(n, 4 * 64))
    elif kind == "attention":
        h = paged.Attention(cache, n_heads=4, max_kv=128, max_q=1, max_tokens=9)
        make = lambda n: (0, bf(n, 4 * 64), bf(n, 4 * 64), i32(3))
    else:
        table = i32(2, 3)
        h = paged.PageMap(table, i32(2), None, None, page_tokens=64, max_tokens=8, n_pages=8)
        h.index = -1
        make = lambda n: (i32(2), i32(2), None)
    device = cache.call if kind == "append" else h.call

    def work(n):
        args = make(n)
        for _ in range(20):
            h(*args)
    threads = [threading.Thread(target=work, args=(n,)) for n in (1, 2, 5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(device.seen) == 3 and not device.torn
