"""Engines with an attention form (cbt_engine_set_attention) at the ends of what it takes."""
import numpy as np
import pytest
import torch

from tests.gpu_harness import ensure_built, to_dev
from tests.test_gpu_attention_form import FORMS, SHAPES, make_engine, run, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("form", [dict(window=2 ** 31 - 1), dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1),
                                  dict(window=2 ** 31 - 1100), dict(window=100, sinks=2 ** 31 - 1),
                                  dict(window=200000, sinks=7)])
def test_windows_and_sinks_that_hide_nothing(form):
    """A window that no row of the arena can outgrow, or as many sinks: every position is seen, to the
    last bit as without a window, also by rows past the tables' first size."""
    w, _ = weights(SHAPES["hd64"])
    lens, steps = [1300, 3], 2
    outs, _ = run(make_engine(w, form)[0], w.shape, lens, steps, chunk=400)
    want, _ = run(make_engine(w, {})[0], w.shape, lens, steps, chunk=400)
    assert all(np.array_equal(a, b) for a, b in zip(outs, want))


def test_growth_under_captured_steps():
    """Rows that outgrow the table and the sums between captured decode steps: the same bits as from an
    engine whose buffers were made for all of it before."""
    w, _ = weights(SHAPES["hd128-gqa"])
    s = w.shape
    g = torch.Generator().manual_seed(2)
    lens = [10, 900, 1500, 5000, 9000, 13000]
    kv = torch.randn(2, s.n_layers, s.n_kv_heads, max(lens), s.head_dim, generator=g).to(torch.bfloat16).cuda()
    toks = to_dev(np.arange(100, 100 + len(lens), dtype=np.int32))

    def add(eng, n):
        slab = eng.kv_slab_alloc(n + 100)
        eng.import_kv(slab, kv[0, :, :, :n].contiguous(), kv[1, :, :, :n].contiguous(), n)
        return slab

    def steps(eng):
        slabs, outs = [], []
        for i, n in enumerate(lens):
            slabs.append(add(eng, n))
            for rows in ([i], list(range(i + 1))):
                lg = torch.empty(len(rows), s.vocab, device="cuda")
                for _ in range(2):  # the second replays what the first captured
                    eng.decode_step_batch([slabs[r] for r in rows], toks[rows], lg)
                    outs.append(lg.clone())
        assert eng.device_error() == (0, 0)
        eng.retire(slabs)
        return outs
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        eng, _ = make_engine(w, FORMS["norm"], stream, arena=256 << 20)
        grown = steps(eng)
        eng, _ = make_engine(w, FORMS["norm"], stream, arena=256 << 20)
        slabs = [add(eng, max(lens)) for _ in lens]
        eng.decode_step_batch(slabs, toks, torch.empty(len(lens), s.vocab, device="cuda"))
        eng.retire(slabs)
        want = steps(eng)
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grown, want)) and torch.isfinite(grown[-1]).all()


def test_scratch_bytes_count_what_grows():
    """The table and the sums of a form are in the engine's statistics, and grow with the rows."""
    w, _ = weights(SHAPES["hd128-gqa"])
    s = w.shape
    eng, _ = make_engine(w, FORMS["norm"], arena=256 << 20)
    counted = [eng.stats().scratch_bytes]
    kv = torch.zeros(2, s.n_layers, s.n_kv_heads, 13000, s.head_dim, dtype=torch.bfloat16, device="cuda")
    lg = torch.empty(3, s.vocab, device="cuda")
    for n in (900, 13000):
        slabs = [eng.kv_slab_alloc(n + 1) for _ in range(3)]
        for slab in slabs:
            eng.import_kv(slab, kv[0, :, :, :n].contiguous(), kv[1, :, :, :n].contiguous(), n)
        eng.decode_step_batch(slabs, to_dev(np.array([1, 2, 3], np.int32)), lg)
        eng.retire(slabs)
        # an entry a page of 8 rows, and partial sums: three rows of 4 heads, in runs of four chunks of 128
        # keys (fewer of short rows), each of head_dim sums with a maximum and a weight
        least = 8 * 4 * -(-(n + 1) // 128) + 3 * 4 * -(-(n + 1) // 512) * (4 * s.head_dim + 8)
        counted.append(eng.stats().scratch_bytes)
        assert counted[0] + least <= counted[-1] <= counted[0] + 16 * least
    assert counted[0] < counted[1] < counted[2]
