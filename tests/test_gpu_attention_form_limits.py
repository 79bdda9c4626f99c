"""Engines with an attention form (cbt_engine_set_attention) at the ends of what it takes."""
import numpy as np
import pytest

from tests.gpu_harness import ensure_built
from tests.test_gpu_attention_form import SHAPES, make_engine, run, weights

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
