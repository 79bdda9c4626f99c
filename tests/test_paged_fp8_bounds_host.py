"""CPU checks of what a paged cache in 8 bits promises to hold, on the reference of its definition."""
import numpy as np

from tests import fp8_reference as F


def growing(seed, n=40, hd=64):
    """Tokens of a block, [n][2][1][hd]: each other one passes what its block's scale holds, some by far; among their
    elements are sizes down to 2^-20 of theirs."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, 2, 1, hd)) * 2.0 ** -r.integers(0, 21, (n, 2, 1, hd))
    top = 1.0
    for t in range(n):
        x[t, :, 0, 0] = top * r.uniform(0.5, 1.0, 2)
        if t % 2:
            top *= 2.0 ** r.choice([1, 1, 1, 2, 5])
    return x.astype(np.float32).astype(np.float64)


def off_at_most(value, held, scale):
    """Whether what is held is within 2^-4 of the value and 2^-9 of the block's scale, together."""
    return np.abs(held - value) <= 2.0 ** -4 * np.abs(value) + 2.0 ** -9 * scale


def test_what_a_growing_block_holds():
    """Each move to a larger scale rounds subnormal codes again: half a step of 2^-9 of the new scale each, in all less than
    2^-10 (1 + 1/2 + 1/4 + ...) of the last one.  Without growth one rounding is all."""
    worst = 0.0
    for seed in range(20):
        x, lay = growing(seed), F.Layout(1, 64, 64)
        pool = np.zeros(lay.page_bytes, np.uint8)
        for t in range(len(x)):
            F.append(pool, lay, x[t:t + 1, 0], x[t:t + 1, 1], [t])
        scales = lay.views(pool)[2][0, :, 0, 0]
        for which, got in enumerate(F.values(pool, lay, [0], len(x))):
            value, held = x[:, which, 0], got[0]
            assert off_at_most(value, held, scales[which]).all()
            once = np.maximum(2.0 ** -4 * np.abs(value), 2.0 ** -10 * scales[which])
            worst = max(worst, (np.abs(held - value) / once).max())
        pool[:] = 0
        F.append(pool, lay, x[:, 0], x[:, 1], list(range(len(x))))  # all at once: the scale does not grow
        scales = lay.views(pool)[2][0, :, 0, 0]
        for which, got in enumerate(F.values(pool, lay, [0], len(x))):
            value = x[:, which, 0]
            assert (np.abs(got[0] - value) <= np.maximum(2.0 ** -4 * np.abs(value), 2.0 ** -10 * scales[which])).all()
    assert worst > 1.2  # one rounding's bound does not hold for a block that has grown


def test_a_weight_as_four_codes():
    """Every fp16 up to 2^8 as the sum of four codes in units of 1, 1 / 16, 1 / 512 and 1 / 131072: each part, formed
    from the last one's rest in fp16, is exact in fp16 and fits a code, and the sum is off by 2^-24 at most."""
    x = np.arange(0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)
    x = x[x <= 256]
    y, unit, total = x, 1.0, np.zeros_like(x)
    for step in (16, 32, 256, 1):
        assert (y.astype(np.float16).astype(np.float64) == y).all() and np.abs(y).max() <= F.TOP
        code = F.VALUES[F.encode(y)]
        total += code * unit
        y, unit = (y - code) * step, unit / step
    assert np.abs(total - x).max() <= 2.0 ** -24
    assert np.abs(total - x)[x >= 2.0 ** -6].max() == 0
