"""Bounds that the operators on a paged cache in 8 bits state, each where it is hardest to hold.

Attention of single tokens: a weight is off by at most 2^-11 of itself and 2^-20 of its row's largest, whatever V's
scales are.  A dim that is zero in the
blocks of the largest scale shows it: what is lost of the others' weights is lost of its whole output.  Each dim has a
tolerance of its own here, made from what it sums itself.
"""
import math

import numpy as np
import pytest
import torch

from tests import fp8_reference as F
from tests import paged_reference as R
from tests.gpu_harness import ensure_built
from tests.test_gpu_paged_fp8 import SCORE, WEIGHT, attend

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -20  # of the row's largest weight


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def row_of(n, hd, exponents, seed):
    """A row whose block b has a V scale near 2^exponents[b]: blocks above the smallest have their values in one
    dim each alone.  Returns pool, table, k, v."""
    r = np.random.default_rng(seed)
    lay = F.Layout(1, hd, 64)
    blocks = -(-n // 64)
    k = r.integers(-8, 9, (n, 1, hd)) / 16.0
    v = r.standard_normal((n, 1, hd))
    least = min(exponents)
    for b in range(blocks):
        e = exponents[b % len(exponents)]
        rows = slice(64 * b, min(n, 64 * b + 64))
        if e > least:
            keep = v[rows, 0, b % 5].copy()
            v[rows] = 0
            v[rows, 0, b % 5] = keep
        v[rows] *= 2.0 ** e
    pool = np.full(blocks * lay.page_bytes, 0x7F, np.uint8)
    F.append(pool, lay, k, v, list(range(n)))
    table = np.arange(blocks, dtype=np.int32)
    return pool, table, *F.values(pool, lay, table, n)


def check(n, new, hd, exponents, decode, seed=0, heads=3, spread=1.0, dtype=torch.float32):
    pool, table, k, v = row_of(n, hd, exponents, seed)
    g = torch.Generator().manual_seed(seed + 1)
    # whole 8ths below 16: two parts of four bits hold them
    q = (torch.randint(-8, 9, (new, heads, hd), generator=g) / 8 * spread).bfloat16()
    got = attend(pool, table, n, q, new, hd, decode, dtype=dtype)
    x, scale = q.double().numpy(), 1 / math.sqrt(hd)
    ref, mag = R.attention(x, k, v, n - new, 0, 0, scale)
    for t in range(new):
        p = n - new + t
        s = scale * (x[t] @ k[0, :p + 1].T)
        w = np.exp(s - s.max(-1, keepdims=True))
        largest = 1 / w.sum(-1)  # of the normalised weights
        # the last rounding, the sum in fp32, each weight's own rounding, and 2^-20 of the largest a position
        tol = (2.0 ** -18 + WEIGHT + SCORE) * mag[t] + FLOOR * largest[:, None] * np.abs(v[0, :p + 1]).sum(0)
        if dtype == torch.bfloat16:
            tol += R.BF16_STEP * np.abs(ref[t])
        off = np.abs(got[t] - ref[t])
        assert (off <= tol).all(), (t, np.nanmax(off / tol), np.argwhere(~(off <= tol))[:5])


# scales of a row's blocks, as exponents, over and over: two in turn (the halves of a chunk of 128 positions), two
# chunks in turn, rising, falling, one large one among many
APART = [[0, 18], [18, 0], [0, 0, 24, 24], [24, 24, 0, 0], [0, 3, 6, 9, 12, 15, 18, 21, 24], [24, 16, 8, 0],
         [40, 0, 0, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 0, 0, 40], [-24, 36], [-24, -24, 0, 0, 36, 36], [2, 0, 1, 0, 3, 0, 0, 0]]


@pytest.mark.parametrize("exponents", APART, ids=str)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,new", [(500, 1), (4000, 1)])
def test_weights_beside_a_far_larger_scale(n, new, hd, exponents):
    """(whole rows and rows cut into runs that are joined)"""
    check(n, new, hd, exponents, decode=True, seed=len(exponents))


@pytest.mark.parametrize("heads", [1, 2, 4, 8, 11])
def test_every_number_of_heads_beside_a_far_larger_scale(heads):
    for exponents in ([0, 30], [30, 30, 0, 0, 15, 0], [0, 5]):
        check(900, 1, 128, exponents, decode=True, heads=heads, seed=heads, spread=6.0)
        check(900, 1, 64, exponents, decode=True, heads=heads, seed=heads, dtype=torch.bfloat16)


@pytest.mark.parametrize("exponents", [[-60, 40], [40, -60], [40, 40, -60, -60], [-60, -30, 0, 40]], ids=str)
def test_scales_as_far_apart_as_there_are(exponents):
    for n in (300, 2500):
        check(n, 1, 128, exponents, decode=True, seed=3)
        check(n, 1, 64, exponents, decode=True, seed=4, heads=8)
