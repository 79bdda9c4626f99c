"""Bounds that the operators on a paged cache in 8 bits state, each where it is hardest to hold.

Attention: a weight is off by at most 2^-11 of itself and 2^-20 of its row's largest, and times its scale of V by no
more than 2^-20 of the largest such product, whatever V's scales are (with more than one token a row: or, where that is
more, 2^-84 of the largest product).  A dim that is zero in the blocks of the largest scale shows the first: what is lost of the others'
weights is lost of its whole output.  Blocks of a large scale and small weights show the second.  Each dim has a
tolerance of its own here, made from what it sums itself.
"""
import math
import random

import numpy as np
import pytest
import torch

from continuous_batching_transformer_gb300 import paged
from tests import fp8_reference as F
from tests import paged_reference as R
from tests.gpu_harness import ensure_built
from tests.test_gpu_paged_fp8 import SCORE, WEIGHT, attend, dev, i32, run_append
from tests.test_paged_fp8_bounds_host import growing, off_at_most

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -20  # of the row's largest weight, or weight times scale


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def row_of(n, hd, exponents, seed, below):
    """A row whose block b has a V scale near 2^exponents[b]: blocks above the smallest have their values in one
    dim each alone, and K's first dim -below.  Returns pool, table, k, v and the exponents of V's scales by position."""
    r = np.random.default_rng(seed)
    lay = F.Layout(1, hd, 64)
    blocks = -(-n // 64)
    k = r.integers(-8, 9, (n, 1, hd)) / 16.0
    k[..., 0] = 0
    v = r.standard_normal((n, 1, hd))
    least = min(exponents)
    for b in range(blocks):
        e = exponents[b % len(exponents)]
        rows = slice(64 * b, min(n, 64 * b + 64))
        if e > least:
            keep = v[rows, 0, b % 5].copy()
            v[rows] = 0
            v[rows, 0, b % 5] = keep
            k[rows, 0, 0] = -below
        v[rows] *= 2.0 ** e
    pool = np.full(blocks * lay.page_bytes, 0x7F, np.uint8)
    F.append(pool, lay, k, v, list(range(n)))
    table = np.arange(blocks, dtype=np.int32)
    held = np.log2(lay.views(pool)[2][:, 1, 0, 0]).repeat(64)[:n]
    return pool, table, *F.values(pool, lay, table, n), held


def check(n, new, hd, exponents, decode, seed=0, heads=3, spread=1.0, dtype=torch.float32, below=0):
    pool, table, k, v, held = row_of(n, hd, exponents, seed, below)
    g = torch.Generator().manual_seed(seed + 1)
    # whole 8ths below 16: two parts of four bits hold them
    q = (torch.randint(-8, 9, (new, heads, hd), generator=g) / 8 * spread).bfloat16()
    q[..., 0] = 8.0
    got = attend(pool, table, n, q, new, hd, decode, dtype=dtype)
    x, scale = q.double().numpy(), 1 / math.sqrt(hd)
    ref, mag = R.attention(x, k, v, n - new, 0, 0, scale)
    for t in range(new):
        p = n - new + t
        s = scale * (x[t] @ k[0, :p + 1].T)
        w = np.exp(s - s.max(-1, keepdims=True))
        product = (w * 2.0 ** held[:p + 1]).max(-1, keepdims=True)  # the largest weight is 1
        part = product / 2.0 ** held[:p + 1]
        floor = FLOOR * np.minimum(np.maximum(1, 0 if decode else part * 2.0 ** -64), part) / w.sum(-1, keepdims=True)
        # the last rounding, the sum in fp32, each weight's own rounding, and what is lost of it beside others
        tol = (2.0 ** -18 + WEIGHT + SCORE) * mag[t] + floor @ np.abs(v[0, :p + 1])
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
@pytest.mark.parametrize("n,new", [(500, 1), (4000, 1), (200, 70), (700, 130), (3000, 4)])
def test_weights_beside_a_far_larger_scale(n, new, hd, exponents):
    """(one token a row, and more; whole rows and rows cut into runs that are joined)"""
    check(n, new, hd, exponents, decode=new == 1, seed=len(exponents))
    if new == 1:
        check(n, 1, hd, exponents, decode=False, seed=7, heads=8)


@pytest.mark.parametrize("heads", [1, 2, 4, 8, 11])
def test_every_number_of_heads_beside_a_far_larger_scale(heads):
    for exponents in ([0, 30], [30, 30, 0, 0, 15, 0], [0, 5]):
        check(900, 1, 128, exponents, decode=True, heads=heads, seed=heads, spread=6.0)
        check(900, 1, 64, exponents, decode=True, heads=heads, seed=heads, dtype=torch.bfloat16)
        check(300, 40, 64, exponents, decode=False, heads=heads, seed=heads, spread=6.0)


@pytest.mark.parametrize("exponents", [[-60, 40], [40, -60], [40, 40, -60, -60], [-60, -30, 0, 40]], ids=str)
def test_scales_as_far_apart_as_there_are(exponents):
    for n in (300, 2500):
        check(n, 9, 128, exponents, decode=False, seed=5)
        check(n, 150, 64, exponents, decode=False, seed=6, heads=8)
        check(n, 1, 128, exponents, decode=True, seed=3)
        check(n, 1, 64, exponents, decode=True, seed=4, heads=8)


@pytest.mark.parametrize("below", [4, 10, 15])
@pytest.mark.parametrize("exponents", [[0, 18], [0, 0, 0, 0, 20, 20, 0, 0], [24, 24, 0, 0], [0, 8, 16, 24]], ids=str)
@pytest.mark.parametrize("n,new", [(700, 1), (4000, 1), (300, 70), (3000, 4)])
def test_small_weights_on_large_blocks(n, new, exponents, below):
    """Blocks whose values are large and whose weights are 2^-6 to 2^-22 of the others' (in heads of 64; 2^-4 to
    2^-15 in those of 128) and still carry the output."""
    for hd in (64, 128):
        check(n, new, hd, exponents, decode=new == 1, seed=below, below=below)


@pytest.mark.parametrize("seed", range(8))
def test_drawn_scales(seed):
    """Any order of scales, within 2^50 of one another, and of weights."""
    r = random.Random(seed)
    for hd in (64, 128):
        exponents = [r.choice([-20, -10, -4, 0, 2, 9, 17, 30]) for _ in range(r.randint(2, 12))]
        for n, new in ((r.randint(65, 1200), 1), (r.randint(2500, 5000), 1), (r.randint(200, 800), r.randint(2, 150))):
            check(n, new, hd, exponents, decode=new == 1, seed=seed, heads=r.choice([1, 2, 5, 8]), below=r.choice([0, 3, 12]),
                  spread=r.choice([1.0, 4.0]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_what_a_growing_block_holds(dtype):
    """Tokens appended one by one, every other one of which raises its block's scale: what is read back is within 2^-4 of
    each value and 2^-9 of the block's scale."""
    hd = 64
    for seed in range(4):
        x = torch.from_numpy(growing(seed)).to(dtype)
        n, lay = len(x), F.Layout(1, hd, 64)
        pool = torch.zeros(lay.page_bytes, dtype=torch.uint8, device=dev())
        cache = paged.PagedKVFp8(pool, i32([[0]]), i32([n]), page_tokens=64, n_kv_heads=1, head_dim=hd)
        app, q = paged.RopeAppend(cache, None, n_heads=1), torch.empty(1, hd, dtype=torch.bfloat16, device=dev())
        qkv = torch.cat([torch.zeros(n, hd, dtype=dtype), x.reshape(n, 2 * hd)], 1).to(dev())
        for t in range(n):
            app(0, qkv[t:t + 1], i32([t]), i32([t]), q)
        out = [torch.empty(n, hd, device=dev()) for _ in range(2)]
        paged.PageRead(cache)(0, *out, i32([0, n]))
        cache.check()
        scales = lay.views(pool.cpu().numpy())[2][0, :, 0, 0]
        for which in (0, 1):
            value, held = x[:, which, 0].double().numpy(), out[which].double().cpu().numpy()
            assert off_at_most(value, held, scales[which]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_of_the_last_positions(dtype):
    """Positions up to 2^31 - 2, the last that 32 bits count with their length: a row whose table names one page over
    and over."""
    kv, hd, n = 2, 64, 150
    lay = F.Layout(kv, hd, 64)
    pool = np.zeros(lay.page_bytes, np.uint8)
    r = np.random.default_rng(3)
    F.append(pool, lay, r.standard_normal((64, kv, hd)), r.standard_normal((64, kv, hd)), list(range(64)))
    want = [x.transpose(1, 0, 2) for x in F.values(pool, lay, [0], 64)]
    table = torch.zeros(1, 1 << 25, dtype=torch.int32, device=dev())
    last = 2 ** 31 - 1
    cache = paged.PagedKVFp8(torch.from_numpy(pool).to(dev()), table, i32([last]), page_tokens=64, n_kv_heads=kv, head_dim=hd)
    out = [torch.full((n, kv, hd), 0.7, dtype=dtype, device=dev()) for _ in range(2)]
    paged.PageRead(cache)(0, *out, i32([0, n]), i32([last - n]))
    cache.check()
    slots = [(last - n + j) % 64 for j in range(n)]
    for got, w in zip(out, want):
        assert (got.double().cpu().numpy() == w[slots]).all()


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("mode,rot", [("half", 64), ("interleaved", 32), ("half", 22), ("none", 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_q_beside_heads_that_are_not_finite(dtype, mode, rot, norm):
    """Infinities and NaN in some of q's heads: they stay what the formula makes of them, and everything else is what it
    is without them."""
    H, kv, hd, n = 5, 1, 64, 40
    r = np.random.default_rng(rot)
    x = torch.from_numpy(r.standard_normal((n, H + 2 * kv, hd))).to(dtype)
    x[::2, 1, 3] = float("inf")
    x[::3, 1, 40] = float("-inf")
    x[::2, 3, 17] = float("nan")
    pos = [int(p) for p in r.integers(0, 5000, n)]
    gain = (1 + 0.1 * torch.from_numpy(r.standard_normal(hd))).to(torch.bfloat16)
    pool = torch.zeros(F.Layout(kv, hd, 64).page_bytes, dtype=torch.uint8, device=dev())
    cache = paged.PagedKVFp8(pool, None, None, page_tokens=64, n_kv_heads=kv, head_dim=hd)
    rope = None if mode == "none" else paged.Rope(hd, rot_dim=rot, layout=mode, theta=1e4)
    q = torch.empty(n, H, hd, dtype=torch.bfloat16, device=dev())
    paged.RopeAppend(cache, rope, n_heads=H, eps=1e-6)(0, x.reshape(n, -1).to(dev()), i32(pos), i32(list(range(n))), q,
                                                       gain.to(dev()) if norm else None)
    cache.check()
    with np.errstate(invalid="ignore"):
        want = R.rope_heads(x[:, :H].double().numpy(), gain.double().numpy() if norm else None, 1e-6, np.array(pos),
                            0 if mode == "none" else rot, mode, R.rope_freqs(rot, 1e4, "none", 1.0, 0)[0], 1.0)
    got, fine = q.double().cpu().numpy(), np.isfinite(want)
    assert not fine.all() and fine[:, [0, 2, 4]].all()
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True)
    got, want = np.where(fine, got, 0), np.where(fine, want, 0)
    size = np.abs(want).max(-1, keepdims=True)
    assert (np.abs(got - want) <= R.BF16_STEP * 1.01 * np.abs(want) + 2.0 ** -18 * size).all()


def test_a_zeroed_page_is_gone_on_with():
    """A block that no append has begun, in a zeroed page, has the smallest scale there is until its first tokens."""
    for page, start in ((64, 9), (128, 70), (64, 63)):
        run_append(runs=[list(range(start, start + 40))], hd=64, page=page, norm=False, mode="none", fill=False)
        run_append(runs=[[start]], hd=128, page=page, fill=False)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("new", [1, 3])
def test_a_row_does_not_depend_on_the_others(new, hd):
    """Rows of every scale, enough of them for several a thread block: each has the bits that it has alone."""
    r = np.random.default_rng(hd + new)
    rows, kv, H, n = 500, 4, 8, 200
    pages = -(-n // 64)
    lay = F.Layout(kv, hd, 64)
    pool = r.integers(0, 256, rows * pages * lay.page_bytes, dtype=np.uint8)
    K, V, S = lay.views(pool)
    for codes in (K, V):
        codes[...] &= 0xBF  # finite, below 2
    S[:, 0] = 2.0 ** -2
    S[:, 1] = 2.0 ** r.integers(-12, 13, (rows * pages, kv, 1))
    S[::7, 1] = 2.0 ** r.integers(-50, 51, (len(S[::7]), kv, 1))
    dpool, table = torch.from_numpy(pool).to(dev()), torch.arange(rows * pages, dtype=torch.int32, device=dev()).view(rows, pages)
    q = torch.randn(rows * new, H, hd, generator=torch.Generator().manual_seed(hd)).bfloat16().to(dev())

    def attend(first, count):
        cache = paged.PagedKVFp8(dpool, table[first:first + count].contiguous(), i32([n] * count), page_tokens=64, n_kv_heads=kv,
                                 head_dim=hd)
        out = torch.empty(count * new, H, hd, device=dev())
        paged.Attention(cache, n_heads=H, max_kv=n, max_q=new, max_tokens=count * new)(
            0, q[first * new:(first + count) * new], out, None if new == 1 else i32([new * i for i in range(count + 1)]))
        cache.check()
        return out
    all_rows = attend(0, rows)
    assert torch.isfinite(all_rows).all()
    for b in range(0, rows, 9):
        assert torch.equal(attend(b, 1), all_rows[b * new:(b + 1) * new]), b
