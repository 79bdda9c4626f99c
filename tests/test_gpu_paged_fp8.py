"""The operators on a paged cache in 8 bits against their definitions in 64 bits (tests/fp8_reference).

Tolerances, from the roundings on the way:
- codes of V: equal (its values are not computed).  Codes of K: a few fp32 roundings and an angle good to
  2^-23, relative to the size of the pair, then one rounding to the code's grid.
- reading back: equal (a code times a power of two is exact in bf16).
- attention: products of codes and q are exact; a score's sum and the exponential are off by a few 2^-24
  of the score's size (SCORE below, for the sizes here) and by what q's rounding moves it; the weights are
  rounded to 2^-11 of each at most, and to 2^-24 of the largest; the output is rounded once.
"""
import math
import random

import numpy as np
import pytest
import torch

from continuous_batching_transformer_gb300 import binding as B
from continuous_batching_transformer_gb300 import paged
from tests import fp8_reference as F
from tests import paged_reference as R
from tests.gpu_harness import ensure_built

pytestmark = pytest.mark.gpu

SCORE = 2.0 ** -14    # |scale q.k| below 64: 64 * 2^-24 * a few dozen roundings
WEIGHT = 2.0 ** -11
KVALUE = 2.0 ** -20   # of a rotated pair's size: norm, product and sum, angle


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def dev():
    return torch.device("cuda:0")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


# ---- append ----------------------------------------------------------------------------------------
def run_append(runs, *, H=4, kv=2, hd=64, page=64, mode="half", rot=None, norm=True, dtype=torch.bfloat16, seed=0,
               layers=1, layer=0, fill=True, edit=None, strided=False, n_pages=None, positions=None, calls=1):
    """Appends runs of slots (lists; -1: skipped) and checks q, codes, scales and everything else."""
    slots = [s for r in runs for s in r]
    n = len(slots)
    n_pages = n_pages or max(max(slots) // page + 1, 1)
    lay = F.Layout(kv, hd, page, layers, layer)
    r = np.random.default_rng(seed)
    pool = np.zeros(n_pages * lay.page_bytes, np.uint8)
    if fill:  # earlier tokens everywhere, NaN codes among them
        pool[:] = r.integers(0, 256, pool.size, dtype=np.uint8)
        for l in range(layers):
            F.Layout(kv, hd, page, layers, l).views(pool)[2][...] = 2.0 ** r.integers(-8, 0, (n_pages, 2, kv, page // 64))
    x = torch.from_numpy(r.standard_normal((n, (H + 2 * kv) * hd))).to(dtype)
    if edit:
        edit(x.view(n, H + 2 * kv, hd))
    pos = positions or [-1 if s < 0 else int(p) for s, p in zip(slots, r.integers(0, 5000, n))]
    gain = (1 + 0.1 * torch.from_numpy(r.standard_normal((2, hd)))).to(torch.bfloat16) if norm else None
    rot = hd if rot is None else rot
    rope = None if mode == "none" else paged.Rope(hd, rot_dim=rot, layout=mode, theta=1e4)

    dpool = torch.from_numpy(pool.copy()).to(dev())
    cache = paged.PagedKVFp8(dpool, None, None, page_tokens=page, n_kv_heads=kv, head_dim=hd, n_layers=layers)
    app = paged.RopeAppend(cache, rope, n_heads=H, eps=1e-6)
    qkv, q = x.to(dev()), torch.full((n, H, hd), 7.0, dtype=torch.bfloat16, device=dev())
    if strided:
        wide = torch.zeros(n, x.shape[1] + 24, dtype=dtype, device=dev())
        wide[:, 8:8 + x.shape[1]] = qkv
        qkv = wide[:, 8:8 + x.shape[1]]
        q = torch.full((n, H * hd + 8), 7.0, dtype=torch.bfloat16, device=dev())[:, :H * hd]
    for _ in range(calls):
        app(layer, qkv, i32(pos), i32(slots), q, None if gain is None else gain[0].to(dev()),
            None if gain is None else gain[1].to(dev()))
    cache.check()
    got = dpool.cpu().numpy()

    # q and k by the formula
    h = x.double().numpy().reshape(n, H + 2 * kv, hd)
    freqs = R.rope_freqs(rot, 1e4, "none", 1.0, 0)[0]
    gains = [None, None] if gain is None else [gain[i].double().numpy() for i in (0, 1)]
    with np.errstate(invalid="ignore"):
        turned = [R.rope_heads(h[:, a:b], gains[i], 1e-6, np.maximum(pos, 0), 0 if mode == "none" else rot, mode,
                               freqs, 1.0) for i, (a, b) in enumerate(((0, H), (H, H + kv)))]
    live = np.array([s >= 0 for s in slots])
    gq = q.reshape(n, H, hd).double().cpu().numpy()
    size = np.abs(turned[0]).max(-1, keepdims=True)
    fine = np.isfinite(turned[0])
    off = np.abs(np.where(fine, gq - turned[0], 0))[live]
    assert (off <= (R.BF16_STEP * 1.01 * np.abs(turned[0]) + 2.0 ** -18 * size)[live][:, :, :][...]).all() or not fine.all()
    assert (gq[~live] == 7.0).all()

    want = pool.copy()
    F.append(want, lay, turned[1], h[:, H + kv:], slots)
    if calls > 1:
        F.append(want, lay, turned[1], h[:, H + kv:], slots)
    K, V, S = lay.views(got)
    Kw, Vw, Sw = lay.views(want)
    # scales: V's equal; K's too but where a largest value lies next to a border
    assert (S[:, 1] == Sw[:, 1]).all()
    differ = np.argwhere(S[:, 0] != Sw[:, 0])
    for pg, g, b in differ:
        mine = [t for t, s in enumerate(slots) if s >= 0 and s // 64 == (pg * page) // 64 + b]
        top = np.abs(turned[1][mine, g]).max()
        border = TOPS(top)
        assert abs(top - border) <= KVALUE * 4 * top, (top, S[pg, 0, g, b], Sw[pg, 0, g, b])
    assert (V == Vw).all()
    wrong = np.argwhere(K != Kw)
    for pg, g, o, d in wrong:  # the value lies next to the border between two codes
        t = max(t for t, s in enumerate(slots) if s == pg * page + o)
        s = S[pg, 0, g, o // 64]
        v, y = F.VALUES[K[pg, g, o, d]] * s, turned[1][t, g, d]
        half = F.step_at(y / s) * s / 2
        assert abs(v - y) <= half * (1 + 1e-9) + KVALUE * np.abs(turned[1][t, g]).max(), (v, y)
    assert len(wrong) <= 2 + 1e-4 * K.size
    # nothing else moved: the pool equals the expected one where no code or scale of this layer lies
    for p in (got, want):
        for view in lay.views(p):
            view[...] = 0
    assert (got == want).all()
    return dpool


def TOPS(x):
    """The border 448 * 2^e nearest to x."""
    e = F.exponent_for(x)
    return min((F.TOP * 2.0 ** e, F.TOP * 2.0 ** (e - 1)), key=lambda b: abs(b - x))


def span(start, n):
    return list(range(start, start + n))


APPENDS = [
    # one token each: in the middle of a block, at its start, at its end
    dict(runs=[[5], [64], [191], [70 + 192]], hd=64, page=64),
    dict(runs=[[5]], hd=128, page=128, H=32, kv=8, mode="none", norm=False),
    # runs over several blocks and pages, from and to odd positions
    dict(runs=[span(3, 200), span(256, 64), span(700, 1)], hd=64, page=64),
    dict(runs=[span(0, 130), [-1] * 5, span(300, 77)], hd=128, page=192, kv=1, H=3),
    dict(runs=[span(1, 63), span(64, 65), span(190, 3)], hd=128, page=64, mode="interleaved", rot=64),
    # parts of a head, odd pairs
    dict(runs=[span(40, 50), span(128, 20)], hd=64, page=64, rot=54),
    dict(runs=[span(40, 50), span(128, 20)], hd=128, page=64, rot=2, norm=False),
    dict(runs=[span(17, 30)], hd=128, page=64, rot=90, dtype=torch.float32),
    dict(runs=[span(64 * i + i, 1 + i) for i in range(40)], hd=64, page=64, kv=4, H=12, dtype=torch.float32),
    # enough tokens for chunks of 64; runs that begin anywhere in them
    dict(runs=[span(7, 701), span(1024, 333), [-1] * 3, span(1601, 500)], hd=64, page=64, kv=8, H=8),
    dict(runs=[span(33, 1300)], hd=128, page=128, kv=8, H=8, mode="interleaved"),
    # layers, strides
    dict(runs=[span(10, 100)], hd=64, page=64, layers=3, layer=1, strided=True),
    dict(runs=[span(10, 100)], hd=128, page=128, layers=2, layer=1, strided=True, dtype=torch.float32),
    # enough heads with them for two a thread block, and one over: short runs and long ones, every form
    dict(runs=[span(7, 701), [-1] * 3, span(1024, 333), span(1601, 200)], hd=64, page=64, kv=37, H=37, rot=54),
    dict(runs=[span(64 * i + i % 58, 3 + i % 4) for i in range(260)], hd=64, page=64, kv=37, H=37, dtype=torch.float32),
    dict(runs=[span(33, 1300)], hd=128, page=128, kv=33, H=33, mode="interleaved", strided=True),
    # norms alone; enough values that some lie beside a border between two codes
    dict(runs=[span(33, 1300)], hd=128, page=128, kv=8, H=8, mode="none"),
    dict(runs=[span(5, 1300)], hd=64, page=128, kv=8, H=8, mode="none", dtype=torch.float32),
    dict(runs=[span(0, 1500)], hd=128, page=64, kv=8, H=8, rot=54, dtype=torch.float32),
    # skipped tokens between runs and at the ends; nothing but skipped tokens
    dict(runs=[[-1], span(30, 3), [-1, -1], span(64, 2), [-1]], hd=64, page=64),
    dict(runs=[[-1] * 20], hd=64, page=64),
]


@pytest.mark.parametrize("case", APPENDS, ids=range(len(APPENDS)))
def test_append(case):
    run_append(**case)


@pytest.mark.parametrize("seed", range(6))
def test_append_drawn(seed):
    r = random.Random(seed)
    page = r.choice([64, 128, 192])
    runs, at = [], 0
    for _ in range(r.randint(1, 12)):
        n = r.randint(1, 150)
        start = at + r.randint(0, 100)
        runs.append(span(start, n))
        at = -(-(start + n) // page) * page
        if r.random() < 0.3:
            runs.append([-1] * r.randint(1, 4))
    run_append(runs=runs, page=page, hd=r.choice([64, 128]), kv=r.choice([1, 2, 5]), H=10, seed=seed,
               mode=r.choice(["none", "half", "interleaved"]), norm=r.random() < 0.5,
               dtype=r.choice([torch.float32, torch.bfloat16]))


def test_append_values_at_the_ends():
    """Zeros, infinities, NaN, the largest and smallest, and a token that raises its block's scale far."""
    def edit(x):  # V heads are the last two
        x[0, -2:] = 0
        x[1, -2] = float("inf")
        x[1, -1, ::2] = float("-inf")
        x[2, -2:, 5] = float("nan")
        x[3, -2:] = 3e38
        x[4, -2:] = 1e-38
        x[5, -2:] = 2.0 ** 40
        x[6, -2:, 0] = -448 * 2.0 ** 3
        x[7, -2:, 0] = 449 * 2.0 ** 3
    runs = [[5], [64 + 5], [128 + 5], [192 + 5], [256 + 5], [320 + 5], [384 + 5], [448 + 5]]
    run_append(runs=runs, hd=64, page=64, edit=edit, norm=False, mode="none")
    run_append(runs=runs, hd=64, page=64, edit=edit, norm=False, mode="none", dtype=torch.float32)
    # all in one block, which starts anew, and which goes on
    run_append(runs=[span(0, 8)], hd=128, page=64, edit=edit, norm=False, mode="none")
    run_append(runs=[span(9, 8)], hd=128, page=64, edit=edit, norm=False, mode="none")
    run_append(runs=[span(9, 8)], hd=128, page=64, edit=lambda x: x.zero_(), norm=False, mode="none", fill=False)


def test_append_again_changes_nothing():
    """The same tokens once more: their block's scale is there already."""
    run_append(runs=[span(3, 100), span(256, 30)], hd=64, page=64, calls=2)


def test_append_one_slot_many_times():
    """Tokens of one slot: the scale holds all of them, each element is one token's."""
    for hd, n in ((64, 300), (128, 300), (128, 40), (64, 2)):
        lay = F.Layout(1, hd, 64)
        pool = torch.zeros(2 * lay.page_bytes, dtype=torch.uint8, device=dev())
        cache = paged.PagedKVFp8(pool, None, None, page_tokens=64, n_kv_heads=1, head_dim=hd)
        x = torch.randn(n, 3 * hd, device=dev(), generator=torch.Generator(device=dev()).manual_seed(n)).bfloat16()
        slots = [64 + 7] * n
        paged.RopeAppend(cache, None, n_heads=1)(0, x, i32([1] * n), i32(slots),
                                                 torch.empty(n, hd, dtype=torch.bfloat16, device=dev()))
        cache.check()
        K, V, S = lay.views(pool.cpu().numpy())
        v = x.double().cpu().numpy().reshape(n, 3, hd)
        for which, got, mine in ((0, K[1, 0, 7], v[:, 1]), (1, V[1, 0, 0, :, 7], v[:, 2])):
            e = F.exponent_for(np.abs(mine).max())
            assert S[1, which, 0, 0] == 2.0 ** e
            choices = F.encode(mine * 2.0 ** -e)
            assert (choices == got[None]).any(0).all()
        assert (pool.cpu().numpy()[:lay.page_bytes] == 0).all()


def test_append_out_of_the_pool():
    lay = F.Layout(2, 64, 64)
    pool = torch.zeros(2 * lay.page_bytes, dtype=torch.uint8, device=dev())
    cache = paged.PagedKVFp8(pool, None, None, page_tokens=64, n_kv_heads=2, head_dim=64)
    app = paged.RopeAppend(cache, paged.Rope(64), n_heads=2)
    q = torch.full((3, 128), 7.0, dtype=torch.bfloat16, device=dev())
    app(0, torch.randn(3, 6 * 64, device=dev()), i32([1, 2, 3]), i32([128, 2 ** 31 - 1, -1]), q)
    with pytest.raises(B.CbtError, match="page id"):
        cache.check()
    assert (pool == 0).all() and (q == 7.0).all()
    app(0, torch.randn(0, 6 * 64, device=dev()), i32([]), i32([]), q[:0])  # no tokens
    cache.check()


# ---- read ------------------------------------------------------------------------------------------
def run_read(rows, *, kv, hd, page, seed=0, dtype=torch.bfloat16, layers=1, layer=0, strided=False, only=None,
             first=True):
    """rows: (first, n, length held)."""
    c = F.Cache([(n, 0) for _, _, n in rows], kv=kv, hd=hd, page=page, window=0, sinks=0, seed=seed, layers=layers,
                layer=layer, poison=False, device=dev())
    cache = paged.PagedKVFp8(c.pool, c.table, c.lens, page_tokens=page, n_kv_heads=kv, head_dim=hd, n_layers=layers)
    counts = [n for _, n, _ in rows]
    cu = [int(x) for x in np.concatenate([[0], np.cumsum(counts)])]
    n, w = cu[-1] + 2, kv * hd
    out = [torch.full((n, w + (16 if strided else 0)), 7.0, dtype=dtype, device=dev())[:, :w].unflatten(1, (kv, hd))
           for _ in range(2)]
    paged.PageRead(cache)(layer, out[0] if only != 1 else None, out[1] if only != 0 else None, i32(cu),
                          i32([a for a, _, _ in rows]) if first else None)
    cache.check()
    for which in (0, 1):
        got = out[which].double().cpu().numpy()
        if only is not None and which != only:
            assert (got == 7.0).all()
            continue
        for b, (a, m, _) in enumerate(rows):
            want = (c.k, c.v)[which][b][:, a:a + m].transpose(1, 0, 2)
            assert (got[cu[b]:cu[b + 1]] == want).all(), (which, b)
        assert (got[cu[-1]:] == 7.0).all()


@pytest.mark.parametrize("rows", [[(0, 1, 1)], [(0, 64, 64)], [(63, 2, 65)], [(5, 300, 310), (0, 0, 0), (100, 1, 500)],
                                  [(64, 64, 129), (0, 200, 200), (130, 0, 130), (17, 90, 107)],
                                  [(i, 3 + i, 110) for i in range(50)]])
@pytest.mark.parametrize("kv,hd,page,dtype", [(1, 64, 64, torch.bfloat16), (3, 128, 128, torch.bfloat16),
                                              (2, 128, 192, torch.float32), (2, 64, 256, torch.float32)])
def test_read(rows, kv, hd, page, dtype):
    run_read(rows, kv=kv, hd=hd, page=page, dtype=dtype)


def test_read_parts():
    rows = [(3, 100, 120), (0, 70, 90)]
    run_read(rows, kv=2, hd=64, page=64, only=0)
    run_read(rows, kv=2, hd=128, page=64, only=1, dtype=torch.float32)
    run_read(rows, kv=2, hd=128, page=64, layers=3, layer=2, strided=True)
    run_read([(0, 50, 60)] * 3, kv=1, hd=64, page=64, first=False)
    run_read([(0, 1, 1)] * 1500, kv=1, hd=64, page=64)  # a search of two rounds


def test_read_of_bad_rows():
    c = F.Cache([(100, 0), (100, 0), (100, 0)], kv=1, hd=64, page=64, window=0, sinks=0, seed=1, poison=False,
                device=dev())
    cache = paged.PagedKVFp8(c.pool, c.table, c.lens, page_tokens=64, n_kv_heads=1, head_dim=64)
    read = paged.PageRead(cache)
    k = torch.full((30, 64), 0.7, device=dev())  # no code times a power of two
    v = k.clone()
    for first in ([0, 91, 0], [0, -1, 0]):  # the second row leaves its positions
        k.fill_(0.7)
        read(0, k, v, i32([0, 10, 20, 30]), i32(first))
        with pytest.raises(B.CbtError, match="length"):
            cache.check()
        assert (k[10:20] == 0.7).all() and (k[:10] != 0.7).all() and (k[20:] != 0.7).all()
    for cu in ([0, 10, 5, 30], [0, 10, 20, 31], [-5, 10, 20, 30], [0, 2 ** 31 - 1, 0, 30]):
        read(0, k, v, i32(cu))
        with pytest.raises(B.CbtError, match="length"):
            cache.check()
    c.table[1, 0] = 99
    k.fill_(0.7)
    read(0, k, v, i32([0, 10, 20, 30]))
    with pytest.raises(B.CbtError, match="page id"):
        cache.check()
    assert (k[10:20] == 0.7).all() and (k[20:] != 0.7).all()
    read(0, k[:0], v[:0], i32([0, 0, 0, 0]))
    cache.check()
    with pytest.raises(ValueError):
        read(0, None, None, i32([0, 0, 0, 0]))
    with pytest.raises(TypeError):
        read(0, k, v.bfloat16(), i32([0, 10, 20, 30]))
    with pytest.raises(ValueError, match="strides"):
        read(0, k, torch.zeros(30, 72, device=dev())[:, :64], i32([0, 10, 20, 30]))


# ---- attention -------------------------------------------------------------------------------------
def check_attention(out, ref, mag, moved, dtype):
    got = out.double().cpu().numpy()
    step = R.BF16_STEP if dtype == torch.bfloat16 else R.F32_STEP
    tol = step * np.abs(ref) + (WEIGHT + SCORE + 2 * moved[..., None]) * mag * 1.01 + 2.0 ** -24 * mag.max(-1, keepdims=True) * 16 + 1e-30
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / tol)} of the tolerance"


def run_attention(rows, H, kv, hd, page, window=0, sinks=0, dtype=torch.bfloat16, seed=0, layers=1, layer=0,
                  decode=False, pad=0, strided=False, slack=0, scale=None, spread=1.0, max_q=None, apart=2, qscale=1.0):
    c = F.Cache(rows, kv=kv, hd=hd, page=page, window=window, sinks=sinks, seed=seed, layers=layers,
                layer=layer, device=dev(), spread=spread, apart=apart)
    g = torch.Generator().manual_seed(seed + 1)
    tokens = c.cu_host[-1]
    q = (torch.randn(tokens + pad, H, hd, generator=g) * qscale).to(torch.bfloat16).to(dev())
    out = torch.full((tokens + pad, H, hd), 7.0, dtype=dtype, device=dev())
    if strided:
        wide = torch.zeros(tokens + pad, H * hd + 64, dtype=torch.bfloat16, device=dev())
        wide[:, 8:8 + H * hd] = q.view(tokens + pad, -1)
        q = wide[:, 8:8 + H * hd].unflatten(1, (H, hd))
        out = torch.full((tokens + pad, H * hd + 16), 7.0, dtype=dtype, device=dev())[:, 8:8 + H * hd]
        out = out.unflatten(1, (H, hd))
    cache = paged.PagedKVFp8(c.pool, c.table, c.lens, page_tokens=page, n_kv_heads=kv, head_dim=hd, n_layers=layers)
    most = max(a + n for a, n in rows)
    attn = paged.Attention(cache, n_heads=H, max_kv=most + slack, window=window, sinks=sinks, scale=scale,
                           max_q=1 if decode else (max_q or max(1, max(n for _, n in rows))),
                           max_tokens=tokens + pad)
    attn(layer, q, out, cu_q=None if decode else c.cu)
    cache.check()
    scale = 1 / math.sqrt(hd) if scale is None else scale
    ref, mag, moved = c.expected(q[:tokens], window, sinks, scale)
    check_attention(out[:tokens], ref, mag, moved, dtype)
    assert (out[tokens:] == 7.0).all()
    return out[:tokens].float().cpu()


DECODE = [
    # lengths (positions held, the new one included), heads, kv heads, head_dim, page, window, sinks
    ([1], 1, 1, 64, 64, 0, 0),
    ([1, 2, 3], 4, 4, 128, 128, 0, 0),
    ([63, 64, 65, 127, 128, 129], 8, 2, 128, 64, 0, 0),
    ([700, 1, 333, 1500], 12, 4, 64, 64, 0, 0),
    ([1000, 257, 4500], 8, 1, 128, 192, 0, 0),
    ([300, 640], 5, 5, 128, 256, 0, 0),
    ([900, 515], 14, 2, 64, 512, 0, 0),
    ([400, 77], 32, 2, 128, 128, 0, 0),          # 16 q heads a kv head
    ([500], 33, 11, 64, 64, 0, 0),
    ([600, 5], 64, 1, 64, 128, 0, 0),
    ([1000, 64, 65, 300], 8, 2, 128, 64, 1, 0),
    ([1000, 64, 65, 300], 8, 2, 128, 64, 64, 0),
    ([1000, 129, 1025], 8, 2, 64, 128, 65, 3),
    ([2000, 300], 4, 2, 128, 64, 500, 70),
    ([2000, 300], 4, 2, 128, 64, 128, 1000),
]


@pytest.mark.parametrize("lens,H,kv,hd,page,window,sinks", DECODE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode(lens, H, kv, hd, page, window, sinks, dtype):
    run_attention([(n - 1, 1) for n in lens], H, kv, hd, page, window, sinks, dtype=dtype, decode=True, seed=len(lens))


PREFILL = [
    # rows (positions held before, new tokens), heads, kv heads, head_dim, page, window, sinks
    ([(0, 1)], 1, 1, 64, 64, 0, 0),
    ([(0, 2), (5, 3)], 4, 4, 128, 128, 0, 0),
    ([(0, 130), (64, 65), (200, 1)], 8, 2, 128, 64, 0, 0),
    ([(0, 257), (0, 63)], 12, 4, 64, 64, 0, 0),
    ([(700, 40), (0, 0), (63, 2)], 8, 1, 128, 192, 0, 0),
    ([(100, 90)], 5, 5, 128, 256, 0, 0),
    ([(300, 50), (0, 7)], 14, 2, 64, 512, 0, 0),
    ([(40, 30)], 64, 1, 64, 64, 0, 0),
    ([(100, 20)], 33, 11, 128, 64, 0, 0),
    ([(500, 100), (0, 200)], 8, 2, 128, 64, 1, 0),
    ([(500, 100), (0, 200)], 8, 2, 64, 128, 64, 3),
    ([(300, 150)], 4, 2, 128, 64, 129, 70),
    ([(900, 60)], 4, 2, 128, 64, 100, 800),
]


@pytest.mark.parametrize("rows,H,kv,hd,page,window,sinks", PREFILL)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill(rows, H, kv, hd, page, window, sinks, dtype):
    run_attention(rows, H, kv, hd, page, window, sinks, dtype=dtype, seed=len(rows), max_q=max(2, max(n for _, n in rows)))


@pytest.mark.parametrize("decode", [True, False])
def test_layers_strides_padding_and_scale(decode):
    rows = [(299, 1), (70, 1)] if decode else [(250, 30), (0, 70)]
    kw = dict(decode=decode, max_q=None)
    run_attention(rows, 8, 2, 128, 128, layers=3, layer=2, strided=True, **kw)
    run_attention(rows, 8, 2, 64, 64, layers=2, layer=0, strided=True, dtype=torch.float32, window=100, sinks=2, **kw)
    if not decode:
        run_attention(rows, 8, 2, 128, 64, pad=7, **kw)
    run_attention(rows, 8, 2, 128, 64, scale=0.0, **kw)
    run_attention(rows, 8, 2, 128, 64, scale=-0.05, **kw)
    run_attention(rows, 8, 2, 64, 64, slack=3000, **kw)


@pytest.mark.parametrize("decode", [True, False])
def test_blocks_of_very_different_sizes(decode):
    """Scales of K and V that differ by up to 2^20 between blocks, and sharp weights."""
    rows = [(699, 1), (300, 1)] if decode else [(300, 60), (0, 140)]
    run_attention(rows, 8, 2, 128, 64, apart=10, spread=0.01, decode=decode, dtype=torch.float32)
    run_attention(rows, 4, 4, 64, 128, apart=10, spread=0.01, decode=decode, dtype=torch.float32)
    run_attention(rows, 8, 2, 128, 64, spread=3.0, decode=decode, dtype=torch.float32, apart=0)


def planted(n, hd, k_of, v_of, page=64):
    """A row of n positions of one kv head with given float64 values (rounded to codes)."""
    lay = F.Layout(1, hd, page)
    pages = -(-n // page)
    pool = np.full(pages * lay.page_bytes, 0x7F, np.uint8)
    k, v = np.stack([k_of(j) for j in range(n)]), np.stack([v_of(j) for j in range(n)])
    F.append(pool, lay, k[:, None], v[:, None], list(range(n)))
    table = np.arange(pages, dtype=np.int32)
    return pool, table, *F.values(pool, lay, table, n)


def attend(pool, table, n, q, new, hd, decode, page=64, dtype=torch.float32):
    cache = paged.PagedKVFp8(torch.from_numpy(pool).to(dev()), torch.from_numpy(table[None]).to(dev()), i32([n]),
                             page_tokens=page, n_kv_heads=1, head_dim=hd)
    out = torch.empty(new, q.shape[1], hd, dtype=dtype, device=dev())
    paged.Attention(cache, n_heads=q.shape[1], max_kv=n, max_q=1 if decode else max(2, new), max_tokens=new)(
        0, q.to(dev()), out, None if decode else i32([0, new]))
    cache.check()
    return out.double().cpu().numpy()


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("hd", [64, 128])
def test_a_far_larger_weight_leaves_the_small_ones(decode, hd):
    """One position with a weight 2^14 times every other's, over 4000 of them: the small ones carry a fifth
    of the sum, and an output that drops or rounds them away is off by as much."""
    n = 4001
    sharp = np.zeros(hd)
    sharp[0] = 1.0
    pool, table, k, v = planted(n, hd, lambda j: sharp * (14.4 if j == 0 else 0.0),
                                lambda j: np.full(hd, -1.0 if j == 0 else 1.0))
    q = torch.zeros(1, 1, hd, dtype=torch.bfloat16)
    q[0, 0, 0] = math.log(2) * math.sqrt(hd)
    ref, _ = R.attention(q.double().numpy(), k, v, n - 1, 0, 0, 1 / math.sqrt(hd))
    got = attend(pool, table, n, q, 1, hd, decode)
    # 14.4 is held as 14 and ln 2 rounds in bf16, so 4000 weights of 2^-13.96 stand against one of 1:
    # (0.251 - 1) / (0.251 + 1) with hd 64, and near it with 128
    assert -0.62 < ref[0, 0, 0] < -0.58
    assert np.abs(got - ref).max() <= 2 * (WEIGHT + SCORE)


@pytest.mark.parametrize("decode", [True, False])
def test_blocks_of_zeros_count(decode):
    """V of a block that is all zero (its scale the smallest there is) still takes its share of the sum."""
    hd, n = 64, 256
    pool, table, k, v = planted(n, hd, lambda j: np.zeros(hd), lambda j: np.full(hd, 0.0 if 64 <= j < 192 else 3.0))
    q = torch.randn(1, 2, hd, generator=torch.Generator().manual_seed(3)).bfloat16()
    got = attend(pool, table, n, q, 1, hd, decode)
    assert np.abs(got - 1.5).max() <= 1.5 * (WEIGHT + SCORE)


@pytest.mark.parametrize("decode", [True, False])
def test_smallest_and_largest_scales(decode):
    hd, n = 128, 200
    for size in (2.0 ** -50, 2.0 ** 50):
        r = np.random.default_rng(5)
        pool, table, k, v = planted(n, hd, lambda j: r.standard_normal(hd) * 0.1, lambda j: r.standard_normal(hd) * size)
        q = torch.randn(1, 2, hd, generator=torch.Generator().manual_seed(3)).bfloat16()
        got = attend(pool, table, n, q, 1, hd, decode)
        ref, mag = R.attention(q.double().numpy(), k, v, n - 1, 0, 0, 1 / math.sqrt(hd))
        assert (np.abs(got - ref) <= 2 * (WEIGHT + SCORE) * mag).all()


@pytest.mark.parametrize("decode", [True, False])
def test_queries_of_any_size(decode):
    """q far from 1 (its parts follow its size), q of zeros, and one that is not finite."""
    rows = [(150, 1), (80, 1)] if decode else [(100, 20), (0, 33)]
    for qscale in (2.0 ** -60, 2.0 ** -12, 2.0 ** 60):
        run_attention(rows, 8, 2, 128, 64, decode=decode, qscale=qscale, scale=1 / qscale / 12, dtype=torch.float32)
    run_attention(rows, 8, 2, 64, 64, decode=decode, qscale=0.0)
    hd, n = 64, 100
    pool, table, k, v = planted(n, hd, lambda j: np.ones(hd), lambda j: np.ones(hd))
    for bad in (float("nan"), float("inf")):
        q = torch.ones(1, 4, hd, dtype=torch.bfloat16)
        q[0, 1, 7] = bad
        got = attend(pool, table, n, q, 1, hd, decode)
        assert np.isnan(got[0, 1]).all() and (np.abs(got[0, [0, 2, 3]] - 1) <= WEIGHT).all()


@pytest.mark.parametrize("decode", [True, False])
def test_long_rows(decode):
    """Rows long enough to be cut into runs of every length."""
    for n in (16500, 9000):
        rows = [(n - 1, 1)] if decode else [(n - 3, 3)]
        run_attention(rows, 2, 1, 128, 512, decode=decode, seed=n)


@pytest.mark.parametrize("decode", [True, False])
def test_bad_rows_and_pages(decode):
    """Lengths and pages out of range are reported; other rows are done."""
    rows = [(99, 1), (150, 1), (70, 1)]
    for what in ("length", "negative", "page"):
        c = F.Cache(rows, kv=2, hd=64, page=64, window=0, sinks=0, seed=3, device=dev())
        q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().to(dev())
        out = torch.full((3, 4, 64), 7.0, device=dev())
        if what == "page":
            c.table[1, 1] = c.n_pages
        else:
            c.lens[1] = 5000 if what == "length" else -3
        cache = paged.PagedKVFp8(c.pool, c.table, c.lens, page_tokens=64, n_kv_heads=2, head_dim=64)
        paged.Attention(cache, n_heads=4, max_kv=200, max_q=1 if decode else 4, max_tokens=3)(
            0, q, out, None if decode else c.cu)
        with pytest.raises(B.CbtError, match="page id" if what == "page" else "length"):
            cache.check()
        ref, mag, moved = c.expected(q, 0, 0, 1 / 8)
        for b in (0, 2):
            check_attention(out[b:b + 1], ref[b:b + 1], mag[b:b + 1], moved[b:b + 1], torch.float32)


def test_queries_before_the_first_position():
    """More query tokens than positions: those that see nothing get zeros."""
    c = F.Cache([(0, 5)], kv=1, hd=64, page=64, window=0, sinks=0, seed=2, device=dev())
    q = torch.randn(9, 2, 64, generator=torch.Generator().manual_seed(1)).bfloat16().to(dev())
    out = torch.full((9, 2, 64), 7.0, device=dev())
    cache = paged.PagedKVFp8(c.pool, c.table, c.lens, page_tokens=64, n_kv_heads=1, head_dim=64)
    paged.Attention(cache, n_heads=2, max_kv=64, max_q=9, max_tokens=9)(0, q, out, i32([0, 9]))
    cache.check()
    ref, mag = R.attention(q.double().cpu().numpy(), c.k[0], c.v[0], -4, 0, 0, 1 / 8)
    assert (out[:4] == 0).all()
    check_attention(out, ref, mag, np.zeros(mag.shape[:2]), torch.float32)


# ---- together --------------------------------------------------------------------------------------
def test_a_served_batch():
    """Prompts admitted, decoded, chunked and retired through PageMap, RopeAppend, Attention and PageRead
    on one cache, each call's outputs against the definition on what the cache then holds."""
    H, kv, hd, page, rows, n_pages = 4, 2, 64, 64, 4, 40
    lay = F.Layout(kv, hd, page)
    pool = torch.randint(0, 256, (n_pages * lay.page_bytes,), dtype=torch.uint8, device=dev(),
                         generator=torch.Generator(device=dev()).manual_seed(9))  # what pages hold before does not count
    table, lens = torch.full((rows, 8), -1, dtype=torch.int32, device=dev()), i32([0] * rows)
    free, count = i32(list(range(n_pages))), i32([n_pages])
    cache = paged.PagedKVFp8(pool, table, lens, page_tokens=page, n_kv_heads=kv, head_dim=hd)
    pages = paged.PageMap(table, lens, free, count, page_tokens=page, max_tokens=512)
    app = paged.RopeAppend(cache, paged.Rope(hd, theta=1e4), n_heads=H)
    attn = {m: paged.Attention(cache, n_heads=H, max_kv=512, max_q=m, max_tokens=512) for m in (1, 200)}
    read = paged.PageRead(cache)
    g = torch.Generator().manual_seed(4)
    held = [[] for _ in range(rows)]  # v rows appended so far, by row
    for new in ([100, 30, 0, 1], [1, 1, 1, 1], [1, 1, 1, 1], [70, 1, 90, 33], [1, -1, 1, -1], [1, 200, 1, 64],
                [1, 1, 1, 1]):
        pages(i32(new))
        n = sum(max(x, 0) for x in new)
        x = torch.randn(n, (H + 2 * kv) * hd, generator=g).bfloat16()
        q = torch.empty(n, H, hd, dtype=torch.bfloat16, device=dev())
        out = torch.zeros(n, H, hd, device=dev())
        app(0, x.to(dev()), pages.positions[:n], pages.slots[:n], q)
        one = all(v == 1 for v in new)
        attn[1 if one else 200](0, q, out, None if one else pages.cu_q)
        at = 0
        for b, m in enumerate(new):
            if m < 0:
                held[b] = []
            for t in range(max(m, 0)):
                held[b].append(x[at + t].double().numpy().reshape(-1, hd)[H + kv:])
            at += max(m, 0)
        ns = [len(h) for h in held]
        cu = [int(v) for v in np.concatenate([[0], np.cumsum(ns)])]
        k_out, v_out = (torch.zeros(cu[-1], kv, hd, dtype=torch.bfloat16, device=dev()) for _ in range(2))
        read(0, k_out, v_out, i32(cu))
        pages.check()
        cache.check()
        assert lens.tolist() == ns
        host, tab = pool.cpu().numpy(), table.cpu().numpy()
        at = 0
        for b, m in enumerate(new):
            if not ns[b]:
                continue
            k, v = F.values(host, lay, tab[b], ns[b])
            assert (k_out[cu[b]:cu[b + 1]].double().cpu().numpy() == k.transpose(1, 0, 2)).all()
            assert (v_out[cu[b]:cu[b + 1]].double().cpu().numpy() == v.transpose(1, 0, 2)).all()
            # what the cache holds is what was appended, to 2^-4 and 2^-8 of the block's scale
            want = np.stack(held[b]).transpose(1, 0, 2)
            top = np.abs(want).max()
            assert (np.abs(v - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -8 * top / F.TOP * 2).all()
            if m > 0:
                ref, mag = R.attention(q[at:at + m].double().cpu().numpy(), k, v, ns[b] - m, 0, 0, 1 / 8)
                check_attention(out[at:at + m], ref, mag, np.full(mag.shape[:2], 2.0 ** -12), torch.float32)
                at += m


def test_a_captured_step():
    """A step captured once and replayed while rows grow equals the calls made one by one."""
    H, kv, hd, page, rows, n_pages = 8, 2, 128, 64, 3, 20
    lay = F.Layout(kv, hd, page)

    def build():
        pool = torch.zeros(n_pages * lay.page_bytes, dtype=torch.uint8, device=dev())
        table, lens = torch.full((rows, 6), -1, dtype=torch.int32, device=dev()), i32([0] * rows)
        cache = paged.PagedKVFp8(pool, table, lens, page_tokens=page, n_kv_heads=kv, head_dim=hd)
        pages = paged.PageMap(table, lens, i32(list(range(n_pages))), i32([n_pages]), page_tokens=page, max_tokens=rows)
        app = paged.RopeAppend(cache, paged.Rope(hd), n_heads=H)
        attn, read = paged.Attention(cache, n_heads=H, max_kv=384), paged.PageRead(cache)
        x = torch.zeros(rows, (H + 2 * kv) * hd, device=dev())
        q, out = (torch.zeros(rows, H, hd, dtype=torch.bfloat16, device=dev()) for _ in range(2))
        k, v = (torch.zeros(rows, kv, hd, dtype=torch.bfloat16, device=dev()) for _ in range(2))
        ones, cu = i32([1] * rows), i32(list(range(rows + 1)))

        def step():
            pages(ones)
            app(0, x, pages.positions, pages.slots, q)
            attn(0, q, out)
            read(0, k, v, cu, first=pages.positions)
        return x, (pool, lens, q, out, k, v), step, (pages, cache, app, attn, read)
    xa, a, step_a, keep_a = build()
    xb, b, step_b, keep_b = build()
    graph = torch.cuda.CUDAGraph()
    step_b()  # once outside, then back to the start
    torch.cuda.synchronize()
    xb, b, step_b, keep_b = build()
    with torch.cuda.graph(graph):
        step_b()
    g = torch.Generator(device=dev()).manual_seed(1)
    for i in range(130):
        new = torch.randn(xa.shape, generator=g, device=dev()) * (1 + i % 7)
        xa.copy_(new)
        xb.copy_(new)
        step_a()
        graph.replay()
        if i % 13 == 0 or i > 126:
            for s, t in zip(a, b):
                assert torch.equal(s, t), i
    for h in (*keep_a[:2], *keep_b[:2]):
        h.check()


def test_the_same_call_gives_the_same_bits():
    """Whatever order blocks run in."""
    rows = [(900, 1), (5000, 1), (77, 1)]
    a = run_attention(rows, 8, 2, 64, 64, decode=True, dtype=torch.float32)
    rows = [(900, 40), (20, 130)]
    b = run_attention(rows, 8, 2, 64, 64, dtype=torch.float32)
    for _ in range(3):
        assert torch.equal(a, run_attention([(900, 1), (5000, 1), (77, 1)], 8, 2, 64, 64, decode=True, dtype=torch.float32))
        assert torch.equal(b, run_attention(rows, 8, 2, 64, 64, dtype=torch.float32))


def test_another_stream():
    c = F.Cache([(200, 1), (90, 1)], kv=2, hd=64, page=64, window=0, sinks=0, seed=3, device=dev())
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().to(dev())
    cache = paged.PagedKVFp8(c.pool, c.table, c.lens, page_tokens=64, n_kv_heads=2, head_dim=64)
    attn, read = paged.Attention(cache, n_heads=4, max_kv=256), paged.PageRead(cache)
    outs = []
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            out = torch.zeros(2, 4, 64, device=dev())
            k, v = (torch.zeros(100, 2, 64, device=dev()) for _ in range(2))
            attn(0, q, out)
            read(0, k, v, i32([0, 60, 100]), i32([30, 2]))
            cache.check()
        outs.append((out, k, v))
    for x, y in zip(*outs):
        assert torch.equal(x, y)


# ---- far sizes ---------------------------------------------------------------------------------------
def test_offsets_past_32_bits():
    """A pool of more than 4 GB, its rows in the last pages: append, read back and attend there."""
    H, kv, hd, page = 4, 2, 128, 64
    lay = F.Layout(kv, hd, page)
    n_pages = (1 << 32) // lay.page_bytes + 40
    if torch.cuda.mem_get_info()[0] < 2 * n_pages * lay.page_bytes:
        pytest.skip("not enough memory")
    pool = torch.empty(n_pages * lay.page_bytes, dtype=torch.uint8, device=dev())
    n = 300
    ids = list(range(n_pages - 1, n_pages - 1 - 5, -1))
    table = torch.tensor([ids], dtype=torch.int32, device=dev())
    cache = paged.PagedKVFp8(pool, table, i32([n]), page_tokens=page, n_kv_heads=kv, head_dim=hd)
    x = torch.randn(n, (H + 2 * kv) * hd, generator=torch.Generator().manual_seed(2)).bfloat16()
    q = torch.empty(n, H, hd, dtype=torch.bfloat16, device=dev())
    paged.RopeAppend(cache, None, n_heads=H)(0, x.to(dev()), i32(list(range(n))),
                                             i32([ids[j // page] * page + j % page for j in range(n)]), q)
    k, v = (torch.zeros(n, kv, hd, device=dev()) for _ in range(2))
    paged.PageRead(cache)(0, k, v, i32([0, n]))
    out = {}
    for new in (1, 70):
        out[new] = torch.zeros(new, H, hd, device=dev())
        paged.Attention(cache, n_heads=H, max_kv=n, max_q=new, max_tokens=new)(
            0, q[n - new:], out[new], None if new == 1 else i32([0, new]))
    cache.check()
    small = np.zeros(5 * lay.page_bytes, np.uint8)
    heads = x.double().numpy().reshape(n, -1, hd)
    F.append(small, lay, heads[:, H:H + kv], heads[:, H + kv:], list(range(n)))
    want_k, want_v = F.values(small, lay, np.arange(5), n)
    assert (k.double().cpu().numpy() == want_k.transpose(1, 0, 2)).all()
    assert (v.double().cpu().numpy() == want_v.transpose(1, 0, 2)).all()
    for new, o in out.items():
        ref, mag = R.attention(heads[n - new:, :H], want_k, want_v, n - new, 0, 0, 1 / math.sqrt(hd))
        check_attention(o, ref, mag, np.full(mag.shape[:2], 2.0 ** -12), torch.float32)


def test_many_rows():
    """More rows than are ranked, and more units than one round of them a block holds."""
    run_attention([(i % 7, 1 + i % 3) for i in range(90)], 2, 1, 64, 64, seed=5)
    r = random.Random(3)
    run_attention([(r.randint(0, 3), r.randint(0, 2)) for _ in range(4096)], 2, 2, 64, 64, max_q=2, seed=6)
    run_attention([(r.randint(0, 200), 1) for _ in range(500)], 3, 1, 64, 64, decode=True, seed=7)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 9, 20, 64])
def test_heads_of_a_kv_head(G):
    run_attention([(130, 1), (64, 1)], 2 * G, 2, 128, 64, decode=True, seed=G)
    run_attention([(130, 40), (0, 70)], 2 * G, 2, 128, 64, seed=G)
    run_attention([(130, 40)], G, 1, 64, 64, seed=G, window=50, sinks=3)


@pytest.mark.parametrize("sinks", [0, 1, 64, 65, 200])
@pytest.mark.parametrize("window", [1, 63, 64, 65, 200])
def test_windows_and_sinks(window, sinks):
    """Tiles whose tokens' windows begin in different steps, sinks that reach into them, runs cut anywhere."""
    run_attention([(700, 100), (0, 300), (129, 1)], 2, 1, 64, 64, window=window, sinks=sinks, seed=window)
    run_attention([(3000, 4)], 2, 1, 64, 64, window=window * 10, sinks=sinks, seed=sinks)
    run_attention([(700, 1), (0, 1), (129, 1)], 2, 1, 64, 64, window=window, sinks=sinks, seed=window, decode=True)


@pytest.mark.parametrize("decode", [True, False])
def test_scores_that_rise_along_the_row(decode):
    """Each step's scores pass the last one's reference, V's exponents change with every block."""
    hd, n = 64, 1400
    r = np.random.default_rng(8)
    sharp = np.zeros(hd)
    sharp[3] = 1.0
    pool, table, k, v = planted(n, hd, lambda j: sharp * (j // 64) * 12.0,
                                lambda j: r.standard_normal(hd) * 2.0 ** (j // 64 * 7 % 23 - 11))
    q = torch.zeros(1, 2, hd, dtype=torch.bfloat16)
    q[0, 0, 3], q[0, 1, 3] = 8.0, -8.0   # rising, and falling
    got = attend(pool, table, n, q, 1, hd, decode)
    ref, mag = R.attention(q.double().numpy(), k, v, n - 1, 0, 0, 1 / math.sqrt(hd))
    # scores up to 252: a few dozen roundings of 2^-24 of that
    assert (np.abs(got - ref) <= (WEIGHT + 4 * SCORE) * mag + 2.0 ** -20 * mag.max()).all()


def test_append_of_every_rotary_form():
    for hd in (64, 128):
        for mode, rot in (("none", hd), ("half", hd), ("half", 8), ("half", hd // 2), ("half", 22), ("interleaved", hd),
                          ("interleaved", 10), ("interleaved", 2)):
            for dtype in (torch.float32, torch.bfloat16):
                run_append(runs=[span(9, 30), span(70, 100), [200]], hd=hd, page=64, mode=mode, rot=rot, dtype=dtype,
                           H=3, kv=1, seed=rot)


def test_append_far_positions():
    """Angles of positions up to 2^31 - 1 keep their fraction of a turn."""
    run_append(runs=[[5], [70], [130], [195], [260]], hd=128, page=64,
               positions=[2 ** 31 - 1, 2 ** 30 + 12345, 1000003, 7, 0])


def test_append_settles_values_beside_a_border():
    """Rotated values that lie within 2^-24 of the middle between two codes, relative, are rounded as the formula's.

    Those that are the larger part of their pair (0.9 of its size): fp32 forms them with errors of at most 1.1 2^-24
    of each element for the angle, half a step for the product and half a step at last, 2.6 steps in all, with the
    distance 3.6, and four steps on either side are looked at.  Closer than 2^-26 is left out: the pairs of fp32
    are good to 2^-28 of the pair."""
    hd, r = 64, np.random.default_rng(7)
    freqs = np.asarray(R.rope_freqs(hd, 1e4, "none", 1.0, 0)[0])
    heads, positions, dims = [], [], []
    for pos in r.integers(1, 5000, 10):
        x = torch.from_numpy(r.standard_normal((50000, hd))).to(torch.bfloat16)
        a, b = (v.double().numpy() for v in (x[:, :hd // 2], x[:, hd // 2:]))
        c, s = np.cos(pos * freqs), np.sin(pos * freqs)
        y = np.concatenate([a * c - b * s, b * c + a * s], 1)
        size = np.tile(np.sqrt(a * a + b * b), 2)
        m, _ = np.frexp(np.abs(y))             # [0.5, 1): codes' middles at odd 32nds
        off = np.abs(m * 32 - (2 * np.floor(m * 16) + 1)) / (m * 32)
        ok = (off > 2.0 ** -26) & (off < 2.0 ** -24) & (np.abs(y) > 0.9 * size)
        ok &= np.abs(y) > 0.1 * np.abs(y).max(1, keepdims=True)  # codes of full length
        for i, d in np.argwhere(ok):
            heads.append(x[i])
            positions.append(int(pos))
            dims.append((d, y[i, d], np.abs(y[i]).max()))
    n = len(heads)
    assert n >= 3
    def edit(x):
        x[:, 1] = torch.stack(heads)
    pool = run_append([[64 * i] for i in range(n)], H=1, kv=1, hd=hd, page=64, norm=False, edit=edit, positions=positions)
    K = F.Layout(1, hd, 64).views(pool.cpu().numpy())[0]
    for i, (d, y, top) in enumerate(dims):
        assert K[i, 0, 0, d] == F.encode(y * 2.0 ** -F.exponent_for(top)), (i, d, y)


def test_append_products_past_the_range():
    """Norms of large rows with a large gain: k is finite, though x times the gain is not, and is held as the largest
    code, never as NaN."""
    n, kv, hd = 1300, 8, 64
    pool = torch.zeros(-(-n // 64) * F.Layout(kv, hd, 64).page_bytes, dtype=torch.uint8, device=dev())
    cache = paged.PagedKVFp8(pool, None, None, page_tokens=64, n_kv_heads=kv, head_dim=hd)
    r = np.random.default_rng(3)
    x = r.choice([-1.0, 1.0], (n, 1 + 2 * kv, hd)) * (1 + 99 * r.random((n, 1 + 2 * kv, hd))) * 2.0 ** 50
    qkv = torch.from_numpy(x.reshape(n, -1)).to(device=dev(), dtype=torch.bfloat16)
    q = torch.empty(n, 1, hd, dtype=torch.bfloat16, device=dev())
    gain = torch.full((hd,), 2.0 ** 100, dtype=torch.bfloat16, device=dev())
    paged.RopeAppend(cache, None, n_heads=1)(0, qkv, i32(list(range(n))), i32(list(range(n))), q, None, gain)
    cache.check()
    K = F.Layout(kv, hd, 64).views(pool.cpu().numpy())[0]
    held = K.transpose(0, 2, 1, 3).reshape(-1, kv, hd)[:n]
    assert (held == np.where(x[:, 1:1 + kv] < 0, 0xFE, 0x7E)).all()
