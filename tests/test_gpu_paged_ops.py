"""The operators on a paged KV cache against their definitions in 64 bits (tests/paged_reference).

Tolerances, from the roundings on the way:
- attention: q, K and V are bf16 and their products exact in fp32; a score's sum of at most 128
  products and the exponential are off by a few 2^-24 of the score's size (SCORE below, for the
  score sizes here), the weights may be rounded to bf16 once (BF16_STEP of each weight, so of
  sum_j p_j |v_j| for the output), the output is rounded once.
- norm and rotation: a few fp32 roundings and an angle good to 2^-22 radians, all relative to the
  size of the pair, then one rounding.
- tables, slots, positions: equal.
"""
import math
import random

import numpy as np
import pytest
import torch

from continuous_batching_transformer_gb300 import binding as B
from continuous_batching_transformer_gb300 import paged
from tests import paged_reference as R
from tests.gpu_harness import ensure_built

pytestmark = pytest.mark.gpu

SCORE = 2.0 ** -14   # |scale q.k| below 64: 64 * 2^-24 * a few dozen roundings


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def dev():
    return torch.device("cuda:0")


def check_attention(out, ref, mag, dtype):
    got = out.double().cpu().numpy()
    step = R.BF16_STEP if dtype == torch.bfloat16 else R.F32_STEP
    tol = step * np.abs(ref) + (R.BF16_STEP + SCORE) * mag * 1.01 + 1e-30
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / tol)} of the tolerance"


def run_attention(rows, H, kv, hd, page, window=0, sinks=0, dtype=torch.bfloat16, seed=0, layers=1, layer=0,
                  poison=True, decode=False, pad=0, strided=False, slack=0, scale=None, spread=1.0,
                  max_q=None):
    """One call; returns the outputs (as a CPU float tensor) after checking them."""
    c = R.Cache(rows, kv=kv, hd=hd, page=page, window=window, sinks=sinks, seed=seed, layers=layers,
                layer=layer, poison=poison, device=dev(), spread=spread)
    g = torch.Generator().manual_seed(seed + 1)
    tokens = c.cu_host[-1]
    q = torch.randn(tokens + pad, H, hd, generator=g).to(torch.bfloat16).to(dev())
    out = torch.full((tokens + pad, H, hd), 7.0, dtype=dtype, device=dev())
    if strided:  # rows inside wider buffers
        wide = torch.zeros(tokens + pad, H * hd + 64, dtype=torch.bfloat16, device=dev())
        wide[:, 8:8 + H * hd] = q.view(tokens + pad, -1)
        q = wide[:, 8:8 + H * hd].unflatten(1, (H, hd))
        out = torch.full((tokens + pad, H * hd + 16), 7.0, dtype=dtype, device=dev())[:, 8:8 + H * hd]
        out = out.unflatten(1, (H, hd))
    cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=page, n_kv_heads=kv, head_dim=hd,
                          n_layers=layers)
    most = max(a + n for a, n in rows)
    attn = paged.Attention(cache, n_heads=H, max_kv=most + slack, window=window, sinks=sinks, scale=scale,
                           max_q=1 if decode else (max_q or max(1, max(n for _, n in rows))),
                           max_tokens=tokens + pad)
    attn(layer, q, out, cu_q=None if decode else c.cu)
    cache.check()
    ref, mag = c.expected(q[:tokens], window, sinks, 1 / math.sqrt(hd) if scale is None else scale)
    check_attention(out[:tokens], ref, mag, dtype)
    assert (out[tokens:] == 7.0).all()
    return out[:tokens].float().cpu()


DECODE = [
    # lengths (positions held, the new one included), heads, kv heads, head_dim, page, window, sinks
    ([1], 1, 1, 64, 64, 0, 0),
    ([1, 2, 3], 4, 4, 128, 128, 0, 0),
    ([63, 64, 65, 127, 128, 129], 8, 2, 128, 64, 0, 0),
    ([100, 1, 777], 12, 4, 64, 192, 0, 0),
    ([300, 513], 16, 1, 64, 128, 0, 0),          # 16 q heads on one kv head
    ([300, 40], 33, 1, 128, 64, 0, 0),           # 33
    ([200, 5], 5, 5, 128, 320, 0, 0),
    ([700, 699, 1, 128], 14, 2, 128, 64, 1, 0),  # a window of the token alone
    ([700, 699, 1, 128], 8, 2, 128, 64, 100, 4),
    ([1025, 600, 30], 8, 4, 64, 128, 128, 128),
    ([1025, 600, 30], 8, 4, 64, 128, 129, 65),
    ([900, 901], 4, 2, 128, 128, 64, 700),       # more sinks than the window hides
    ([900, 901], 4, 2, 128, 128, 5000, 3),       # a window longer than the rows
    ([2500, 1], 4, 1, 128, 256, 1000, 300),
]


@pytest.mark.parametrize("case", DECODE, ids=[str(i) for i in range(len(DECODE))])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_new_token(case, dtype):
    lens, H, kv, hd, page, w, s = case
    run_attention([(n - 1, 1) for n in lens], H, kv, hd, page, w, s, dtype, decode=True)


@pytest.mark.parametrize("hd", [64, 128])
def test_one_new_token_long_ragged_rows(hd):
    run_attention([(n - 1, 1) for n in (9000, 17, 4096, 12289, 1)], 4, 2, hd, 128, decode=True, seed=3)


@pytest.mark.parametrize("decode", [True, False])
def test_strided_rows_layers_and_slack(decode):
    rows = [(150, 1), (3, 1)] if decode else [(150, 20), (0, 33)]
    run_attention(rows, 8, 2, 128, 64, strided=True, layers=3, layer=1, slack=5000, decode=decode)
    run_attention(rows, 8, 2, 64, 64, 40, 2, strided=True, layers=2, layer=1, slack=1, decode=decode,
                  dtype=torch.float32)


PREFILL = [
    # (positions before, new tokens) of the rows, heads, kv heads, head_dim, page, window, sinks
    ([(0, 1)], 1, 1, 64, 64, 0, 0),
    ([(0, 5), (0, 17), (0, 32), (0, 9)], 4, 4, 64, 64, 0, 0),
    ([(0, 130), (7, 1), (200, 65)], 8, 2, 128, 128, 0, 0),
    ([(0, 260)], 4, 1, 128, 64, 0, 0),
    ([(77, 129), (0, 1), (500, 3)], 12, 4, 64, 192, 0, 0),
    ([(10, 40), (0, 21)], 33, 1, 128, 64, 0, 0),
    ([(10, 40), (0, 21)], 7, 1, 64, 64, 0, 0),
    ([(300, 200), (0, 90)], 8, 2, 128, 64, 1, 0),
    ([(300, 200), (0, 90), (1, 2)], 8, 2, 128, 64, 100, 4),
    ([(500, 140), (0, 300)], 8, 4, 64, 128, 128, 64),
    ([(500, 140), (0, 300)], 4, 2, 128, 128, 129, 65),
    ([(400, 130)], 4, 2, 128, 128, 30, 300),
    ([(600, 70), (0, 0), (128, 64)], 4, 2, 128, 128, 5000, 3),
    ([(1500, 200)], 2, 1, 128, 256, 700, 10),
]


@pytest.mark.parametrize("case", PREFILL, ids=[str(i) for i in range(len(PREFILL))])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_runs_of_tokens(case, dtype):
    rows, H, kv, hd, page, w, s = case
    run_attention(rows, H, kv, hd, page, w, s, dtype, pad=3)


def test_large_scores_and_scale():
    # peaked rows: scores up to about 60, so one key takes nearly all the weight
    run_attention([(200, 1), (511, 1)], 4, 2, 128, 64, decode=True, spread=4.0)
    run_attention([(100, 70)], 4, 2, 128, 64, spread=4.0)
    run_attention([(100, 1)], 4, 2, 64, 64, decode=True, scale=0.0)
    run_attention([(100, 50)], 4, 2, 64, 64, scale=-0.3)


def test_rows_that_see_nothing_get_zeros():
    """A row of length 0, and query tokens before a row's first position."""
    c = R.Cache([(0, 0), (9, 1), (0, 0)], kv=2, hd=64, page=64, window=0, sinks=0, seed=5, device=dev())
    cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=64, n_kv_heads=2, head_dim=64)
    q = torch.randn(3, 4, 64, device=dev()).to(torch.bfloat16)
    out = torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device=dev())
    paged.Attention(cache, n_heads=4, max_kv=64)(0, q, out)
    cache.check()
    assert (out[0] == 0).all() and (out[2] == 0).all() and torch.isfinite(out).all() and (out[1] != 0).any()
    # five query tokens of a row with three positions: the first two are at -2 and -1
    c = R.Cache([(-2, 5)], kv=2, hd=64, page=64, window=0, sinks=0, seed=6, device=dev())
    cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=64, n_kv_heads=2, head_dim=64)
    q = torch.randn(5, 4, 64, device=dev()).to(torch.bfloat16)
    out = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device=dev())
    paged.Attention(cache, n_heads=4, max_kv=3, max_q=5, max_tokens=5)(0, q, out, cu_q=c.cu)
    cache.check()
    ref, mag = c.expected(q, 0, 0, 0.125)
    assert (out[:2] == 0).all()
    check_attention(out, ref, mag, torch.bfloat16)


def test_row_results_do_not_depend_on_the_batch():
    rows = [(1200, 1), (5, 1), (640, 1), (127, 1)]
    c = R.Cache(rows, kv=2, hd=128, page=128, window=0, sinks=0, seed=8, device=dev())
    q = torch.randn(4, 8, 128, device=dev()).to(torch.bfloat16)
    for max_q in (1, 4):  # both forms of the call
        def run(sel):
            cache = paged.PagedKV(c.pool, c.table[sel].contiguous(), c.lens[sel].contiguous(),
                                  page_tokens=128, n_kv_heads=2, head_dim=128)
            out = torch.empty(len(sel), 8, 128, dtype=torch.float32, device=dev())
            cu = torch.arange(len(sel) + 1, dtype=torch.int32, device=dev())
            paged.Attention(cache, n_heads=8, max_kv=1300, max_q=max_q, max_tokens=len(sel))(
                0, q[sel].contiguous(), out, cu_q=cu)
            cache.check()
            return out
        together = run([0, 1, 2, 3])
        for b in range(4):
            assert torch.equal(run([b])[0], together[b])


def expect_error(cache, code, info):
    assert cache.err.tolist() == [code, info]
    with pytest.raises(B.CbtError):
        cache.check()
    cache.check()


@pytest.mark.parametrize("decode", [True, False])
def test_attention_reports_bad_rows_and_pages(decode):
    rows = [(100, 1), (150, 1), (20, 1)] if decode else [(100, 30), (150, 20), (20, 10)]
    c = R.Cache(rows, kv=2, hd=128, page=64, window=0, sinks=0, seed=9, device=dev())
    q = torch.randn(c.cu_host[-1], 4, 128, device=dev()).to(torch.bfloat16)
    ref, mag = c.expected(q, 0, 0, 1 / math.sqrt(128))

    def run(lens=None, table=None, cu=None, max_kv=256):
        cache = paged.PagedKV(c.pool, c.table if table is None else table, c.lens if lens is None else lens,
                              page_tokens=64, n_kv_heads=2, head_dim=128)
        out = torch.zeros(c.cu_host[-1], 4, 128, dtype=torch.bfloat16, device=dev())
        paged.Attention(cache, n_heads=4, max_kv=max_kv, max_q=1 if decode else 32, max_tokens=len(q))(
            0, q, out, cu_q=None if decode else (c.cu if cu is None else cu))
        torch.cuda.synchronize()
        good = [i for b in (0, 2) for i in range(c.cu_host[b], c.cu_host[b + 1])]
        check_attention(out[good], ref[good], mag[good], torch.bfloat16)
        return cache
    for bad in (257, -1, 2 ** 31 - 1):
        lens = c.lens.clone()
        lens[1] = bad
        expect_error(run(lens=lens), B.DEV_LENGTH, 1)
    lens = c.lens.clone()
    lens[1] = c.max_pages * 64 + 1           # within max_kv, past the table
    expect_error(run(lens=lens, max_kv=1 << 20), B.DEV_LENGTH, 1)
    for bad in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[1, 1] = bad
        expect_error(run(table=table), B.DEV_PAGE_ID, 1)
    if not decode:
        for at, bad in ((3, c.cu_host[-1] + 1), (3, c.cu_host[2] - 1), (3, 2 ** 31 - 1)):
            cu = c.cu.clone()
            cu[at] = bad
            cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=64, n_kv_heads=2, head_dim=128)
            out = torch.zeros(c.cu_host[-1], 4, 128, dtype=torch.bfloat16, device=dev())
            paged.Attention(cache, n_heads=4, max_kv=256, max_q=32, max_tokens=len(q))(0, q, out, cu_q=cu)
            torch.cuda.synchronize()
            n = c.cu_host[2]
            check_attention(out[:n], ref[:n], mag[:n], torch.bfloat16)
            assert cache.err.tolist() == [B.DEV_LENGTH, 2]


# ---- norm, rotation, append --------------------------------------------------------------------
ROPE = [
    # tokens, heads, kv heads, head_dim, page, layout, rot, scaling, factor, norm, dtype
    (1, 1, 1, 64, 64, "half", 64, "none", 1.0, False, torch.bfloat16),
    (8, 32, 8, 128, 128, "half", 128, "none", 1.0, False, torch.float32),
    (7, 4, 4, 128, 64, "half", 64, "linear", 4.0, True, torch.bfloat16),
    (65, 12, 4, 64, 192, "interleaved", 64, "by_parts", 8.0, True, torch.float32),
    (130, 3, 1, 128, 128, "interleaved", 2, "base", 2.0, True, torch.bfloat16),
    (33, 5, 5, 64, 64, "half", 6, "none", 1.0, True, torch.float32),
    (260, 8, 2, 128, 64, "half", 54, "by_parts", 40.0, False, torch.bfloat16),
    (200, 8, 2, 64, 128, "half", 32, "linear", 2.5, False, torch.float32),
    (50, 16, 1, 128, 64, None, 0, "none", 1.0, True, torch.bfloat16),
    (3, 2, 2, 64, 64, None, 0, "none", 1.0, False, torch.bfloat16),
]


@pytest.mark.parametrize("case", ROPE, ids=[str(i) for i in range(len(ROPE))])
@pytest.mark.parametrize("one_gain", [None, "q", "k"])
def test_rope_append(case, one_gain):
    n, H, kv, hd, page, layout, rot, scaling, factor, norm, dtype = case
    if one_gain and not norm:
        pytest.skip("no norm in this case")
    layers, layer = 2, 1
    g = torch.Generator().manual_seed(n)
    rng = random.Random(n)
    # runs of positions, some skipped tokens, slots spread over shuffled pages
    positions, slots = [], []
    n_pages = 2 * n + 4
    ids = list(range(n_pages))
    rng.shuffle(ids)
    t = 0
    while t < n:
        k = min(n - t, rng.choice([1, 3, 40, 150]))
        p0 = rng.choice([0, 5, 63, 64, 1000, 999_983])
        for p in range(p0, p0 + k):
            if (p - p0) % page == 0 or p % page == 0:
                pg = ids.pop()
            positions.append(p)
            slots.append(pg * page + p % page)
        t += k
    for t in range(0, n, 11):
        if t % 2:
            slots[t] = -1
        elif t:
            positions[t] = -5
    live = [t for t in range(n) if slots[t] >= 0 and positions[t] >= 0]
    width = (H + 2 * kv) * hd
    wide = torch.randn(n, width + 16, generator=g).to(dtype).to(dev())
    qkv = wide[:, 8:8 + width]
    qg = (1 + 0.2 * torch.randn(hd, generator=g)).to(torch.bfloat16) if norm and one_gain != "k" else None
    kg = (1 + 0.2 * torch.randn(hd, generator=g)).to(torch.bfloat16) if norm and one_gain != "q" else None
    pool = torch.randn(n_pages * layers * 2 * kv * page * hd, generator=g).to(torch.bfloat16)
    before = pool.clone()
    pool = pool.to(dev())
    q_out = torch.full((n, H * hd + 24), 3.0, dtype=torch.bfloat16, device=dev())
    rope = None if layout is None else paged.Rope(hd, rot_dim=rot, layout=layout, theta=1e4, scaling=scaling,
                                                  factor=factor, original_len=4096)
    cache = paged.PagedKV(pool, None, None, page_tokens=page, n_kv_heads=kv, head_dim=hd, n_layers=layers)
    d = lambda x: None if x is None else x.to(dev())
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())
    paged.RopeAppend(cache, rope, n_heads=H, eps=1e-5)(
        layer, qkv, i32(positions), i32(slots), q_out[:, 16:16 + H * hd], d(qg), d(kg))
    cache.check()

    x = qkv.double().cpu().numpy().reshape(n, H + 2 * kv, hd)
    f, m = R.rope_freqs(rot, 1e4, scaling, factor, 4096) if rot else ([], 1.0)
    num = lambda v: None if v is None else v.double().numpy()
    q = R.rope_heads(x[:, :H], num(qg), 1e-5, positions, rot, layout, f, m)
    k = R.rope_heads(x[:, H:H + kv], num(kg), 1e-5, positions, rot, layout, f, m)

    def close(got, ref, size):
        got = got.double().cpu().numpy()
        # the rounding to bf16, and fp32 roundings relative to the head's largest value
        tol = R.BF16_STEP * np.abs(ref) + 2.0 ** -18 * size
        assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)
    size = lambda y: np.abs(y).max(-1, keepdims=True) * 2
    close(q_out[:, 16:16 + H * hd].reshape(n, H, hd)[live], q[live], size(q[live]))
    dead = [t for t in range(n) if t not in set(live)]
    assert (q_out[dead] == 3.0).all() and (q_out[:, :16] == 3.0).all() and (q_out[:, 16 + H * hd:] == 3.0).all()
    after = pool.cpu()
    K, V = (fn(after, n_pages, layers, kv, page, hd, layer) for fn in (R.k_view, R.v_view))
    K0, V0 = (fn(before, n_pages, layers, kv, page, hd, layer) for fn in (R.k_view, R.v_view))
    for t in live:
        pg, o = slots[t] // page, slots[t] % page
        close(K[pg, :, o], k[t], size(k[t]))
        assert torch.equal(V[pg, :, o // 64, :, o % 64],
                           torch.from_numpy(x[t, H + kv:]).to(torch.bfloat16))
        K0[pg, :, o] = K[pg, :, o]
        V0[pg, :, o // 64, :, o % 64] = V[pg, :, o // 64, :, o % 64]
    assert torch.equal(after, before)  # nothing else in the pool was written


def test_rope_far_positions():
    """Angles near position 2^31: the fraction of a turn is exact, so the rotation stays as good as
    the 64-bit definition (position * f in double, 2^-22 radians there)."""
    n, hd = 6, 128
    pos = [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 30 + 1, 123_456_789, 2 ** 24 + 1, 0]
    x = torch.randn(n, 3 * hd, device=dev())
    pool = torch.zeros(paged.page_bytes(64, 1, hd) // 2, dtype=torch.bfloat16, device=dev())
    cache = paged.PagedKV(pool, None, None, page_tokens=64, n_kv_heads=1, head_dim=hd)
    q = torch.empty(n, hd, dtype=torch.bfloat16, device=dev())
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())
    paged.RopeAppend(cache, paged.Rope(hd, theta=1e6), n_heads=1)(0, x, i32(pos), i32(list(range(n))), q)
    cache.check()
    f, m = R.rope_freqs(hd, 1e6, "none", 1.0, 0)
    ref = R.rope_heads(x[:, None, :hd].double().cpu().numpy(), None, 0, pos, hd, "half", f, m)[:, 0]
    got = q.double().cpu().numpy()
    tol = R.BF16_STEP * np.abs(ref) + 2.0 ** -17 * np.abs(ref).max(-1, keepdims=True)
    assert (np.abs(got - ref) <= tol).all()


def test_append_reports_slots_outside_the_pool():
    pool = torch.zeros(2 * paged.page_bytes(64, 1, 64) // 2, dtype=torch.bfloat16, device=dev())
    cache = paged.PagedKV(pool, None, None, page_tokens=64, n_kv_heads=1, head_dim=64)
    x = torch.ones(3, 192, dtype=torch.bfloat16, device=dev())
    q = torch.zeros(3, 64, dtype=torch.bfloat16, device=dev())
    for bad in (128, 2 ** 31 - 1):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())
        paged.RopeAppend(cache, None, n_heads=1)(0, x, i32([0, 1, 2]), i32([0, bad, 5]), q)
        expect_error(cache, B.DEV_PAGE_ID, 1)
        assert (q[0] == 1).all() and (q[1] == 0).all() and (q[2] == 1).all()


# ---- tables and slots ---------------------------------------------------------------------------
def map_inputs(rows, page, max_pages, max_tokens, seed, grow=None):
    rng = random.Random(seed)
    lens = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, page * max_pages // 2)]) for _ in range(rows)]
    lens = [min(x, page * max_pages) for x in lens]
    new, room = [], max_tokens
    for n in lens:
        k = rng.choice([0, 1, 1, 1, -1, rng.randint(0, page * 2)]) if grow is None else grow
        k = min(k, page * max_pages - n, room)
        room -= max(k, 0)
        new.append(k)
    n_pages = rows * max_pages
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table = [[-9] * max_pages for _ in range(rows)]
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            table[b][j] = ids.pop()
    return lens, new, table, ids + [-7] * (n_pages - len(ids)), len(ids), n_pages


@pytest.mark.parametrize("rows,page,max_pages,max_tokens", [
    (1, 64, 2, 1), (3, 64, 4, 40), (8, 128, 8, 8), (37, 1, 9, 300), (100, 192, 6, 5000),
    (256, 64, 16, 2048), (256, 64, 16, 2049), (1024, 16, 4, 3000), (1025, 16, 4, 700), (4096, 64, 3, 9000)])
@pytest.mark.parametrize("inplace", [False, True])
def test_page_map(rows, page, max_pages, max_tokens, inplace):
    lens, new, table, stack, count, n_pages = map_inputs(rows, page, max_pages, max_tokens, rows + page)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())
    tl, tt, ts, tc = i32(lens), i32(table), i32(stack), i32([count])
    pm = paged.PageMap(tt, tl, ts, tc, page_tokens=page, max_tokens=max_tokens)
    lo, co = (None, None) if inplace else (torch.empty_like(tl), torch.empty_like(tc))
    for step in range(2 if inplace else 1):
        want = R.page_map(table, lens, new, stack, count, page, max_tokens)
        pm(i32(new), lo, co)
        pm.check()
        table, lens, stack, count, cu, pos, slots = want
        assert tt.tolist() == table and ts.tolist() == stack
        assert (tl if inplace else lo).tolist() == lens and (tc if inplace else co).tolist() == [count]
        assert pm.cu_q.tolist() == cu and pm.positions.tolist() == pos and pm.slots.tolist() == slots
        new = [1 if n < page * max_pages else 0 for n in lens]
        if sum(new) > max_tokens:
            break


def test_page_map_without_a_free_stack():
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())
    table = i32([[3, 1, 0], [2, 4, -1], [5, 5, 5]])
    lens = i32([60, 64, 7])
    pm = paged.PageMap(table, lens, None, None, page_tokens=64, max_tokens=16, n_pages=6)
    pm(i32([6, 2, -1]))
    pm.check()
    assert pm.cu_q.tolist() == [0, 6, 8, 8] and lens.tolist() == [66, 66, 0]
    assert pm.slots.tolist() == [3 * 64 + 60, 3 * 64 + 61, 3 * 64 + 62, 3 * 64 + 63, 64, 65, 4 * 64, 4 * 64 + 1] + [-1] * 8
    lens2 = i32([128, 128, 0])
    pm = paged.PageMap(i32([[0, 1, 9], [2, 4, -1], [5, 5, 5]]), lens2, None, None, page_tokens=64, max_tokens=16, n_pages=6)
    pm(i32([1, 2, 3]))
    assert pm.slots.tolist() == [-1, -1, -1, 320, 321, 322] + [-1] * 10
    assert pm.positions.tolist() == [128, 128, 129, 0, 1, 2] + [-1] * 10
    assert pm.err.tolist()[0] == B.DEV_PAGE_ID and pm.err.tolist()[1] in (0, 1)


@pytest.mark.parametrize("rows", [4, 1500])
def test_page_map_changes_nothing_on_errors(rows):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())
    page, max_pages, n_pages = 64, 4, rows * 4
    base_lens = [10] * rows
    ids = list(range(n_pages))
    base_table = [[ids.pop()] + [-1] * 3 for _ in range(rows)]

    def run(lens=base_lens, new=None, count=None, max_tokens=2 * rows):
        stack = ids + [-7] * (n_pages - len(ids))
        t, l, s, c = i32(base_table), i32(lens), i32(stack), i32([len(ids) if count is None else count])
        pm = paged.PageMap(t, l, s, c, page_tokens=page, max_tokens=max_tokens)
        pm(i32(new or [1] * rows))
        torch.cuda.synchronize()
        assert t.tolist() == base_table and s.tolist() == stack and l.tolist() == list(lens)
        assert c.tolist() == [len(ids) if count is None else count]
        assert pm.cu_q.tolist() == [0] * (rows + 1)
        assert set(pm.positions.tolist()) == {-1} and set(pm.slots.tolist()) == {-1}
        return tuple(pm.err.tolist())
    put = lambda v, at, x: v[:at] + [x] + v[at + 1:]
    assert run(lens=put(base_lens, 2, -1)) == (B.DEV_LENGTH, 2)
    assert run(lens=put(base_lens, 3, 257)) == (B.DEV_LENGTH, 3)
    assert run(new=put(put([1] * rows, 1, 247), 3, 2 ** 31 - 1)) == (B.DEV_LENGTH, 1)
    assert run(max_tokens=rows - 1) == (B.DEV_TOKENS, rows - 1)
    assert run(new=put([1] * rows, 0, 246), count=2, max_tokens=rows + 300) == (B.DEV_PAGES, 1)
    assert run(count=-1)[0] == B.DEV_PAGES
    assert run(count=n_pages, new=put([1] * rows, 0, -1))[0] == B.DEV_PAGES
    assert run(count=2 ** 31 - 1)[0] == B.DEV_PAGES


# ---- together -------------------------------------------------------------------------------------
def serve(steps, layers=2, H=8, kv=2, hd=64, page=64, window=70, sinks=3, graph=False):
    """A few continuous-batching steps on device state: rows admit prompts, decode and retire; every
    step maps pages, then appends and attends per layer.  Returns each step's outputs."""
    rows, max_pages, max_tokens = 4, 6, 128
    n_pages = 14
    g = torch.Generator(device=dev()).manual_seed(1)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())
    table = torch.full((rows, max_pages), -1, dtype=torch.int32, device=dev())
    lens, free, count = i32([0] * rows), i32(list(range(n_pages))), i32([n_pages])
    pool = torch.zeros(n_pages * paged.page_bytes(page, kv, hd, layers) // 2, dtype=torch.bfloat16, device=dev())
    cache = paged.PagedKV(pool, table, lens, page_tokens=page, n_kv_heads=kv, head_dim=hd, n_layers=layers)
    pm = paged.PageMap(table, lens, free, count, page_tokens=page, max_tokens=max_tokens)
    rope = paged.Rope(hd, theta=1e4, layout="interleaved")
    app = paged.RopeAppend(cache, rope, n_heads=H)
    attn = paged.Attention(cache, n_heads=H, max_kv=page * max_pages, max_q=100, max_tokens=max_tokens,
                           window=window, sinks=sinks)
    gain = (1 + 0.1 * torch.randn(2, layers, hd, device=dev(), generator=g)).to(torch.bfloat16)
    new = i32([0] * rows)
    qkv = torch.zeros(layers, max_tokens, (H + 2 * kv) * hd, device=dev())
    q = torch.zeros(max_tokens, H, hd, dtype=torch.bfloat16, device=dev())
    out = torch.zeros(layers, max_tokens, H, hd, dtype=torch.float32, device=dev())

    def step():
        pm(new)
        for l in range(layers):
            app(l, qkv[l], pm.positions, pm.slots, q, gain[0, l], gain[1, l])
            attn(l, q, out[l], cu_q=pm.cu_q)
    captured = None
    results, hist = [], [[] for _ in range(rows)]
    for s, n in enumerate(steps):
        new.copy_(i32(n))
        qkv.copy_(torch.randn(qkv.shape, device=dev(), generator=g))
        out.fill_(9.0)
        if graph:
            if captured is None:
                state = [t.clone() for t in (table, lens, free, count, pool)]
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    step()
                torch.cuda.current_stream().wait_stream(side)
                for t, v in zip((table, lens, free, count, pool), state):
                    t.copy_(v)
                out.fill_(9.0)
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    step()
                out.fill_(9.0)
            captured.replay()
        else:
            step()
        pm.check()
        cache.check()
        # the same step from the history of every row's QKV, in 64 bits
        at = 0
        f, m = R.rope_freqs(hd, 1e4, "none", 1.0, 0)
        for b in range(rows):
            if n[b] < 0:
                hist[b] = []
            k = max(n[b], 0)
            hist[b] += [qkv[:, at + i].double().cpu().numpy() for i in range(k)]
            L = len(hist[b])
            for l in range(layers):
                if not k:
                    continue
                x = np.stack([h[l] for h in hist[b]]).reshape(L, H + 2 * kv, hd)
                bf = lambda y: torch.from_numpy(y).to(torch.bfloat16).double().numpy()
                pos = list(range(L))
                G = gain[:, l].double().cpu().numpy()
                qr = bf(R.rope_heads(x[L - k:, :H], G[0], 1e-6, pos[L - k:], hd, "interleaved", f, m))
                kr = bf(R.rope_heads(x[:, H:H + kv], G[1], 1e-6, pos, hd, "interleaved", f, m))
                o, mag = R.attention(qr, kr.transpose(1, 0, 2), bf(x[:, H + kv:]).transpose(1, 0, 2), L - k,
                                     window, sinks, 1 / math.sqrt(hd))
                got = out[l, at:at + k].double().cpu().numpy()
                # a value next to a bf16 border may round the other way in q or k: its step moves a
                # score by at most 2 BF16_STEP |q||k| scale, here below 2^-3 and rarely; bound by
                # what all scores together could move
                sc = 4 * R.BF16_STEP * math.sqrt(hd) * 2
                assert (np.abs(got - o) <= (R.BF16_STEP + SCORE + sc) * mag + 1e-6).all()
            at += k
        assert (out[:, at:] == 9.0).all()
        assert lens.tolist() == [len(h) for h in hist]
        used = [x for b in range(rows) for x in table[b, :-(-len(hist[b]) // page)].tolist()]
        left = free[:int(count)].tolist()
        assert sorted(used + left) == list(range(n_pages))
        results.append(out.clone())
    return results


STEPS = [[60, 0, 0, 1], [1, 70, 0, 1], [1, 1, 0, 1], [-1, 1, 100, 1], [5, 1, 1, -1], [1, 1, 30, 90],
         [1, -1, 1, 1], [1, 33, -1, 1]]


def test_a_served_batch():
    serve(STEPS)


def test_a_served_batch_as_a_replayed_graph():
    a, b = serve(STEPS), serve(STEPS, graph=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_other_streams_and_two_handles():
    """Two attention handles on two streams at once: each has a workspace of its own."""
    rows = [(3000, 1), (2500, 1)]
    c = R.Cache(rows, kv=2, hd=128, page=128, window=0, sinks=0, seed=2, device=dev())
    cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=128, n_kv_heads=2, head_dim=128)
    q = torch.randn(2, 2, 8, 128, device=dev()).to(torch.bfloat16)
    out = torch.zeros(2, 2, 8, 128, device=dev())
    handles = [paged.Attention(cache, n_heads=8, max_kv=4096) for _ in range(2)]
    want = torch.zeros_like(out)
    for i in range(2):
        handles[i](0, q[i], want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                handles[i](0, q[i], out[i])
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_handles_refuse_wrong_tensors():
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev())
    pool = torch.zeros(4 * paged.page_bytes(64, 2, 64) // 2, dtype=torch.bfloat16, device=dev())
    cache = paged.PagedKV(pool, i32([[0, 1]]), i32([5]), page_tokens=64, n_kv_heads=2, head_dim=64)
    attn = paged.Attention(cache, n_heads=4, max_kv=128)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=dev())
    for bad in (lambda: attn(0, q.float(), q), lambda: attn(0, q.cpu(), q), lambda: attn(0, q, q.half()),
                lambda: attn(0, q[:, :, ::2], q), lambda: attn(1, q, q.clone()), lambda: attn(0, q.expand(2, 4, 64), q),
                lambda: attn(0, q, q.clone(), cu_q=i32([0])), lambda: attn(0, q, q.clone(), cu_q=i32([0, 1]).long()),
                lambda: paged.PagedKV(pool, i32([[0, 1]]), i32([5, 6]), page_tokens=64, n_kv_heads=2, head_dim=64),
                lambda: paged.PagedKV(pool[:100], None, None, page_tokens=64, n_kv_heads=2, head_dim=64),
                lambda: paged.PageMap(i32([[0]]), i32([1]), i32([0]), None, page_tokens=64, max_tokens=1),
                lambda: paged.PageMap(i32([[0]]), i32([1]), None, None, page_tokens=64, max_tokens=1)):
        with pytest.raises((TypeError, ValueError, IndexError)):
            bad()
    with pytest.raises(B.CbtError):
        paged.Attention(cache, n_heads=5, max_kv=128)(0, torch.zeros(1, 5, 64, dtype=torch.bfloat16, device=dev()),
                                                      torch.zeros(1, 5, 64, dtype=torch.bfloat16, device=dev()))
