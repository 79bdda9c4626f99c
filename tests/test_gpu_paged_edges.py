"""The operators on a paged KV cache at the ends of their ranges: few query tokens over long rows (cut
into runs and joined), more rows and units than a launch's first pass takes, the most q heads on a kv
head, offsets past 32 bits, captured calls side by side.  Checks and tolerances are those of
tests/test_gpu_paged_ops."""
import pytest
import torch

from continuous_batching_transformer_gb300 import binding as B
from continuous_batching_transformer_gb300 import paged
from tests import paged_reference as R
from tests.gpu_harness import ensure_built
from tests.test_gpu_paged_ops import check_attention, dev, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


LONG = [
    # (positions before, new tokens) of the rows, heads, kv heads, head_dim, page, window, sinks
    ([(449, 2)], 4, 1, 64, 64, 0, 0),             # one step above a single run
    ([(510, 2)], 4, 1, 128, 64, 0, 0),            # 8 steps, exactly
    ([(511, 2)], 4, 1, 128, 64, 0, 0),            # and a key more
    ([(6000, 5)], 4, 1, 64, 192, 0, 0),
    ([(8127, 2)], 2, 1, 128, 128, 0, 0),          # 127 + 1 steps, in runs that do not divide them
    ([(8060, 4)], 14, 2, 64, 64, 0, 0),
    ([(5000, 3), (0, 0), (17, 4), (2500, 0), (3000, 1)], 8, 2, 128, 128, 0, 0),
    ([(3000, 200), (700, 100)], 4, 1, 128, 64, 0, 0),
    ([(6000, 7), (900, 3)], 8, 2, 64, 64, 1500, 100),
    ([(6000, 7), (900, 3)], 4, 1, 128, 128, 5000, 2000),
    ([(4000, 2), (-3, 5)], 4, 2, 64, 64, 0, 0),   # and tokens before their row's first position
]


@pytest.mark.parametrize("case", range(len(LONG)))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_tokens_over_long_rows(case, dtype):
    rows, H, kv, hd, page, w, s = LONG[case]
    run_attention(rows, H, kv, hd, page, w, s, dtype, pad=3, seed=case)


@pytest.mark.parametrize("max_q", [3, 50, 20000])
def test_bounds_above_the_call(max_q):
    """Bounds larger than any row's: other cuts, and none at all, of the same sums."""
    run_attention([(4500, 3), (100, 2)], 8, 2, 128, 128, slack=30000, max_q=max_q)
    run_attention([(4500, 3), (100, 2)], 8, 2, 64, 64, 700, 90, strided=True, max_q=max_q, dtype=torch.float32)


def test_large_scores_across_runs():
    run_attention([(3000, 3)], 4, 2, 128, 64, spread=4.0)
    run_attention([(3000, 3)], 4, 2, 64, 64, scale=-0.3)
    run_attention([(3000, 3)], 4, 2, 64, 64, scale=0.0)


def test_more_rows_than_are_ranked():
    rows = [(7 * b % 90, b % 10) for b in range(80)] + [(400, 150)]
    run_attention(rows, 4, 2, 64, 64, pad=1)
    run_attention(rows, 8, 1, 128, 64, 33, 5)


@pytest.mark.parametrize("rows", [60, 100])
def test_more_units_than_the_sms_take(rows):
    """Each (row, kv head) is a unit: above 48 for each SM the grid grows."""
    run_attention([(b % 11, 1 + b % 2) for b in range(rows)], 128, 128, 64, 64)


@pytest.mark.parametrize("rows", [33, 1100, 4096])
def test_many_rows_of_one_new_token(rows):
    lens = [(37 * b) % 23 if rows > 100 else (311 * b) % 1500 for b in range(rows)]
    run_attention([(n, 1) for n in lens], 4, 2, 64, 64, decode=True)


@pytest.mark.parametrize("group", [43, 64])
def test_most_heads_on_a_kv_head(group):
    run_attention([(700, 1), (5, 1)], group, 1, 128, 64, decode=True)
    run_attention([(700, 1), (5, 1)], 2 * group, 2, 64, 64, 100, 3, decode=True)
    run_attention([(700, 9), (5, 3)], group, 1, 128, 64)
    run_attention([(1700, 9), (5, 3)], 2 * group, 2, 64, 64, 900, 3)


@pytest.mark.parametrize("new", [1, 3, 150])
def test_a_row_does_not_depend_on_what_the_others_hold(new):
    """Two calls of the same sizes, with one row in common."""
    n = 2000
    q = torch.randn(3 * new, 4, 64, device=dev()).to(torch.bfloat16)
    outs = []
    for other in (n, 3):
        rows = [(other, new), (n, new), (other // 2, new)]
        c = R.Cache(rows, kv=2, hd=64, page=64, window=0, sinks=0, seed=8, device=dev())
        own = R.Cache([(n, new)], kv=2, hd=64, page=64, window=0, sinks=0, seed=9, device=dev())
        pool = torch.cat([c.pool, own.pool])  # the row in the middle from a pool of its own
        table = torch.full((3, 60), -1, dtype=torch.int32, device=dev())
        table[:, :c.table.shape[1]] = c.table
        table[1] = -1
        table[1, :own.table.shape[1]] = torch.where(own.table[0] < 0, -1, own.table[0] + c.n_pages)
        cache = paged.PagedKV(pool, table, c.lens, page_tokens=64, n_kv_heads=2, head_dim=64)
        out = torch.empty(3 * new, 4, 64, device=dev())
        paged.Attention(cache, n_heads=4, max_kv=2200, max_q=new, max_tokens=3 * new)(0, q, out, cu_q=c.cu)
        cache.check()
        outs.append(out[new:2 * new].clone())
    assert torch.equal(*outs)


@pytest.mark.parametrize("new", [1, 4])
def test_two_captured_calls_side_by_side(new):
    rows = [(3000, new), (2500, new)]
    c = R.Cache(rows, kv=2, hd=128, page=128, window=0, sinks=0, seed=2, device=dev())
    cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=128, n_kv_heads=2, head_dim=128)
    q = torch.randn(2, 2 * new, 8, 128, device=dev()).to(torch.bfloat16)
    out, want = torch.zeros(2, 2 * new, 8, 128, device=dev()), torch.zeros(2, 2 * new, 8, 128, device=dev())
    handles = [paged.Attention(cache, n_heads=8, max_kv=4096, max_q=new, max_tokens=2 * new) for _ in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        handles[i](0, q[i], want[i], cu_q=c.cu)
    torch.cuda.synchronize()
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            for _ in range(5):
                handles[i](0, q[i], out[i], cu_q=c.cu)
    assert (out == 0).all()
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    q.neg_()  # a replay reads what the buffers hold then
    for i in range(2):
        handles[i](0, q[i], want[i], cu_q=c.cu)
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    cache.check()


def test_pages_past_32_bit_offsets():
    """A pool of 5 * 2^30 elements, whose last pages are the ones in use."""
    kv, hd, page, H = 2, 128, 128, 8
    elems = 2 * kv * page * hd
    n_pages = 5 * 2 ** 30 // elems
    pool = torch.empty(n_pages * elems, dtype=torch.bfloat16, device=dev())
    for rows in ([(300, 1), (129, 1)], [(300, 40), (129, 1)], [(2000, 2)]):
        c = R.Cache(rows, kv=kv, hd=hd, page=page, window=0, sinks=0, seed=4, device=dev())
        base = n_pages - c.n_pages
        pool[base * elems:].copy_(c.pool)
        table = torch.where(c.table < 0, c.table, c.table + base)
        cache = paged.PagedKV(pool, table, c.lens, page_tokens=page, n_kv_heads=kv, head_dim=hd)
        most = max(n for _, n in rows)
        q = torch.randn(c.cu_host[-1], H, hd, device=dev()).to(torch.bfloat16)
        out = torch.zeros(c.cu_host[-1], H, hd, device=dev())
        paged.Attention(cache, n_heads=H, max_kv=2100, max_q=most, max_tokens=len(q))(0, q, out, cu_q=c.cu)
        cache.check()
        check_attention(out, *c.expected(q, 0, 0, hd ** -0.5), torch.float32)
    # and the append, without a norm or a rotation: K and V land as they are
    append = paged.RopeAppend(cache, n_heads=H, rope=None)
    slots = torch.tensor([n_pages * page - 1, (n_pages - 1) * page, 5], dtype=torch.int32, device=dev())
    qkv = torch.randn(3, (H + 2 * kv) * hd, device=dev()).to(torch.bfloat16)
    append(0, qkv, torch.zeros(3, dtype=torch.int32, device=dev()), slots,
           torch.empty(3, H, hd, dtype=torch.bfloat16, device=dev()))
    cache.check()
    x = qkv.view(3, H + 2 * kv, hd)
    for t, s in enumerate(slots.tolist()):
        page_of = pool[s // page * elems:(s // page + 1) * elems]
        K, V = R.k_view(page_of, 1, 1, kv, page, hd), R.v_view(page_of, 1, 1, kv, page, hd)
        o = s % page
        assert torch.equal(K[0, :, o], x[t, H:H + kv])
        assert torch.equal(V[0, :, o // 64, :, o % 64], x[t, H + kv:])


@pytest.mark.parametrize("new", [1, 3, 200])
@pytest.mark.parametrize("hd", [64, 128])
def test_infinite_scores(new, hd):
    """A score of -inf is a weight of 0, wherever it falls: all that a run of the row's keys holds (the
    last key, alone in its chunk), the first keys, a chunk in the middle.  A query all of whose scores
    are -inf has no softmax: NaN."""
    page, H = 64, 4
    for n, hidden in ((641, [640]), (641, range(0, 130)), (1300, range(128, 256)), (70, [0]), (1, [0])):
        if n < new:
            continue
        c = R.Cache([(n - new, new)], kv=2, hd=hd, page=page, window=0, sinks=0, seed=3, device=dev())
        K = R.k_view(c.pool, c.n_pages, 1, 2, page, hd)
        for j in hidden:
            K[int(c.table[0, j // page]), :, j % page, 0] = float("-inf")
            c.k[0][:, j, 0] = float("-inf")
        q = torch.randn(new, H, hd, device=dev()).to(torch.bfloat16)
        q[..., 0] = q[..., 0].abs() + 0.5
        cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=page, n_kv_heads=2, head_dim=hd)
        for max_q in {new, 20000 if new > 1 else 1}:  # cut and whole
            out = torch.zeros(new, H, hd, device=dev())
            paged.Attention(cache, n_heads=H, max_kv=n, max_q=max_q, max_tokens=new)(0, q, out, cu_q=c.cu)
            cache.check()
            if n == 1:
                assert torch.isnan(out).all()
            else:
                check_attention(out, *c.expected(q, 0, 0, hd ** -0.5), torch.float32)
