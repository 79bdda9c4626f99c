"""Calls of the operators on a paged KV cache that the documentation allows and that lie off the usual
path: CTAs that hold every unit they may, ranges of tokens that are none, handles that are
dropped early and streams other than their own.  Tolerances are those of tests/test_gpu_paged_ops."""
import numpy as np
import pytest
import torch

from continuous_batching_transformer_gb300 import binding as B
from continuous_batching_transformer_gb300 import paged
from tests import paged_reference as R
from tests.gpu_harness import ensure_built
from tests.test_gpu_paged_ops import STEPS, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def dev():
    return torch.device("cuda:0")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [57, 228])
def test_ctas_full_of_units(rows, hd):
    """7296 units of (row, kv head) on 152 SMs: 48 for each CTA, the most it may hold.  Through a window
    of the token alone every output is its own V: off by the rounding of its one weight, which the sum
    does not share, and by that of the output."""
    kv = 7296 // rows
    n_pages = rows
    shape = (n_pages, 2, kv, 64 * hd)
    pool = torch.randn(shape, device=dev()).to(torch.bfloat16)
    table = torch.randperm(n_pages, device=dev()).int()[:, None].contiguous()
    lens, new = [1 + 7 * b % 64 for b in range(rows)], [1 + b % 2 for b in range(rows)]
    lens = [max(a, n) for a, n in zip(lens, new)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    cache = paged.PagedKV(pool.view(-1), table, i32(lens), page_tokens=64, n_kv_heads=kv, head_dim=hd)
    attn = paged.Attention(cache, n_heads=kv, max_kv=64, max_q=2, max_tokens=cu[-1], window=1)
    q = torch.randn(cu[-1], kv, hd, device=dev()).to(torch.bfloat16)
    out = torch.empty_like(q)
    attn(0, q, out, cu_q=i32(cu))
    cache.check()
    V = pool[:, 1].view(n_pages, kv, hd, 64)
    row = [b for b in range(rows) for _ in range(new[b])]
    pos = [lens[b] - new[b] + i for b in range(rows) for i in range(new[b])]
    want = V[table[row, 0].long(), :, :, torch.tensor(pos, device=dev())]
    tol = (2 * R.BF16_STEP + 2.0 ** -15) * want.float().abs()
    assert ((out.float() - want.float()).abs() <= tol).all()


@pytest.mark.parametrize("cut", [True, False])
@pytest.mark.parametrize("cu,good", [([0, 5, 1000, 10, 15], [0, 3]),    # rows 1 and 2 leave the call's tokens
                                     ([10, 15, 3, 8], [0, 2]),          # in another order
                                     ([-1, 4, 9, 2 ** 31 - 1, 12, 15], [1, 4]),
                                     ([-2 ** 31, 0, 5, -2 ** 31, 12, 15], [1, 4])])
def test_bad_ranges_in_the_middle(cu, good, cut):
    """A row whose range of tokens is no range is reported and skipped, whether the others' long rows
    are cut into runs or not; the tokens that no row takes stay as they are."""
    n = len(cu) - 1
    c = R.Cache([(3000 + 100 * b, 5) for b in range(n)], kv=2, hd=64, page=64, window=0, sinks=0, seed=4,
                device=dev())
    q = torch.randn(15, 8, 64, device=dev()).to(torch.bfloat16)
    out = torch.full((15, 8, 64), 7.0, device=dev())
    cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=64, n_kv_heads=2, head_dim=64)
    paged.Attention(cache, n_heads=8, max_kv=3500, max_q=5 if cut else 20000, max_tokens=15)(0, q, out, cu_q=i32(cu))
    torch.cuda.synchronize()
    assert cache.err.tolist()[0] == B.DEV_LENGTH and cache.err.tolist()[1] not in good
    left = set(range(15))
    for b in good:
        t = range(cu[b], cu[b + 1])
        first = 3000 + 100 * b + 5 - len(t)  # the last of them is the row's last position
        ref, mag = R.attention(q[cu[b]:cu[b + 1]].double().cpu().numpy(), c.k[b], c.v[b], first, 0, 0, 64 ** -0.5)
        check_attention(out[cu[b]:cu[b + 1]], ref, mag, torch.float32)
        left -= set(t)
    assert (out[sorted(left)] == 7.0).all()


@pytest.mark.parametrize("rows,max_kv", [(63, 4000), (63, 64), (4095, 64)])
def test_ranges_that_overlap(rows, max_kv):
    """Every other row takes all of the call's tokens, many more units than its launch is made for: it
    is reported, nothing but the call's rows is written, and the next call is right."""
    tokens, hd = 200, 64
    pool = torch.randn(2 * 2 * 64 * hd, device=dev()).to(torch.bfloat16)
    table = torch.zeros(rows, 1 + max_kv // 64, dtype=torch.int32, device=dev())
    lens = torch.full((rows,), max_kv, dtype=torch.int32, device=dev())
    cache = paged.PagedKV(pool, table, lens, page_tokens=64, n_kv_heads=1, head_dim=hd)
    attn = paged.Attention(cache, n_heads=4, max_kv=max_kv, max_q=tokens, max_tokens=tokens + 5)
    q = torch.randn(tokens + 5, 4, hd, device=dev()).to(torch.bfloat16)
    out = torch.full((tokens + 9, 4, hd), 7.0, device=dev())
    attn(0, q, out[:tokens + 5], cu_q=i32([0, tokens] * ((rows + 1) // 2)))
    torch.cuda.synchronize()
    assert (out[tokens:] == 7.0).all()
    assert cache.err.tolist()[0] == B.DEV_LENGTH and cache.err.tolist()[1] % 2 == 1
    cache.err.zero_()
    attn(0, q, out[:tokens + 5], cu_q=i32([0] * rows + [tokens]))
    cache.check()
    K, V = (R.k_view(pool, 2, 1, 1, 64, hd)[0], R.v_view(pool, 2, 1, 1, 64, hd)[0])
    n = max_kv // 64
    k = K.double().cpu().repeat(1, n + 1, 1)[:, :max_kv].numpy()
    v = V.permute(0, 1, 3, 2).reshape(1, 64, hd).double().cpu().repeat(1, n + 1, 1)[:, :max_kv].numpy()
    check_attention(out[:tokens], *R.attention(q[:tokens].double().cpu().numpy(), k, v, max_kv - tokens, 0, 0,
                                               hd ** -0.5), torch.float32)


def busy():
    torch.cuda._sleep(1_000_000_000)  # some 0.5 s, for the host to be ahead of


def taken_from(ptrs, sizes):
    """Whether new tensors of these sizes, made on the current stream, take any of the addresses."""
    held = [torch.empty(n, dtype=torch.uint8, device=dev()) for n in sizes for _ in range(50)]
    return {t.data_ptr() for t in held} & set(ptrs)


@pytest.mark.parametrize("new", [1, 3])
def test_memory_of_dropped_handles(new):
    """Handles that are dropped while another stream has yet to run their calls: what they made themselves
    is not handed out again before."""
    rows = [(3000, new), (2500, new)]
    c = R.Cache(rows, kv=2, hd=128, page=128, window=0, sinks=0, seed=2, device=dev())
    q = torch.randn(2 * new, 8, 128, device=dev()).to(torch.bfloat16)
    out, want = torch.zeros(2 * new, 8, 128, device=dev()), torch.zeros(2 * new, 8, 128, device=dev())
    table, lens, fresh = torch.zeros(2, 5, dtype=torch.int32, device=dev()), i32([0, 0]), i32([1, 2])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def handles():
        cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=128, n_kv_heads=2, head_dim=128)
        pm = paged.PageMap(table, lens, None, None, page_tokens=128, max_tokens=700, n_pages=4)
        return cache, paged.Attention(cache, n_heads=8, max_kv=4096, max_q=new, max_tokens=2 * new), pm
    cache, attn, pm = handles()
    attn(0, q, want, cu_q=c.cu)
    pm(fresh)  # (a kernel's first call loads it, which may wait for the device)
    cache.check()
    del cache, attn, pm
    busy()
    torch.cuda.synchronize()
    cache, attn, pm = handles()
    own = [cache.err, attn.workspace, pm.err, pm.cu_q, pm.positions, pm.slots]
    ptrs, sizes = [t.data_ptr() for t in own], [t.numel() * t.element_size() for t in own]
    with torch.cuda.stream(side):
        busy()
        attn(0, q, out, cu_q=c.cu)
        pm(fresh)
        done = side.record_event()
    del cache, attn, pm, own
    taken = taken_from(ptrs, sizes)
    assert not done.query(), "the other stream was done too early for this test to see anything"
    assert not taken
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_the_first_call_waits_for_the_error_word():
    """A cache made on a stream that is busy: a call on another one waits until its error word is zeroed,
    so that the error it finds is not wiped out afterwards."""
    c = R.Cache([(100, 1)], kv=2, hd=64, page=64, window=0, sinks=0, seed=2, device=dev())
    c.table.fill_(-1)
    q = torch.randn(1, 4, 64, device=dev()).to(torch.bfloat16)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        busy()
        cache = paged.PagedKV(c.pool, c.table, c.lens, page_tokens=64, n_kv_heads=2, head_dim=64)
        attn = paged.Attention(cache, n_heads=4, max_kv=128)
    attn(0, q, out)
    torch.cuda.synchronize()
    assert cache.err.tolist() == [B.DEV_PAGE_ID, 0]


@pytest.mark.parametrize("own", [True, False])
def test_a_map_of_no_rows(own):
    """No rows take no tokens: positions and slots say so, and the append that follows writes nothing."""
    given = {} if own else dict(cu_q=i32([5]), positions=i32([3, 2, 1]), slots=i32([0, 1, 2]))
    pm = paged.PageMap(i32([[0]])[:0], i32([]), None, None, page_tokens=64, max_tokens=3, n_pages=2, **given)
    # (before any call the handle's own outputs name no token either)
    assert not own or (pm.positions.tolist() == pm.slots.tolist() == [-1] * 3 and pm.cu_q.tolist() == [0])
    pm(i32([]))
    pm.check()
    assert pm.cu_q.tolist() == [0] and pm.positions.tolist() == pm.slots.tolist() == [-1] * 3
    pool = torch.full((2 * 2 * 64 * 64,), 7.0, dtype=torch.bfloat16, device=dev())
    cache = paged.PagedKV(pool, None, None, page_tokens=64, n_kv_heads=1, head_dim=64)
    qkv = torch.randn(3, 3 * 64, device=dev()).to(torch.bfloat16)
    q = torch.full((3, 1, 64), 7.0, dtype=torch.bfloat16, device=dev())
    paged.RopeAppend(cache, None, n_heads=1)(0, qkv, pm.positions, pm.slots, q)
    cache.check()
    assert (pool == 7.0).all() and (q == 7.0).all()


@pytest.mark.parametrize("rows", [5, 1500])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, "past", 2 ** 31 - 1])
def test_a_page_id_that_may_not_be_returned(rows, bad):
    """Rows that retire with an id outside the pool in their table: the call changes nothing, and no later
    one is handed that id."""
    page, mp = 64, 3
    n_pages = rows * mp + 8
    bad = n_pages if bad == "past" else bad
    table = torch.arange(rows * mp, dtype=torch.int32, device=dev()).view(rows, mp)
    lens = i32([130] * rows)
    stack = i32(list(range(rows * mp, n_pages)) + [-7] * (rows * mp))
    count = i32([8])
    pm = paged.PageMap(table, lens, stack, count, page_tokens=page, max_tokens=2 * rows)
    new = torch.where(torch.arange(rows, device=dev()) % 5 == 3, -1, 1).int()
    last = (rows - 4) // 5 * 5 + 3
    for where in ([3], [last], [last, 3]):
        t = table.clone()
        for r in where:
            table[r, r % 3] = bad
        before = [x.clone() for x in (table, lens, stack[:8], count)]
        pm(new)
        torch.cuda.synchronize()
        assert pm.err.tolist() == [B.DEV_PAGE_ID, min(where)]
        assert all(torch.equal(x, y) for x, y in zip(before, (table, lens, stack[:8], count)))
        assert set(pm.cu_q.tolist()) == {0} and set(pm.positions.tolist()) == set(pm.slots.tolist()) == {-1}
        pm.err.zero_()
        table.copy_(t)
    want = R.page_map(table.tolist(), lens.tolist(), new.tolist(), stack.tolist(), 8, page, 2 * rows)
    pm(new)
    pm.check()
    t, l, s, c, cu, pos, slots = want
    assert (table.tolist(), lens.tolist(), stack[:c].tolist(), count.tolist()) == (t, l, s[:c], [c])
    assert (pm.cu_q.tolist(), pm.positions.tolist(), pm.slots.tolist()) == (cu, pos, slots)
    # ids beyond a row's length are not looked at, nor those of rows that stay
    table[3, 1:] = bad
    table[0, 2] = bad
    lens[3] = 5
    pm(i32([0, 0, 0, -1] + [0] * (rows - 4)))
    pm.check()


@pytest.mark.parametrize("graph", [False, True])
def test_a_served_batch_from_what_was_cached(graph):
    """Steps of map, append and attention on device state, each part against 64 bits from what the part
    before it really left: q and the new K and V from the QKV rows, the attention from the q and the
    pages that it read.  So its tolerance is that of one call, which a lost sink, a window off by one or a
    stale page passes by far."""
    rows, H, kv, hd, page, window, sinks, layers, top, n_pages, mp = 4, 8, 2, 64, 64, 70, 3, 2, 128, 14, 6
    g = torch.Generator(device=dev()).manual_seed(1)
    table = torch.full((rows, mp), -1, dtype=torch.int32, device=dev())
    lens, free, count = i32([0] * rows), i32(list(range(n_pages))), i32([n_pages])
    pool = torch.zeros(n_pages * paged.page_bytes(page, kv, hd, layers) // 2, dtype=torch.bfloat16, device=dev())
    cache = paged.PagedKV(pool, table, lens, page_tokens=page, n_kv_heads=kv, head_dim=hd, n_layers=layers)
    pm = paged.PageMap(table, lens, free, count, page_tokens=page, max_tokens=top)
    app = paged.RopeAppend(cache, paged.Rope(hd, theta=1e4), n_heads=H)
    attn = paged.Attention(cache, n_heads=H, max_kv=page * mp, max_q=100, max_tokens=top, window=window, sinks=sinks)
    gain = (1 + 0.1 * torch.randn(2, layers, hd, device=dev(), generator=g)).to(torch.bfloat16)
    new = i32([0] * rows)
    qkv = torch.zeros(layers, top, (H + 2 * kv) * hd, device=dev())
    q = torch.zeros(layers, top, H, hd, dtype=torch.bfloat16, device=dev())
    out = torch.zeros(layers, top, H, hd, device=dev())

    def step():
        pm(new)
        for l in range(layers):
            app(l, qkv[l], pm.positions, pm.slots, q[l], gain[0, l], gain[1, l])
            attn(l, q[l], out[l], cu_q=pm.cu_q)
    captured = None
    f, m = R.rope_freqs(hd, 1e4, "none", 1.0, 0)
    blind = {"sinks": 0, "late window": 0, "early window": 0, "stale key": 0}
    held = [0] * rows
    for n in STEPS:
        new.copy_(i32(n))
        qkv.copy_(torch.randn(qkv.shape, device=dev(), generator=g))
        if graph and captured is None:
            state = [t.clone() for t in (table, lens, free, count, pool)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            for t, v in zip((table, lens, free, count, pool), state):
                t.copy_(v)
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
        out.fill_(9.0)
        captured.replay() if graph else step()
        pm.check()
        cache.check()
        held = [0 if k < 0 else h + k for h, k in zip(held, n)]
        assert lens.tolist() == held
        at = 0
        for b in range(rows):
            k, L = max(n[b], 0), held[b]
            if not k:
                continue
            ids = table[b, :-(-L // page)].long()
            pos = list(range(L - k, L))
            for l in range(layers):
                K = R.k_view(pool, n_pages, layers, kv, page, hd, l)[ids].permute(1, 0, 2, 3).reshape(kv, -1, hd)
                V = R.v_view(pool, n_pages, layers, kv, page, hd, l)[ids].permute(1, 0, 2, 4, 3).reshape(kv, -1, hd)
                K, V = K[:, :L].double().cpu().numpy(), V[:, :L].double().cpu().numpy()
                x = qkv[l, at:at + k].double().cpu().numpy().reshape(k, H + 2 * kv, hd)
                G = gain[:, l].double().cpu().numpy()
                got_q = q[l, at:at + k].double().cpu().numpy()
                for got, heads, gn in ((got_q, x[:, :H], G[0]),
                                       (K[:, L - k:].transpose(1, 0, 2), x[:, H:H + kv], G[1])):
                    ref = R.rope_heads(heads, gn, 1e-6, pos, hd, "half", f, m)
                    # the rounding to bf16, and fp32 roundings relative to the head's largest value
                    tol = R.BF16_STEP * np.abs(ref) + 2.0 ** -17 * np.abs(ref).max(-1, keepdims=True)
                    assert (np.abs(got - ref) <= tol).all()
                v_in = torch.from_numpy(x[:, H + kv:]).to(torch.bfloat16).double().numpy()
                assert np.array_equal(V[:, L - k:].transpose(1, 0, 2), v_in)
                o = out[l, at:at + k]
                scale = hd ** -0.5
                check_attention(o, *R.attention(got_q, K, V, L - k, window, sinks, scale), torch.float32)
                # mistakes planted in the reference are seen
                if L > window + sinks:
                    stale = K.copy()
                    stale[:, L - window // 2] = K[:, L - 1]
                    for name, (K2, w2, s2) in {"sinks": (K, window, 0), "late window": (K, window - 1, sinks),
                                               "early window": (K, window + 1, sinks),
                                               "stale key": (stale, window, sinks)}.items():
                        wrong = R.attention(got_q, K2, V, L - k, w2, s2, scale)
                        with pytest.raises(AssertionError):
                            check_attention(o, *wrong, torch.float32)
                        blind[name] += 1
            at += k
        assert (out[:, at:] == 9.0).all()
    assert all(v >= 10 for v in blind.values()), blind
