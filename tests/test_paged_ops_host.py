"""CPU checks of the paged operators: the frequencies of cbt_rope_init, every refusal of the C
entries (before anything reaches a device) and the checks of the Python handles."""
import ctypes
import math

import numpy as np
import pytest
import torch

import continuous_batching_transformer_gb300 as cbt
from continuous_batching_transformer_gb300 import binding as B
from continuous_batching_transformer_gb300 import paged
from tests.paged_reference import rope_freqs

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    cbt.build()
    return B.lib()


@pytest.mark.parametrize("hd,rot", [(64, 64), (128, 128), (128, 2), (128, 54), (64, 16)])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("base", 8.0),
                                            ("by_parts", 1.0), ("by_parts", 40.0)])
@pytest.mark.parametrize("theta", [1e4, 1e6])
def test_rope_init_frequencies(lib, hd, rot, scaling, factor, theta):
    r = paged.Rope(hd, rot_dim=rot, theta=theta, scaling=scaling, factor=factor, original_len=4096).desc
    f, m = rope_freqs(rot, theta, scaling, factor, 4096)
    got = [r.turns[i] / 2.0 ** 64 * 2 * math.pi for i in range(rot // 2)]
    # pow, a division by 2 pi and the conversion: a few roundings of 2^-53 each
    assert np.allclose(got, f, rtol=32 * 2.0 ** -53, atol=2.0 ** -60)
    assert all(r.turns[i] == 0 for i in range(rot // 2, 64))
    assert r.mscale == pytest.approx(m, rel=2.0 ** -23)
    assert (r.rot_dim, r.head_dim) == (rot, hd)


def test_rope_init_refusals(lib):
    ok = dict(layout=0, rot_dim=64, scaling=3, original_len=4096, theta=1e4, factor=2.0)
    out = B.RopeDesc()

    def rc(hd=128, **kw):
        c = B.RopeConfig()
        for k, v in {**ok, **kw}.items():
            setattr(c, k, v)
        return lib.cbt_rope_init(ctypes.byref(c), hd, ctypes.byref(out))
    assert rc() == 0
    assert lib.cbt_rope_init(None, 128, ctypes.byref(out)) == -2
    nan, inf = float("nan"), float("inf")
    for bad in (dict(layout=2), dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=130), dict(scaling=4),
                dict(scaling=-1), dict(theta=1.0), dict(theta=nan), dict(theta=inf), dict(factor=0.5),
                dict(factor=nan), dict(original_len=0), dict(beta_fast=1.0, beta_slow=2.0),
                dict(beta_fast=nan), dict(mscale=-1.0), dict(mscale=nan), dict(hd=96)):
        assert rc(**bad) == -1, bad


def kv_desc(**kw):
    d = dict(pool=FAKE, pool_bytes=16 * 65536, page_bytes=65536, k_offset=0, v_offset=32768, n_pages=16,
             page_tokens=64, n_kv_heads=2, head_dim=128)
    d.update(kw)
    r = B.PagedKvDesc()
    for k, v in d.items():
        setattr(r, k, v)
    return r


BAD_KV = [(dict(pool=None), -2), (dict(pool=FAKE + 16), -1), (dict(head_dim=96), -11),
          (dict(page_tokens=32), -1), (dict(page_tokens=0), -1), (dict(n_pages=0), -1),
          (dict(n_pages=17), -1), (dict(page_bytes=65536 + 8), -1), (dict(page_bytes=0), -1),
          (dict(k_offset=-256), -1), (dict(v_offset=32768 + 256), -1), (dict(v_offset=1 << 62), -1),
          (dict(pool_bytes=1 << 40), -12), (dict(n_pages=1 << 26), -12), (dict(n_kv_heads=0), -1),
          (dict(n_kv_heads=1 << 30), -1)]


def test_append_refusals(lib):
    def rc(kv=None, **kw):
        a = B.RopeAppendArgs()
        d = dict(qkv=FAKE, qkv_dtype=0, qkv_stride=(8 + 4) * 128, tokens=3, n_heads=8, eps=1e-6,
                 positions=FAKE, slots=FAKE, q_out=FAKE, q_stride=1024, err=FAKE)
        d.update(kw)
        a.kv = kv_desc(**(kv or {}))
        for k, v in d.items():
            setattr(a, k, v)
        return lib.cbt_rope_append(ctypes.byref(a), None)
    for bad, code in BAD_KV:
        assert rc(kv=bad) == code, bad
    assert rc(tokens=0) == 0
    assert rc(tokens=0, qkv=None) == 0
    wrong = paged.Rope(64).desc
    for bad, code in ((dict(tokens=-1), -1), (dict(n_heads=0), -1), (dict(qkv_dtype=2), -1),
                      (dict(qkv_stride=12 * 128 - 8), -1), (dict(qkv_stride=12 * 128 + 4), -1),
                      (dict(q_stride=1016), -1), (dict(q_stride=1028), -1), (dict(eps=-1.0), -1),
                      (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(qkv=None), -2),
                      (dict(q_out=None), -2), (dict(positions=None), -2), (dict(slots=None), -2),
                      (dict(err=None), -2), (dict(qkv=FAKE + 8), -1), (dict(q_out=FAKE + 2), -1),
                      (dict(q_gain=FAKE + 2), -1), (dict(k_gain=FAKE + 8), -1),
                      (dict(rope=ctypes.pointer(wrong)), -1),
                      (dict(n_heads=1 << 29, q_stride=1 << 40, qkv_stride=1 << 40), -12)):
        assert rc(**bad) == code, bad
    assert lib.cbt_rope_append(None, None) == -2


def attn_args(kv=None, **kw):
    a = B.PagedAttentionArgs()
    d = dict(block_table=FAKE, max_pages=4, rows=3, kv_lens=FAKE, tokens=3, max_q=1, max_kv=256,
             n_heads=8, q=FAKE, q_stride=1024, scale=0.1, out=FAKE, out_stride=1024, workspace=FAKE,
             workspace_bytes=1 << 40, err=FAKE)
    d.update(kw)
    a.kv = kv_desc(**(kv or {}))
    for k, v in d.items():
        setattr(a, k, v)
    return a


def test_attention_refusals(lib):
    def rc(kv=None, **kw):
        return lib.cbt_paged_attention(ctypes.byref(attn_args(kv, **kw)), None)
    for bad, code in BAD_KV:
        if bad != dict(n_kv_heads=1 << 30):
            assert rc(kv=bad) == code, bad
    assert rc(rows=0, tokens=0) == 0
    assert rc(tokens=0, cu_q=FAKE) == 0
    for bad, code in ((dict(rows=-1), -1), (dict(tokens=-1), -1), (dict(max_q=0), -1),
                      (dict(max_q=2), -1), (dict(tokens=4), -1), (dict(max_kv=-1), -1),
                      (dict(n_heads=9), -1), (dict(n_heads=0), -1), (dict(window=-1), -1),
                      (dict(sinks=-1), -1), (dict(scale=float("nan")), -1),
                      (dict(scale=float("inf")), -1), (dict(out_dtype=2), -1), (dict(max_pages=0), -1),
                      (dict(q_stride=1016), -1), (dict(q_stride=1020), -1), (dict(out_stride=1020), -1),
                      (dict(n_heads=130, q_stride=1 << 20, out_stride=1 << 20), -11),
                      (dict(rows=5000, tokens=5000), -12), (dict(max_kv=2 ** 31 - 1, window=1), -12),
                      (dict(max_kv=2 ** 31 - 1, sinks=1), -12), (dict(q=None), -2), (dict(out=None), -2),
                      (dict(block_table=None), -2), (dict(kv_lens=None), -2), (dict(err=None), -2),
                      (dict(q=FAKE + 2), -1), (dict(out=FAKE + 4), -1), (dict(workspace=FAKE + 16), -1)):
        assert rc(**bad) == code, bad
    assert lib.cbt_paged_attention(None, None) == -2


def test_attention_workspace_grows_with_the_bounds(lib):
    size = lambda **kw: lib.cbt_paged_attention_workspace(ctypes.byref(attn_args(**kw)))
    assert lib.cbt_paged_attention_workspace(None) == 0
    assert size(n_heads=9) == 0
    for small, big in ((dict(max_kv=100), dict(max_kv=100000)), (dict(max_kv=50000), dict(max_kv=60000)),
                       (dict(max_kv=50000, rows=1, tokens=1), dict(max_kv=50000)),
                       (dict(max_kv=50000, window=500), dict(max_kv=50000))):
        assert size(**small) <= size(**big), (small, big)
    # a workspace that is too small, or missing, is refused where one is needed
    n = size(max_kv=100000)
    if n:
        assert lib.cbt_paged_attention(ctypes.byref(attn_args(max_kv=100000, workspace_bytes=n - 1)), None) == -1
        assert lib.cbt_paged_attention(ctypes.byref(attn_args(max_kv=100000, workspace=None)), None) == -2


def test_page_map_refusals(lib):
    def rc(**kw):
        a = B.PageMapArgs()
        d = dict(block_table=FAKE, max_pages=8, page_tokens=64, n_pages=32, rows=4, kv_lens=FAKE,
                 new_lens=FAKE, free_pages=FAKE, free_count=FAKE, max_tokens=8, kv_lens_out=FAKE,
                 free_count_out=FAKE, cu_q=FAKE, positions=FAKE, slots=FAKE, err=FAKE)
        d.update(kw)
        for k, v in d.items():
            setattr(a, k, v)
        return lib.cbt_page_map(ctypes.byref(a), None)
    assert rc(rows=0) == 0
    for bad, code in ((dict(rows=-1), -1), (dict(max_pages=0), -1), (dict(page_tokens=0), -1),
                      (dict(n_pages=0), -1), (dict(max_tokens=-1), -1), (dict(rows=4097), -12),
                      (dict(max_pages=1 << 26), -12), (dict(n_pages=1 << 26), -12),
                      (dict(block_table=None), -2), (dict(kv_lens=None), -2), (dict(new_lens=None), -2),
                      (dict(free_count=None), -2), (dict(free_count_out=None), -2),
                      (dict(kv_lens_out=None), -2), (dict(cu_q=None), -2), (dict(positions=None), -2),
                      (dict(slots=None), -2), (dict(err=None), -2)):
        assert rc(**bad) == code, bad
    assert lib.cbt_page_map(None, None) == -2


def test_handles_refuse_host_tensors():
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        paged.PagedKV(torch.zeros(1 << 16, dtype=torch.bfloat16), None, None, page_tokens=64,
                      n_kv_heads=1, head_dim=64)
    with pytest.raises(TypeError):
        paged.PagedKV(i32, None, None, page_tokens=64, n_kv_heads=1, head_dim=64)
    with pytest.raises(ValueError):
        paged.PageMap(i32.view(2, 2), i32, None, None, page_tokens=64, max_tokens=4, n_pages=4)
    with pytest.raises(ValueError):
        paged.Rope(128, layout="quarter")
    with pytest.raises(B.CbtError):
        paged.Rope(128, rot_dim=7)
    assert paged.page_bytes(128, 8, 128, 32) == 2 * 32 * 8 * 128 * 128 * 2


def test_set_attention_refuses_a_null_engine(lib):
    assert lib.cbt_engine_set_attention(None, None) == -2
    c = B.AttentionConfig()
    assert lib.cbt_engine_set_attention(None, ctypes.byref(c)) == -2


def test_sizes_past_the_kernels_counters_are_refused(lib):
    """Each call also lacks its err, so that none could be queued if its sizes were taken."""
    def page_map(**kw):
        a = B.PageMapArgs()
        d = dict(block_table=FAKE, max_pages=8, page_tokens=1, n_pages=32, rows=4, kv_lens=FAKE,
                 new_lens=FAKE, max_tokens=8, kv_lens_out=FAKE, cu_q=FAKE, positions=FAKE, slots=FAKE)
        for k, v in {**d, **kw}.items():
            setattr(a, k, v)
        return lib.cbt_page_map(ctypes.byref(a), None)
    for ok in (dict(), dict(max_tokens=1 << 30), dict(n_pages=1 << 30)):
        assert page_map(**ok) == -2, ok
    for bad in (dict(max_tokens=(1 << 30) + 1), dict(max_tokens=2 ** 31 - 1), dict(n_pages=(1 << 30) + 1)):
        assert page_map(**bad) == -12, bad

    def append(tokens):
        a = B.RopeAppendArgs()
        a.kv = kv_desc()
        for k, v in dict(qkv=FAKE, qkv_stride=(8 + 4) * 128, tokens=tokens, n_heads=8, eps=1e-6,
                         positions=FAKE, slots=FAKE, q_out=FAKE, q_stride=1024).items():
            setattr(a, k, v)
        return lib.cbt_rope_append(ctypes.byref(a), None)
    assert append(1 << 30) == -2
    assert append((1 << 30) + 1) == -12 and append(2 ** 31 - 1) == -12


def test_sizes_of_multi_token_calls(lib):
    big = dict(n_heads=16, rows=1, tokens=65536, max_q=65536, max_kv=1 << 20, max_pages=1 << 20, cu_q=FAKE,
               q_stride=2048, out_stride=2048, err=None)
    rc = lambda **kw: lib.cbt_paged_attention(ctypes.byref(attn_args(**{**big, **kw})), None)
    size = lambda **kw: lib.cbt_paged_attention_workspace(ctypes.byref(attn_args(**{**big, **kw})))
    assert rc() == -2                                     # taken, but for err
    assert rc(tokens=(1 << 25)) == -12 and rc(tokens=2 ** 31 - 1) == -12
    assert size() == 0                                    # units enough to stay whole
    # few tokens over long rows are cut: a workspace, which is looked for before the launch
    few = dict(tokens=4, max_q=4, err=FAKE)
    n = size(**few)
    assert 0 < n <= 152 * 256 * (128 * 4 + 8)
    assert size(**{**few, "max_kv": 500}) == 0
    assert size(**{**few, "window": 200}) <= n and size(**{**few, "tokens": 3}) <= n
    assert rc(**few, workspace_bytes=n - 1) == -1
    assert rc(**few, workspace=None) == -2


def test_a_call_of_fewer_tokens_needs_no_more_workspace(lib):
    """A workspace for the most tokens serves every call with the same bounds."""
    for rows, max_q, max_kv in ((1, 4096, 100000), (3, 200, 40000), (10, 4, 8192), (64, 7, 3000), (1, 2, 1 << 20)):
        kw = dict(rows=rows, max_q=max_q, max_kv=max_kv, cu_q=FAKE)
        most = rows * max_q
        sizes = [lib.cbt_paged_attention_workspace(ctypes.byref(attn_args(**kw, tokens=t)))
                 for t in sorted({1, 2, 3, most // 7 + 1, most // 2 + 1, most - 1, most})]
        assert sizes == sorted(sizes), kw
