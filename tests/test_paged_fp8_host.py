"""CPU checks of the operators on a paged cache in 8 bits: the reference's own rounding, every refusal of
the C entries (before anything reaches a device) and of the Python handles."""
import ctypes

import numpy as np
import pytest
import torch

import continuous_batching_transformer_gb300 as cbt
from continuous_batching_transformer_gb300 import binding as B
from continuous_batching_transformer_gb300 import paged
from tests import fp8_reference as F

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    cbt.build()
    return B.lib()


def test_reference_codes():
    """Every code is its own value's, and values between two go to the nearer, ties to the even one."""
    fine = [c for c in range(128) if c != 127]
    assert list(F.encode(F.VALUES[fine])) == fine
    assert list(F.encode(-F.VALUES[fine[1:]])) == [c | 128 for c in fine[1:]]
    lo, hi = F.VALUES[fine[:-1]], F.VALUES[fine[1:]]
    even = [a if a % 2 == 0 else a + 1 for a in fine[:-1]]
    assert list(F.encode((lo + hi) / 2)) == even
    assert list(F.encode(lo * 0.49 + hi * 0.51)) == fine[1:]
    assert list(F.encode([449.0, 1e30, np.inf, -np.inf, np.nan, -0.0])) == [126, 126, 126, 254, 127, 128]
    # torch's type agrees
    x = torch.randn(10000, generator=torch.Generator().manual_seed(1)).mul(50).clamp(-448, 448)
    assert (x.to(torch.float8_e4m3fn).view(torch.uint8).numpy() == F.encode(x.double().numpy())).all()


def test_reference_exponents():
    assert [F.exponent_for(x) for x in (0.0, 448.0, 448.1, 896.0, 897.0, 1e-30, 1e30)] == [-56, 0, 1, 1, 2, -56, 56]
    assert [F.held_exponent(x) for x in (0.0, 1.0, 3.0, 0.5, np.inf, 2.0 ** -100)] == [-56, 0, 1, -1, 56, -56]


def kv_desc(**kw):
    d = dict(pool=FAKE, pool_bytes=16 * 33024, page_bytes=33024, k_offset=0, v_offset=16384, s_offset=32768,
             n_pages=16, page_tokens=64, n_kv_heads=2, head_dim=128)
    d.update(kw)
    r = B.PagedKvFp8Desc()
    for k, v in d.items():
        setattr(r, k, v)
    return r


BAD_KV = [(dict(pool=None), -2), (dict(pool=FAKE + 16), -1), (dict(head_dim=96), -11),
          (dict(page_tokens=32), -1), (dict(page_tokens=0), -1), (dict(page_tokens=96), -1), (dict(n_pages=0), -1),
          (dict(n_pages=17), -1), (dict(page_bytes=33024 + 8), -1), (dict(page_bytes=0), -1),
          (dict(k_offset=-256), -1), (dict(v_offset=16384 + 512), -1), (dict(v_offset=1 << 62), -1),
          (dict(s_offset=32768 + 256), -1), (dict(s_offset=-256), -1), (dict(s_offset=1 << 62), -1),
          (dict(s_offset=32768 + 16), -1), (dict(pool_bytes=1 << 40), -12), (dict(n_pages=1 << 26), -12),
          (dict(n_kv_heads=0), -1), (dict(n_kv_heads=1 << 30), -1)]


def setall(a, kv, d, kw):
    a.kv = kv_desc(**(kv or {}))
    for k, v in {**d, **kw}.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def test_append_refusals(lib):
    d = dict(qkv=FAKE, qkv_dtype=0, qkv_stride=(8 + 4) * 128, tokens=3, n_heads=8, eps=1e-6,
             positions=FAKE, slots=FAKE, q_out=FAKE, q_stride=1024, err=FAKE)
    rc = lambda kv=None, **kw: lib.cbt_rope_append_fp8(setall(B.RopeAppendFp8Args(), kv, d, kw), None)
    for bad, code in BAD_KV:
        assert rc(kv=bad) == code, bad
    assert rc(tokens=0) == 0
    assert rc(tokens=0, qkv=None) == 0
    wrong = paged.Rope(64).desc
    for bad, code in ((dict(tokens=-1), -1), (dict(n_heads=0), -1), (dict(qkv_dtype=2), -1),
                      (dict(qkv_stride=12 * 128 - 8), -1), (dict(qkv_stride=12 * 128 + 4), -1),
                      (dict(q_stride=1016), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
                      (dict(qkv=None), -2), (dict(q_out=None), -2), (dict(positions=None), -2),
                      (dict(slots=None), -2), (dict(err=None), -2), (dict(qkv=FAKE + 8), -1),
                      (dict(q_out=FAKE + 2), -1), (dict(q_gain=FAKE + 2), -1), (dict(k_gain=FAKE + 8), -1),
                      (dict(rope=ctypes.pointer(wrong)), -1),
                      (dict(n_heads=1 << 29, q_stride=1 << 40, qkv_stride=1 << 40), -12),
                      (dict(tokens=(1 << 30) + 1), -12)):
        assert rc(**bad) == code, bad
    assert lib.cbt_rope_append_fp8(None, None) == -2


def test_read_refusals(lib):
    d = dict(block_table=FAKE, max_pages=4, rows=3, kv_lens=FAKE, first=FAKE, cu=FAKE, tokens=9, k_out=FAKE,
             v_out=FAKE, out_stride=256, err=FAKE)
    rc = lambda kv=None, **kw: lib.cbt_paged_read_fp8(setall(B.PagedReadFp8Args(), kv, d, kw), None)
    for bad, code in BAD_KV:
        assert rc(kv=bad) == code, bad
    assert rc(tokens=0) == 0 and rc(rows=0) == 0 and rc(k_out=None, v_out=None) == 0
    for bad, code in ((dict(tokens=-1), -1), (dict(rows=-1), -1), (dict(max_pages=0), -1), (dict(out_stride=248), -1),
                      (dict(out_stride=260), -1), (dict(out_dtype=2), -1), (dict(rows=4097), -12),
                      (dict(tokens=(1 << 30) + 1), -12), (dict(block_table=None), -2), (dict(kv_lens=None), -2),
                      (dict(cu=None), -2), (dict(err=None), -2), (dict(k_out=FAKE + 8), -1),
                      (dict(v_out=FAKE + 2), -1)):
        assert rc(**bad) == code, bad
    assert lib.cbt_paged_read_fp8(None, None) == -2


ATTN = dict(block_table=FAKE, max_pages=4, rows=3, kv_lens=FAKE, tokens=3, max_q=1, max_kv=256,
            n_heads=8, q=FAKE, q_stride=1024, scale=0.1, out=FAKE, out_stride=1024, workspace=FAKE,
            workspace_bytes=1 << 40, err=FAKE)


def attn(kv=None, **kw):
    return setall(B.PagedAttentionFp8Args(), kv, ATTN, kw)


def test_attention_refusals(lib):
    rc = lambda kv=None, **kw: lib.cbt_paged_attention_fp8(attn(kv, **kw), None)
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
                      (dict(q=FAKE + 2), -1), (dict(out=FAKE + 4), -1)):
        assert rc(**bad) == code, bad
    assert lib.cbt_paged_attention_fp8(None, None) == -2


def test_attention_workspace(lib):
    size = lambda **kw: lib.cbt_paged_attention_fp8_workspace(attn(**kw))
    assert lib.cbt_paged_attention_fp8_workspace(None) == 0
    assert size(n_heads=9) == 0
    for kw in (dict(max_kv=100000), dict(max_kv=50000, rows=1, tokens=1),
               dict(max_kv=100000, rows=2, max_q=4, tokens=8, cu_q=FAKE)):
        n = size(**kw)
        assert size(**{**kw, "max_kv": 100}) <= n
        if n:  # too small, or missing, where one is needed
            assert lib.cbt_paged_attention_fp8(attn(**kw, workspace_bytes=n - 1), None) == -1
            assert lib.cbt_paged_attention_fp8(attn(**kw, workspace=None), None) == -2
            assert lib.cbt_paged_attention_fp8(attn(**kw, workspace=FAKE + 16), None) == -1
    # a workspace for the most tokens serves every call with the same bounds
    for rows, max_q, max_kv in ((1, 4096, 100000), (3, 200, 40000), (10, 4, 8192), (64, 7, 3000), (1, 2, 1 << 20)):
        kw, most = dict(rows=rows, max_q=max_q, max_kv=max_kv, cu_q=FAKE), rows * max_q
        sizes = [size(**kw, tokens=t) for t in sorted({1, 2, 3, most // 7 + 1, most // 2 + 1, most - 1, most})]
        assert sizes == sorted(sizes), kw


def test_handles_refuse_what_they_cannot_take():
    kv = dict(page_tokens=64, n_kv_heads=1, head_dim=64)
    with pytest.raises(ValueError):
        paged.PagedKVFp8(torch.zeros(1 << 16, dtype=torch.uint8), None, None, **kv)  # on the host
    with pytest.raises(TypeError):
        paged.PagedKVFp8(torch.zeros(1 << 16, dtype=torch.bfloat16), None, None, **kv)
    with pytest.raises(TypeError, match="PagedKVFp8"):
        paged.PageRead(object())
    for name in kv:
        with pytest.raises(ValueError, match=name):
            paged.PagedKVFp8(torch.zeros(1 << 16, dtype=torch.uint8), None, None, **{**kv, name: 2 ** 32 + 64})


def test_page_sizes():
    # 7B shape: a page of 128 positions, 32 layers; scales take 2 * 8 * 2 * 4 = 128 bytes, padded to 256
    assert paged.page_bytes_fp8(128, 8, 128, 32) == 32 * (2 * 8 * 128 * 128 + 256)
    assert paged.page_bytes_fp8(64, 1, 64) == 2 * 64 * 64 + 256
    assert paged.page_bytes_fp8(512, 8, 128) == 2 * 8 * 512 * 128 + 512
    for kv, hd, page in ((1, 64, 64), (8, 128, 512), (5, 64, 192)):
        assert F.Layout(kv, hd, page).page_bytes == paged.page_bytes_fp8(page, kv, hd)
