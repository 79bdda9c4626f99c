"""Calls of the operators on a paged KV cache that the documentation allows and that lie off the usual
path: CTAs that hold every unit they may."""
import pytest
import torch

from continuous_batching_transformer_gb300 import paged
from tests.gpu_harness import ensure_built
from tests.paged_reference import BF16_STEP

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
    tol = (2 * BF16_STEP + 2.0 ** -15) * want.float().abs()
    assert ((out.float() - want.float()).abs() <= tol).all()
