"""The operators on a paged KV cache from their definitions, in 64 bits on the CPU, and builders of
small paged caches for the tests."""
from __future__ import annotations

import math

import numpy as np
import torch

BF16_STEP = torch.finfo(torch.bfloat16).eps / 2   # a rounding to bf16 is off by at most this, relative
F32_STEP = torch.finfo(torch.float32).eps / 2


def k_view(pool, n_pages, layers, kv, page, hd, layer=0):
    """[page][kv head][position][dim] of a layer's K in a flat pool."""
    return pool.view(n_pages, layers, 2, kv, page * hd)[:, layer, 0].view(n_pages, kv, page, hd)


def v_view(pool, n_pages, layers, kv, page, hd, layer=0):
    """[page][kv head][position / 64][dim][position % 64] of a layer's V in a flat pool."""
    return pool.view(n_pages, layers, 2, kv, page * hd)[:, layer, 1].view(n_pages, kv, page // 64, hd, 64)


def visible(p, n, window, sinks):
    j = np.arange(n)
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def attention(q, k, v, first, window, sinks, scale):
    """One row: q [new][heads][hd] at positions first, first + 1, ...; k, v [kv][n][hd] (float64).
    Returns the outputs and sum_j p_j |v_j| (what a relative error of the weights is relative to)."""
    new, H, hd = q.shape
    kv, n, _ = k.shape
    G = H // kv
    out = np.zeros((new, H, hd))
    mag = np.zeros((new, H, hd))
    for i in range(new):
        see = visible(first + i, n, window, sinks) if first + i >= 0 else np.zeros(n, bool)
        if not see.any():
            continue
        for h in range(H):
            s = (k[h // G][see] @ q[i, h]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ v[h // G][see]
            mag[i, h] = w @ np.abs(v[h // G][see])
    return out, mag


class Cache:
    """A pool of shuffled pages for rows of given lengths, filled with seeded values; positions that
    no query of the call may see (and pages no row holds) are poisoned with NaN and infinities."""

    def __init__(self, rows, *, kv, hd, page, window, sinks, seed, layers=1, layer=0, poison=True,
                 device="cpu", spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.kv, self.hd, self.page = rows, kv, hd, page
        lens = [a + n for a, n in rows]
        need = [-(-x // page) for x in lens]
        self.n_pages = sum(need) + 2
        self.max_pages = max(1, max(need, default=1)) + 1
        ids = torch.randperm(self.n_pages, generator=g).tolist()
        pool = torch.full((self.n_pages * layers * 2 * kv * page * hd,), float("nan"), dtype=torch.bfloat16)
        if not poison:
            pool.zero_()
        table = torch.full((len(rows), self.max_pages), -1, dtype=torch.int32)
        K, V = (f(pool, self.n_pages, layers, kv, page, hd, layer) for f in (k_view, v_view))
        self.k, self.v = [], []
        at = 0
        for b, (prev, new) in enumerate(rows):
            n = prev + new
            table[b, :need[b]] = torch.tensor(ids[at:at + need[b]], dtype=torch.int32)
            at += need[b]
            k = (torch.randn(kv, n, hd, generator=g) * spread).to(torch.bfloat16)
            v = torch.randn(kv, n, hd, generator=g).to(torch.bfloat16)
            self.k.append(k.double().numpy().copy())
            self.v.append(v.double().numpy().copy())
            seen = np.zeros(n, bool)
            for p in range(max(0, prev), n):
                seen |= visible(p, n, window, sinks)
            hidden = torch.from_numpy(~seen)
            if poison and hidden.any():
                bad = torch.tensor([float("nan"), float("inf"), float("-inf")], dtype=torch.bfloat16)
                fill = bad[torch.arange(int(hidden.sum())) % 3][None, :, None]
                k[:, hidden], v[:, hidden] = fill, fill
            for j in range(n):
                pg, o = int(table[b, j // page]), j % page
                K[pg, :, o] = k[:, j]
                V[pg, :, o // 64, :, o % 64] = v[:, j]
        self.pool, self.table = pool.to(device), table.to(device)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)
        cu = np.concatenate([[0], np.cumsum([n for _, n in rows])])
        self.cu_host = [int(x) for x in cu]
        self.cu = torch.tensor(self.cu_host, dtype=torch.int32, device=device)

    def expected(self, q, window, sinks, scale):
        outs, mags = [], []
        for b, (prev, new) in enumerate(self.rows):
            o, m = attention(q[self.cu_host[b]:self.cu_host[b + 1]].double().cpu().numpy(), self.k[b],
                             self.v[b], prev, window, sinks, scale)
            outs.append(o)
            mags.append(m)
        return np.concatenate(outs), np.concatenate(mags)


def rope_freqs(rot, theta, scaling, factor, original, fast=32.0, slow=1.0):
    """(radians per position of each pair, factor on cos and sin)."""
    if scaling == "base" and rot > 2:
        theta = theta * factor ** (rot / (rot - 2))
    u = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in u], 1.0
    if scaling == "by_parts":
        c = lambda n: rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(theta))
        lo, hi = max(0, math.floor(c(fast))), min(rot - 1, math.ceil(c(slow)))
        if hi <= lo:
            hi = lo + 0.001
        r = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(rot // 2)]
        return ([x * (1 - a) + x / factor * a for x, a in zip(u, r)],
                0.1 * math.log(factor) + 1 if factor > 1 else 1.0)
    return u, 1.0


def rope_heads(x, gain, eps, positions, rot, layout, freqs, mscale):
    """x [tokens][heads][hd] float64: norm (gain or None), then rotation."""
    x = x.copy()
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain
    if not rot:
        return x
    y = x.copy()
    for i, f in enumerate(freqs):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        ang = np.asarray(positions, np.float64) * f
        c, s = (np.cos(ang) * mscale)[:, None], (np.sin(ang) * mscale)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def page_map(table, lens, new, stack, count, page, max_tokens):
    """One step on Python lists; returns (table, lens, stack, count, cu, positions, slots)."""
    table = [list(r) for r in table]
    lens, stack = list(lens), list(stack)
    for b, n in enumerate(new):
        if n < 0:
            for j in range(-(-lens[b] // page)):
                stack[count] = table[b][j]
                count += 1
    cu, positions, slots = [0], [], []
    after = []
    for b, n in enumerate(new):
        if n >= 0:
            for j in range(-(-lens[b] // page), -(-(lens[b] + n) // page)):
                count -= 1
                table[b][j] = stack[count]
            for p in range(lens[b], lens[b] + n):
                positions.append(p)
                slots.append(table[b][p // page] * page + p % page)
        cu.append(cu[-1] + max(n, 0))
        after.append(0 if n < 0 else lens[b] + n)
    pad = [-1] * (max_tokens - len(positions))
    return table, after, stack, count, cu, positions + pad, slots + pad
