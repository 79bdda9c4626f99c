"""A paged KV cache in 8 bits from its definition, in 64 bits on the CPU: codes, scales, the append, and
builders of small caches for the tests.  Nothing here uses torch's own 8-bit types."""
from __future__ import annotations

import numpy as np
import torch

from tests import paged_reference as R

TOP, LOW, HIGH = 448.0, -56, 56


def _decode_table():
    out = np.zeros(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = m / 512 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = np.nan if b & 127 == 127 else -v if b >> 7 else v
    return out


VALUES = _decode_table()


def step_at(x):
    """The distance between neighbouring e4m3 values around |x|."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)


def encode(x):
    """Codes of float64 values: nearest, ties to even, beyond 448 the largest, NaN 127."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), TOP)
    s = step_at(a)
    v = np.minimum(np.rint(a / s) * s, TOP)
    e = np.floor(np.log2(np.maximum(v, 2.0 ** -6)))
    m = np.rint(v / 2.0 ** (e - 3))  # 8 .. 15, below 8 for subnormal values (e = -6)
    code = np.where(v < 2.0 ** -6, np.rint(v * 512), (e + 7) * 8 + m - 8).astype(np.uint8)
    code |= (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(127), code)


def exponent_for(top):
    e = LOW
    while e < HIGH and top > TOP * 2.0 ** e:
        e += 1
    return e


def held_exponent(scale):
    """The exponent that a stored fp32 scale stands for."""
    bits = int(np.float32(scale).view(np.uint32))
    return min(max((bits >> 23 & 255) - 127, LOW), HIGH)


class Layout:
    def __init__(self, kv, hd, page, layers=1, layer=0):
        self.kv, self.hd, self.page, self.nb = kv, hd, page, page // 64
        codes = 2 * kv * page * hd
        scales = -(-8 * kv * self.nb // 256) * 256
        self.page_bytes = layers * (codes + scales)
        self.at, self.codes = layer * (codes + scales), codes

    def views(self, pool):
        """K codes [page][kv][position][dim], V codes [page][kv][position / 64][dim][64] and scales
        [page][2][kv][position / 64] in a flat uint8 numpy array."""
        p = pool.reshape(-1, self.page_bytes)
        n, a = self.codes // 2, self.at
        k = np.lib.stride_tricks.as_strided(p[:, a:], (len(p), self.kv, self.page, self.hd),
                                            (self.page_bytes, self.page * self.hd, self.hd, 1))
        v = np.lib.stride_tricks.as_strided(p[:, a + n:], (len(p), self.kv, self.nb, self.hd, 64),
                                            (self.page_bytes, self.page * self.hd, 64 * self.hd, 64, 1))
        f = pool.view(np.float32)
        s = np.lib.stride_tricks.as_strided(f[(a + 2 * n) // 4:], (len(p), 2, self.kv, self.nb),
                                            (self.page_bytes, 4 * self.kv * self.nb, 4 * self.nb, 4))
        return k, v, s


def append(pool, lay, k, v, slots):
    """One append of float64 rows k, v [tokens][kv][hd] into a flat uint8 pool, in place.  Returns the
    codes' exact values before rounding, {(slot, which): values}, and touched blocks."""
    K, V, S = lay.views(pool)
    runs = []
    for t, s in enumerate(slots):
        if s < 0:
            continue
        if runs and runs[-1][-1] == t - 1 and slots[t - 1] // 64 == s // 64:
            runs[-1].append(t)
        else:
            runs.append([t])
    for run in runs:
        s0 = slots[run[0]]
        pg, b = s0 // lay.page, s0 % lay.page // 64
        anew = any(slots[t] % 64 == 0 for t in run)
        for which, x in ((0, k), (1, v)):
            for h in range(lay.kv):
                y = x[run, h]
                fine = np.abs(y[np.isfinite(y)])
                e = exponent_for(fine.max() if fine.size else 0.0)
                if not anew:
                    old = held_exponent(S[pg, which, h, b])
                    codes = K[pg, h, 64 * b:64 * b + 64] if which == 0 else V[pg, h, b]
                    if e > old:
                        codes[...] = encode(VALUES[codes] * 2.0 ** (old - e))
                    e = max(e, old)
                S[pg, which, h, b] = 2.0 ** e
                with np.errstate(invalid="ignore"):
                    c = encode(y * 2.0 ** -e)
                for i, t in enumerate(run):
                    o = slots[t] % lay.page
                    if which == 0:
                        K[pg, h, o] = c[i]
                    else:
                        V[pg, h, b, :, o % 64] = c[i]
    return runs


def values(pool, lay, table_row, n):
    """K and V of a row's first n positions, [kv][n][hd]."""
    K, V, S = lay.views(pool)
    k, v = np.zeros((lay.kv, n, lay.hd)), np.zeros((lay.kv, n, lay.hd))
    for j in range(n):
        pg, o = int(table_row[j // lay.page]), j % lay.page
        sk = np.array([2.0 ** held_exponent(x) for x in S[pg, 0, :, o // 64]])
        sv = np.array([2.0 ** held_exponent(x) for x in S[pg, 1, :, o // 64]])
        k[:, j] = VALUES[K[pg, :, o]] * sk[:, None]
        v[:, j] = VALUES[V[pg, :, o // 64, :, o % 64]] * sv[:, None]
    return k, v


class Cache:
    """A pool of shuffled pages for rows of (positions held, new) lengths, filled with seeded values whose
    blocks differ in size; what no query of the call may see is poisoned with NaN codes and odd scales."""

    def __init__(self, rows, *, kv, hd, page, window, sinks, seed, layers=1, layer=0, poison=True,
                 device="cpu", spread=1.0, apart=2):
        r = np.random.default_rng(seed)
        self.rows, self.kv, self.hd, self.page = rows, kv, hd, page
        self.lay = lay = Layout(kv, hd, page, layers, layer)
        lens = [a + n for a, n in rows]
        need = [-(-x // page) for x in lens]
        self.n_pages = sum(need) + 2
        self.max_pages = max(1, max(need, default=1)) + 1
        ids = r.permutation(self.n_pages)
        pool = np.full(self.n_pages * lay.page_bytes, 0x7F if poison else 0, np.uint8)
        K, V, S = lay.views(pool)
        table = np.full((len(rows), self.max_pages), -1, np.int32)
        self.k, self.v, at = [], [], 0
        for b, (prev, new) in enumerate(rows):
            n = prev + new
            table[b, :need[b]] = ids[at:at + need[b]]
            at += need[b]
            seen = np.zeros(n, bool)
            for p in range(max(0, prev), n):
                seen |= R.visible(p, n, window, sinks)
            for j0 in range(0, n, 64):
                pg, o = int(table[b, j0 // page]), j0 % page
                m = min(64, n - j0)
                for h in range(kv):
                    for which in (0, 1):
                        x = r.standard_normal((m, hd)) * 2.0 ** r.uniform(-apart, apart) * (spread if which == 0 else 1)
                        e = exponent_for(np.abs(x).max())
                        if not seen[j0:j0 + m].any() and poison:
                            S[pg, which, h, o // 64] = [np.nan, np.inf, 0, -1][h % 4]
                        else:
                            S[pg, which, h, o // 64] = 2.0 ** e
                        c = encode(x * 2.0 ** -e)
                        if poison:
                            c[~seen[j0:j0 + m]] = [0x7F, 0xFF][which]
                        if which == 0:
                            K[pg, h, o:o + m] = c
                        else:
                            V[pg, h, o // 64, :, :m] = c.T
            k, v = values(pool, lay, table[b], n)
            self.k.append(k)
            self.v.append(v)
        self.host = pool
        self.pool, self.table = torch.from_numpy(pool).to(device), torch.from_numpy(table).to(device)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=device)
        self.cu_host = [int(x) for x in np.concatenate([[0], np.cumsum([n for _, n in rows])])]
        self.cu = torch.tensor(self.cu_host, dtype=torch.int32, device=device)

    def expected(self, q, window, sinks, scale):
        """Outputs, sum_j p_j |v_j|, and a bound on what q's rounding may move a score by."""
        outs, mags, moved = [], [], []
        for b, (prev, new) in enumerate(self.rows):
            x = q[self.cu_host[b]:self.cu_host[b + 1]].double().cpu().numpy()
            k = np.nan_to_num(self.k[b])
            o, m = R.attention(x, self.k[b], self.v[b], prev, window, sinks, scale)
            outs.append(o)
            mags.append(m)
            # q is taken as two e4m3 parts: exact down to 2^-10 of the head's largest element, and
            # off by at most 2^-18 of that below
            top = np.abs(x).max(-1, keepdims=True)
            off = np.where(np.abs(x) < top * 2.0 ** -9, top * 2.0 ** -17, 0)
            kmax = np.abs(k).max(1, initial=0).repeat(x.shape[1] // self.kv, 0)  # [head][hd]
            moved.append(np.abs(scale) * (off * kmax[None]).sum(-1))
        return np.concatenate(outs), np.concatenate(mags), np.concatenate(moved)
