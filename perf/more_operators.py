"""What is measured of the operators on a paged KV cache in 8 bits, and what each of them computes.

A serving loop that holds its KV cache as 8-bit floats runs, per layer, the operators of the bf16
cache over codes instead, and reads positions back where a prefix leaves the GPU or goes to other
kernels:

  append   QKV rows -> norms and rotary positions as for a bf16 cache, q out in bf16, k and v rounded
           to e4m3 codes in their slots; then the blocks that the tokens lie in read back, with the
           tokens held there before
  read     positions of each row -> K and V in bf16
  decode   attention of one new token per row over the row's pages
  prefill  attention of ragged runs of new tokens over the row's pages

A value is a code times its block's scale.  A block is 64 positions of one kv head (of K, or of V); its
scale is 2^e, e the smallest whole number in [-56, 56] with every value of the block within 448 2^e at
the time.  Tokens that exceed it raise e, and the codes held there are rounded anew to the new scale
(exact but for the smallest); a token in the first position of a block starts it anew.

A page holds K codes [kv head][position][dim], V codes [kv head][position / 64][dim][64], then the scales
of K and of V, fp32 [kv head][position / 64] each, and is padded to whole 256 bytes.
"""
import math
import random

import torch

own = False  # False: plain torch forms; True: the framework's operators

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TOP = 448.0          # the largest e4m3
LOW, HIGH = -56, 56  # exponents of a scale


# ---- cases -----------------------------------------------------------------------------------
def listed():
    return [
        # the decode step's rows of the 7B shape, each in a block that holds earlier tokens (latency)
        dict(name="append-decode-8", op="append", rows=8, new_lo=1, new_hi=1, pad=0, heads=32, kv_heads=8,
             hd=128, page=128, dtype="f32", norm=False, layout="half", rot=128, scaling="none", theta=1e6,
             factor=1.0, far=4096, lens_seed=11),
        # packed prompts and chunks of the 7B shape with per-head norms and positions scaled by parts
        dict(name="append-prompts-8192", op="append", rows=8, new_lo=1024, new_hi=1024, pad=0, heads=32,
             kv_heads=8, hd=128, page=128, dtype="bf16", norm=True, layout="half", rot=128,
             scaling="by_parts", theta=1e6, factor=8.0, far=100000, lens_seed=12),
        # odd runs of tokens, interleaved pairs over half of a 64-wide head, padded rows
        dict(name="append-odd-64", op="append", rows=9, new_lo=1, new_hi=177, pad=23, heads=12, kv_heads=4,
             hd=64, page=64, dtype="bf16", norm=True, layout="interleaved", rot=32, scaling="linear",
             theta=1e4, factor=4.0, far=30000, lens_seed=13),
        # the last positions of three short rows (latency)
        dict(name="read-3-short", op="read", rows=3, lo=40, hi=130, first=17, kv_heads=4, hd=64, page=64,
             lens_seed=14),
        # four long prefixes of the 7B shape that leave for another machine (all their positions)
        dict(name="read-4-prefixes", op="read", rows=4, lo=8192, hi=16384, first=0, kv_heads=8, hd=128,
             page=128, lens_seed=15),
        # one short sequence (latency)
        dict(name="decode-1-short", op="decode", rows=1, lo=100, hi=100, heads=4, kv_heads=4, hd=64,
             page=64, window=0, sinks=0, lens_seed=1),
        # the 7B decode workload: 8 rows of 512 to 4096 positions
        dict(name="decode-8-ragged", op="decode", rows=8, lo=512, hi=4096, heads=32, kv_heads=8,
             hd=128, page=128, window=0, sinks=0, lens_seed=2),
        # long-context decode: 32 rows of 8192 to 16384 positions (the most bytes)
        dict(name="decode-32-long", op="decode", rows=32, lo=8192, hi=16384, heads=32, kv_heads=8,
             hd=128, page=128, window=0, sinks=0, lens_seed=3),
        # the same contexts through a window of 4096 and four sinks: most pages are not read
        dict(name="decode-16-window", op="decode", rows=16, lo=8192, hi=16384, heads=32, kv_heads=8,
             hd=128, page=128, window=4096, sinks=4, lens_seed=4),
        # admission: four 1024-token prompts of the 7B shape
        dict(name="prefill-4x1024", op="prefill", rows=4, new_lo=1024, new_hi=1024, lo=0, hi=0,
             heads=32, kv_heads=8, hd=128, page=128, window=0, sinks=0, lens_seed=5),
        # chunks of prompts that continue long contexts, through a window with sinks
        dict(name="chunks-window", op="prefill", rows=4, new_lo=500, new_hi=1030, lo=3000, hi=9000,
             heads=32, kv_heads=8, hd=128, page=128, window=4096, sinks=4, lens_seed=6),
        # ragged odd prompts of a 64-wide head with three q heads per kv head
        dict(name="prefill-odd-64", op="prefill", rows=7, new_lo=1, new_hi=700, lo=0, hi=300,
             heads=12, kv_heads=4, hd=64, page=64, window=129, sinks=65, lens_seed=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "prefill"])
    page = rng.choice([64, 128, 192, 256, 512])
    hd = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    window = 0 if rng.random() < 0.4 else _log(rng, 1, 5000)
    sinks = rng.choice([0, 1, 4, rng.randint(2, 300)]) if window else 0
    seed = rng.randrange(1 << 30)
    if op == "append":
        rows = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, 4000 // rows))
        return dict(op=op, rows=rows, new_lo=rng.randint(1, hi), new_hi=hi, pad=rng.choice([0, 0, 1, 37]),
                    heads=heads, kv_heads=kv_heads, hd=hd, page=page, dtype=rng.choice(["f32", "bf16"]),
                    norm=rng.random() < 0.6, layout=rng.choice(["half", "interleaved"]),
                    rot=rng.choice([hd, hd // 2, hd // 4, 2 * rng.randint(1, hd // 2)]),
                    scaling=rng.choice(["none", "linear", "base", "by_parts"]),
                    theta=rng.choice([1e4, 5e5, 1e6]), factor=rng.choice([1.0, 2.5, 8.0, 40.0]),
                    far=_log(rng, 100, 1000000), lens_seed=seed)
    if op == "read":
        rows = _log(rng, 1, 32)
        hi = _log(rng, 2, max(4, 16384 // rows))
        lo = rng.randint(1, hi)
        return dict(op=op, rows=rows, lo=lo, hi=hi, first=rng.choice([0, 0, rng.randint(0, lo - 1)]),
                    kv_heads=kv_heads, hd=hd, page=page, lens_seed=seed)
    if op == "decode":
        hi = _log(rng, 1, 16384)
        most = max(1, (1 << 22) * 1024 // (hi * kv_heads * hd * 4))  # bounds the cache
        return dict(op=op, rows=_log(rng, 1, min(48, most) + 1), lo=rng.randint(1, hi), hi=hi, heads=heads,
                    kv_heads=kv_heads, hd=hd, page=page, window=window, sinks=sinks, lens_seed=seed)
    new_hi = _log(rng, 2, 1024)
    hi = rng.choice([0, _log(rng, 1, 6000)])
    return dict(op=op, rows=rng.randint(1, 4), new_lo=rng.randint(1, new_hi), new_hi=new_hi,
                lo=rng.randint(0, hi), hi=hi, heads=min(heads, 4 * kv_heads), kv_heads=kv_heads, hd=hd, page=page,
                window=window, sinks=sinks, lens_seed=seed)


def _lens(case):
    """(positions before the call's tokens, the call's tokens) of every row.  Of a read: (the first
    position that is read, how many are)."""
    r = random.Random(case["lens_seed"])
    rows = range(case["rows"])
    if case["op"] == "append":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in rows]
        return [(r.randint(0, max(0, case["far"] - n)), n) for n in new]
    if case["op"] == "read":
        lens = [r.randint(case["lo"], case["hi"]) for _ in rows]
        return [(min(case["first"], n), n - min(case["first"], n)) for n in lens]
    if case["op"] == "decode":
        return [(r.randint(case["lo"], case["hi"]) - 1, 1) for _ in rows]
    return [(r.randint(case["lo"], case["hi"]), r.randint(case["new_lo"], case["new_hi"])) for _ in rows]


def _visible(p, window, sinks):
    """Positions that the token at position p attends to."""
    if not window or p + 1 <= window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def work(case):
    lens = _lens(case)
    KV, hd = case["kv_heads"], case["hd"]
    per = 2 * KV * hd  # elements of K and V of a position
    if case["op"] == "append":
        # qkv in, q and codes out; the blocks' earlier codes in, all their values out
        n, back = sum(k for _, k in lens), sum(p % 64 + k for p, k in lens)
        width = case["heads"] * hd
        return {"bytes": n * (width + per) * (4 if case["dtype"] == "f32" else 2) + n * width * 2 + n * per
                + (back - n) * per + back * per * 2, "flops": n * (width + per) * 8}
    if case["op"] == "read":
        return {"bytes": sum(n for _, n in lens) * per * 3, "flops": 0}
    H, W, S = (case[k] for k in ("heads", "window", "sinks"))
    keys = pairs = tokens = 0
    for prev, new in lens:
        last = prev + new - 1
        first = max(0, prev - W + 1) if W else 0
        keys += last + 1 - first + min(S, first)
        pairs += sum(_visible(p, W, S) for p in range(prev, last + 1))
        tokens += new
    return {"bytes": keys * per + tokens * H * hd * 4, "flops": 4 * pairs * H * hd}


# ---- rotary frequencies ------------------------------------------------------------------------
ORIGINAL = 4096  # positions the unscaled frequencies were made for (scaled cases)


def _rope_freqs(case):
    """Radians per position of each rotated pair, and the factor on cos and sin."""
    rot, theta, s = case["rot"], case["theta"], case["factor"]
    kind = case["scaling"]
    if kind == "base":
        theta = theta * s ** (rot / (rot - 2)) if rot > 2 else theta
    f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        return [x / s for x in f], 1.0
    if kind == "by_parts":
        # pairs that turn more than 32 times over the original length keep their frequency, those
        # that turn less than once are slowed by the factor, a ramp over the index joins them
        def index(turns):
            return rot * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(0, math.floor(index(32.0))), min(rot - 1, math.ceil(index(1.0)))
        hi = hi if hi > lo else lo + 0.001
        out = []
        for i, x in enumerate(f):
            ramp = min(1.0, max(0.0, (i - lo) / (hi - lo)))
            out.append(x / s * ramp + x * (1 - ramp))
        return out, (0.1 * math.log(s) + 1.0 if s > 1 else 1.0)
    return f, 1.0


# ---- inputs ------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed & 0x7FFFFFFF)


def _randn(shape, g, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _exponents(top):
    """The scales' exponents of blocks whose largest magnitudes are `top`."""
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    return (e - 9 + (m > 0.875).int()).clamp(LOW, HIGH)


def _pow2(e):
    """2^e in fp32, from its bits (exp2 and ldexp need not be exact on a GPU)."""
    return (e.int() + 127 << 23).view(torch.float32)


def _page(c):
    """Bytes of a page, and of its K or V codes."""
    n = c["kv_heads"] * c["page"] * c["hd"]
    return -(-(2 * n + 8 * c["kv_heads"] * (c["page"] // 64)) // 256) * 256, n


def _views(c, pool):
    """K codes [page][kv][position][dim], V codes [page][kv][position / 64][dim][64], scales
    [page][2][kv][position / 64] in the pool."""
    size, n = _page(c)
    p, KV, hd, nb = pool.view(-1, size), c["kv_heads"], c["hd"], c["page"] // 64
    return (p[:, :n].view(E4M3).unflatten(1, (KV, c["page"], hd)),
            p[:, n:2 * n].view(E4M3).unflatten(1, (KV, nb, hd, 64)),
            p[:, 2 * n:2 * n + 8 * KV * nb].view(torch.float32).unflatten(1, (2, KV, nb)))


def _fill(c, n_pages, g):
    """A pool whose blocks hold normal values of K and V, some blocks larger than others."""
    size, _ = _page(c)
    pool = torch.zeros(n_pages * size, dtype=torch.uint8, device=DEV)
    K, V, S = _views(c, pool)
    KV, hd, nb, page = c["kv_heads"], c["hd"], c["page"] // 64, c["page"]
    for i in range(0, n_pages, 256):  # a few pages at a time: their values in fp32 are large
        n = min(256, n_pages - i)
        for which, codes in ((0, K), (1, V)):
            shape = (n, KV, nb, 64, hd) if which == 0 else (n, KV, nb, hd, 64)
            size_of = torch.exp2(torch.rand((n, KV, nb, 1, 1), generator=g, device=DEV) * 2 - 1)
            x = torch.randn(shape, generator=g, device=DEV) * size_of
            e = _exponents(x.abs().amax((3, 4)))
            x = (x * _pow2(-e)[..., None, None]).clamp(-TOP, TOP).to(E4M3)
            codes[i:i + n] = x.reshape(n, KV, page, hd) if which == 0 else x
            S[i:i + n, which] = _pow2(e)
    return pool


def _table(lens, page, r, only_last=None):
    """Shuffled pages for rows of (first, number of) positions; with only_last, a row's pages before
    the one with position only_last(row) are not there."""
    spans = [(0 if only_last is None else only_last(b) // page, -(-(a + n) // page)) for b, (a, n) in enumerate(lens)]
    ids = list(range(sum(hi - lo for lo, hi in spans) + 1))
    r.shuffle(ids)
    table = torch.full((len(lens), max(1, max(hi for _, hi in spans))), -1, dtype=torch.int32)
    at = 0
    for b, (lo, hi) in enumerate(spans):
        table[b, lo:hi] = torch.tensor(ids[at:at + hi - lo], dtype=torch.int32)
        at += hi - lo
    return table, len(ids)


def _cache(st):
    from continuous_batching_transformer_gb300 import paged
    c = st["case"]
    return paged.PagedKVFp8(st["pool"], st["table"], st["lens"], page_tokens=c["page"],
                            n_kv_heads=c["kv_heads"], head_dim=c["hd"])


def _cu(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def _out_kv(st, n):
    c = st["case"]
    for name in ("k", "v"):
        st[name] = torch.zeros((n, c["kv_heads"], c["hd"]), dtype=torch.bfloat16, device=DEV)


def _prepare_append(case, seed):
    r, g = random.Random(seed), _gen(seed)
    pad, page, H, KV, hd = (case[k] for k in ("pad", "page", "heads", "kv_heads", "hd"))
    lens = _lens(case)
    table, n_pages = _table(lens, page, r, lambda b: lens[b][0])
    n = sum(k for _, k in lens)
    positions = [p for a, k in lens for p in range(a, a + k)] + [-1] * pad
    host = table.tolist()
    slots = [host[b][p // page] * page + p % page for b, (a, k) in enumerate(lens) for p in range(a, a + k)]
    st = dict(case=case, table=table.to(DEV), lens=_i32([a + k for a, k in lens]), tokens=n, qg=None, kg=None,
              qkv=_randn((n + pad, (H + 2 * KV) * hd), g,
                         dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16),
              pool=_fill(case, n_pages, g), positions=_i32(positions), slots=_i32(slots + [-1] * pad),
              q=torch.zeros((n + pad, H, hd), dtype=torch.bfloat16, device=DEV))
    # what is read back: from the start of the block that holds a row's first new token
    first = [a // 64 * 64 for a, _ in lens]
    st["back"] = [(f, a + k - f) for f, (a, k) in zip(first, lens)]
    st["first"], st["cu"] = _i32(first), _i32(_cu([m for _, m in st["back"]]))
    _out_kv(st, sum(m for _, m in st["back"]))
    if case["norm"]:
        st["qg"] = (1 + 0.1 * torch.randn(hd, generator=g, device=DEV)).to(torch.bfloat16)
        st["kg"] = (1 + 0.1 * torch.randn(hd, generator=g, device=DEV)).to(torch.bfloat16)
    f, st["mscale"] = _rope_freqs(case)
    st["freqs"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    if own:
        from continuous_batching_transformer_gb300 import paged
        cache = _cache(st)
        rope = paged.Rope(hd, rot_dim=case["rot"], layout=case["layout"], theta=case["theta"],
                          scaling=case["scaling"], factor=case["factor"], original_len=ORIGINAL)
        st["append"] = paged.RopeAppend(cache, rope, n_heads=H, eps=1e-6)
        st["read"] = paged.PageRead(cache)
    return st


def _prepare_read(case, seed):
    r, g = random.Random(seed), _gen(seed)
    back = _lens(case)
    table, n_pages = _table(back, case["page"], r)
    st = dict(case=case, table=table.to(DEV), lens=_i32([a + n for a, n in back]), back=back,
              first=_i32([a for a, _ in back]), cu=_i32(_cu([n for _, n in back])), pool=_fill(case, n_pages, g))
    _out_kv(st, sum(n for _, n in back))
    if own:
        from continuous_batching_transformer_gb300 import paged
        st["read"] = paged.PageRead(_cache(st))
    return st


def _prepare_attention(case, seed):
    r, g = random.Random(seed), _gen(seed)
    lens = _lens(case)
    table, n_pages = _table(lens, case["page"], r)
    cu = _cu([n for _, n in lens])
    q = _randn((cu[-1], case["heads"], case["hd"]), g, 1.5)
    st = dict(case=case, pool=_fill(case, n_pages, g), table=table.to(DEV), lens=_i32([a + n for a, n in lens]),
              host=lens, cu=_i32(cu), q=q, out=torch.zeros_like(q), max_q=max(n for _, n in lens))
    if own:
        from continuous_batching_transformer_gb300 import paged
        st["attn"] = paged.Attention(_cache(st), n_heads=case["heads"], max_kv=max(a + n for a, n in lens),
                                     max_q=st["max_q"], max_tokens=cu[-1],
                                     window=case["window"], sinks=case["sinks"])
    return st


def prepare(case, seed):
    if case["op"] == "append":
        return _prepare_append(case, seed)
    if case["op"] == "read":
        return _prepare_read(case, seed)
    return _prepare_attention(case, seed)


# ---- the plain forms -----------------------------------------------------------------------------
def _plain_append(st):
    c = st["case"]
    H, KV, hd, page, rot = c["heads"], c["kv_heads"], c["hd"], c["page"], c["rot"]
    ok = st["slots"] >= 0
    x = st["qkv"].float().reshape(-1, H + 2 * KV, hd)
    q, k, v = x[:, :H], x[:, H:H + KV], x[:, H + KV:]
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * st["qg"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-6) * st["kg"].float()
    ang = st["positions"].double()[:, None] * st["freqs"][None, :]
    cos, sin = (ang.cos() * st["mscale"]).float()[:, None], (ang.sin() * st["mscale"]).float()[:, None]

    def turn(y):
        y = y.clone()
        if c["layout"] == "half":
            a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        return y

    q, k = turn(q), turn(k)
    st["q"][ok] = q[ok].to(torch.bfloat16)
    K, V, S = _views(c, st["pool"])
    slot = st["slots"][ok].long()
    pg, off, nb = slot // page, slot % page, page // 64
    block = slot // 64
    # per block and kv head: the largest magnitude among the call's tokens
    blocks, mine = torch.unique(block, return_inverse=True)
    anew = torch.zeros(len(blocks), dtype=torch.bool, device=DEV)
    anew[mine[slot % 64 == 0]] = True
    at = (blocks // nb, blocks % nb)
    for which, y in ((0, k[ok]), (1, v[ok])):
        top = torch.zeros((len(blocks), KV), device=DEV).scatter_reduce_(
            0, mine[:, None].expand(-1, KV), y.abs().amax(-1), "amax")
        e_call = _exponents(top)
        held = S[at[0], which, :, at[1]]
        e_old = (torch.frexp(held)[1] - 1).clamp(LOW, HIGH)
        e = torch.where(anew[:, None], e_call, torch.maximum(e_call, e_old))
        S[at[0], which, :, at[1]] = _pow2(e)
        down = _pow2(torch.where(anew[:, None], torch.zeros_like(e), e_old - e))[..., None, None]
        if which == 0:
            old = K.unflatten(2, (nb, 64))[at[0], :, at[1]].float()
            K.unflatten(2, (nb, 64))[at[0], :, at[1]] = (old * down).to(E4M3)
        else:
            old = V[at[0], :, at[1]].float()
            V[at[0], :, at[1]] = (old * down).to(E4M3)
        code = (y * _pow2(-e)[mine][..., None]).clamp(-TOP, TOP).to(E4M3)
        if which == 0:
            K[pg, :, off] = code
        else:
            V[pg, :, off // 64, :, off % 64] = code
    return dict(q=st["q"], **_plain_read(st))


def _values(st, b, first, n):
    """K and V of a row's positions [first, first + n), [kv head][position][dim] in fp32."""
    c = st["case"]
    KV, hd, page = c["kv_heads"], c["hd"], c["page"]
    K, V, S = _views(c, st["pool"])
    lo, hi = first // page, -(-(first + n) // page)
    ids = st["table"][b, lo:hi].long()
    scale = S[ids].transpose(0, 1).transpose(1, 2)  # [2][kv][page][block]
    k = K[ids].float().transpose(0, 1).reshape(KV, -1, 64, hd) * scale[0].reshape(KV, -1)[..., None, None]
    v = V[ids].float().transpose(0, 1).reshape(KV, -1, hd, 64) * scale[1].reshape(KV, -1)[..., None, None]
    at = slice(first - lo * page, first - lo * page + n)
    return k.reshape(KV, -1, hd)[:, at], v.transpose(2, 3).reshape(KV, -1, hd)[:, at]


def _plain_read(st):
    at = 0
    for b, (first, n) in enumerate(st["back"]):
        if not n:
            continue
        k, v = _values(st, b, first, n)
        st["k"][at:at + n] = k.transpose(0, 1).to(torch.bfloat16)
        st["v"][at:at + n] = v.transpose(0, 1).to(torch.bfloat16)
        at += n
    return dict(k=st["k"], v=st["v"])


def _plain_attention(st):
    c = st["case"]
    KV, hd, W, S = c["kv_heads"], c["hd"], c["window"], c["sinks"]
    G, scale, at = c["heads"] // KV, 1 / math.sqrt(hd), 0
    for b, (prev, new) in enumerate(st["host"]):
        n = prev + new
        k, v = _values(st, b, 0, n)
        q = st["q"][at:at + new].float().reshape(new, KV, G, hd).permute(1, 2, 0, 3).reshape(KV, G * new, hd)
        s = torch.matmul(q, k.transpose(1, 2)).reshape(KV, G, new, n) * scale
        p = torch.arange(prev, n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None, :]
        see = j <= p
        if W:
            see = see & ((j > p - W) | (j < S))
        s = torch.where(see, s, torch.full_like(s, -math.inf))
        e = torch.exp(s - s.amax(-1, keepdim=True))
        w = (e / e.sum(-1, keepdim=True)).reshape(KV, G * new, n)
        o = torch.matmul(w, v).reshape(KV, G, new, hd)
        st["out"][at:at + new] = o.permute(2, 0, 1, 3).reshape(new, KV * G, hd).to(torch.bfloat16)
        at += new
    return st["out"]


def run(st):
    op = st["case"]["op"]
    if op == "append":
        if not own:
            return _plain_append(st)
        st["append"](0, st["qkv"], st["positions"], st["slots"], st["q"], q_gain=st["qg"], k_gain=st["kg"])
        st["read"](0, st["k"], st["v"], st["cu"], first=st["first"])
        return dict(q=st["q"], k=st["k"], v=st["v"])
    if op == "read":
        if not own:
            return _plain_read(st)
        st["read"](0, st["k"], st["v"], st["cu"], first=st["first"])
        return dict(k=st["k"], v=st["v"])
    if not own:
        return _plain_attention(st)
    if st["max_q"] == 1:
        st["attn"](0, st["q"], st["out"])
    else:
        st["attn"](0, st["q"], st["out"], cu_q=st["cu"])
    return st["out"]


# ---- the operators from their definitions, in 64 bits ----------------------------------------------
def _floor2(x):
    """The power of two at or below each positive float64: its bits without the mantissa."""
    return (x.contiguous().view(torch.int64) >> 52 << 52).view(torch.float64)


def _round_e4m3(x):
    """The nearest e4m3 to each float64, ties to even, larger ones the largest: steps of 2^-3 of the power
    of two below, of 2^-9 below 2^-6."""
    step = _floor2(x.abs().clamp(min=2.0 ** -6)) / 8
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def _bytes_value(code):
    """What bytes stand for as e4m3: sign, four bits of exponent, three of mantissa."""
    b = code.long()
    e, m = b >> 3 & 15, (b & 7).double()
    power = (e + (1023 - 7) << 52).view(torch.float64)
    mag = torch.where(e > 0, (1 + m / 8) * power, m / 512)
    return torch.where(b >> 7 > 0, -mag, mag)


def _at(case, table, b, j):
    """Byte offsets of positions j of row b, kv head 0, dim 0: K [j], V [j], and the scale's index
    (in fp32 from the pool's start, K's)."""
    size, n = _page(case)
    page, hd, nb = case["page"], case["hd"], case["page"] // 64
    start, o = table[b].long()[j // page] * size, j % page
    return start + o * hd, start + n + (o // 64) * hd * 64 + o % 64, (start + 2 * n) // 4 + o // 64


def _exact_values(case, st, pool, scales, b, j, h):
    page, hd, nb, KV = case["page"], case["hd"], case["page"] // 64, case["kv_heads"]
    ka, va, sa = _at(case, st["table"], b, j)
    d = torch.arange(hd, device=DEV)[None]
    k = _bytes_value(pool[ka[:, None] + h * page * hd + d]) * scales[sa + h * nb].double()[:, None]
    v = _bytes_value(pool[va[:, None] + h * page * hd + d * 64]) * scales[sa + (KV + h) * nb].double()[:, None]
    return k, v


def _exact_read(case, st):
    out = {x: torch.zeros(st[x].shape, dtype=torch.float64, device=DEV) for x in ("k", "v")}
    scales, at = st["pool"].view(torch.float32), 0
    for b, (first, n) in enumerate(st["back"]):
        j = torch.arange(first, first + n, device=DEV)
        for h in range(case["kv_heads"]):
            out["k"][at:at + n, h], out["v"][at:at + n, h] = _exact_values(case, st, st["pool"], scales, b, j, h)
        at += n
    return out


def _exact_append(case, st):
    """Every head as complex numbers turned by e^(i angle): a pair (a, b) is a + ib.  Then each block as
    the values that it held and those that it gets."""
    H, KV, hd, rot = (case[k] for k in ("heads", "kv_heads", "hd", "rot"))
    n = st["tokens"]
    x = st["qkv"][:n].double().reshape(n, H + 2 * KV, hd)
    if case["norm"]:
        gain = torch.cat([st["qg"].double().expand(H, hd), st["kg"].double().expand(KV, hd)])
        y = x[:, :H + KV]
        x = torch.cat([gain * y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / hd + 1e-6), x[:, H + KV:]], 1)
    turns = torch.polar(torch.full((n, rot // 2), st["mscale"], dtype=torch.float64, device=DEV),
                        torch.outer(st["positions"][:n].double(), st["freqs"]))
    y = x[:, :H + KV, :rot]
    if case["layout"] == "half":
        z = torch.complex(*[h.contiguous() for h in y.split(rot // 2, -1)]) * turns[:, None]
        y = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(y.reshape(n, H + KV, rot // 2, 2).contiguous()) * turns[:, None]
        y = torch.view_as_real(z).reshape(n, H + KV, rot)
    head = torch.cat([y, x[:, :H + KV, rot:]], -1)
    q = st["q"].double()
    q[:n] = head[:, :H]
    out = _exact_read(case, st)  # the values held before the call
    at = t = 0
    for (first, m), (a, new) in zip(st["back"], _lens(case)):
        for p0 in range(first, first + m, 64):
            rows = slice(at + p0 - first, at + min(m, p0 - first + 64))  # the block's part of the output
            lo, hi = max(a, p0), min(a + new, p0 + 64)                   # its new tokens
            for name, z in (("k", head[t + lo - a:t + hi - a, H:]), ("v", x[t + lo - a:t + hi - a, H + KV:])):
                have = out[name][rows]
                top = z.abs().amax((0, 2)) / TOP
                size = _floor2(top.clamp(2.0 ** LOW, 2.0 ** HIGH))
                size = torch.where(top > size, 2 * size, size).clamp(max=2.0 ** HIGH)
                if lo > p0:  # the scale that the block has
                    size = torch.maximum(size, st["scale"][name][at + lo - 1 - first])
                size = size[None, :, None]
                have = _round_e4m3(have / size) * size
                have[lo - p0:hi - p0] = _round_e4m3(z / size) * size
                out[name][rows] = have
        at += m
        t += new
    return dict(q=q, **out)


def _scales_held(case, st):
    """Scale of every (output row, kv head), K and V, before the call."""
    scales, nb, KV = st["pool"].view(torch.float32), case["page"] // 64, case["kv_heads"]
    h = torch.arange(KV, device=DEV)[None] * nb
    held = {"k": [], "v": []}
    for b, (first, n) in enumerate(st["back"]):
        # rows behind the tokens held before have nothing to say; their pages exist
        sa = _at(case, st["table"], b, torch.arange(first, first + n, device=DEV))[2]
        held["k"].append(scales[sa[:, None] + h].double())
        held["v"].append(scales[sa[:, None] + h + KV * nb].double())
    return {x: torch.cat(y) for x, y in held.items()}


def _exact_attention(case, st):
    """Per row and kv head, over the visible positions of 128 queries at a time."""
    KV, W, S, hd = (case[k] for k in ("kv_heads", "window", "sinks", "hd"))
    G = case["heads"] // KV
    out, at = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV), 0
    scales = st["pool"].view(torch.float32)
    for b, (prev, new) in enumerate(st["host"]):
        for q0 in range(0, new, 128):
            pos = torch.arange(prev + q0, prev + min(new, q0 + 128), device=DEV)
            j = torch.arange(int(pos[-1]) + 1, device=DEV)
            if W:
                j = j[(j < S) | (j > int(pos[0]) - W)]
            hidden = j[None] > pos[:, None]
            if W:
                hidden |= (j[None] <= pos[:, None] - W) & (j[None] >= S)
            rows = slice(at + q0, at + q0 + len(pos))
            for h in range(KV):
                k, v = _exact_values(case, st, st["pool"], scales, b, j, h)
                q = st["q"][rows, h * G:(h + 1) * G].double()
                s = torch.einsum("tgd,kd->tgk", q, k) / hd ** 0.5
                s = s.masked_fill(hidden[:, None], -math.inf)
                out[rows, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", torch.softmax(s, -1), v)
        at += new
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        st["scale"] = _scales_held(case, st)
        return _exact_append(case, st)
    if case["op"] == "read":
        return _exact_read(case, st)
    return _exact_attention(case, st)
