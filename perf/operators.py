"""What is measured of the paged-attention operators, and what each of them computes.

A serving loop that keeps its KV cache in pages runs four operators per step, the first once and
the others once per layer:

  page_map     request lengths -> pages taken from (and returned to) a free stack, the block table,
               and each new token's row offset, position and cache slot;
  rope_append  QKV rows -> RMS norm of every q and k head (optional), rotary positions (half or
               interleaved pairs, part of the head, scaled for long contexts), q out in bf16, k and
               v into their cache slots;
  attention    one new token per row ("decode"), or ragged runs of new tokens ("prefill"), over the
               row's pages: causal, optionally with a sliding window and first tokens that stay
               visible (sinks).

The page layout is the engine's: per layer a K block and a V block of every kv head; K is
[position][head_dim], V is [position / 64][head_dim][64].
"""
import math
import random

import torch

own = False  # False: plain torch forms; True: the framework's operators

DEV = "cuda"


# ---- cases -----------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a small batch: every row takes one token (latency)
        dict(name="map-decode-8", op="page_map", rows=8, page=128, max_pages=64, ctx=4096, prompt=0,
             prompts=0, retire=0, max_tokens=8),
        # a busy serving step: most rows decode, some admit ragged prompts, some retire
        dict(name="map-serve-256", op="page_map", rows=256, page=64, max_pages=128, ctx=6000,
             prompt=2048, prompts=24, retire=9, max_tokens=32768),
        # the decode step's rows of the 7B shape (latency)
        dict(name="append-decode-8", op="rope_append", tokens=8, pad=0, heads=32, kv_heads=8, hd=128,
             page=128, dtype="f32", norm=False, layout="half", rot=128, scaling="none", theta=1e6,
             factor=1.0, far=4096),
        # packed prompts of the 7B shape with per-head norms and positions scaled by parts
        dict(name="append-prompts-8192", op="rope_append", tokens=8192, pad=0, heads=32, kv_heads=8,
             hd=128, page=128, dtype="bf16", norm=True, layout="half", rot=128, scaling="by_parts",
             theta=1e6, factor=8.0, far=100000),
        # an odd number of tokens, interleaved pairs over half of a 64-wide head, padded rows
        dict(name="append-odd-777", op="rope_append", tokens=777, pad=23, heads=12, kv_heads=4, hd=64,
             page=64, dtype="bf16", norm=True, layout="interleaved", rot=32, scaling="linear",
             theta=1e4, factor=4.0, far=30000),
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
    op = rng.choice(["page_map", "rope_append", "decode", "prefill"])
    page = rng.choice([64, 128, 192, 256, 512])
    hd = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    window = 0 if rng.random() < 0.4 else _log(rng, 1, 5000)
    sinks = rng.choice([0, 1, 4, rng.randint(2, 300)]) if window else 0
    seed = rng.randrange(1 << 30)
    if op == "page_map":
        rows = _log(rng, 1, 512)
        max_pages = _log(rng, 4, 128)
        ctx = max(1, page * max_pages * 3 // 4)
        prompts = rng.randint(0, rows // 4)
        return dict(op=op, rows=rows, page=page, max_pages=max_pages, ctx=ctx,
                    prompt=max(1, min(2000, page * max_pages // 4)), prompts=prompts,
                    retire=rng.randint(0, rows // 8), max_tokens=_log(rng, max(64, rows), 32768))
    if op == "rope_append":
        tokens = _log(rng, 1, 6000)
        return dict(op=op, tokens=tokens, pad=rng.choice([0, 0, 1, 37]), heads=heads,
                    kv_heads=kv_heads, hd=hd, page=page, dtype=rng.choice(["f32", "bf16"]),
                    norm=rng.random() < 0.6, layout=rng.choice(["half", "interleaved"]),
                    rot=rng.choice([hd, hd // 2, hd // 4, 2 * rng.randint(1, hd // 2)]),
                    scaling=rng.choice(["none", "linear", "base", "by_parts"]),
                    theta=rng.choice([1e4, 5e5, 1e6]), factor=rng.choice([1.0, 2.5, 8.0, 40.0]),
                    far=_log(rng, 100, 1000000))
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
    """(positions held before the call, new tokens) of every row of an attention case."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "decode":
        return [(r.randint(case["lo"], case["hi"]) - 1, 1) for _ in range(case["rows"])]
    return [(r.randint(case["lo"], case["hi"]), r.randint(case["new_lo"], case["new_hi"]))
            for _ in range(case["rows"])]


def _visible(p, window, sinks):
    """Positions that the token at position p attends to."""
    if not window or p + 1 <= window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def work(case):
    if case["op"] == "page_map":
        rows, tok = case["rows"], case["max_tokens"]
        # lengths in and out, new lengths, offsets, a table entry a row, a position and a slot a token
        return {"bytes": rows * 4 * 5 + tok * 8, "flops": 0}
    if case["op"] == "rope_append":
        n, width = case["tokens"], (case["heads"] + 2 * case["kv_heads"]) * case["hd"]
        return {"bytes": n * width * ((4 if case["dtype"] == "f32" else 2) + 2) + 8 * (n + case["pad"]),
                "flops": n * width * 8}
    H, KV, hd, W, S = (case[k] for k in ("heads", "kv_heads", "hd", "window", "sinks"))
    keys = pairs = tokens = 0
    for prev, new in _lens(case):
        last = prev + new - 1
        first = max(0, prev - W + 1) if W else 0
        keys += last + 1 - first + min(S, first)
        pairs += sum(_visible(p, W, S) for p in range(prev, last + 1))
        tokens += new
    return {"bytes": keys * KV * hd * 4 + tokens * H * hd * 4, "flops": 4 * pairs * H * hd}


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


def _prepare_map(case, seed):
    r = random.Random(seed)
    rows, page, mp = case["rows"], case["page"], case["max_pages"]
    lens = [r.randint(0, min(case["ctx"], page * mp - 1)) for _ in range(rows)]
    new = [1] * rows
    order = list(range(rows))
    r.shuffle(order)
    for b in order[:case["prompts"]]:
        new[b] = min(r.randint(1, case["prompt"]), page * mp - lens[b])
    for b in order[case["prompts"]:case["prompts"] + case["retire"]]:
        new[b] = -1
    room = case["max_tokens"]
    for b in range(rows):
        if new[b] > 0:
            new[b] = min(new[b], room)
            room -= new[b]
    pages = list(range(rows * mp))
    r.shuffle(pages)
    table = torch.full((rows, mp), -1, dtype=torch.int32)
    at = 0
    for b in range(rows):
        k = -(-lens[b] // page)
        table[b, :k] = torch.tensor(pages[at:at + k], dtype=torch.int32)
        at += k
    free = torch.full((rows * mp,), -1, dtype=torch.int32)
    free[:rows * mp - at] = torch.tensor(pages[at:], dtype=torch.int32)
    st = dict(case=case, lens=_i32(lens), new=_i32(new), table=table.to(DEV), free=free.to(DEV),
              count=_i32([rows * mp - at]))
    if own:
        from continuous_batching_transformer_gb300 import paged
        st["lens_out"] = torch.empty_like(st["lens"])
        st["count_out"] = torch.empty_like(st["count"])
        st["map"] = paged.PageMap(st["table"], st["lens"], st["free"], st["count"], page_tokens=page,
                                  max_tokens=case["max_tokens"])
    return st


def _prepare_append(case, seed):
    r, g = random.Random(seed), _gen(seed)
    n, pad, page = case["tokens"], case["pad"], case["page"]
    H, KV, hd = case["heads"], case["kv_heads"], case["hd"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    qkv = _randn((n + pad, (H + 2 * KV) * hd), g, dtype=dt)
    # the tokens are runs of consecutive positions (prompts); short calls are decode rows
    run = 1 if n <= 64 else max(1, n // 5)
    pos = []
    for t in range(0, n, run):
        k = min(run, n - t)
        pos.append((r.randint(0, max(0, case["far"] - k)), k))
    n_pages = sum((k - 1) // page + 2 for _, k in pos)  # most pages that the runs can touch
    ids = list(range(n_pages))
    r.shuffle(ids)
    positions, slots, at = [], [], 0
    for p0, k in pos:
        for p in range(p0, p0 + k):
            positions.append(p)
            slots.append(ids[at + p // page - p0 // page] * page + p % page)
        at += (p0 + k - 1) // page - p0 // page + 1
    positions += [-1] * pad
    slots += [-1] * pad
    pool = _randn((n_pages * 2 * KV * page * hd,), g)
    st = dict(case=case, qkv=qkv, pool=pool, positions=_i32(positions), slots=_i32(slots),
              q=torch.zeros((n + pad, H, hd), dtype=torch.bfloat16, device=DEV), qg=None, kg=None)
    if case["norm"]:
        st["qg"] = (1 + 0.1 * torch.randn(hd, generator=g, device=DEV)).to(torch.bfloat16)
        st["kg"] = (1 + 0.1 * torch.randn(hd, generator=g, device=DEV)).to(torch.bfloat16)
    f, st["mscale"] = _rope_freqs(case)
    st["freqs"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    if own:
        from continuous_batching_transformer_gb300 import paged
        rope = paged.Rope(hd, rot_dim=case["rot"], layout=case["layout"], theta=case["theta"],
                          scaling=case["scaling"], factor=case["factor"], original_len=ORIGINAL)
        cache = paged.PagedKV(pool, None, None, page_tokens=page, n_kv_heads=KV, head_dim=hd)
        st["append"] = paged.RopeAppend(cache, rope, n_heads=H, eps=1e-6)
    return st


def _prepare_attention(case, seed):
    r, g = random.Random(seed), _gen(seed)
    H, KV, hd, page = (case[k] for k in ("heads", "kv_heads", "hd", "page"))
    lens = _lens(case)
    need = [-(-(a + n) // page) for a, n in lens]
    n_pages = sum(need) + 1
    ids = list(range(n_pages))
    r.shuffle(ids)
    mp = max(need)
    table, at = torch.full((len(lens), mp), -1, dtype=torch.int32), 0
    for b, k in enumerate(need):
        table[b, :k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
        at += k
    pool = torch.randn((n_pages * 2 * KV * page * hd,), generator=g, device=DEV,
                       dtype=torch.bfloat16)
    cu = [0]
    for _, n in lens:
        cu.append(cu[-1] + n)
    q = _randn((cu[-1], H, hd), g, 1.5)
    st = dict(case=case, pool=pool, table=table.to(DEV), lens=_i32([a + n for a, n in lens]),
              host=lens, cu=_i32(cu), q=q, out=torch.zeros_like(q))
    if own:
        from continuous_batching_transformer_gb300 import paged
        cache = paged.PagedKV(pool, st["table"], st["lens"], page_tokens=page, n_kv_heads=KV,
                              head_dim=hd)
        st["attn"] = paged.Attention(cache, n_heads=H, max_kv=max(a + n for a, n in lens),
                                     max_q=max(n for _, n in lens), max_tokens=cu[-1],
                                     window=case["window"], sinks=case["sinks"])
    return st


def prepare(case, seed):
    if case["op"] == "page_map":
        return _prepare_map(case, seed)
    if case["op"] == "rope_append":
        return _prepare_append(case, seed)
    return _prepare_attention(case, seed)


# ---- the plain forms -----------------------------------------------------------------------------
def _plain_map(st):
    c = st["case"]
    page, mp, top = c["page"], c["max_pages"], c["max_tokens"]
    lens, new = st["lens"].long(), st["new"].long()
    retired = new < 0
    grow = new.clamp(min=0)
    held = (lens + page - 1) // page
    after = torch.where(retired, torch.zeros_like(lens), lens + grow)
    need = torch.where(retired, torch.zeros_like(lens), (after + page - 1) // page - held)
    idx = torch.arange(mp, device=DEV)[None, :]
    # retired rows' pages go onto the stack in row order, new pages come off its top in row order
    back = retired[:, None] & (idx < held[:, None])
    rank = torch.cumsum(back.reshape(-1).long(), 0) - 1
    count, released = st["count"].long(), back.sum()
    n = st["free"].numel()
    stack = torch.cat([st["free"], st["free"].new_zeros(1)])
    at = torch.where(back.reshape(-1), count + rank, torch.full_like(rank, n))
    stack.scatter_(0, at, torch.where(back, st["table"], stack[n]).reshape(-1))
    stack = stack[:n]
    take = (idx >= held[:, None]) & (idx < (held + need)[:, None])
    rank = torch.cumsum(take.reshape(-1).long(), 0) - 1
    got = stack[(count + released - 1 - rank).clamp(0, n - 1)].reshape(take.shape)
    table = torch.where(take, got, st["table"])
    cu = torch.zeros(len(lens) + 1, dtype=torch.int64, device=DEV)
    cu[1:] = torch.cumsum(grow, 0)
    t = torch.arange(top, device=DEV)
    row = (t[:, None] >= cu[None, 1:]).sum(1) if len(lens) <= 16 else torch.searchsorted(cu[1:], t, right=True)
    row = row.clamp(max=len(lens) - 1)
    live = t < cu[-1]
    pos = lens[row] + t - cu[row]
    slot = table[row, (pos // page).clamp(0, mp - 1)].long() * page + pos % page
    none = torch.full_like(t, -1)
    return dict(table=table, free=stack, count=(count + released - need.sum()).int(), lens=after.int(),
                cu=cu.int(), positions=torch.where(live, pos, none).int(),
                slots=torch.where(live, slot, none).int())


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
    pool = st["pool"].reshape(-1, 2, KV, page * hd)
    slot = st["slots"][ok].long()
    pg, off = slot // page, slot % page
    pool[:, 0].view(-1, KV, page, hd)[pg, :, off] = k[ok].to(torch.bfloat16)
    pool[:, 1].view(-1, KV, page // 64, hd, 64)[pg, :, off // 64, :, off % 64] = v[ok].to(torch.bfloat16)
    return dict(q=st["q"], pool=st["pool"])


def _gather(st, b, n):
    """K and V of a row's first n positions, [kv head][position][head_dim] in fp32."""
    c = st["case"]
    KV, hd, page = c["kv_heads"], c["hd"], c["page"]
    pool = st["pool"].reshape(-1, 2, KV, page * hd)
    ids = st["table"][b, :-(-n // page)].long()
    pages = pool[ids]
    k = pages[:, 0].reshape(-1, KV, page, hd).permute(1, 0, 2, 3).reshape(KV, -1, hd)[:, :n]
    v = pages[:, 1].reshape(-1, KV, page // 64, hd, 64).permute(1, 0, 2, 4, 3).reshape(KV, -1, hd)[:, :n]
    return k.float(), v.float()


def _plain_attention(st):
    c = st["case"]
    KV, hd, W, S = c["kv_heads"], c["hd"], c["window"], c["sinks"]
    G, scale, at = c["heads"] // KV, 1 / math.sqrt(hd), 0
    for b, (prev, new) in enumerate(st["host"]):
        n = prev + new
        k, v = _gather(st, b, n)
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
    if op == "page_map":
        if not own:
            return _plain_map(st)
        m = st["map"]
        m(st["new"], kv_lens_out=st["lens_out"], free_count_out=st["count_out"])
        return dict(table=st["table"], free=st["free"], count=st["count_out"], lens=st["lens_out"],
                    cu=m.cu_q, positions=m.positions, slots=m.slots)
    if op == "rope_append":
        if not own:
            return _plain_append(st)
        st["append"](0, st["qkv"], st["positions"], st["slots"], st["q"], q_gain=st["qg"], k_gain=st["kg"])
        return dict(q=st["q"], pool=st["pool"])
    if not own:
        return _plain_attention(st)
    if op == "decode":
        st["attn"](0, st["q"], st["out"])
    else:
        st["attn"](0, st["q"], st["out"], cu_q=st["cu"])
    return st["out"]


# ---- the operators from their definitions, in 64 bits ----------------------------------------------
def _exact_append(case, st):
    """Every head as complex numbers turned by e^(i angle): a pair (a, b) is a + ib."""
    H, KV, hd, page, rot = (case[k] for k in ("heads", "kv_heads", "hd", "page", "rot"))
    n = case["tokens"]
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
    # flat element offsets of every (token, kv head, dim) in the pool
    slot = st["slots"][:n].long()[:, None, None]
    h = torch.arange(KV, device=DEV)[None, :, None]
    d = torch.arange(hd, device=DEV)[None, None, :]
    base, o = (slot // page) * (2 * KV * page * hd), slot % page
    pool = st["pool"].double()
    pool[(base + h * page * hd + o * hd + d).reshape(-1)] = head[:, H:].reshape(-1)
    pool[(base + (KV + h) * page * hd + ((o // 64) * hd + d) * 64 + o % 64).reshape(-1)] = \
        x[:, H + KV:].reshape(-1)
    return dict(q=q, pool=pool)


def _exact_attention(case, st):
    """Per row and kv head, over the visible positions of 128 queries at a time."""
    KV, hd, page, W, S = (case[k] for k in ("kv_heads", "hd", "page", "window", "sinks"))
    G = case["heads"] // KV
    out, at = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV), 0
    for b, (prev, new) in enumerate(st["host"]):
        for q0 in range(0, new, 128):
            pos = torch.arange(prev + q0, prev + min(new, q0 + 128), device=DEV)
            j = torch.arange(int(pos[-1]) + 1, device=DEV)
            if W:
                j = j[(j < S) | (j > int(pos[0]) - W)]
            hidden = j[None] > pos[:, None]
            if W:
                hidden |= (j[None] <= pos[:, None] - W) & (j[None] >= S)
            page_at = st["table"][b].long()[j // page] * (2 * KV * page * hd)
            o, d = (j % page)[:, None], torch.arange(hd, device=DEV)[None]
            rows = slice(at + q0, at + q0 + len(pos))
            for h in range(KV):
                k = st["pool"][page_at[:, None] + h * page * hd + o * hd + d].double()
                v = st["pool"][page_at[:, None] + (KV + h) * page * hd + ((o // 64) * hd + d) * 64 + o % 64].double()
                q = st["q"][rows, h * G:(h + 1) * G].double()
                s = torch.einsum("tgd,kd->tgk", q, k) / hd ** 0.5
                s = s.masked_fill(hidden[:, None], -math.inf)
                out[rows, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", torch.softmax(s, -1), v)
        at += new
    return out


def exact(case, seed):
    if case["op"] == "page_map":
        return None  # whole numbers: compared for equality
    st = prepare(case, seed)
    if case["op"] == "rope_append":
        return _exact_append(case, st)
    return _exact_attention(case, st)
