"""Engines with an attention form of their own (cbt_engine_set_attention): per-head q and k norms,
rotary forms, a sliding window and sinks, against a 64-bit composition of the whole model and, where
the form is the built-in one, against the CPU oracle and the built-in path."""
import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

import oracle
from continuous_batching_transformer_gb300 import binding as B
from continuous_batching_transformer_gb300 import paged
from continuous_batching_transformer_gb300.model import DeviceWeights, Engine
from synth.recipes import ModelShape
from tests import paged_reference as R
from tests.gpu_harness import TOL, check_logits, ensure_built, to_dev

pytestmark = pytest.mark.gpu

SHAPES = {
    "hd64": ModelShape("form-hd64", 2, 256, 4, 4, 64, 768, 1024, 1e-6, 1e4, gain_sigma=0.1),
    "hd128-gqa": ModelShape("form-gqa", 2, 512, 4, 2, 128, 1024, 2048, 1e-5, 1e6, gain_sigma=0.1),
    "affine4": ModelShape("form-affine4", 2, 512, 4, 2, 128, 1024, 2048, 1e-5, 1e6, gain_sigma=0.1,
                          weight_format="affine4"),
}
FORMS = {
    "plain": dict(),
    "window": dict(window=20, sinks=3),
    "window-page": dict(window=130, sinks=0),
    "norm": dict(norm=True),
    "all": dict(norm=True, window=33, sinks=5, layout="interleaved", rot=32, scaling="by_parts", factor=8.0),
    "k-norm-linear": dict(norm="k", layout="half", rot=64, scaling="linear", factor=3.0),
}
_weights = {}


def weights(shape):
    if shape.name not in _weights:
        _weights[shape.name] = (DeviceWeights(shape, torch.device("cuda:0")), oracle.OracleModel(shape))
    return _weights[shape.name]


def f32(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def reference(m, tokens, form, gains):
    """Logits of every position of one sequence in float64; K and V rounded to bf16 as cached."""
    s, dt = m.shape, torch.float64
    W = lambda lin: torch.tensor(f32(lin.w) if lin.w is not None else oracle.dequantize_affine4(
        lin.packed, lin.scales, lin.biases, s.group_size), dtype=dt)
    g = lambda b: torch.tensor(f32(b), dtype=dt)
    hd, T = s.head_dim, len(tokens)
    rot, theta = form.get("rot", hd), s.rope_theta
    f, ms = R.rope_freqs(rot, theta, form.get("scaling", "none"), form.get("factor", 1.0), 4096)
    pos = list(range(T))
    x = torch.tensor(f32(m.embed[np.asarray(tokens)]), dtype=dt)
    for l, L in enumerate(m.layers):
        h = F.rms_norm(x, (s.d_model,), weight=g(L["attn_norm"]), eps=s.rms_eps)
        heads = lambda w, n: (h @ W(L[w]).T).view(T, n, hd).numpy()
        norm = form.get("norm")
        gq = gains[0][l].double().cpu().numpy() if norm in (True, "q") else None
        gk = gains[1][l].double().cpu().numpy() if norm in (True, "k") else None
        q = R.rope_heads(heads("wq", s.n_heads), gq, 1e-5, pos, rot, form.get("layout", "half"), f, ms)
        k = R.rope_heads(heads("wk", s.n_kv_heads), gk, 1e-5, pos, rot, form.get("layout", "half"), f, ms)
        bf = lambda y: torch.from_numpy(y).float().to(torch.bfloat16).double().numpy().transpose(1, 0, 2)
        o, _ = R.attention(q, bf(k), bf(heads("wv", s.n_kv_heads)), 0, form.get("window", 0), form.get("sinks", 0),
                           1 / math.sqrt(hd))
        x = x + torch.from_numpy(o.reshape(T, -1)) @ W(L["wo"]).T
        h = F.rms_norm(x, (s.d_model,), weight=g(L["ffn_norm"]), eps=s.rms_eps)
        x = x + (F.silu(h @ W(L["wg"]).T) * (h @ W(L["wu"]).T)) @ W(L["wd"]).T
    h = F.rms_norm(x, (s.d_model,), weight=g(m.final_norm), eps=s.rms_eps)
    return (h @ W(m.lm_head).T).numpy()


def make_engine(w, form, stream=None, arena=64 << 20, max_batch=8):
    eng = Engine(w, arena_bytes=arena, max_batch=max_batch, max_prefill_tokens=512, page_tokens=128, stream=stream)
    s = w.shape
    g = torch.Generator().manual_seed(3)
    gains = [[(1 + 0.2 * torch.randn(s.head_dim, generator=g)).to(torch.bfloat16).cuda() for _ in range(s.n_layers)]
             for _ in range(2)]
    rope = None
    if "layout" in form:
        rope = paged.Rope(s.head_dim, rot_dim=form["rot"], layout=form["layout"], theta=s.rope_theta,
                          scaling=form["scaling"], factor=form["factor"], original_len=4096)
    norm = form.get("norm")
    eng.set_attention(rope, gains[0] if norm in (True, "q") else None, gains[1] if norm in (True, "k") else None,
                      1e-5, form.get("window", 0), form.get("sinks", 0))
    return eng, gains


def run(eng, shape, lens, steps, chunk=None):
    """Prefill (whole or in chunks), then `steps` decode steps of fixed tokens; returns the logits of
    each prompt's end and of each step, with the tokens fed."""
    toks = [np.random.default_rng(50 + r).integers(0, shape.vocab, n + steps).astype(np.int32)
            for r, n in enumerate(lens)]
    slabs = [eng.kv_slab_alloc(n + steps) for n in lens]
    lg = torch.empty(len(lens), shape.vocab, device="cuda")
    outs = []
    if chunk is None:
        eng.prefill_segmented(slabs, lens, to_dev(np.concatenate([t[:n] for t, n in zip(toks, lens)])), lg)
    else:
        for a in range(0, max(lens), chunk):
            idx = [r for r in range(len(lens)) if lens[r] > a]
            part = [min(chunk, lens[r] - a) for r in idx]
            o = torch.empty(len(idx), shape.vocab, device="cuda")
            eng.prefill_segmented([slabs[r] for r in idx], part,
                                  to_dev(np.concatenate([toks[r][a:a + k] for r, k in zip(idx, part)])), o)
            lg[idx] = o
    outs.append(lg.cpu().numpy().copy())
    feed = torch.empty(len(lens), dtype=torch.int32, device="cuda")
    for s in range(steps):
        feed.copy_(to_dev(np.array([t[n + s] for t, n in zip(toks, lens)], np.int32)))
        eng.decode_step_batch(slabs, feed, lg)
        outs.append(lg.cpu().numpy().copy())
    assert eng.device_error() == (0, 0)
    assert [eng.position(s) for s in slabs] == [n + steps for n in lens]
    eng.retire(slabs)
    return outs, toks


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("form", FORMS)
def test_form_matches_the_composition(shape, form):
    ensure_built()
    w, m = weights(SHAPES[shape])
    fm = FORMS[form]
    lens, steps = [150, 1, 37], 3
    eng, gains = make_engine(w, fm)
    outs, toks = run(eng, w.shape, lens, steps)
    tol = TOL[w.shape.weight_format]
    refs = [reference(m, t, fm, gains) for t in toks]
    for s, lg in enumerate(outs):
        check_logits(lg, np.stack([r[n - 1 + s] for r, n in zip(refs, lens)]), tol, f"{shape} {form} step {s}")
    # the same prompts in chunks, on a stream of its own (captured steps)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        eng2, _ = make_engine(w, fm, stream)
        outs2, _ = run(eng2, w.shape, lens, steps, chunk=64)
    for s, lg in enumerate(outs2):
        check_logits(lg, np.stack([r[n - 1 + s] for r, n in zip(refs, lens)]), tol, f"{shape} {form} chunked step {s}")


def test_the_form_changes_the_result():
    """Each option moves the logits far beyond the tolerance, so a dropped one cannot pass above."""
    ensure_built()
    w, m = weights(SHAPES["hd128-gqa"])
    toks = np.random.default_rng(50).integers(0, w.shape.vocab, 150)
    _, gains = make_engine(w, {})
    base = reference(m, toks, {}, gains)[-1]
    for fm in (dict(window=20, sinks=3), dict(norm=True), dict(layout="interleaved", rot=32)):
        assert np.abs(reference(m, toks, fm, gains)[-1] - base).max() > 5e-2, fm


def test_builtin_form_through_the_operators_matches_the_oracle():
    ensure_built()
    w, m = weights(SHAPES["hd128-gqa"])
    lens, steps = [9, 130, 64], 4
    outs, toks = run(make_engine(w, {})[0], w.shape, lens, steps)
    plain = Engine(w, arena_bytes=64 << 20, max_batch=8, max_prefill_tokens=512, page_tokens=128)
    outs2, _ = run(plain, w.shape, lens, steps)
    caches = [oracle.KVCache(w.shape, n + steps) for n in lens]
    ref = oracle.prefill_segmented(m, caches, lens, np.concatenate([t[:n] for t, n in zip(toks, lens)]))
    for s in range(steps + 1):
        check_logits(outs[s], ref, TOL["bf16"], f"step {s}")
        check_logits(outs2[s], ref, TOL["bf16"], f"built-in step {s}")
        if s < steps:
            ref = oracle.decode_step_batch(m, caches, [int(t[n + s]) for t, n in zip(toks, lens)])


def test_rows_and_growth():
    """More rows than one projection tile takes, contexts past the first size of the tables, slabs
    freed and taken again, a prefix shared copy-on-write: all against the composition."""
    ensure_built()
    w, m = weights(SHAPES["hd64"])
    fm = FORMS["window"]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        eng, gains = make_engine(w, fm, stream, arena=256 << 20, max_batch=40)
        # 40 rows decode together
        lens = [1 + (7 * r) % 12 for r in range(40)]
        outs, toks = run(eng, w.shape, lens, 2)
        refs = [reference(m, t, fm, gains) for t in toks]
        for s, lg in enumerate(outs):
            check_logits(lg, np.stack([r[n - 1 + s] for r, n in zip(refs, lens)]), TOL["bf16"], f"40 rows, step {s}")
        # a row past 1024 positions, in chunks; then a row sharing its first 1000 positions
        n = 1100
        t = np.random.default_rng(5).integers(0, w.shape.vocab, n + 3).astype(np.int32)
        a = eng.kv_slab_alloc(2000)
        lg = torch.empty(1, w.shape.vocab, device="cuda")
        for i in range(0, n, 300):
            eng.prefill_segmented([a], [min(300, n - i)], to_dev(t[i:min(n, i + 300)]), lg)
        ref = reference(m, t, fm, gains)
        check_logits(lg.cpu().numpy(), ref[n - 1:n], TOL["bf16"], "long prompt")
        b = eng.kv_slab_alloc(2000)
        eng.share_prefix(a, b, 1000)
        t2 = np.concatenate([t[:1000], np.random.default_rng(6).integers(0, w.shape.vocab, 30).astype(np.int32)])
        lg2 = torch.empty(1, w.shape.vocab, device="cuda")
        eng.prefill_segmented([b], [30], to_dev(t2[1000:]), lg2)
        check_logits(lg2.cpu().numpy(), reference(m, t2, fm, gains)[-1:], TOL["bf16"], "shared prefix")
        eng.decode_step_batch([a], to_dev(t[n:n + 1]), lg)
        check_logits(lg.cpu().numpy(), ref[n:n + 1], TOL["bf16"], "after sharing")
        assert eng.device_error() == (0, 0)


def test_refusals():
    ensure_built()
    w, _ = weights(SHAPES["hd64"])
    code = lambda f: pytest.raises(B.CbtError, match=f)
    contiguous = Engine(w, arena_bytes=64 << 20, max_batch=4, max_prefill_tokens=64)
    with code("UNSUPPORTED"):
        contiguous.set_attention(window=5)
    quant = Engine(w, arena_bytes=64 << 20, max_batch=4, max_prefill_tokens=64, page_tokens=128, kv_bits=8)
    with code("UNSUPPORTED"):
        quant.set_attention(window=5)
    eng = Engine(w, arena_bytes=64 << 20, max_batch=4, max_prefill_tokens=64, page_tokens=128)
    for bad in (dict(window=-1), dict(sinks=-1), dict(eps=-1.0), dict(eps=float("nan"))):
        with code("INVALID"):
            eng.set_attention(**bad)
    with pytest.raises(ValueError):
        eng.set_attention(q_norm=[torch.ones(64, dtype=torch.bfloat16, device="cuda")])
    with pytest.raises(ValueError):
        eng.set_attention(q_norm=[torch.ones(64, device="cuda")] * 2)
    slab = eng.kv_slab_alloc(10)
    with code("INVALID"):
        eng.set_attention(window=5)
    with code("INVALID"):
        B.engine_set_attention(eng.handle, None)
    eng.kv_slab_free(slab)
    eng.set_attention(window=5)
    B.engine_set_attention(eng.handle, None)  # back to the built-in form
    lens = [40, 3]
    outs, toks = run(eng, w.shape, lens, 2)
    plain = Engine(w, arena_bytes=64 << 20, max_batch=4, max_prefill_tokens=64, page_tokens=128)
    outs2, _ = run(plain, w.shape, lens, 2)
    assert all(np.array_equal(x, y) for x, y in zip(outs, outs2))


def test_few_tokens_after_long_prompts():
    """A few tokens admitted behind a long context, whose keys are taken in several runs, next to a row
    that has none yet; then decode steps over both."""
    ensure_built()
    w, m = weights(SHAPES["hd128-gqa"])
    fm = FORMS["norm"]
    eng, gains = make_engine(w, fm, arena=256 << 20)
    n, few = 1300, 5
    t = np.random.default_rng(7).integers(0, w.shape.vocab, n + few + 2).astype(np.int32)
    u = np.random.default_rng(8).integers(0, w.shape.vocab, 4).astype(np.int32)
    a, b = eng.kv_slab_alloc(2000), eng.kv_slab_alloc(100)
    one, two = (torch.empty(k, w.shape.vocab, device="cuda") for k in (1, 2))
    for i in range(0, n, 500):
        eng.prefill_segmented([a], [min(500, n - i)], to_dev(t[i:min(n, i + 500)]), one)
    ref, ref2 = reference(m, t, fm, gains), reference(m, u, fm, gains)
    check_logits(one.cpu().numpy(), ref[n - 1:n], TOL["bf16"], "long prompt")
    eng.prefill_segmented([a, b], [few, 2], to_dev(np.concatenate([t[n:n + few], u[:2]])), two)
    check_logits(two.cpu().numpy(), np.stack([ref[n + few - 1], ref2[1]]), TOL["bf16"], "few tokens")
    for s in range(2):
        eng.decode_step_batch([a, b], to_dev(np.array([t[n + few + s], u[2 + s]], np.int32)), two)
        check_logits(two.cpu().numpy(), np.stack([ref[n + few + s], ref2[2 + s]]), TOL["bf16"], f"step {s}")
    assert eng.device_error() == (0, 0)
