"""pa_prefill against the definition in 64 bits: ragged batches, every cache
format, capped and biased scores, document and prefix masks, split keys, rows
without a visible key, bad pages and lengths, refusals.

Tolerance. The output is rounded to bf16 (at most 2^-8 of it), every weight is
rounded to bf16 before the second product (2^-8 of each term p |s (c - shift)|,
whose weighted mean is `mag`), and a weight carries the error of its score, in
the numerator and the denominator: 2 max|v| delta with
  delta = 2^-21 + 2^-23 (D / 16 + 8) s_abs + 2^-22 cap + 96 * 2^-24 (bias)
as for the decode (s_abs: scale times the sum of the magnitudes that are added).
The roundings of different weights are independent: in the 2-norm they and the
output's stay within 2^-8 of the result together. The log-sum-exp carries delta
and two fp32 roundings of its own size.
"""
import ctypes

import pytest
import torch

from paged_kv_cache_466_b200 import (PA_DERR_BAD_CTX, PA_DERR_BAD_PAGE, PA_DERR_BAD_SEQ, KVPool, Rope,
                                     _lib, pa_decode_scored, pa_kv_append_rope, pa_prefill,
                                     pa_prefill_workspace_bytes)
from paged_kv_cache_466_b200._lib import (PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE,
                                          PA_OK, pa_kv_pool_t, pa_score_t)
from tests.helpers import DEV
from tests.scored_ref import attend64, make_batch, pool_rows, slopes_for

gpu = pytest.mark.gpu
SPARE = 3   # rows behind the last sequence


def _queries(g, qlens, Hq, D, amp=1.0):
    begin = torch.tensor([0] + qlens).cumsum(0).to(torch.int32).to(DEV)
    n = sum(qlens)
    q = (torch.randn(n + SPARE, Hq, D, generator=g, device=DEV) * amp).to(torch.bfloat16)
    return q, begin, n


def _check(pool, q, begin, bt, ctx, scale, n, got, lse, softcap=0.0, slopes=None, doc_begin=None,
           prefix_end=None, d_rel=2.0 ** -8):
    D = q.shape[2]
    lens = ctx.tolist()
    want, wlse, s_abs, mag = attend64(pool, q[:n], begin.tolist(), bt, lens, scale, softcap, slopes,
                                      doc_begin, prefix_end, weighted=True)
    vmax = max([float(pool_rows(pool, bt[b], c)[1].abs().max()) for b, c in enumerate(lens) if c] + [0.0])
    delta = (2.0 ** -21 + 2.0 ** -23 * (D / 16 + 8) * s_abs + 2.0 ** -22 * softcap
             + (96 * 2.0 ** -24 if slopes is not None else 0))
    tol = 1.01 * 2.0 ** -8 * (want.abs() + mag) + 2 * vmax * delta
    err = (got[:n].double() - want).abs()
    assert torch.isfinite(got[:n]).all()
    rel = float(err.norm() / want.norm().clamp_min(1e-30))
    print(f"max err/tol {float((err / tol.clamp_min(1e-30)).max()) if n else 0:.3f}, rel {rel:.2e}")
    assert torch.all(err <= tol) and rel <= d_rel
    assert torch.all(got[n:] == 7.0)                       # rows behind the last sequence
    empty = wlse == -float("inf")
    assert torch.equal(lse[:n] == -float("inf"), empty) and torch.all(got[:n][empty] == 0)
    e = (lse[:n].double() - wlse)[~empty].abs()
    assert torch.all(e <= delta + 2.0 ** -22 * (1 + wlse[~empty].abs()))
    assert torch.all(lse[n:] == 7.0)


def _run(pool, q, begin, bt, ctx, scale, kw, **more):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    N = q.shape[0]
    # the masks hold one entry per row of q, spare rows included
    pad = lambda t: None if t is None else torch.cat([t, t.new_zeros(N - t.numel())])
    got = pa_prefill(pool, q, begin, bt, ctx, scale, softcap=kw.get("softcap", 0.0),
                     alibi_slopes=kw.get("slopes"), doc_begin=pad(kw.get("doc_begin")),
                     prefix_end=pad(kw.get("prefix_end")), out=out, lse_out=lse, **more)
    assert got is out
    return out, lse


def _mods(name, Hq, qlens, lens):
    """Score changes and masks by name; positions of every query token come from the lengths."""
    pos = torch.cat([torch.arange(c - n, c) for n, c in zip(qlens, lens)]).to(DEV) if sum(qlens) else \
        torch.zeros(0, dtype=torch.long, device=DEV)
    i32 = lambda t: t.to(torch.int32).contiguous()
    kw = {}
    if "cap" in name:
        kw["softcap"] = 15.0
    if "tight" in name:
        kw["softcap"] = 0.25
    if "bias" in name:
        kw["slopes"] = slopes_for(Hq)
    if "doc" in name:
        kw["doc_begin"] = i32(pos // 100 * 100)
    if "pre" in name:
        kw["prefix_end"] = i32(pos // 100 * 100 + 37)
    if "empty" in name:     # every third token sees nothing, the others only the far past or all
        kw["doc_begin"] = i32(torch.where(pos % 3 == 0, pos + 1, torch.where(pos % 3 == 1, -4, pos)))
    if "image" in name:     # everything sees the whole sequence and more
        kw["prefix_end"] = i32(pos * 0 + 100_000)
    return kw


QLENS = [1, 17, 128, 300, 0, 5, 257, 64]
LENS = [1, 17, 300, 300, 50, 1000, 259, 70]


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
@pytest.mark.parametrize("D,P,G", [(128, 16, 4), (64, 32, 8), (128, 32, 1), (64, 16, 3), (128, 16, 7)])
@pytest.mark.parametrize("mod", ["none", "cap", "bias doc", "cap bias doc pre", "empty"])
def test_ragged_batches(kind, D, P, G, mod):
    pool, bt, ctx, g = make_batch(LENS, 2 * G, 2, D, P, kind)
    q, begin, n = _queries(g, QLENS, 2 * G, D)
    kw = _mods(mod, 2 * G, QLENS, LENS)
    got, lse = _run(pool, q, begin, bt, ctx, D ** -0.5, kw, num_splits=1)
    _check(pool, q, begin, bt, ctx, D ** -0.5, n, got, lse, **kw)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u4"])
@pytest.mark.parametrize("mod", ["none", "tight", "pre", "bias pre", "bias image", "doc pre", "empty bias"])
@pytest.mark.parametrize("splits", [0, 1, 2, 5, 64])
def test_masks_and_splits(kind, mod, splits):
    qlens, lens = [33, 1, 260, 9], [1500, 700, 400, 9]
    pool, bt, ctx, g = make_batch(lens, 6, 2, 128, 16, kind, seed=3)
    q, begin, n = _queries(g, qlens, 6, 128)
    kw = _mods(mod, 6, qlens, lens)
    got, lse = _run(pool, q, begin, bt, ctx, 128 ** -0.5, kw, num_splits=splits)
    _check(pool, q, begin, bt, ctx, 128 ** -0.5, n, got, lse, **kw)


@gpu
@pytest.mark.parametrize("qlen,ctx_", [(1, 1), (1, 128), (1, 129), (2, 127), (128, 128), (129, 129),
                                       (1000, 1000), (2111, 2111), (63, 4001), (511, 16)])
def test_single_sequence_lengths(qlen, ctx_):
    ctx_ = max(qlen, ctx_)
    pool, bt, ctx, g = make_batch([ctx_], 4, 1, 64, 16, "bf16", max_pages=300)
    q, begin, n = _queries(g, [qlen], 4, 64)
    got, lse = _run(pool, q, begin, bt, ctx, 0.125, {})
    _check(pool, q, begin, bt, ctx, 0.125, n, got, lse)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8"])
@pytest.mark.parametrize("amp,scale", [(6.0, 1.0), (0.01, 1.0), (1.0, 0.0), (1.0, -0.1)])
def test_score_sizes(kind, amp, scale):
    """One-hot rows, flat rows, a scale of zero and a negative one."""
    qlens, lens = [70, 130], [200, 130]
    pool, bt, ctx, g = make_batch(lens, 2, 2, 128, 16, kind)
    q, begin, n = _queries(g, qlens, 2, 128, amp)
    for kw in ({}, {"softcap": 8.0}):
        got, lse = _run(pool, q, begin, bt, ctx, scale, kw)
        _check(pool, q, begin, bt, ctx, scale, n, got, lse, **kw)


@gpu
def test_many_sequences_and_none():
    g0 = torch.Generator().manual_seed(1)
    qlens = torch.randint(0, 9, (77,), generator=g0).tolist()
    lens = [n + int(p) for n, p in zip(qlens, torch.randint(0, 60, (77,), generator=g0))]
    pool, bt, ctx, g = make_batch(lens, 3, 1, 64, 32, "fp8")
    q, begin, n = _queries(g, qlens, 3, 64)
    got, lse = _run(pool, q, begin, bt, ctx, 0.125, {})
    _check(pool, q, begin, bt, ctx, 0.125, n, got, lse)
    none = pa_prefill(pool, q[:0], begin[:1] * 0, bt[:0], ctx[:0], 0.125)
    assert none.shape == (0, 3, 64)
    got, lse = _run(pool, q, begin * 0, bt, ctx, 0.125, {})   # no sequence has a query
    assert torch.all(got == 7.0) and torch.all(lse == 7.0)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8"])
@pytest.mark.parametrize("splits", [1, 3])
def test_bad_pages_lengths_and_rows(kind, splits):
    qlens, lens = [40, 40, 40, 40], [600, 600, 600, 600]
    pool, bt, ctx, g = make_batch(lens, 4, 2, 128, 16, kind)
    q, begin, n = _queries(g, qlens, 4, 128)
    bad_bt, bad_ctx, bad_begin = bt.clone(), ctx.clone(), begin.clone()
    bad_bt[0, 3] = -7                  # tokens 48..63 of sequence 0
    bad_bt[0, 37] = pool.num_pages     # the page that its context ends in
    bad_ctx[1] = 39                    # fewer than its query tokens
    bad_ctx[2] = 16 * bt.shape[1] + 1  # past the table
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got, lse = _run(pool, q, begin, bad_bt, bad_ctx, 0.1, {}, num_splits=splits, d_err=err)
    assert int(err.item()) == PA_DERR_BAD_PAGE | PA_DERR_BAD_CTX
    good, glse = _run(pool, q, begin, bt, ctx, 0.1, {}, num_splits=splits)
    assert torch.all(got[40:120] == 0) and torch.all(lse[40:120] == -float("inf"))
    assert torch.equal(got[120:], good[120:]) and torch.equal(lse[120:], glse[120:])
    # sequence 0 without the tokens of its two bad pages, in 64 bits
    K, V = pool_rows(pool, bt[0], 600)
    j = torch.arange(600, device=DEV)
    dead = (j // 16 == 3) | (j // 16 == 37)
    for h in range(4):
        x = q[:40, h].double() @ K[:, h // 2].T * 0.1
        x = x.masked_fill(dead | (j > 560 + torch.arange(40, device=DEV)[:, None]), -float("inf"))
        want = torch.softmax(x, -1) @ V[:, h // 2]
        assert (got[:40, h].double() - want).abs().max() <= 2.0 ** -7 * float(V.abs().max())
    # entries of q_begin out of order or out of range: flagged, every access in range
    err.zero_()
    bad_begin[1] = 200_000
    out, _ = _run(pool, q, bad_begin, bt, ctx, 0.1, {}, num_splits=splits, d_err=err)
    assert int(err.item()) & PA_DERR_BAD_SEQ
    assert torch.equal(pa_prefill(pool, q, begin, bt, ctx, 0.1, num_splits=splits)[:n], good[:n])


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
@pytest.mark.parametrize("D,P,splits", [(128, 16, 1), (128, 32, 3), (64, 32, 1)])
def test_pages_before_the_first_document_may_be_dropped(kind, D, P, splits):
    """Pages that end before the first key any query sees: entries outside the pool, or pages
    that hold NaN by now. Neither is read; the results are those of the whole table, bit for bit."""
    lens, firsts, qlens = [700, 333, 129, 520], [333, 200, 128, 256], [90, 40, 1, 200]
    pool, bt, ctx, g = make_batch(lens, 4, 2, D, P, kind)
    q, begin, n = _queries(g, qlens, 4, D)
    doc = torch.cat([torch.full((m,), f, dtype=torch.int32) for m, f in zip(qlens, firsts)]).to(DEV)
    doc[80:90] = 690                                         # a second document
    got, lse = _run(pool, q, begin, bt, ctx, 0.1, {"doc_begin": doc}, num_splits=splits)
    _check(pool, q, begin, bt, ctx, 0.1, n, got, lse, doc_begin=doc)
    last = torch.tensor([90, 130, 131, 331], device=DEV) - 1
    step = pa_decode_scored(pool, q[last], bt, ctx, 0.1, doc_begin=doc[last], num_splits=splits)
    dropped = bt.clone()
    for b, f in enumerate(firsts):
        gone = bt[b, :f // P].long()
        for t in pool.tensors():
            t[gone] = float("nan") if t.is_floating_point() else 0xFF
        dropped[b, :f // P:2] = -1
        dropped[b, 1:f // P:4] = pool.num_pages
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got2, lse2 = _run(pool, q, begin, dropped, ctx, 0.1, {"doc_begin": doc}, num_splits=splits, d_err=err)
    assert int(err.item()) == 0 and torch.equal(got, got2) and torch.equal(lse, lse2)
    step2 = pa_decode_scored(pool, q[last], dropped, ctx, 0.1, doc_begin=doc[last], num_splits=splits,
                             d_err=err)
    assert int(err.item()) == 0 and torch.equal(step, step2)


@gpu
def test_garbage_behind_the_context_is_not_read():
    """Rows behind the context in its last page, and pages behind it, hold NaN."""
    pool = KVPool(4, 1, 16, 128, "bf16", DEV, fill_byte=0xFF)
    assert torch.isnan(pool.k.float()).all()
    g = torch.Generator(device=DEV).manual_seed(0)
    pool.k[1, :, :5] = torch.randn(1, 5, 128, generator=g, device=DEV).to(torch.bfloat16)
    pool.v[1, :, :5] = torch.randn(1, 5, 128, generator=g, device=DEV).to(torch.bfloat16)
    bt = torch.tensor([[1, 2, 3]], dtype=torch.int32, device=DEV)
    ctx = torch.tensor([5], dtype=torch.int32, device=DEV)
    q, begin, n = _queries(g, [5], 2, 128)
    got, lse = _run(pool, q, begin, bt, ctx, 0.1, {})
    _check(pool, q, begin, bt, ctx, 0.1, n, got, lse)


@gpu
def test_pool_past_two_to_the_31_elements():
    P, Hkv, D = 16, 8, 128
    pages = 2 ** 31 // (P * Hkv * D) + 40
    pool = KVPool(pages, Hkv, P, D, "bf16", DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    bt = torch.tensor([[pages - 1, 3, pages - 9]], dtype=torch.int32, device=DEV)
    ctx = torch.tensor([41], dtype=torch.int32, device=DEV)
    n = 41
    q, k, v = (torch.randn(n, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (16, Hkv, Hkv))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    rope = Rope.from_base(64, 128, 10000.0, DEV)
    qr = pa_kv_append_rope(pool, rope, q, k, v, pos * 0, pos, bt)
    begin = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    qs = torch.cat([qr, qr[:SPARE]])
    got, lse = _run(pool, qs, begin, bt, ctx, 0.09, {})
    _check(pool, qs, begin, bt, ctx, 0.09, n, got, lse)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
def test_a_prompt_in_chunks_then_steps(kind):
    """The set as it is used: chunks of a prompt written with their rotation and attended, then
    fused decode steps; every result against one 64-bit attention over the final cache."""
    D, P, Hq, Hkv, T, B = 128, 16, 8, 2, 221, 2
    g = torch.Generator(device=DEV).manual_seed(4)
    pool = KVPool(B * 15 + 1, Hkv, P, D, kind, DEV, fill_byte=0xFF)
    bt = torch.randperm(B * 15, generator=g, device=DEV).to(torch.int32).view(B, 15).contiguous()
    rope = Rope.from_base(300, 64, 10000.0, DEV)
    rand = lambda h: torch.randn(B, T, h, D, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = rand(Hq), rand(Hkv), rand(Hkv)
    slopes = slopes_for(Hq)
    outs = torch.zeros(B, T, Hq, D, device=DEV)
    rotated = torch.zeros_like(q)
    at = 0
    for n in (100, 7, 112):
        seq = torch.arange(B, device=DEV).repeat_interleave(n).to(torch.int32)
        pos = torch.arange(at, at + n, device=DEV).repeat(B).to(torch.int32)
        flat = lambda t: t[:, at:at + n].reshape(B * n, -1, D).contiguous()
        qr = pa_kv_append_rope(pool, rope, flat(q), flat(k), flat(v), seq, pos, bt)
        begin = torch.arange(B + 1, device=DEV, dtype=torch.int32) * n
        ctx = torch.full((B,), at + n, dtype=torch.int32, device=DEV)
        o = pa_prefill(pool, qr, begin, bt, ctx, D ** -0.5, softcap=30.0, alibi_slopes=slopes)
        outs[:, at:at + n] = o.view(B, n, Hq, D).float()
        rotated[:, at:at + n] = qr.view(B, n, Hq, D)
        at += n
    while at < T:
        ctx = torch.full((B,), at + 1, dtype=torch.int32, device=DEV)
        tok = lambda t: t[:, at].contiguous()
        outs[:, at] = pa_decode_scored(pool, tok(q), bt, ctx, D ** -0.5, softcap=30.0, alibi_slopes=slopes,
                                       rope=rope, k_new=tok(k), v_new=tok(v))
        rotated[:, at] = pa_kv_append_rope(pool, rope, tok(q), tok(k), tok(v),
                                           torch.arange(B, dtype=torch.int32, device=DEV), ctx - 1, bt)
        at += 1
    want, _, _, mag = attend64(pool, rotated.flatten(0, 1), [0, T, 2 * T], bt, [T, T], D ** -0.5, 30.0,
                               slopes, weighted=True)
    tol = 1.01 * 2.0 ** -8 * (want.abs() + mag) + 1e-4
    assert torch.all((outs.flatten(0, 1).double() - want).abs() <= tol)


@gpu
def test_graph_replay_shared_workspace_and_determinism():
    qlens, lens = [20, 3], [3000, 900]
    pool, bt, ctx, g = make_batch(lens, 8, 2, 128, 16, "bf16")
    q, begin, n = _queries(g, qlens, 8, 128)
    need = pa_prefill_workspace_bytes(pool, q.shape[0], 2, 8, bt.shape[1])
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
    graphs = []
    for cap in (0.0, 9.0):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            pa_prefill(pool, q, begin, bt, ctx, 0.09, softcap=cap, out=out, lse_out=lse, workspace=ws)
        graphs.append(gr)
    for _ in range(2):
        q.copy_(torch.randn(q.shape, generator=g, device=DEV).to(torch.bfloat16))
        for gr, cap in zip(graphs, (0.0, 9.0)):
            gr.replay()
            _check(pool, q, begin, bt, ctx, 0.09, n, out, lse, softcap=cap)
            first = out.clone()
            gr.replay()
            assert torch.equal(first, out)
    # the split counters that the decode keeps at the workspace's start are untouched
    lenb = torch.tensor([3000, 900], dtype=torch.int32, device=DEV)
    a = pa_decode_scored(pool, q[:2].contiguous(), bt, lenb, 0.09, workspace=ws, num_splits=2)
    b = pa_decode_scored(pool, q[:2].contiguous(), bt, lenb, 0.09, num_splits=2)
    assert torch.equal(a, b)


@gpu
def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, beside a busy default stream."""
    cases = []
    for seed, (qlens, lens, kind) in enumerate([([700, 33], [900, 2000], "bf16"), ([5, 6, 7], [3000, 40, 7], "u8")]):
        pool, bt, ctx, g = make_batch(lens, 8, 2, 128, 16, kind, seed=seed)
        q, begin, n = _queries(g, qlens, 8, 128)
        ws = torch.zeros(1 << 25, dtype=torch.uint8, device=DEV)
        cases.append((pool, q, begin, bt, ctx, n, ws, torch.full_like(q, 7.0),
                      torch.full(q.shape[:2], 7.0, device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device=DEV)
    for _ in range(4):
        busy = busy @ busy * 1e-3
        for pool, q, begin, bt, ctx, n, ws, out, lse, stream in cases:
            pa_prefill(pool, q, begin, bt, ctx, 0.09, softcap=20.0, out=out, lse_out=lse, workspace=ws,
                       num_splits=3, stream=stream)
    torch.cuda.synchronize()
    for pool, q, begin, bt, ctx, n, ws, out, lse, stream in cases:
        _check(pool, q, begin, bt, ctx, 0.09, n, out, lse, softcap=20.0)


# ---- refusals, without a GPU -------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_466_b200 import build
    build.build()
    return _lib.load()


def _pool(**kw):
    d = dict(num_pages=8, page_size=16, num_kv_heads=2, head_dim=128, dtype=0, k_pool=0x1000,
             v_pool=0x2000, k_sz=None, v_sz=None)
    d.update(kw)
    return pa_kv_pool_t(**d)


def _call(lib, pool=None, score=None, n=9, hq=4, B=2, max_pages=40, splits=1, **kw):
    pool = pool or _pool()
    ptr = lambda k, d: kw.get(k, d)
    return lib.pa_prefill(ctypes.byref(pool), None if score is None else ctypes.byref(score),
                          ptr("q", 0x3000), n, hq, ptr("begin", 0x4000), B, ptr("bt", 0x5000), max_pages,
                          ptr("ctx", 0x6000), kw.get("scale", 0.1), ptr("out", 0x7000), None,
                          kw.get("ws"), kw.get("ws_bytes", 0), splits, None, None)


def test_refusals(lib):
    assert _call(lib, n=0) == PA_OK and _call(lib, B=0) == PA_OK
    assert _call(lib, pool=_pool(head_dim=96)) == PA_ERR_UNSUPPORTED
    assert _call(lib, pool=_pool(page_size=8)) == PA_ERR_UNSUPPORTED
    assert _call(lib, pool=_pool(dtype=1)) == PA_ERR_INVALID_ARG
    assert _call(lib, hq=5) == PA_ERR_INVALID_ARG
    assert _call(lib, hq=18) == PA_ERR_UNSUPPORTED
    assert _call(lib, n=-1) == PA_ERR_INVALID_ARG
    assert _call(lib, n=(1 << 24) + 1) == PA_ERR_UNSUPPORTED
    assert _call(lib, pool=_pool(num_kv_heads=32), n=1 << 24, hq=256) == PA_ERR_UNSUPPORTED
    assert _call(lib, max_pages=0) == PA_ERR_INVALID_ARG
    assert _call(lib, splits=-1) == PA_ERR_INVALID_ARG
    assert _call(lib, scale=float("nan")) == PA_ERR_INVALID_ARG
    assert _call(lib, score=pa_score_t(-2.0, None, None, None)) == PA_ERR_INVALID_ARG
    for k in ("q", "begin", "bt", "ctx", "out"):
        assert _call(lib, **{k: None}) == PA_ERR_INVALID_ARG
    assert _call(lib, q=0x3008) == PA_ERR_INVALID_ARG
    assert _call(lib, out=0x7008) == PA_ERR_INVALID_ARG
    assert _call(lib, splits=3) == PA_ERR_WORKSPACE
    need = lib.pa_prefill_workspace_bytes(ctypes.byref(_pool()), 9, 2, 4, 40, 3)
    parts = 9 * 4 * 3 * 4
    assert need >= parts * 128 + parts and need % 256 == 0
    assert _call(lib, splits=3, ws=0x10010, ws_bytes=need) == PA_ERR_WORKSPACE
    assert _call(lib, splits=3, ws=0x10000, ws_bytes=parts * 128) == PA_ERR_WORKSPACE
    assert lib.pa_prefill_workspace_bytes(ctypes.byref(_pool()), 9, 2, 4, 40, 1) == 0
    assert lib.pa_prefill_workspace_bytes(ctypes.byref(_pool(head_dim=32)), 9, 2, 4, 40, 3) == 0
