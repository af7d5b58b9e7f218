"""pa_decode_scored: capped and biased scores, document masks, the rotation and
the cache write in the same launch, against the definition in 64 bits.

Tolerance. A weight is exp(x): its relative error is the error of x, plus the
2^-17 that a weight cut to two 16-bit halves may lose (none does here) and the
2^-22 of ex2. x carries the fp32 accumulation of q.k (at most D / 16 + 8
roundings of 2^-23 of s_abs = scale sum |q||k|), the cap's (2^-22 cap), the
bias' (three roundings of the bias of the keys that matter, below 32).
Numerator and denominator each carry it once, against values up to max|v|:
  |err| <= 2 max|v| (2^-17 + 2^-22 + 2^-23 (D / 16 + 8) s_abs + 2^-22 cap + 3 * 32 * 2^-24)
The errors of single keys are independent, so in the 2-norm they stay within
2e-5 of the result (the largest, 2^-17, is 7.6e-6).
"""
import ctypes

import pytest
import torch

from paged_kv_cache_466_b200 import (PA_DERR_BAD_CTX, PA_DERR_BAD_PAGE, PA_DERR_BAD_POS, Rope, _lib,
                                     pa_decode_append, pa_decode_scored, pa_decode_workspace_bytes, pa_kv_append_rope)
from paged_kv_cache_466_b200._lib import (PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE,
                                          PA_OK, pa_kv_pool_t, pa_rope_t, pa_score_t)
from tests.helpers import DEV
from tests.scored_ref import attend64, make_batch, pool_rows, slopes_for

gpu = pytest.mark.gpu


def _check(pool, q, bt, ctx, scale, got, softcap=0.0, slopes=None, doc_begin=None):
    B, Hq, D = q.shape
    lens = ctx.tolist()
    begin = [0]
    for c in lens:
        begin.append(begin[-1] + (c > 0))
    live = [b for b in range(B) if lens[b] > 0]
    want, _, s_abs = attend64(pool, q[live], begin, bt, lens, scale, softcap, slopes,
                              None if doc_begin is None else doc_begin[live])
    vmax = max([float(pool_rows(pool, bt[b], lens[b])[1].abs().max()) for b in live] + [0.0])
    tol = 2 * vmax * (2.0 ** -17 + 2.0 ** -22 + 2.0 ** -23 * (D / 16 + 8) * s_abs
                      + 2.0 ** -22 * softcap + (96 * 2.0 ** -24 if slopes is not None else 0))
    err = (got[live].double() - want).abs().max() if live else torch.zeros(())
    rel = (got[live].double() - want).norm() / want.norm().clamp_min(1e-30) if live else 0
    print(f"max err {float(err):.2e} of {tol:.2e}, rel {float(rel):.2e}")
    assert torch.isfinite(got).all()
    assert float(err) <= tol and float(rel) <= 2e-5
    for b in range(B):
        if lens[b] == 0:
            assert torch.all(got[b] == 0)


MODS = {
    "none": dict(),
    "cap": dict(softcap=20.0),
    "tightcap": dict(softcap=0.5),
    "bias": dict(slopes=True),
    "all": dict(softcap=30.0, slopes=True, doc=True),
    "doc": dict(doc=True),
}


def _mods(name, Hq, ctx, P):
    m = MODS[name]
    kw = dict(softcap=m.get("softcap", 0.0), slopes=slopes_for(Hq) if m.get("slopes") else None)
    kw["doc_begin"] = None
    if m.get("doc"):
        # inside a page, on its border, the newest token alone, before the start
        pick = [lambda c: c // 2, lambda c: c // 2 // P * P, lambda c: max(c - 1, 0), lambda c: -5]
        kw["doc_begin"] = torch.tensor([pick[b % 4](c) for b, c in enumerate(ctx)],
                                       dtype=torch.int32, device=DEV)
    return kw


def _run(pool, q, bt, ctx, scale, kw, **more):
    return pa_decode_scored(pool, q, bt, ctx, scale, softcap=kw["softcap"], alibi_slopes=kw["slopes"],
                            doc_begin=kw["doc_begin"], **more)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
@pytest.mark.parametrize("D,P,G", [(128, 16, 4), (64, 32, 8), (128, 32, 1), (64, 16, 3)])
@pytest.mark.parametrize("mod", list(MODS))
def test_scores(kind, D, P, G, mod):
    lens = [1, P, P + 1, 0, 333, 1000, 47]
    pool, bt, ctx, g = make_batch(lens, 2 * G, 2, D, P, kind)
    q = torch.randn(len(lens), 2 * G, D, generator=g, device=DEV).to(torch.bfloat16)
    kw = _mods(mod, 2 * G, lens, P)
    for S in (0, 1, 3):
        got = _run(pool, q, bt, ctx, D ** -0.5, kw, num_splits=S)
        _check(pool, q, bt, ctx, D ** -0.5, got, **kw)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8"])
def test_large_scores_reach_the_cap(kind):
    """Scores far past the cap on both sides (tanh at 1 and -1) and around the border of its
    two forms."""
    lens = [200, 64, 3]
    pool, bt, ctx, g = make_batch(lens, 4, 2, 128, 16, kind, amp=3.0)
    q = (torch.randn(3, 4, 128, generator=g, device=DEV) * 3).to(torch.bfloat16)
    for cap in (0.1, 5.0, 1000.0):
        got = pa_decode_scored(pool, q, bt, ctx, 0.5, softcap=cap)
        _check(pool, q, bt, ctx, 0.5, got, softcap=cap)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
def test_without_changes_it_attends_as_the_plain_decode(kind):
    """No change of the scores: the plain decode's definition; the stored rows are its bits."""
    lens = [5, 300, 1, 64]
    pool, bt, ctx, g = make_batch(lens, 8, 2, 128, 16, kind)
    other, _, _, _ = make_batch(lens, 8, 2, 128, 16, kind)
    q = torch.randn(4, 8, 128, generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn(4, 2, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
    for S in (1, 2):
        _check(pool, q, bt, ctx, 0.1, pa_decode_scored(pool, q, bt, ctx, 0.1, num_splits=S))
        got = pa_decode_scored(pool, q, bt, ctx, 0.1, k_new=k, v_new=v, num_splits=S)
        pa_decode_append(other, q, k, v, bt, ctx, 0.1, num_splits=S)
        _check(other, q, bt, ctx, 0.1, got)
        for x, y in zip(pool.tensors(), other.tensors()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
def test_long_contexts_do_not_drift(kind):
    """30,000 tokens in as few splits as there can be: sums of blocks are added rounded, not
    cut off, and zero points do not cancel most of the output (codes enter centred)."""
    pool, bt, ctx, g = make_batch([30000, 12345], 8, 1, 64, 32, kind, seed=2)
    q = torch.randn(2, 8, 64, generator=g, device=DEV).to(torch.bfloat16)
    for cap in (0.0, 30.0):
        _check(pool, q, bt, ctx, 0.125, pa_decode_scored(pool, q, bt, ctx, 0.125, softcap=cap, num_splits=1),
               softcap=cap)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
@pytest.mark.parametrize("D,rot,interleaved,axes", [(128, 128, False, 1), (128, 64, True, 1),
                                                    (64, 32, False, 3), (64, 64, True, 3)])
def test_rotation_and_write_in_one_launch(kind, D, rot, interleaved, axes):
    """The fused step's stored bits and outputs are those of pa_kv_append_rope followed by the
    call without rope and rows, bit for bit; and those are the definition's."""
    lens = [1, 16, 17, 400, 0, 33]
    pool, bt, ctx, g = make_batch(lens, 6, 2, D, 16, kind)
    other, _, _, _ = make_batch(lens, 6, 2, D, 16, kind)
    B = len(lens)
    q = torch.randn(B, 6, D, generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn(B, 2, D, generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
    pairs = rot // 2
    rope = Rope.from_base(500, rot, 100.0, DEV, interleaved=interleaved,
                          axis_of_pair=[j * axes // pairs for j in range(pairs)])
    rp = torch.randint(0, 500, (axes, B), generator=g, device=DEV, dtype=torch.int32) if axes > 1 else None
    doc = torch.tensor([0, 20, 5, 100, 0, 33], dtype=torch.int32, device=DEV)  # two see nothing
    slopes = slopes_for(6)
    live = torch.tensor([b for b in range(B) if lens[b] > 0], dtype=torch.int32, device=DEV)
    i = live.long()
    qr = torch.zeros_like(q)
    qr[i] = pa_kv_append_rope(other, rope, q[i], k[i], v[i], live, (ctx - 1)[i].contiguous(), bt,
                              rope_pos=None if rp is None else rp[:, i].contiguous())
    for S in (1, 2):
        got = pa_decode_scored(pool, q, bt, ctx, 0.1, softcap=10.0, alibi_slopes=slopes, doc_begin=doc,
                               rope=rope, rope_pos=rp, k_new=k, v_new=v, num_splits=S)
        for a, b in zip(pool.tensors(), other.tensors()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        want = pa_decode_scored(other, qr, bt, ctx, 0.1, softcap=10.0, alibi_slopes=slopes,
                                doc_begin=doc, num_splits=S)
        assert torch.equal(got, want)
        _check(other, qr, bt, ctx, 0.1, got, softcap=10.0, slopes=slopes, doc_begin=doc)


@gpu
def test_bad_pages_lengths_and_positions():
    lens = [40, 40, 40, 40]
    pool, bt, ctx, g = make_batch(lens, 4, 2, 64, 16, "bf16")
    q = torch.randn(4, 4, 64, generator=g, device=DEV).to(torch.bfloat16)
    k, v = (torch.randn(4, 2, 64, generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
    good = pa_decode_scored(pool, q, bt, ctx, 0.1, softcap=5.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = pool.k.clone()
    rope = Rope.from_base(100, 64, 100.0, DEV)
    rp = torch.tensor([-1, 100, 3, 4], dtype=torch.int32, device=DEV)
    bad_bt, bad_ctx = bt.clone(), ctx.clone()
    bad_bt[2, 2] = pool.num_pages                         # the page of the newest token
    bad_ctx[3] = 49                                       # past the table
    out = pa_decode_scored(pool, q, bad_bt, bad_ctx, 0.1, softcap=5.0, rope=rope, rope_pos=rp, k_new=k,
                           v_new=v, d_err=err)
    assert int(err.item()) == PA_DERR_BAD_POS | PA_DERR_BAD_PAGE | PA_DERR_BAD_CTX
    assert torch.all(out[[0, 1, 3]] == 0) and torch.isfinite(out).all()
    assert torch.equal(pool.k.view(torch.int16), before.view(torch.int16))   # nothing was stored
    assert torch.equal(pa_decode_scored(pool, q, bt, ctx, 0.1, softcap=5.0), good)


@gpu
def test_two_graphs_share_a_workspace():
    lens = [700, 90, 411]
    pool, bt, ctx, g = make_batch(lens, 8, 2, 128, 16, "fp8")
    q = torch.randn(3, 8, 128, generator=g, device=DEV).to(torch.bfloat16)
    ws = torch.zeros(pa_decode_workspace_bytes(3, 8, 128, 8), dtype=torch.uint8, device=DEV)
    outs, graphs = [], []
    for cap, S in ((0.0, 8), (7.0, 4)):
        out = torch.empty(3, 8, 128, device=DEV)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            pa_decode_scored(pool, q, bt, ctx, 0.1, softcap=cap, out=out, workspace=ws, num_splits=S)
        outs.append(out)
        graphs.append(gr)
    for _ in range(3):
        q.copy_(torch.randn(3, 8, 128, generator=g, device=DEV).to(torch.bfloat16))
        for gr in graphs:
            gr.replay()
        for out, cap in zip(outs, (0.0, 7.0)):
            _check(pool, q, bt, ctx, 0.1, out, softcap=cap)


# ---- refusals, without a GPU -------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_466_b200 import build
    build.build()
    return _lib.load()


def _call(lib, score=None, rope=None, k=None, v=None, rp=None, B=2, hq=4, splits=1, dtype=0, **kw):
    pool = pa_kv_pool_t(num_pages=8, page_size=16, num_kv_heads=2, head_dim=128, dtype=dtype,
                        k_pool=0x1000, v_pool=0x2000, k_sz=None, v_sz=None)
    return lib.pa_decode_scored(ctypes.byref(pool), None if score is None else ctypes.byref(score),
                                None if rope is None else ctypes.byref(rope), kw.get("q", 0x3000), k, v,
                                rp, B, hq, 0x5000, 4, 0x6000, 0.1, kw.get("out", 0x4000), None, 0, splits,
                                None, None)


def test_refusals(lib):
    assert _call(lib, B=0) == PA_OK
    for cap in (-1.0, float("nan"), float("inf")):
        assert _call(lib, pa_score_t(cap, None, None, None)) == PA_ERR_INVALID_ARG
    rope = pa_rope_t(0x1000, 10, 136, 0, 1, (ctypes.c_uint8 * 64)())
    assert _call(lib, rope=rope) == PA_ERR_UNSUPPORTED
    rope.rotary_dim, rope.table = 128, 0x1004
    assert _call(lib, rope=rope) == PA_ERR_INVALID_ARG
    assert _call(lib, rp=0x7000) == PA_ERR_INVALID_ARG                 # positions without a rotation
    assert _call(lib, k=0x7000) == PA_ERR_INVALID_ARG                  # keys without values
    assert _call(lib, v=0x7000) == PA_ERR_INVALID_ARG
    assert _call(lib, k=0x7004, v=0x8000) == PA_ERR_INVALID_ARG
    assert _call(lib, hq=3) == PA_ERR_INVALID_ARG
    assert _call(lib, hq=18) == PA_ERR_UNSUPPORTED
    assert _call(lib, q=None) == PA_ERR_INVALID_ARG
    assert _call(lib, out=0x4004) == PA_ERR_INVALID_ARG
    assert _call(lib, splits=2) == PA_ERR_WORKSPACE
    assert _call(lib, dtype=9) == PA_ERR_UNSUPPORTED
