"""The edges of the rotating cache write, prompt attention and scored decode:
malformed batches, queries that are not numbers, rows that see nothing, caps and
scales at the ends of their range, storage that a call allocates. The 64-bit
definitions and the tolerances are those of test_prefill.py and
test_decode_scored.py."""
import contextlib
import ctypes
import types

import pytest
import torch

import paged_kv_cache_466_b200 as pa
from paged_kv_cache_466_b200 import (PA_DERR_BAD_SEQ, KVPool, Rope, _lib, pa_decode_scored,
                                     pa_kv_append_rope, pa_prefill, pa_prefill_workspace_bytes)
from paged_kv_cache_466_b200._lib import PA_ERR_INVALID_ARG, PA_OK, pa_kv_pool_t, pa_score_t
from tests.helpers import DEV
from tests.scored_ref import attend64, make_batch
from tests.test_decode_scored import _check as _check_step
from tests.test_prefill import _check, _queries, _run

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8"])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("entries,whole", [
    ({3: -5}, [(0, 40)]),                 # the last entry negative
    ({3: -2 ** 31}, [(0, 40)]),
    ({3: 17}, [(0, 23), (23, 40)]),       # the last sequence descends into the others' rows
    ({2: 3}, [(0, 23)]),                  # an interior entry descends
    ({0: -7, 3: 10 ** 9}, [(23, 40)]),    # both ends out of range
    ({0: 2 ** 31 - 1}, [(23, 40), (40, 41)]),
])
def test_malformed_query_ranges_stay_inside_the_outputs(kind, splits, entries, whole):
    """No row outside the outputs is written (41 x 6 rows: the last CTA of a merge is not full),
    the call is flagged, and sequences whose own entries are in order, and whose rows no other
    sequence claims, keep their results bit for bit."""
    qlens, lens, Hq = [23, 17, 1], [900, 700, 300], 6
    pool, bt, ctx, g = make_batch(lens, Hq, 2, 128, 16, kind)
    q, begin, n = _queries(g, qlens, Hq, 128)
    q = q[:n].contiguous()
    bad = begin.clone()
    for i, x in entries.items():
        bad[i] = x

    def run(b, err):
        out = torch.full((n * Hq + 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((n * Hq + 8,), 7.0, device=DEV)
        pa_prefill(pool, q, b, bt, ctx, 0.1, out=out[:n * Hq].view(n, Hq, 128),
                   lse_out=lse[:n * Hq].view(n, Hq), num_splits=splits, d_err=err)
        assert torch.all(out[n * Hq:] == 7.0) and torch.all(lse[n * Hq:] == 7.0)
        return out[:n * Hq].view(n, Hq, 128), lse[:n * Hq].view(n, Hq)

    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    good, glse = run(begin, err)
    assert int(err.item()) == 0 and not torch.any(good == 7.0)
    out, lse = run(bad, err)
    assert int(err.item()) & PA_DERR_BAD_SEQ
    b = [min(max(int(x), 0), n) for x in bad.tolist()]
    claimed = torch.zeros(n, dtype=torch.int32)
    for s, e in zip(b, b[1:]):
        claimed[s:max(e, s)] += 1
    for s, e in whole:
        for i in range(s, e):
            if claimed[i] == 1:
                assert torch.equal(out[i], good[i]) and torch.equal(lse[i], glse[i])
    idle = (claimed == 0).to(DEV)
    assert torch.all(out[idle] == 7.0) and torch.all(lse[idle] == 7.0)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "u4"])
@pytest.mark.parametrize("D,P", [(128, 16), (64, 32)])
def test_blocks_whose_rows_all_see_nothing(kind, D, P):
    """Blocks of 256 rows without a single key: their zeros go out through shared memory that no
    query may still be on its way to. Many blocks, several times; queries far from zero."""
    qlens, lens, Hq = [1500, 200, 900], [1600, 333, 900], 8
    pool, bt, ctx, g = make_batch(lens, Hq, 2, D, P, kind)
    q, begin, n = _queries(g, qlens, Hq, D, 100.0)
    pos = torch.cat([torch.arange(c - m, c) for m, c in zip(qlens, lens)]).to(DEV)
    blind = (torch.arange(n, device=DEV) < 1500) | (torch.arange(n, device=DEV) >= 1700)
    doc = torch.where(blind, pos + 1, 0).to(torch.int32)
    for _ in range(10):
        got, lse = _run(pool, q, begin, bt, ctx, 1e-3, {"doc_begin": doc}, num_splits=1)
        assert torch.all(got[:n][blind] == 0) and torch.all(lse[:n][blind] == -float("inf"))
    _check(pool, q, begin, bt, ctx, 1e-3, n, got, lse, doc_begin=doc)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
@pytest.mark.parametrize("splits", [1, 3, 0])
def test_a_query_that_is_not_a_number_gives_nan(kind, splits):
    """NaN in one head, in all heads of a token, an infinity: out and lse of those rows are NaN
    however the keys are split, and the others hold their result."""
    qlens, lens = [40, 3], [1500, 700]
    pool, bt, ctx, g = make_batch(lens, 6, 2, 128, 16, kind)
    q, begin, n = _queries(g, qlens, 6, 128)
    sick = torch.zeros(n, 6, dtype=torch.bool, device=DEV)
    sick[5, 1] = sick[41] = sick[17, 4] = True
    bad = q.clone()
    bad[5, 1, 7] = bad[41] = float("nan")
    bad[17, 4, 3] = float("inf")
    clean, clse = _run(pool, q, begin, bt, ctx, 0.1, {}, num_splits=splits)
    got, lse = _run(pool, bad, begin, bt, ctx, 0.1, {}, num_splits=splits)
    assert torch.isnan(got[:n][sick]).all() and torch.isnan(lse[:n][sick]).all()
    got[:n][sick], lse[:n][sick] = clean[:n][sick], clse[:n][sick]
    _check(pool, q, begin, bt, ctx, 0.1, n, got, lse)


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
@pytest.mark.parametrize("G", [3, 8])
def test_a_step_whose_query_is_not_a_number_gives_nan(kind, G):
    lens = [1500, 700, 1, 400]
    pool, bt, ctx, g = make_batch(lens, 2 * G, 2, 128, 16, kind)
    q = torch.randn(4, 2 * G, 128, generator=g, device=DEV).to(torch.bfloat16)
    sick = torch.zeros(4, 2 * G, dtype=torch.bool, device=DEV)
    sick[0, 1] = sick[1] = sick[2, 4] = True
    bad = q.clone()
    bad[0, 1, 7] = bad[1] = bad[2, 4, 3] = float("nan")
    doc = torch.tensor([0, 0, 0, 400], dtype=torch.int32, device=DEV)   # the last sees nothing
    bad[3] = float("nan")
    for splits in (1, 3):
        kw = dict(softcap=9.0, doc_begin=doc)
        clean = pa_decode_scored(pool, q, bt, ctx, 0.1, num_splits=splits, **kw)
        got = pa_decode_scored(pool, bad, bt, ctx, 0.1, num_splits=splits, **kw)
        assert torch.isnan(got[sick]).all() and torch.all(got[3] == 0)
        got[sick] = clean[sick]
        _check_step(pool, q, bt, ctx, 0.1, got, **kw)


@gpu
@pytest.mark.parametrize("kind,most", [("bf16", 1.5e-6), ("fp8", 1.5e-6), ("u8", 1.5e-6), ("u4", 5e-6)])
@pytest.mark.parametrize("D", [64, 128])
def test_long_contexts_keep_the_bits_of_their_weights(kind, most, D):
    """The scored step's error in the 2-norm at 30,000 keys in one split. Independent errors:
    a weight carries its score's (the sum of q.k, about 2e-7 rms) and the exponential's (2^-22 at
    most, 1.5e-7 rms); a block's 16 products are summed with 1.2e-7; the 235 sums of a warp's
    blocks, which grow as their square root, are added with roundings of 2^-24, together
    2^-24 sqrt(235 / 2) / sqrt(3) = 3.7e-7. In all 4.6e-7, a third of the bound. Weights cut to
    two bf16 operands alone are 2.4e-6 off, sums cut off toward zero in place 9e-6.
    INT4: a row's centre z + 8 s lies half a step (0.16 of the deviation) beside 0, so the sum of
    p z grows to 0.16 sqrt(30000) = 28 times the output; a lane's 120 additions of it round with
    2^-24 sqrt(120 / 3) of it at most, 1e-5 for one lane, which 64 lanes' independent signs make
    1.3e-6; the same again for the terms that it meets in O."""
    pool, bt, ctx, g = make_batch([30000, 12345], 8, 1, D, 32, kind, seed=2)
    q = torch.randn(2, 8, D, generator=g, device=DEV).to(torch.bfloat16)
    for cap in (0.0, 30.0):
        got = pa_decode_scored(pool, q, bt, ctx, D ** -0.5, softcap=cap, num_splits=1)
        want, _, _ = attend64(pool, q, [0, 1, 2], bt, ctx.tolist(), D ** -0.5, cap)
        rel = float((got.double() - want).norm() / want.norm())
        print(f"rel {rel:.2e}")
        assert rel <= most


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8"])
@pytest.mark.parametrize("scale,cap", [(1e-5, 50.0), (1e-8, 30.0), (1e-12, 30.0), (0.09, 1e6),
                                       (1e-3, 50.0)])
def test_caps_with_small_scales(kind, scale, cap):
    """Scores of ordinary size made of large products and a small scale (and a large cap): the
    short polynomial of the cap is left before one of its coefficients loses bits."""
    qlens, lens = [300, 40], [900, 640]
    amp = (0.1 * min(cap, 60.0) / (scale * 128 ** 0.5)) ** 0.5   # a tenth of the cap
    pool, bt, ctx, g = make_batch(lens, 4, 2, 128, 16, kind, amp=amp)
    q, begin, n = _queries(g, qlens, 4, 128, amp)
    got, lse = _run(pool, q, begin, bt, ctx, scale, {"softcap": cap}, num_splits=1)
    _check(pool, q, begin, bt, ctx, scale, n, got, lse, softcap=cap)


@gpu
@pytest.mark.parametrize("cap", [2.0 ** 125, 2.0 ** -126])
def test_largest_and_smallest_cap(cap):
    """The largest cap changes nothing, the smallest makes all scores equal; a query of zeros
    has scores of exactly 0 (whose product with an infinite factor would be NaN)."""
    lens = [500, 130]
    pool, bt, ctx, g = make_batch(lens, 4, 2, 128, 16, "bf16")
    q, begin, n = _queries(g, [40, 130], 4, 128)
    q[39, 1] = 0
    got, lse = _run(pool, q, begin, bt, ctx, 0.1, {"softcap": cap})
    as_if = 0.0 if cap > 1 else cap
    _check(pool, q, begin, bt, ctx, 0.1, n, got, lse, softcap=as_if)
    last = q[[39, 169]].contiguous()
    step = pa_decode_scored(pool, last, bt, ctx, 0.1, softcap=cap)
    _check_step(pool, last, bt, ctx, 0.1, step, softcap=as_if)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_466_b200 import build
    build.build()
    return _lib.load()


def test_caps_out_of_range_are_refused(lib):
    """softcap * log2(e) and its reciprocal have to be normal fp32 numbers (no call launches)."""
    pool = pa_kv_pool_t(num_pages=8, page_size=16, num_kv_heads=2, head_dim=128, dtype=0, k_pool=0x1000,
                        v_pool=0x2000, k_sz=None, v_sz=None)
    for cap, status in ((2.0 ** 125, PA_OK), (1.01 * 2.0 ** 125, PA_ERR_INVALID_ARG),
                        (2.5e38, PA_ERR_INVALID_ARG), (2.0 ** -126, PA_OK),
                        (0.99 * 2.0 ** -126, PA_ERR_INVALID_ARG), (1e-44, PA_ERR_INVALID_ARG),
                        (0.0, PA_OK), (50.0, PA_OK)):
        score = ctypes.byref(pa_score_t(cap, None, None, None))
        assert lib.pa_prefill(ctypes.byref(pool), score, None, 0, 4, None, 0, None, 4, None, 0.1, None,
                              None, None, 0, 1, None, None) == status
        assert lib.pa_decode_scored(ctypes.byref(pool), score, None, None, None, None, None, 0, 4, None, 4,
                                    None, 0.1, None, None, 0, 1, None, None) == status


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8"])
def test_a_workspace_for_the_largest_batch_serves_the_smaller_ones(kind):
    """The automatic split count rises as the batch shrinks: what the workspace cannot hold is
    not split, and nothing behind the given size is written."""
    pool, bt, ctx, g = make_batch([3000], 8, 2, 128, 16, kind)
    size = lambda n, s=0: pa_prefill_workspace_bytes(pool, n, 1, 8, bt.shape[1], s)
    q, begin, n = _queries(g, [4], 8, 128)
    N = q.shape[0]
    whole = size(N)
    assert size(3000) < whole                  # else there is nothing to lower here
    for given in (size(3000), 256, size(N, 2), size(N, 3) - 256, size(N, 5), whole):
        ws = torch.full((given + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        got, lse = _run(pool, q, begin, bt, ctx, 0.1, {}, workspace=ws[:given])
        _check(pool, q, begin, bt, ctx, 0.1, n, got, lse)
        assert torch.all(ws[given:] == 0x5A)
    with pytest.raises(pa.PagedAttnError):     # an explicit count is not lowered
        _run(pool, q, begin, bt, ctx, 0.1, {}, workspace=ws[:size(N, 2)], num_splits=3)


@gpu
def test_calls_on_a_stream_allocate_for_that_stream():
    """Only stream= is given, while the current stream is busy and then refills what it can get
    of the freed storage: outputs and workspaces of the calls must not meet either."""
    B, Hq, D = 3, 8, 128
    lens, qlens = [3000, 900, 17], [9, 4, 1]
    pool, bt, ctx, g = make_batch(lens, Hq, 2, D, 16, "bf16")
    q, begin, n = _queries(g, qlens, Hq, D)
    q = q[:n].contiguous()
    step = torch.randn(B, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    rope = Rope.from_base(4000, D, 10000.0, DEV)
    k, v = (torch.randn(n, 2, D, generator=g, device=DEV).to(torch.bfloat16) for _ in "kv")
    spare = KVPool(8, 2, 16, D, "bf16", DEV, fill_byte=0)
    seq = torch.zeros(n, dtype=torch.int32, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None].contiguous()

    def calls(stream):
        return (pa_prefill(pool, q, begin, bt, ctx, 0.09, num_splits=4, stream=stream),
                pa_decode_scored(pool, step, bt, ctx, 0.09, softcap=9.0, num_splits=4, stream=stream),
                pa_kv_append_rope(spare, rope, q, k, v, seq, pos, table, stream=stream),
                pa.pa_decode(pool, step, bt, ctx, 0.09, num_splits=4, stream=stream),
                pa.pa_decode_range(pool, step, bt, ctx, 0.09, 0, 3008, num_splits=4, stream=stream)[0])

    want = [t.clone() for t in calls(None)]
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for _ in range(5):
        busy = busy @ busy * 1e-3                     # the current stream is behind
        got = calls(side)
        for size in (1 << 12, 1 << 16, 1 << 20, 1 << 22):
            for _ in range(8):
                torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
        torch.cuda.current_stream().wait_stream(side)
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        del got, x


class Library:
    """A library whose every call succeeds: sizes are 4096, split counts 2."""

    def __getattr__(self, name):
        return lambda *a: (4096 if name.endswith("_bytes") else 2 if "splits" in name else 0)


def test_workspaces_elsewhere_are_refused(monkeypatch):
    """A workspace on another device than the pool, or with gaps, never reaches a kernel."""
    monkeypatch.setattr(_lib, "load", Library)
    monkeypatch.setattr(pa, "_need_device", lambda *a: None)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    pool = KVPool(2, 1, 16, 64, "bf16", "cpu")
    z = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    one, bt = i32(1), i32(0).view(1, 1)
    for ws in (torch.empty(4096, dtype=torch.uint8, device="meta"),
               torch.empty(8192, dtype=torch.uint8)[::2]):
        kw = dict(workspace=ws, stream=types.SimpleNamespace(cuda_stream=0))
        out = torch.zeros(1, 1, 64)
        for call in (lambda: pa_prefill(pool, z, i32(0, 1), bt, one, 0.1, out=z.clone(), **kw),
                     lambda: pa_decode_scored(pool, z, bt, one, 0.1, out=out, **kw),
                     lambda: pa.pa_decode(pool, z, bt, one, 0.1, out=out, **kw),
                     lambda: pa.pa_decode_append(pool, z, z, z, bt, one, 0.1, out=out, **kw),
                     lambda: pa.pa_decode_shared_prefix(pool, z, one, 16, bt, one, 0.1, out=out, **kw),
                     lambda: pa.pa_decode_window(pool, z, bt, one, 0.1, 1, 1, out=out, **kw),
                     lambda: pa.pa_decode_range(pool, z, bt, one, 0.1, 0, 1, o_out=out,
                                                lse_out=torch.zeros(1, 1), **kw)):
            with pytest.raises(ValueError, match="workspace"):
                call()


def test_storage_of_a_call_is_allocated_on_its_stream(monkeypatch):
    """Without a GPU: every tensor that a call with stream= makes is made with that stream as the
    current one, and its outputs are recorded on the caller's."""
    current, made, recorded = ["the current stream"], [], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def watched(make):
        def f(*a, **kw):
            made.append(current[-1])
            return make(*a, **kw)
        return f

    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    pool = KVPool(2, 1, 16, 64, "bf16", "cpu")
    rope = Rope(torch.zeros(4, 64))
    z = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    one, bt = i32(1), i32(0).view(1, 1)
    parts, lse = torch.zeros(2, 1, 1, 64), torch.zeros(2, 1, 1)
    packet = types.SimpleNamespace(shape=(1, 1, 1, 1), dev=z, host=z, nbytes=1)
    out_host = torch.zeros(1, 1, 64)
    monkeypatch.setattr(_lib, "load", Library)
    monkeypatch.setattr(_lib, "check", lambda *a: None)
    monkeypatch.setattr(pa, "_need_device", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append(s))
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, watched(getattr(torch, name)))
    monkeypatch.setattr(torch.Tensor, "new_empty", watched(torch.Tensor.new_empty))
    side = types.SimpleNamespace(cuda_stream=5)
    for call, outputs in (
            (lambda: pa_prefill(pool, z, i32(0, 1), bt, one, 0.1, stream=side), 1),
            (lambda: pa_decode_scored(pool, z, bt, one, 0.1, stream=side), 1),
            (lambda: pa_kv_append_rope(pool, rope, z, z, z, one, one, bt, stream=side), 1),
            (lambda: pa.pa_decode(pool, z, bt, one, 0.1, stream=side), 1),
            (lambda: pa.pa_decode_append(pool, z, z, z, bt, one, 0.1, stream=side), 1),
            (lambda: pa.pa_decode_shared_prefix(pool, z, one, 16, bt, one, 0.1, stream=side), 1),
            (lambda: pa.pa_decode_window(pool, z, bt, one, 0.1, 1, 1, stream=side), 1),
            (lambda: pa.pa_decode_range(pool, z, bt, one, 0.1, 0, 1, stream=side), 2),
            (lambda: pa.pa_decode_step_host(pool, packet, 0.1, out_host, stream=side), 1),
            (lambda: pa.pa_splitkv_reduce(parts[None, 0], lse[None, 0], stream=side), 1),
            (lambda: pa.pa_merge_partials(parts, lse, stream=side), 2)):
        made.clear()
        recorded.clear()
        call()
        assert made and all(s is side for s in made)
        assert recorded == ["the current stream"] * outputs
