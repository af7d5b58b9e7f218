"""pa_kv_append_rope: the rotation against its formula in 64 bits and, bit for
bit, against rotating first and calling pa_kv_append; positions on several
axes, strides, in-place rotation, bad tokens, refusals.

Tolerance of the rotated queries: one bf16 rounding (half a step, 2^-8 of the
value) plus the fp32 roundings of two products and their sum, each half a step
(2^-24) of terms bounded by |a| + |b|: 2^-8 |x'| + 3 * 2^-24 (|a| + |b|), and
the bf16 step of what those add: a factor 1.01 covers both.
"""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_466_b200 import (PA_DERR_BAD_PAGE, PA_DERR_BAD_POS, PA_DERR_BAD_SEQ, KVPool,
                                     Rope, _lib, pa_kv_append, pa_kv_append_rope)
from paged_kv_cache_466_b200._lib import (PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_OK, pa_kv_pool_t,
                                          pa_rope_t)
from tests.helpers import DEV

gpu = pytest.mark.gpu


def _split(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _join(x, a, b, rot, interleaved):
    y = x.clone()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a, b
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a, b
    return y


def rotate(x, table, rope_pos, axes, interleaved, dtype):
    """x [N, H, D] rotated in `dtype`, unrounded; also |a| + |b| per element."""
    rot = table.shape[1]
    j = torch.arange(rot // 2, device=x.device)
    at = rope_pos[torch.tensor(axes, device=x.device)].long().T
    c, s = table[at, j].to(dtype)[:, None], table[at, rot // 2 + j].to(dtype)[:, None]
    x = x.to(dtype)
    a, b = _split(x, rot, interleaved)
    y = _join(x, a * c - b * s, b * c + a * s, rot, interleaved)
    m = _join(x * 0, a.abs() + b.abs(), a.abs() + b.abs(), rot, interleaved)
    return y, m


def _batch(N, Hq, Hkv, D, P, kind, rot, interleaved=False, axes=1, seed=0, B=3, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *sh: (torch.randn(*sh, generator=g, device=DEV) * scale).to(torch.bfloat16)
    max_pages = -(-(N + 5) // P)
    pool = KVPool(B * max_pages + 2, Hkv, P, D, kind, DEV, fill_byte=0x5A)
    bt = torch.randperm(pool.num_pages, generator=g, device=DEV)[:B * max_pages]
    bt = bt.to(torch.int32).view(B, max_pages).contiguous()
    slots = torch.randperm(B * max_pages * P, generator=g, device=DEV)[:N]  # no slot twice
    seq, pos = (slots // (max_pages * P)).to(torch.int32), (slots % (max_pages * P)).to(torch.int32)
    table_len = max_pages * P + 7
    t = 3 if axes > 1 else 1
    axis_of_pair = ([0] * (rot // 2) if axes == 1 else
                    [(j * 3) // (rot // 2) for j in range(rot // 2)] if axes == 3 else
                    [j % 3 for j in range(rot // 2)])                       # axes == 4: alternating
    rope = Rope.from_base(table_len, rot, 10000.0, DEV, interleaved=interleaved,
                          axis_of_pair=axis_of_pair)
    rp = pos[None].clone() if t == 1 else torch.randint(0, table_len, (3, N), generator=g,
                                                        device=DEV, dtype=torch.int32)
    return pool, rope, randn(N, Hq, D), randn(N, Hkv, D), randn(N, Hkv, D), seq, pos, bt, rp.contiguous()


def _check(pool, rope, q, k, v, seq, pos, bt, rp, got):
    axes = list(rope.c.axis_of_pair)[:rope.table.shape[1] // 2]
    want, mag = rotate(q, rope.table, rp, axes, rope.interleaved, torch.float64)
    tol = 1.01 * (want.abs() * 2.0 ** -8 + 3 * 2.0 ** -24 * mag)
    assert torch.all((got.double() - want).abs() <= tol)
    # bit for bit: rotate in fp32, operation by operation, then the plain cache write
    k32, _ = rotate(k, rope.table, rp, axes, rope.interleaved, torch.float32)
    other = KVPool(pool.num_pages, pool.num_kv_heads, pool.page_size, pool.head_dim, pool.kind, DEV,
                   fill_byte=0x5A)
    pa_kv_append(other, k32.to(torch.bfloat16).contiguous(), v.contiguous(), seq, pos, bt)
    for mine, ref in zip(pool.tensors(), other.tensors()):
        assert torch.equal(mine.view(torch.uint8), ref.view(torch.uint8))


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u8", "fp8", "u4"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 16), (64, 64), (64, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_and_cache_bits(kind, D, rot, interleaved):
    b = _batch(37, 6, 2, D, 16, kind, rot, interleaved)
    got = pa_kv_append_rope(b[0], *b[1:8], rope_pos=b[8])
    _check(*b, got)


@gpu
@pytest.mark.parametrize("N,Hq,Hkv,P", [(1, 1, 1, 16), (1, 64, 8, 32), (2, 7, 7, 16), (700, 32, 8, 16),
                                        (5000, 5, 5, 32), (3, 40, 33, 16)])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_sizes(N, Hq, Hkv, P, kind):
    b = _batch(N, Hq, Hkv, 128, P, kind, 128, seed=N)
    _check(*b, pa_kv_append_rope(b[0], *b[1:8]))


@gpu
@pytest.mark.parametrize("axes", [3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 48)])
def test_positions_on_three_axes(axes, interleaved, D, rot):
    """Blocks of pairs per axis (block borders inside a thread's eight pairs
    included) and axes alternating pair by pair."""
    b = _batch(61, 4, 2, D, 16, "bf16", rot, interleaved, axes=axes, seed=axes)
    _check(*b, pa_kv_append_rope(b[0], *b[1:8], rope_pos=b[8]))


@gpu
@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_extreme_magnitudes(scale):
    b = _batch(29, 4, 2, 128, 16, "bf16", 128, scale=scale)
    _check(*b, pa_kv_append_rope(b[0], *b[1:8]))


@gpu
@pytest.mark.parametrize("kind", ["u8", "fp8", "u4"])
@pytest.mark.parametrize("span", [0, 18, 30, 60, 62, 100])
def test_quantiser_bits_over_the_range_of_scales(kind, span):
    """60,000 rows of every spread of magnitudes, 2^-span .. 2^span: each quotient by the row's
    scale rounds as the division does, on both sides of where the quick form is left."""
    b = _batch(7500, 1, 4, 64, 32, kind, 16, seed=span)
    pool, rope, q, k, v, seq, pos, bt, rp = b
    g = torch.Generator(device=DEV).manual_seed(span)
    e = (torch.rand(7500, 4, 1, generator=g, device=DEV) * 2 - 1) * span
    k = (k.float() * torch.exp2(e)).to(torch.bfloat16)
    v = (v.float() * torch.exp2(-e)).to(torch.bfloat16)
    got = pa_kv_append_rope(pool, rope, q, k, v, seq, pos, bt)
    _check(pool, rope, q, k, v, seq, pos, bt, rp, got)


@gpu
def test_slices_of_a_fused_projection_and_in_place():
    pool, rope, q, k, v, seq, pos, bt, rp = _batch(53, 8, 2, 128, 16, "bf16", 128)
    qkv = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).contiguous()
    qs = qkv[:, :8 * 128].view(53, 8, 128)
    ks = qkv[:, 8 * 128:10 * 128].view(53, 2, 128)
    vs = qkv[:, 10 * 128:].view(53, 2, 128)
    got = pa_kv_append_rope(pool, rope, qs, ks, vs, seq, pos, bt)
    _check(pool, rope, q, k, v, seq, pos, bt, rp, got)
    mine = q.clone()
    again = pa_kv_append_rope(pool, rope, mine, k, v, seq, pos, bt, q_out=mine)
    assert again is mine and torch.equal(mine.view(torch.int16), got.view(torch.int16))
    with pytest.raises(Exception):
        pa_kv_append_rope(pool, rope, qs, ks, vs, seq, pos, bt, q_out=qs)   # not dense


@gpu
def test_keys_only_and_empty():
    b = _batch(20, 4, 2, 64, 16, "u8", 64)
    pool, rope, q, k, v, seq, pos, bt, rp = b
    assert pa_kv_append_rope(pool, rope, None, k, v, seq, pos, bt) is None
    _check(*b, rotate(q, rope.table, rp, [0] * 32, False, torch.float64)[0].to(torch.bfloat16))
    before = [t.clone() for t in pool.tensors()]
    none = pa_kv_append_rope(pool, rope, q[:0], k[:0], v[:0], seq[:0], pos[:0], bt)
    assert none.shape == (0, 4, 64)
    for x, y in zip(before, pool.tensors()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@gpu
@pytest.mark.parametrize("kind", ["bf16", "u4"])
def test_bad_tokens_are_flagged_and_not_stored(kind):
    pool, rope, q, k, v, seq, pos, bt, rp = _batch(6, 4, 2, 128, 16, kind, 128)
    before = [t.clone() for t in pool.tensors()]
    seq = torch.tensor([-1, 3, 0, 1, 2, 2], dtype=torch.int32, device=DEV)
    pos = torch.tensor([0, 0, 100_000, 3, 1, 2], dtype=torch.int32, device=DEV)
    bt = bt.clone()
    bt[1, 0] = pool.num_pages
    rp = torch.tensor([[1, 2, 3, 4, -1, rope.table.shape[0]]], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 9.0)
    pa_kv_append_rope(pool, rope, q, k, v, seq, pos, bt, rope_pos=rp, q_out=out, d_err=err)
    assert int(err.item()) == PA_DERR_BAD_SEQ | PA_DERR_BAD_POS | PA_DERR_BAD_PAGE
    for x, y in zip(before, pool.tensors()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # the first four queries are rotated, the two without an angle are left as they were
    want, mag = rotate(q[:4], rope.table, rp[:, :4], [0] * 64, False, torch.float64)
    tol = 1.01 * (want.abs() * 2.0 ** -8 + 3 * 2.0 ** -24 * mag)
    assert torch.all((out[:4].double() - want).abs() <= tol)
    assert torch.all(out[4:] == 9.0)


@gpu
def test_replayed_in_a_graph_and_on_another_stream():
    b = _batch(33, 4, 2, 128, 16, "fp8", 128)
    pool, rope, q, k, v, seq, pos, bt, rp = b
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pa_kv_append_rope(pool, rope, q, k, v, seq, pos, bt, q_out=out)
    q.copy_(torch.randn_like(q))
    k.mul_(0.5)
    graph.replay()
    _check(pool, rope, q, k, v, seq, pos, bt, rp, out)


# ---- refusals, without a GPU -------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_466_b200 import build
    build.build()
    return _lib.load()


def _c_rope(**kw):
    axes = kw.pop("axes", [0] * 64)
    d = dict(table=0x1000, table_len=10, rotary_dim=128, interleaved=0, num_axes=1)
    d.update(kw)
    return pa_rope_t(d["table"], d["table_len"], d["rotary_dim"], d["interleaved"], d["num_axes"],
                     (ctypes.c_uint8 * 64)(*axes))


def _call(lib, rope="default", D=128, q=0x1000, q_stride=512, hq=4, q_out=0x2000, k=0x3000, ks=256, v=0x4000,
          vs=256, n=2, max_pages=4, seq=0x5000):
    pool = pa_kv_pool_t(num_pages=8, page_size=16, num_kv_heads=2, head_dim=D, dtype=0, k_pool=0x1000,
                        v_pool=0x2000, k_sz=None, v_sz=None)
    rope = _c_rope() if rope == "default" else rope
    return lib.pa_kv_append_rope(ctypes.byref(pool), None if rope is None else ctypes.byref(rope), q,
                                 q_stride, hq, q_out, k, ks, v, vs, seq, 0x6000, None, n, 0x7000, 2,
                                 max_pages, None, None)


def test_refusals(lib):
    assert _call(lib, n=0) == PA_OK
    assert _call(lib, rope=None) == PA_ERR_INVALID_ARG
    assert _call(lib, rope=_c_rope(table=None)) == PA_ERR_INVALID_ARG
    assert _call(lib, rope=_c_rope(table=0x1008)) == PA_ERR_INVALID_ARG
    assert _call(lib, rope=_c_rope(table_len=0)) == PA_ERR_INVALID_ARG
    for rot in (0, -16, 24, 144):
        assert _call(lib, rope=_c_rope(rotary_dim=rot)) == PA_ERR_UNSUPPORTED
    assert _call(lib, D=64) == PA_ERR_UNSUPPORTED                      # rotary_dim 128 of 64
    for n in (0, 5):
        assert _call(lib, rope=_c_rope(num_axes=n)) == PA_ERR_UNSUPPORTED
    assert _call(lib, rope=_c_rope(axes=[0] * 63 + [1])) == PA_ERR_INVALID_ARG
    assert _call(lib, n=-1) == PA_ERR_INVALID_ARG
    assert _call(lib, hq=-1) == PA_ERR_INVALID_ARG
    assert _call(lib, max_pages=0) == PA_ERR_INVALID_ARG
    assert _call(lib, q=None) == PA_ERR_INVALID_ARG
    assert _call(lib, q_out=None) == PA_ERR_INVALID_ARG
    assert _call(lib, k=None) == PA_ERR_INVALID_ARG
    assert _call(lib, seq=None) == PA_ERR_INVALID_ARG
    assert _call(lib, q=0x1002) == PA_ERR_INVALID_ARG
    assert _call(lib, q_stride=504) == PA_ERR_INVALID_ARG              # under one row
    assert _call(lib, q_stride=516) == PA_ERR_INVALID_ARG              # not a multiple of 8
    assert _call(lib, ks=248) == PA_ERR_INVALID_ARG
    assert _call(lib, vs=260) == PA_ERR_INVALID_ARG
    assert _call(lib, q_out=0x1000, q_stride=1024) == PA_ERR_INVALID_ARG  # in place, not dense


def test_rope_arguments_are_checked():
    t = torch.zeros(4, 64)
    assert Rope(t).num_axes == 1
    assert Rope(t, axis_of_pair=[0] * 8 + [1] * 12 + [2] * 12).num_axes == 3
    for bad in (dict(axis_of_pair=[0] * 31), dict(axis_of_pair=[4] * 32), dict(axis_of_pair=[-1] * 32)):
        with pytest.raises(ValueError):
            Rope(t, **bad)
    with pytest.raises(TypeError):
        Rope(t.double())
    with pytest.raises(ValueError):
        Rope(torch.zeros(4, 256))
    with pytest.raises(ValueError):
        Rope(t.T)
    got = Rope.from_base(100, 64, 500.0, "cpu").table
    ang = np.arange(100)[:, None] * 500.0 ** (-np.arange(0, 64, 2) / 64)
    np.testing.assert_allclose(got[:, :32].numpy(), np.cos(ang), atol=2.0 ** -23)
    np.testing.assert_allclose(got[:, 32:].numpy(), np.sin(ang), atol=2.0 ** -23)
    cpu_pool = KVPool(2, 1, 16, 64, "bf16", "cpu")
    z, i = torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa_kv_append_rope(cpu_pool, Rope(t), z, z, z, i, i, i.view(1, 1))
