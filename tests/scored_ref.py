"""Attention with changed scores in 64 bits, from the definition, over a paged
pool's contents (a loop over sequences and heads; torch only)."""
from __future__ import annotations

import math

import torch

from paged_kv_cache_466_b200 import KVPool, pa_kv_append
from tests.helpers import DEV


def pool_rows(pool, table_row, ctx, magnitudes=False):
    """K and V rows of tokens 0 .. ctx - 1, fp64 [ctx, Hkv, D] each; with `magnitudes` also, for
    K and V, |scale (code - shift)| and |zero + shift scale|, whose sum a quantised row is."""
    P = pool.page_size
    pages = table_row[:-(-ctx // P)].long()
    shift = {"bf16": 0, "fp8": 0, "u8": 128, "u4": 8}[pool.kind]
    out, mags = [], []
    for codes, sz in ((pool.k, pool.k_sz), (pool.v, pool.v_sz)):
        x = codes[pages]                                        # [n, Hkv, P, D or D / 2]
        if pool.kind == "u4":
            x = torch.stack([x & 15, x >> 4], -1).flatten(-2)
        if pool.kind == "fp8":
            x = x.view(torch.float8_e4m3fn)
        x = x.double()
        m = (x.abs(), torch.zeros_like(x))
        if sz is not None:
            s, z = sz[pages][..., :1].double(), sz[pages][..., 1:].double()
            m = ((s * (x - shift)).abs(), (z + shift * s).abs().expand_as(x))
            x = x * s + z
        flat = lambda t: t.transpose(1, 2).flatten(0, 1)[:ctx]
        out.append(flat(x))
        mags.append([flat(t) for t in m])
    return (*out, *mags) if magnitudes else out


def attend64(pool, q, q_begin, bt, ctx, scale, softcap=0.0, slopes=None, doc_begin=None,
             prefix_end=None, weighted=False):
    """(out [N, Hq, D], lse [N, Hq], largest |scale| sum |q k| over the visible pairs), fp64; the
    last tokens of sequence b are its query tokens q_begin[b] .. q_begin[b + 1]. With `weighted`
    also the softmax-weighted mean of |scale (code - shift)| of the values, [N, Hq, D]."""
    N, Hq, D = q.shape
    G = Hq // pool.num_kv_heads
    out = torch.zeros(N, Hq, D, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64, device=q.device)
    s_abs = 0.0
    for b in range(len(ctx)):
        i0, i1, c = int(q_begin[b]), int(q_begin[b + 1]), int(ctx[b])
        n = i1 - i0
        if n == 0 or c == 0:
            continue
        K, V, mk, mv = pool_rows(pool, bt[b], c, magnitudes=True)
        mk = mk[0] + mk[1]
        j = torch.arange(c, device=q.device)
        pos = c - n + torch.arange(n, device=q.device)[:, None]
        see = j <= pos
        if prefix_end is not None:
            see = see | (j < prefix_end[i0:i1].long()[:, None])
        if doc_begin is not None:
            see = see & (j >= doc_begin[i0:i1].long()[:, None])
        for h in range(Hq):
            qh = q[i0:i1, h].double()
            x = qh @ K[:, h // G].T * scale
            if see.any():
                s_abs = max(s_abs, float((qh.abs() @ mk[:, h // G].T)[see].max()) * abs(scale))
            if softcap:
                x = softcap * torch.tanh(x / softcap)
            if slopes is not None:
                x = x - slopes[h].double() * (pos - j).abs()
            x = x.masked_fill(~see, -math.inf)
            lse[i0:i1, h] = torch.logsumexp(x, -1)
            p = torch.where(see.any(-1, keepdim=True), torch.softmax(x, -1), torch.zeros_like(x))
            p = torch.where(p > 0, p, torch.zeros_like(p))
            out[i0:i1, h] = p @ V[:, h // G]
            mag[i0:i1, h] = p @ mv[0][:, h // G]
    return (out, lse, s_abs, mag) if weighted else (out, lse, s_abs)


def make_batch(ctx, Hq, Hkv, D, P, kind, seed=0, slack=3, max_pages=None, amp=1.0):
    """A pool holding random rows for sequences of the given lengths, its tables, a generator."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-c // P) for c in ctx]
    pool = KVPool(sum(need) + slack, Hkv, P, D, kind, DEV, fill_byte=0x7F)  # NaN where nothing is stored
    ids = torch.randperm(pool.num_pages, generator=g, device=DEV).to(torch.int32)
    bt = torch.full((len(ctx), max_pages or max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    counts = torch.tensor(ctx)
    n = int(counts.sum())
    if n:
        seq = torch.repeat_interleave(torch.arange(len(ctx)), counts)
        pos = torch.arange(n) - (counts.cumsum(0) - counts)[seq]
        rows = lambda: (torch.randn(n, Hkv, D, generator=g, device=DEV) * amp).to(torch.bfloat16)
        pa_kv_append(pool, rows(), rows(), seq.to(DEV, torch.int32), pos.to(DEV, torch.int32), bt)
    return pool, bt, torch.tensor(ctx, dtype=torch.int32, device=DEV), g


def slopes_for(Hq):
    return 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32) / Hq)
