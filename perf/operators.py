"""The serving operators around the paged cache, as cases to measure.

* ``append``  rotary positions applied to the queries and keys of new tokens, the
              rotated keys and the values written into their cache pages
* ``prefill`` attention of the new tokens of a ragged batch over the paged cache,
              with capped scores, a distance bias, document and prefix masks
* ``decode``  the same scores for one token per sequence, with the rotation and
              the cache write of that token in the same call

``run`` computes them in elementary torch operations (fp32, rounded once at the
end) or, where ``own`` is true, by this repository's entry points. Shapes are
those of the repository's own workloads: tiny (4/2 heads of 64), the
Llama-3-8B-shaped layer (32/8 heads of 128, pages of 16) and the
Llama-3-70B-shaped one (64/8 heads of 128, pages of 32).
"""
import math

import torch

own = False

DEV = "cuda"
ROPE_BASE = 500000.0


def listed():
    return [
        # one decode step of eight sequences of the 70B-shaped layer: launch latency
        _append("rotate step", B=8, new=1, past=8191, Hq=64, Hkv=8, D=128, P=32, kind="bf16", rot=128),
        # a whole prompt of the 8B-shaped layer, q/k/v still side by side in the projection's output
        _append("rotate prompt", B=1, new=8192, past=0, Hq=32, Hkv=8, D=128, P=16, kind="bf16", rot=128),
        # image tokens placed on three axes (time, height, width), FP8 cache
        _append("rotate images fp8", B=3, new=5477, past=211, Hq=64, Hkv=8, D=128, P=16, kind="fp8",
                rot=128, axes=3, ragged=True),
        # many short ragged chunks, small heads of which half is rotated, neighbouring elements paired
        _append("rotate ragged partial", B=29, new=701, past=300, Hq=8, Hkv=4, D=64, P=32, kind="bf16",
                rot=32, interleaved=True, ragged=True),
        # a few short prompts of the tiny layer: launch latency
        _prefill("prefill tiny", B=3, new=33, past=64, Hq=4, Hkv=2, D=64, P=16, kind="bf16", ragged=True),
        # one long prompt of the 8B-shaped layer with capped scores
        _prefill("prefill prompt capped", B=1, new=8192, past=0, Hq=32, Hkv=8, D=128, P=16, kind="bf16",
                 softcap=50.0),
        # packed documents, each with a beginning that all of its tokens see
        _prefill("prefill documents", B=4, new=4099, past=0, Hq=32, Hkv=8, D=128, P=16, kind="bf16",
                 doc=1500, prefix=257, ragged=True),
        # chunked prefill deep into long contexts, distance bias, FP8 cache
        _prefill("prefill chunk biased fp8", B=2, new=512, past=32000, Hq=64, Hkv=8, D=128, P=32,
                 kind="fp8", alibi=True),
        # a handful of draft tokens per sequence checked against long contexts, INT8 cache
        _prefill("prefill drafts int8", B=4, new=5, past=16001, Hq=32, Hkv=8, D=128, P=16, kind="u8"),
        # one short sequence: launch latency of the fused step
        _decode("decode one", B=1, ctx=100, Hq=32, Hkv=8, D=128, P=16, kind="bf16", rot=128, append=True),
        # the 70B-shaped long-context step, capped, with rotation and cache write
        _decode("decode long capped", B=32, ctx=8192, Hq=64, Hkv=8, D=128, P=32, kind="bf16", rot=128,
                append=True, softcap=30.0),
        # ragged batch over an INT8 cache, distance bias, only the current document visible
        _decode("decode ragged biased int8", B=64, ctx=4095, Hq=32, Hkv=8, D=128, P=16, kind="u8",
                alibi=True, doc=3001, ragged=True),
    ]


def _append(name, *, B, new, past, Hq, Hkv, D, P, kind, rot, axes=1, interleaved=False, ragged=False):
    return dict(name=name, op="append", B=B, new=new, past=past, Hq=Hq, Hkv=Hkv, D=D, P=P, kind=kind,
                rot=rot, axes=axes, interleaved=interleaved, ragged=ragged)


def _prefill(name, *, B, new, past, Hq, Hkv, D, P, kind, softcap=0.0, alibi=False, doc=0, prefix=0,
             ragged=False):
    return dict(name=name, op="prefill", B=B, new=new, past=past, Hq=Hq, Hkv=Hkv, D=D, P=P, kind=kind,
                softcap=softcap, alibi=alibi, doc=doc, prefix=prefix, ragged=ragged)


def _decode(name, *, B, ctx, Hq, Hkv, D, P, kind, rot=0, append=False, softcap=0.0, alibi=False, doc=0,
            ragged=False):
    return dict(name=name, op="decode", B=B, new=1, past=ctx - 1, Hq=Hq, Hkv=Hkv, D=D, P=P, kind=kind,
                rot=rot, append=append, softcap=softcap, alibi=alibi, doc=doc, ragged=ragged)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "prefill", "decode"])
    D = rng.choice([64, 128, 128])
    P = rng.choice([16, 32])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.randint(1, 8)
    ragged = rng.random() < 0.7
    if op == "append":
        kind = rng.choice(["bf16", "fp8"])
        B = log(1, 64)
        new = max(1, min(log(1, 8192), 16384 // B))
        axes = rng.choice([1, 3])
        rot = rng.choice([r for r in (32, 64, 128) if r <= D])
        c = _append("", B=B, new=new, past=log(1, 8192) - 1, Hq=Hq, Hkv=Hkv, D=D, P=P, kind=kind, rot=rot,
                    axes=axes, interleaved=rng.random() < 0.4, ragged=ragged)
    elif op == "prefill":
        kind = rng.choice(["bf16", "bf16", "fp8", "u8", "u4"])
        B = log(1, 8)
        past = log(1, 32000) - 1
        # at most the scores of the long prompt
        new = max(1, min(log(1, 8192), 60_000_000 // (B * (past + 8192)), 16384 // B))
        doc = rng.choice([0, 0, log(100, 6000)])
        c = _prefill("", B=B, new=new, past=past, Hq=min(Hq, 32) // Hkv * Hkv, Hkv=Hkv, D=D, P=P, kind=kind,
                     softcap=rng.choice([0.0, 30.0, 50.0]), alibi=rng.random() < 0.3, doc=doc,
                     prefix=rng.choice([0, 0, log(1, 600)]), ragged=ragged)
    else:
        kind = rng.choice(["bf16", "fp8", "u8", "u4"])
        B = log(1, 128)
        ctx = max(1, min(log(1, 32000), 262144 // B))
        append = kind in ("bf16", "fp8") and rng.random() < 0.6
        rot = rng.choice([r for r in (32, 64, 128) if r <= D]) if append or rng.random() < 0.5 else 0
        c = _decode("", B=B, ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, P=P, kind=kind, rot=rot, append=append,
                    softcap=rng.choice([0.0, 30.0, 50.0]), alibi=rng.random() < 0.3,
                    doc=rng.choice([0, 0, log(100, 6000)]), ragged=ragged)
    del c["name"]
    return c


# ---- lengths: whole numbers that follow from the case alone ----------------------


def _lens(case):
    """(new tokens, cached tokens before them) of every sequence."""
    B, new, past = case["B"], case["new"], case["past"]
    if not case["ragged"]:
        return [new] * B, [past] * B
    frac = [((b + 1) * 0.6180339887498949) % 1.0 for b in range(B)]
    frac2 = [((b + 1) * 0.7548776662466927) % 1.0 for b in range(B)]
    return ([max(1, new - int(f * 0.9 * new)) for f in frac],
            [past - int(f * 0.9 * past) for f in frac2])


def _doc_begin(case, pos):
    return pos // case["doc"] * case["doc"] if case["doc"] else pos * 0


def _visible(case):
    """Visible (query token, key) pairs, and keys visible to any query token, over the batch."""
    new, past = (torch.tensor(x) for x in _lens(case))
    seq = torch.repeat_interleave(torch.arange(len(new)), new)
    pos = torch.arange(len(seq)) - (new.cumsum(0) - new)[seq] + past[seq]
    lo = _doc_begin(case, pos)
    hi = pos + 1
    if case.get("prefix"):
        hi = torch.minimum(torch.maximum(hi, lo + case["prefix"]), (new + past)[seq])
    first = torch.full_like(new, 1 << 40).scatter_reduce(0, seq, lo, "amin")
    last = torch.zeros_like(new).scatter_reduce(0, seq, hi, "amax")
    return int((hi - lo).sum()), int((last - first).sum())


def _row_bytes(case):
    """Bytes of one cached row (one token, one KV head, K or V)."""
    D = case["D"]
    return {"bf16": 2 * D, "fp8": D + 8, "u8": D + 8, "u4": D // 2 + 8}[case["kind"]]


def work(case):
    new, past = _lens(case)
    N = sum(new)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        rows = N * (Hq + 2 * Hkv) * D * 2 + N * case["rot"] * 4  # q, k, v and the angles
        return {"bytes": rows + N * Hq * D * 2 + N * Hkv * 2 * _row_bytes(case),
                "flops": 3 * N * (Hq + Hkv) * case["rot"]}
    pairs, keys = _visible(case)
    w = {"bytes": keys * Hkv * 2 * _row_bytes(case), "flops": 4 * D * Hq * pairs}
    if case["op"] == "prefill":
        w["bytes"] += N * Hq * D * (2 + 2)
    else:
        w["bytes"] += N * Hq * D * (2 + 4)
        if case["append"]:
            w["bytes"] += N * Hkv * 2 * (2 * D + _row_bytes(case))
    return w


# ---- inputs -----------------------------------------------------------------------


def _quantise(x, kind):
    """(codes as stored, (scale, zero)) of rows x [..., D] fp32; the cache's per-row formats."""
    x = x + 0.0  # -0 is stored as +0
    if kind == "fp8":
        s = x.abs().amax(-1, keepdim=True)
        s = s / torch.full_like(s, 448.0)  # a quotient: by a plain number torch multiplies by its inverse
        y = torch.where(s == 0, torch.zeros_like(x), x / torch.where(s == 0, torch.ones_like(s), s))
        codes = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        return codes, torch.cat([s, torch.zeros_like(s)], -1)
    top = 255.0 if kind == "u8" else 15.0
    z = x.amin(-1, keepdim=True)
    s = (x.amax(-1, keepdim=True) - z) / torch.full_like(z, top)
    c = torch.round((x - z) / torch.where(s == 0, torch.ones_like(s), s)).clamp(0.0, top)
    c = torch.where(s == 0, torch.zeros_like(c), c).to(torch.uint8)
    if kind == "u4":
        c = c[..., 0::2] | (c[..., 1::2] << 4)
    return c.contiguous(), torch.cat([s, z], -1)


def _dequantise(codes, sz, kind, dtype):
    """The rows that the codes [..., D] stand for."""
    if kind == "bf16":
        return codes.to(dtype)
    if kind == "fp8":
        return codes.view(torch.float8_e4m3fn).to(dtype) * sz[..., :1].to(dtype)
    if kind == "u4":
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return codes.to(dtype) * sz[..., :1].to(dtype) + sz[..., 1:].to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)

    B, Hq, Hkv, D, P, kind = (case[k] for k in ("B", "Hq", "Hkv", "D", "P", "kind"))
    new, past = _lens(case)
    N = sum(new)
    pages = [-(-(n + p) // P) for n, p in zip(new, past)]
    num_pages = sum(pages) + 3
    st = dict(case=case, N=N, scale=1.0 / math.sqrt(D))
    # the page pool, already holding the cached tokens (and arbitrary rows elsewhere)
    for t in ("k", "v"):
        rows = randn(num_pages, Hkv, P, D)
        if kind == "bf16":
            st[t], st[t + "_sz"] = rows, None
        else:
            st[t], st[t + "_sz"] = _quantise(rows.float(), kind)
        del rows
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    bt = torch.full((B, max(pages)), -1, dtype=torch.int32)
    at = 0
    perm_h = perm.cpu()
    for b, n in enumerate(pages):
        bt[b, :n] = perm_h[at:at + n]
        at += n
    st["block_tables"] = bt.to(DEV)
    # new tokens: sequence, position, and where each sequence's tokens begin
    counts = torch.tensor(new)
    seq = torch.repeat_interleave(torch.arange(B), counts)
    begin = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    pos = torch.arange(N) - begin[seq] + torch.tensor(past)[seq]
    ctx = counts + torch.tensor(past)

    def ints(t):
        return t.to(torch.int32).to(DEV)

    st.update(seq_idx=ints(seq), pos=ints(pos), q_begin=ints(begin), context_lens=ints(ctx),
              max_new=max(new))
    # q, k and v as the projection leaves them: side by side in one row per token
    qkv = randn(N, (Hq + 2 * Hkv) * D)
    st["q"] = qkv[:, :Hq * D].view(N, Hq, D)
    st["k_new"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(N, Hkv, D)
    st["v_new"] = qkv[:, (Hq + Hkv) * D:].view(N, Hkv, D)
    if case["op"] != "append":
        st["q"], st["k_new"], st["v_new"] = (st[k].contiguous() for k in ("q", "k_new", "v_new"))
    rot = case.get("rot", 0)
    if rot:
        # angles in 64 bits, rounded once: row p is cos then sin of p / base^(2 j / rot)
        inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        ang = torch.arange(int(ctx.max()) + 8, dtype=torch.float64, device=DEV)[:, None] * inv
        st["table"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        axes = case.get("axes", 1)
        st["axis_of_pair"] = [0] * (rot // 2)
        st["rope_pos"] = st["pos"][None].contiguous()
        if axes == 3:
            # a quarter of the pairs follow time, the others height and width; the
            # tokens are pictures of 37 columns, one after another
            t = rot // 8
            hw = (rot // 2 - t) // 2
            st["axis_of_pair"] = [0] * t + [1] * hw + [2] * (rot // 2 - t - hw)
            grid = torch.stack([pos // 1369, pos % 1369 // 37, pos % 37])
            st["rope_pos"] = ints(grid + torch.tensor(past)[seq] // 64)
    st["slopes"] = None
    if case.get("alibi"):
        st["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=DEV, dtype=torch.float32) / Hq)
    st["doc_begin"] = st["prefix_end"] = None
    if case.get("doc"):
        st["doc_begin"] = ints(_doc_begin(case, pos))
    if case.get("prefix"):
        st["prefix_end"] = ints(_doc_begin(case, pos) + case["prefix"])
    if own:
        _handles(st)
    return st


# ---- the plain forms ----------------------------------------------------------------


def _rotate(x, table, rope_pos, axis_of_pair, interleaved, dtype=torch.float32):
    """x [N, H, D] with its first rot elements rotated, in `dtype`, not rounded further."""
    half = table.shape[1] // 2
    axis = torch.tensor(axis_of_pair, device=x.device)
    at = rope_pos[axis].long().T                                # [N, half]: the row of each pair
    j = torch.arange(half, device=x.device)
    c, s = table[at, j].to(dtype)[:, None], table[at, half + j].to(dtype)[:, None]
    x = x.to(dtype)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


def _write(st, k, v):
    """k, v [N, Hkv, D] bf16 into the page slots of the new tokens."""
    P, kind = st["case"]["P"], st["case"]["kind"]
    pos = st["pos"].long()
    page = st["block_tables"][st["seq_idx"].long(), pos // P].long()
    for t, rows in (("k", k), ("v", v)):
        if kind == "bf16":
            st[t][page, :, pos % P] = rows
        else:
            codes, sz = _quantise(rows.float(), kind)
            st[t][page, :, pos % P] = codes
            st[t + "_sz"][page, :, pos % P] = sz


def _cache(st):
    """The cache as outputs: FP8 codes as the numbers that they are, beside their scales."""
    if st["case"]["kind"] == "bf16":
        return {"k": st["k"], "v": st["v"]}
    return {"k": st["k"].view(torch.float8_e4m3fn), "v": st["v"].view(torch.float8_e4m3fn),
            "k_sz": st["k_sz"], "v_sz": st["v_sz"]}


def _rope_args(st):
    return st["table"], st["rope_pos"], st["axis_of_pair"], st["case"].get("interleaved", False)


def _attend(st, q, dtype=torch.float32):
    """Attention of q [N, Hq, D] over the paged cache: [N, Hq, D] in `dtype`. Sequences are
    padded to the longest: query slot l of sequence b is token q_begin[b] + l."""
    case = st["case"]
    B, Hq, Hkv, D, P = (case[k] for k in ("B", "Hq", "Hkv", "D", "P"))
    G, L, T = Hq // Hkv, st["max_new"], st["block_tables"].shape[1] * P
    begin, ctx = st["q_begin"].long(), st["context_lens"].long()
    slot = torch.arange(L, device=q.device)[None]
    live = slot < (begin[1:] - begin[:-1])[:, None]                         # [B, L]
    tok = torch.where(live, begin[:-1, None] + slot, torch.zeros_like(slot))
    pages = st["block_tables"].long().clamp_min(0)

    def gather(t):                                                        # [B, Hkv, T, D]
        sz = st[t + "_sz"]
        rows = _dequantise(st[t][pages], None if sz is None else sz[pages], case["kind"], dtype)
        return rows.transpose(1, 2).reshape(B, Hkv, T, D)

    qp = q.to(dtype)[tok].view(B, L, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * L, D)
    x = torch.matmul(qp, gather("k").transpose(2, 3)).view(B, Hkv, G, L, T)
    x *= st["scale"]
    if case["softcap"]:
        x /= case["softcap"]
        x.tanh_().mul_(case["softcap"])
    j = torch.arange(T, device=q.device)
    pos = st["pos"].long()[tok]                                             # [B, L]
    if st["slopes"] is not None:
        dist = (pos[..., None] - j).abs().to(dtype)[:, None, None]
        x -= st["slopes"].to(dtype).view(1, Hkv, G, 1, 1) * dist
    hi = pos + 1
    if st["prefix_end"] is not None:
        hi = torch.maximum(hi, st["prefix_end"].long()[tok])
    see = (j < torch.minimum(hi, ctx[:, None])[..., None]) & live[..., None]
    if st["doc_begin"] is not None:
        see &= j >= st["doc_begin"].long()[tok][..., None]
    x.masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x -= torch.where(top == -math.inf, torch.zeros_like(top), top)
    x.exp_()
    den = x.sum(-1, keepdim=True)
    x /= torch.where(den == 0, torch.ones_like(den), den)
    o = torch.matmul(x.view(B, Hkv, G * L, T), gather("v")).view(B, Hkv, G, L, D)
    return o.permute(0, 3, 1, 2, 4).reshape(B, L, Hq, D)[live]              # in token order


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    if case["op"] == "append":
        q = _rotate(st["q"], *_rope_args(st)).to(torch.bfloat16)
        _write(st, _rotate(st["k_new"], *_rope_args(st)).to(torch.bfloat16), st["v_new"])
        return {"q": q, **_cache(st)}
    if case["op"] == "prefill":
        return {"out": _attend(st, st["q"]).to(torch.bfloat16)}
    q = st["q"]
    if case["rot"]:
        q = _rotate(q, *_rope_args(st)).to(torch.bfloat16)
    if case["append"]:
        _write(st, _rotate(st["k_new"], *_rope_args(st)).to(torch.bfloat16), st["v_new"])
    out = {"out": _attend(st, q)}
    return {**out, **_cache(st)} if case["append"] else out


# ---- this repository's calls -----------------------------------------------------------


def _handles(st):
    """What a user's program keeps: the pool, the rotation and a workspace."""
    import paged_kv_cache_466_b200 as pa
    case = st["case"]
    st["pa"] = pa
    pool = pa.KVPool(st["k"].shape[0], case["Hkv"], case["P"], case["D"], case["kind"], DEV)
    for mine, its in (("k", pool.k), ("v", pool.v), ("k_sz", pool.k_sz), ("v_sz", pool.v_sz)):
        if its is not None:
            its.copy_(st[mine])
            st[mine] = its
    st["pool"] = pool
    st["rope"] = None
    if case.get("rot"):
        st["rope"] = pa.Rope(st["table"], interleaved=case.get("interleaved", False),
                             axis_of_pair=st["axis_of_pair"])
    max_pages = st["block_tables"].shape[1]
    need = 0
    if case["op"] == "prefill":
        need = pa.pa_prefill_workspace_bytes(pool, st["N"], case["B"], case["Hq"], max_pages)
    elif case["op"] == "decode":
        need = pa.pa_decode_workspace_bytes(case["B"], case["Hq"], case["D"],
                                            pa.pa_decode_num_splits(pool, case["B"], max_pages))
    st["workspace"] = torch.zeros(need, dtype=torch.uint8, device=DEV) if need else None


def _run_own(st):
    pa, case, pool = st["pa"], st["case"], st["pool"]
    if case["op"] == "append":
        q = pa.pa_kv_append_rope(pool, st["rope"], st["q"], st["k_new"], st["v_new"], st["seq_idx"],
                                 st["pos"], st["block_tables"], rope_pos=st["rope_pos"])
        return {"q": q, **_cache(st)}
    if case["op"] == "prefill":
        return {"out": pa.pa_prefill(pool, st["q"], st["q_begin"], st["block_tables"],
                                     st["context_lens"], st["scale"], softcap=case["softcap"],
                                     alibi_slopes=st["slopes"], doc_begin=st["doc_begin"],
                                     prefix_end=st["prefix_end"], workspace=st["workspace"])}
    new = dict(k_new=st["k_new"], v_new=st["v_new"]) if case["append"] else {}
    out = {"out": pa.pa_decode_scored(pool, st["q"], st["block_tables"], st["context_lens"],
                                      st["scale"], softcap=case["softcap"], alibi_slopes=st["slopes"],
                                      doc_begin=st["doc_begin"], rope=st["rope"],
                                      workspace=st["workspace"], **new)}
    return {**out, **_cache(st)} if case["append"] else out


# ---- in 64 bits, from the definitions -----------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    D, P, Hkv, kind = case["D"], case["P"], case["Hkv"], case["kind"]
    G = case["Hq"] // Hkv
    pos = st["pos"].long()

    def turn(x, rounded):
        """The rotation as complex multiplication by e^{i angle}; `rounded`: with the roundings that
        belong to a stored row (each product and each sum to 32 bits, the result to 16)."""
        half = case["rot"] // 2
        ang = st["table"].to(f64)
        c, s = (torch.stack([ang[st["rope_pos"][axis].long(), part + j]
                             for j, axis in enumerate(st["axis_of_pair"])], -1)[:, None]
                for part in (0, half))
        a = torch.arange(half, device=DEV)
        a, b = (2 * a, 2 * a + 1) if case.get("interleaved") else (a, a + half)
        y = x.to(f64)
        if not rounded:
            z = torch.complex(y[..., a], y[..., b]) * torch.complex(c, s)
            y[..., a], y[..., b] = z.real, z.imag
            return y

        def r32(t):
            return t.float().to(f64)

        y[..., a], y[..., b] = (r32(r32(y[..., a] * c) - r32(y[..., b] * s)),
                                r32(r32(y[..., b] * c) + r32(y[..., a] * s)))
        return y.float().to(torch.bfloat16).to(f64)

    def stored(t, rows):
        """The whole cache as outputs, rows [N, Hkv, D] f64 at the new tokens' slots."""
        page = st["block_tables"].long()[st["seq_idx"].long(), pos // P]
        if kind == "bf16":
            k = st[t].to(f64)
            k[page, :, pos % P] = rows
            return {t: k}
        k, sz = st[t].view(torch.float8_e4m3fn).to(f64), st[t + "_sz"].to(f64)
        s = rows.abs().amax(-1, keepdim=True) / 448
        k[page, :, pos % P] = rows / s
        sz[page, :, pos % P] = torch.cat([s, torch.zeros_like(s)], -1)
        return {t: k, t + "_sz": sz}

    def meant(codes, sz):
        """The rows that cached rows [n, ...] stand for: scale times code plus zero."""
        if kind == "bf16":
            return codes.to(f64)
        if kind == "u4":
            nibbles = torch.empty(codes.shape[0], D, dtype=torch.uint8, device=DEV)
            nibbles[:, 0::2], nibbles[:, 1::2] = codes % 16, codes // 16
            codes = nibbles
        if kind == "fp8":
            codes = codes.view(torch.float8_e4m3fn)
        return torch.addcmul(sz[:, 1:].to(f64), sz[:, :1].to(f64), codes.to(f64))

    if case["op"] == "append":
        return {"q": turn(st["q"], False), **stored("k", turn(st["k_new"], kind != "bf16")),
                **stored("v", st["v_new"].to(f64))}

    # the rotated rows and the cache's codes are roundings that belong to the definition
    q = turn(st["q"], True) if case.get("rot") else st["q"].to(f64)
    out = {"out": torch.zeros(st["N"], case["Hq"], D, dtype=f64, device=DEV)}
    if case.get("append"):
        k_new = turn(st["k_new"], True)
        for t, rows in (("k", k_new), ("v", st["v_new"].to(f64))):
            out.update(stored(t, rows))
        _write(st, k_new.to(torch.bfloat16), st["v_new"])
    begin = st["q_begin"].tolist()
    for b, ctx in enumerate(st["context_lens"].tolist()):
        i = torch.arange(begin[b], begin[b + 1], device=DEV)
        pages = st["block_tables"][b, :-(-ctx // P)].long()
        j = torch.arange(ctx, device=DEV)
        hi = pos[i] + 1
        if st["prefix_end"] is not None:
            hi = torch.maximum(hi, st["prefix_end"][i].long())
        lo = st["doc_begin"][i].long() if st["doc_begin"] is not None else torch.zeros_like(hi)
        seen = (j >= lo[:, None]) & (j < hi[:, None])
        for h in range(Hkv):
            rows = {}
            for t in ("k", "v"):
                sz = st[t + "_sz"]
                sz = None if sz is None else sz[pages, h].reshape(-1, 2)[:ctx]
                codes = st[t][pages, h]
                rows[t] = meant(codes.reshape(-1, codes.shape[-1])[:ctx], sz)
            for hq in range(h * G, h * G + G):
                x = q[i, hq] @ rows["k"].T * st["scale"]
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if st["slopes"] is not None:
                    x = x - st["slopes"][hq].to(f64) * (pos[i][:, None] - j).abs()
                p = torch.softmax(x.masked_fill(~seen, -math.inf), -1).nan_to_num(0.0)
                out["out"][i, hq] = p @ rows["v"]
    return out
