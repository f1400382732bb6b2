"""The serving-step operators beside the paged cache, as cases to measure.

One decode or chunked-prefill step over the paged cache runs them in this order:

  advance    block tables, slot mapping and positions of the step's tokens, from request lengths
  norm_rope  RMS norm of the query and key heads, rotary positions, and the cache write
  bounds     the smallest and largest key of each touched block (per KV head and dimension)
  scores     per query token and KV head: an upper bound of every block's logits
  select     the k blocks each query token attends, exactly, in ascending order
  sparse     attention over the selected blocks

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true
it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
GQA = dict(hq=32, hkv=8, dim=128)  # the repository's grouped-query workloads
BF16, F32, E4M3 = "bf16", "f32", "e4m3"
TORCH = {BF16: torch.bfloat16, F32: torch.float32, E4M3: torch.float8_e4m3fn}
BYTES = {BF16: 2, F32: 4, E4M3: 1}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's metadata at the default request limit: 256 requests, one token each
        dict(name="advance decode 256", op="advance", seqs=256, chunks=0, chunk=1, empty=0, block=16, median=1024, pad=0),
        # continuous batching: 480 decodes beside 32 prompt chunks of 2048 tokens
        dict(name="advance mixed 66k tokens", op="advance", seqs=512, chunks=32, chunk=2048, empty=0, block=16,
             median=1024, pad=0),
        # a decode step's query/key/value rows, sliced out of one fused projection
        dict(name="norm rope decode 256", op="norm_rope", tokens=256, **GQA, rot=128, axes=1, interleaved=False,
             norm=True, dtype=BF16, cache=BF16, fused=True, block=16, pad=0),
        # a prompt of text and images: positions with time, height and width
        dict(name="norm rope prompt 16384 3-axis", op="norm_rope", tokens=16384, **GQA, rot=128, axes=3,
             interleaved=False, norm=True, dtype=BF16, cache=BF16, fused=True, block=16, pad=0),
        # the blocks a decode step wrote one key into
        dict(name="bounds decode 256", op="bounds", seqs=256, query=1, median=4096, hkv=8, dim=128, block=16, cache=BF16),
        # the blocks of sixteen 8192-token prompts, over an E4M3 cache with wide blocks
        dict(name="bounds prompt 16x8192 e4m3", op="bounds", seqs=16, query=8192, median=8192, hkv=8, dim=128, block=64,
             cache=E4M3),
        # every block of 64 long requests, scored for one query token each
        dict(name="scores decode 64x32k", op="scores", seqs=64, query=1, median=32768, **GQA, block=16),
        # four 512-token chunks scored against 8192 earlier positions
        dict(name="scores chunk 4x512", op="scores", seqs=4, query=512, median=8192, **GQA, block=16),
        # 128 of about 2048 blocks for each of 64 x 8 rows
        dict(name="select decode 64x2048", op="select", seqs=64, query=1, median=32768, hkv=8, block=16, k=128, init=1,
             local=2, ties=False),
        # 64 of about 512 blocks for each row of four 512-token chunks
        dict(name="select chunk 4x512", op="select", seqs=4, query=512, median=8192, hkv=8, block=16, k=64, init=1,
             local=2, ties=False),
        # two requests verifying four drafted tokens each: few rows, latency-bound
        dict(name="sparse draft 2x4 e4m3", op="sparse", seqs=2, query=4, median=40000, **GQA, block=16, k=128, cache=E4M3),
        # a full decode batch over 64 blocks (1024 keys) of each row's choice
        dict(name="sparse decode 256 k64", op="sparse", seqs=256, query=1, median=4096, **GQA, block=16, k=64, cache=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["advance", "norm_rope", "bounds", "scores", "select", "sparse"])
    hq, hkv, dim = rng.choice([(32, 8, 128), (32, 32, 128), (32, 4, 128), (16, 2, 64), (8, 4, 64), (4, 1, 128), (8, 1, 128)])
    if op == "advance":
        seqs = _log(rng, 1, 1024)
        chunks = rng.randint(0, min(seqs, 32))
        return dict(op=op, seqs=seqs, chunks=chunks, chunk=_log(rng, 2, 1800), empty=rng.randint(0, seqs - chunks),
                    block=rng.choice([4, 8, 16, 32, 64]), median=_log(rng, 1, 4000), pad=rng.choice([0, 1, 37, 300]))
    if op == "norm_rope":
        dtype, cache = rng.choice([(BF16, BF16), (BF16, BF16), (F32, F32), (BF16, E4M3), (F32, E4M3)])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        return dict(op=op, tokens=_log(rng, 1, 4000), hq=hq, hkv=hkv, dim=dim, rot=rot, axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8, dtype=dtype, cache=cache,
                    fused=rng.random() < 0.6, block=rng.choice([4, 16, 64]), pad=rng.choice([0, 0, 1, 9]))
    cache, block = rng.choice([BF16, BF16, E4M3]), rng.choice([16, 16, 32, 64, 128])
    if op == "bounds":
        query = rng.choice([1, 1, _log(rng, 2, 2000)])
        return dict(op=op, seqs=_log(rng, 1, 100 if query == 1 else 6), query=query, median=_log(rng, 16, 4000), hkv=hkv,
                    dim=dim, block=block, cache=cache)
    if op == "scores":
        query = rng.choice([1, 1, _log(rng, 2, 300)])
        return dict(op=op, seqs=_log(rng, 1, 48 if query == 1 else 4), query=query, median=_log(rng, 30, 12000), hq=hq,
                    hkv=min(hkv, 8), dim=dim, block=block) if hkv <= 8 else \
            dict(op=op, seqs=_log(rng, 1, 12), query=1, median=_log(rng, 30, 12000), hq=hq, hkv=hkv, dim=dim, block=block)
    if op == "select":
        query = rng.choice([1, 1, _log(rng, 2, 200)])
        k = _log(rng, 2, 256)
        return dict(op=op, seqs=_log(rng, 1, 64 if query == 1 else 6), query=query,
                    median=_log(rng, 20, 30000 if query == 1 else 2500), hkv=hkv, block=block, k=k,
                    init=rng.randint(0, min(2, k // 2)), local=rng.randint(0, min(4, k // 2)), ties=rng.random() < 0.5)
    query = rng.choice([1, 1, 1, _log(rng, 2, 16)])
    k = max(2, _log(rng, 2, 64) * 16 // block)
    return dict(op=op, seqs=_log(rng, 1, 64 if query == 1 else 4), query=query, median=_log(rng, 20, 9000), hq=hq, hkv=hkv,
                dim=dim, block=block, k=k, cache=cache)


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _lens(c, seqs, g):
    """Context lengths: lognormal around the median (a quarter of an octave each way at most)."""
    x = torch.randn(seqs, generator=g, device=DEV).mul(0.1).clamp(-0.17, 0.17).exp().mul(c["median"])
    return x.round().clamp_(min=1).to(torch.int32)


def _batch(c, g):
    """Requests of `query` new tokens at the end of their context: tables over a shuffled pool."""
    S, Q, B = c["seqs"], c["query"], c["block"]
    lens = torch.maximum(_lens(c, S, g), torch.tensor(Q, dtype=torch.int32, device=DEV))
    W = -(-int(math.ceil(c["median"] * math.exp(0.17)) + 1) // B)
    W = max(W, -(-Q // B))
    NB = S * W + 3
    table = torch.randperm(NB, generator=g, device=DEV)[: S * W].to(torch.int32).view(S, W)
    qsl = torch.arange(S + 1, device=DEV, dtype=torch.int32) * Q
    return dict(S=S, Q=Q, B=B, W=W, NB=NB, T=S * Q, seq_lens=lens, block_table=table, query_start_loc=qsl,
                max_seq_len=W * B)


def _keys(shape, g, cache):
    """Keys with channels of different spread, as projected keys have them."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if math.prod(shape) < 1 << 28 else torch.bfloat16)
    x *= torch.rand(shape[-1], generator=g, device=DEV).mul(1.5).add(0.25).to(x.dtype)
    if cache == E4M3:
        return (x.float() / 2 ** -5).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return x.to(TORCH[cache])


def _sections(c):
    half = c["rot"] // 2
    return [half] if c["axes"] == 1 else [half - half // 2, half // 2] if c["axes"] == 2 else \
        [half - 2 * (half * 3 // 8), half * 3 // 8, half * 3 // 8]


def prepare(c, seed):
    g = _gen(seed)
    op = c["op"]
    if op == "advance":
        S, B = c["seqs"], c["block"]
        ctx = _lens(c, S, g)
        q = torch.ones(S, dtype=torch.int32, device=DEV)
        perm = torch.randperm(S, generator=g, device=DEV)
        q[perm[: c["chunks"]]] = c["chunk"]
        q[perm[c["chunks"]: c["chunks"] + c["empty"]]] = 0
        T = c["chunks"] * c["chunk"] + (S - c["chunks"] - c["empty"]) + c["pad"]
        W = -(-(int(c["median"] * math.exp(0.17)) + 2 + c["chunk"]) // B)
        have = (ctx + B - 1) // B
        table = torch.randint(0, S * W, (S, W), generator=g, device=DEV, dtype=torch.int32)
        table[torch.arange(W, device=DEV)[None, :] >= have[:, None]] = -1
        free = torch.randperm(S * W + 8, generator=g, device=DEV).to(torch.int32)
        i32 = dict(dtype=torch.int32, device=DEV)
        return dict(c=c, S=S, B=B, W=W, T=T, NB=S * W + 8, block_table=table, seq_lens=ctx, query_lens=q, free_blocks=free,
                    free_head=torch.full((1,), 5, **i32), seq_lens_out=torch.empty(S, **i32),
                    free_head_out=torch.empty(1, **i32), query_start_loc=torch.empty(S + 1, **i32),
                    slot_mapping=torch.empty(T, dtype=torch.int64, device=DEV), positions=torch.empty(T, **i32))
    if op == "norm_rope":
        T, hq, hkv, D, dt = c["tokens"], c["hq"], c["hkv"], c["dim"], TORCH[c["dtype"]]
        qkv = torch.randn((T, hq + 2 * hkv, D), generator=g, device=DEV).mul_(2.0).to(dt)
        q, k, v = qkv[:, :hq], qkv[:, hq: hq + hkv], qkv[:, hq + hkv:]
        if not c["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        w = [(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(dt) if c["norm"] else None for _ in range(2)]
        limit = 32768
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        ang = torch.arange(limit, device=DEV, dtype=torch.float64)[:, None] * inv
        cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
        shape = (T,) if c["axes"] == 1 else (c["axes"], T)
        positions = torch.randint(0, limit, shape, generator=g, device=DEV, dtype=torch.int32)
        NB = -(-T // c["block"]) + 2
        slots = torch.randperm(NB * c["block"], generator=g, device=DEV)[:T].contiguous()
        slots[T - min(c["pad"], T):] = -1
        kc = torch.zeros((NB, c["block"], hkv, D), dtype=TORCH[c["cache"]], device=DEV)
        return dict(c=c, q=q, k=k, v=v, q_weight=w[0], k_weight=w[1], cos_sin=cos_sin, positions=positions, slots=slots,
                    k_cache=kc, v_cache=torch.zeros_like(kc), q_out=torch.empty((T, hq, D), dtype=dt, device=DEV),
                    sections=None if c["axes"] == 1 else tuple(_sections(c)), eps=1e-6,
                    k_scale=2 ** -5 if c["cache"] == E4M3 else 1.0, v_scale=0.0173 if c["cache"] == E4M3 else 1.0)
    b = _batch(c, g)
    b["c"] = c
    if op == "bounds":
        b["k_cache"] = _keys((b["NB"], b["B"], c["hkv"], c["dim"]), g, c["cache"])
        b["bounds"] = torch.zeros((b["NB"], c["hkv"], 2, c["dim"]), dtype=torch.bfloat16, device=DEV)
        return b
    if op == "scores":
        mid = _keys((b["NB"], c["hkv"], 1, c["dim"]), g, BF16)
        half = torch.rand((b["NB"], c["hkv"], 1, c["dim"]), generator=g, device=DEV).mul_(1.7).to(torch.bfloat16)
        b["bounds"] = torch.cat([mid - half, mid + half], 2)
        b["q"] = torch.randn((b["T"], c["hq"], c["dim"]), generator=g, device=DEV).to(torch.bfloat16)
        b["scores"] = torch.empty((b["T"], c["hkv"], b["W"]), dtype=torch.float32, device=DEV)
        return b
    last = (_positions(b) // b["B"]).view(-1, 1, 1)
    blocks = torch.arange(b["W"], device=DEV).view(1, 1, -1)
    if op == "select":
        s = torch.randn((b["T"], c["hkv"], b["W"]), generator=g, device=DEV).mul_(4.0)
        if c["ties"]:
            s = s.mul_(2).round_().div_(2)
        b["scores"] = torch.where(blocks <= last, s, -math.inf)
        b["block_idx"] = torch.empty((b["T"], c["hkv"], c["k"]), dtype=torch.int32, device=DEV)
        return b
    r = torch.rand((b["T"], c["hkv"], b["W"]), generator=g, device=DEV)
    r = torch.where(blocks == last, 2.0, torch.where(blocks < last, r, -1.0))
    k = min(c["k"], b["W"])
    top = r.topk(k, dim=2)
    idx = torch.where(top.values >= 0, top.indices, b["W"]).sort(dim=2).values
    idx = torch.where(idx == b["W"], -1, idx).to(torch.int32)
    b["block_idx"] = torch.full((b["T"], c["hkv"], c["k"]), -1, dtype=torch.int32, device=DEV)
    b["block_idx"][:, :, :k] = idx
    b["k_cache"] = _keys((b["NB"], b["B"], c["hkv"], c["dim"]), g, c["cache"])
    b["v_cache"] = _keys((b["NB"], b["B"], c["hkv"], c["dim"]), g, c["cache"])
    b["q"] = torch.randn((b["T"], c["hq"], c["dim"]), generator=g, device=DEV).to(torch.bfloat16)
    b["out"] = torch.empty_like(b["q"])
    b["scale"] = c["dim"] ** -0.5
    b["k_scale"], b["v_scale"] = (2 ** -5, 2 ** -5) if c["cache"] == E4M3 else (1.0, 1.0)
    return b


def _positions(b):
    """Position of every query token: the last Q positions of its request."""
    j = torch.arange(b["Q"], device=DEV)
    return (b["seq_lens"][:, None] - b["Q"] + j).view(-1).long()


# ------------------------------------------------------------------------------- one pass
def run(st):
    op = st["c"]["op"]
    if own:
        return _own(op, st)
    return {"advance": _advance, "norm_rope": _norm_rope, "bounds": _bounds, "scores": _scores, "select": _select,
            "sparse": _sparse}[op](st)


def _own(op, st):
    import paged_kv_cache_161_gb300 as pa

    if op == "advance":
        pa.advance_batch(st["block_table"], st["seq_lens"], st["query_lens"], st["free_blocks"], st["free_head"],
                         st["seq_lens_out"], st["free_head_out"], st["query_start_loc"], st["slot_mapping"],
                         st["positions"], block_size=st["B"], num_blocks=st["NB"])
        return [st[n] for n in ("block_table", "seq_lens_out", "free_head_out", "query_start_loc", "slot_mapping",
                                "positions")]
    if op == "norm_rope":
        pa.norm_rope_write(st["q_out"], st["q"], st["k"], st["v"], st["q_weight"], st["k_weight"], st["cos_sin"],
                           st["positions"], st["slots"], st["k_cache"], st["v_cache"], eps=st["eps"],
                           interleaved=st["c"]["interleaved"], sections=st["sections"], k_scale=st["k_scale"],
                           v_scale=st["v_scale"])
        return [st["q_out"], _values(st["k_cache"]), _values(st["v_cache"])]
    meta = (st["block_table"], st["seq_lens"], st["query_start_loc"])
    if op == "bounds":
        pa.block_bounds(st["bounds"], st["k_cache"], *meta, max_query_len=st["Q"], max_seq_len=st["max_seq_len"])
        return st["bounds"]
    if op == "scores":
        pa.block_scores(st["scores"], st["q"], st["bounds"], *meta, block_size=st["B"], max_query_len=st["Q"],
                        max_seq_len=st["max_seq_len"])
        return st["scores"]
    if op == "select":
        pa.select_blocks(st["block_idx"], st["scores"], st["seq_lens"], st["query_start_loc"], block_size=st["B"],
                         init_blocks=st["c"]["init"], local_blocks=st["c"]["local"])
        return st["block_idx"]
    pa.attention_sparse(st["out"], st["q"], st["k_cache"], st["v_cache"], *meta, st["block_idx"],
                        max_seq_len=st["max_seq_len"], scale=st["scale"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    return st["out"]


def _values(cache):
    """A cache's content: E4M3 codes as the values they stand for (exact in bfloat16)."""
    return cache.bfloat16() if cache.dtype == torch.float8_e4m3fn else cache


def _advance(st):
    S, B, W, T = st["S"], st["B"], st["W"], st["T"]
    ctx, q = st["seq_lens"].long(), st["query_lens"].long()
    have = (ctx + B - 1) // B
    need = (ctx + q + B - 1) // B - have
    qsl = torch.nn.functional.pad(q.cumsum(0), (1, 0))
    off = need.cumsum(0) - need + st["free_head"]
    t = torch.arange(T, device=DEV)
    s = torch.searchsorted(qsl[1:], t, right=True).clamp_(max=S - 1)
    valid = t < qsl[-1]
    pos = torch.where(valid, ctx[s] + t - qsl[s], 0)
    b = pos // B
    new = b - have[s]
    ids = torch.where(new >= 0, st["free_blocks"][torch.where(valid & (new >= 0), off[s] + new, 0)],
                      st["block_table"][s, b])
    flat = torch.nn.functional.pad(st["block_table"].view(-1), (0, 1))
    flat[torch.where(valid, s * W + b, S * W)] = ids
    slots = torch.where(valid, ids.long() * B + pos % B, -1)
    i32 = torch.int32
    return [flat[:-1].view(S, W), (ctx + q).to(i32), (st["free_head"] + need.sum()).to(i32), qsl.to(i32), slots,
            pos.to(i32)]


def _rotate(x, cos, sin, rot, interleaved):
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rot // 2], r[..., rot // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _norm(x, w, eps):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _encode(x, scale, dtype):
    return (x / scale).clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _norm_rope(st):
    c = st["c"]
    rot = c["rot"]
    pos = st["positions"].long()
    if st["sections"] is None:
        table = st["cos_sin"][pos]
    else:
        axis = torch.repeat_interleave(torch.arange(len(st["sections"]), device=DEV),
                                       torch.tensor(st["sections"], device=DEV), output_size=rot // 2).repeat(2)
        table = st["cos_sin"][pos[axis].t(), torch.arange(rot, device=DEV)]
    cos, sin = table[:, None, : rot // 2], table[:, None, rot // 2:]
    q = _rotate(_norm(st["q"], st["q_weight"], st["eps"]), cos, sin, rot, c["interleaved"])
    k = _rotate(_norm(st["k"], st["k_weight"], st["eps"]), cos, sin, rot, c["interleaved"])
    dt = st["k_cache"].dtype
    rows, hkv, D = st["k_cache"].shape[0] * c["block"], c["hkv"], c["dim"]
    kv = []
    for x, scale, cache in ((k, st["k_scale"], st["k_cache"]), (st["v"].float(), st["v_scale"], st["v_cache"])):
        y = _encode(x, scale, dt)
        if c["pad"]:  # padding tokens write nothing: their rows go to a spare row that is cut off
            z = torch.zeros((rows + 1, hkv, D), dtype=dt, device=DEV)
            z[torch.where(st["slots"] < 0, rows, st["slots"])] = y
            z = z[:-1].view_as(cache)
        else:
            z = cache
            z.view(rows, hkv, D)[st["slots"]] = y
        kv.append(_values(z))
    return [q.to(st["q_out"].dtype), *kv]


def _bounds(st):
    B, Q = st["B"], st["Q"]
    L = st["seq_lens"].long()
    first = (L - Q) // B
    n = min((Q - 1) // B + 2, st["W"])
    b = first[:, None] + torch.arange(n, device=DEV)
    live = b * B < L[:, None]
    b = b.clamp(max=st["W"] - 1)
    blk = st["block_table"].long().gather(1, b)
    k = st["k_cache"][blk].float()  # [S, n, B, hkv, D]
    pos = b[:, :, None] * B + torch.arange(B, device=DEV)
    out = (pos >= L[:, None, None])[..., None, None]
    lo, hi = k.masked_fill(out, math.inf).amin(2), k.masked_fill(out, -math.inf).amax(2)
    new = torch.stack([lo, hi], 3).to(torch.bfloat16)
    # entries past the last block repeat the request's first touched one
    st["bounds"][torch.where(live, blk, blk[:, :1])] = torch.where(live[..., None, None, None], new, new[:, :1])
    return st["bounds"]


def _scores(st):
    c, S, Q, W = st["c"], st["S"], st["Q"], st["W"]
    hkv, G, D = c["hkv"], c["hq"] // c["hkv"], c["dim"]
    bd = st["bounds"][st["block_table"].long()].float()  # [S, W, hkv, 2, D]
    bd = bd.permute(0, 2, 3, 4, 1).reshape(S, hkv, 2 * D, W)
    q = st["q"].float().view(S, Q, hkv, G, D)
    q = torch.cat([q.clamp(max=0), q.clamp(min=0)], -1).permute(0, 2, 1, 3, 4).reshape(S, hkv, Q * G, 2 * D)
    s = torch.matmul(q, bd).view(S, hkv, Q, G, W).amax(3).transpose(1, 2).reshape(S * Q, hkv, W)
    last = (_positions(st) // st["B"]).view(-1, 1, 1)
    return s.masked_fill(torch.arange(W, device=DEV) > last, -math.inf)


def _select(st):
    c = st["c"]
    W, k = st["W"], c["k"]
    last = (_positions(st) // st["B"]).view(-1, 1, 1)
    b = torch.arange(W, device=DEV).view(1, 1, -1)
    s = st["scores"]
    forced = (b <= last) & ((b < c["init"]) | (b > last - c["local"]))
    key = s.masked_fill(forced, math.inf)
    order = key.sort(dim=2, descending=True, stable=True)  # equal scores: the lowest block first
    idx = torch.where(order.values > -math.inf, order.indices, W)[:, :, :k].sort(dim=2).values
    idx = torch.where(idx == W, -1, idx).to(torch.int32)
    return torch.nn.functional.pad(idx, (0, k - idx.shape[2]), value=-1)


def _sparse(st):
    c, B, Q = st["c"], st["B"], st["Q"]
    hkv, G, D = c["hkv"], c["hq"] // c["hkv"], c["dim"]
    T, K = st["T"], c["k"]
    idx = st["block_idx"].long()
    live = idx >= 0
    at = idx.clamp(min=0)
    blk = st["block_table"].long().repeat_interleave(Q, 0)[:, None, :].expand(T, hkv, -1).gather(2, at)
    h = torch.arange(hkv, device=DEV).view(1, -1, 1)
    k = st["k_cache"].transpose(1, 2)[blk, h].float().view(T, hkv, K * B, D)
    v = st["v_cache"].transpose(1, 2)[blk, h].float().view(T, hkv, K * B, D)
    pos = (at[..., None] * B + torch.arange(B, device=DEV)).view(T, hkv, K * B)
    seen = live.repeat_interleave(B, 2) & (pos <= _positions(st).view(-1, 1, 1))
    q = st["q"].float().view(T, hkv, G, D)
    s = torch.matmul(q, k.transpose(2, 3)) * (st["scale"] * st["k_scale"])
    s = s.masked_fill(~seen[:, :, None], -math.inf)
    p = (s - s.amax(3, keepdim=True)).exp()
    o = torch.matmul(p, v) / p.sum(3, keepdim=True) * st["v_scale"]
    return o.view(T, c["hq"], D).to(torch.bfloat16)


# ------------------------------------------------------------------------------- what a pass needs
def work(c):
    op = c["op"]
    if op == "advance":
        S = c["seqs"]
        T = c["chunks"] * c["chunk"] + (S - c["chunks"] - c["empty"])
        return dict(bytes=16 * S + 12 * (T + c["pad"]) + 8 * (T / c["block"]) + 4 * S, flops=0)
    if op == "norm_rope":
        T, D = c["tokens"], c["dim"]
        e, w = BYTES[c["dtype"]], BYTES[c["cache"]]
        rows = c["hq"] + c["hkv"]
        return dict(bytes=T * D * (c["hq"] * 2 * e + c["hkv"] * 2 * (e + w)) + T * (4 * c["rot"] + 8 + 4 * c["axes"]),
                    flops=T * rows * (4 * D + 3 * c["rot"]))
    S, Q, B, hkv = c["seqs"], c["query"], c["block"], c["hkv"]
    T, n = S * Q, max(c["median"], Q) / B
    if op == "bounds":
        touched = min(Q / B + 1, n)
        return dict(bytes=S * touched * hkv * c["dim"] * (min(B, max(c["median"], Q)) * BYTES[c["cache"]] + 4), flops=0)
    if op == "scores":
        return dict(bytes=S * n * hkv * 4 * c["dim"] + T * c["hq"] * c["dim"] * 2 + T * hkv * n * 4,
                    flops=4.0 * T * c["hq"] * n * c["dim"])
    if op == "select":
        return dict(bytes=T * hkv * 4 * (n + c["k"]), flops=0)
    keys = min(c["k"], n) * B
    distinct = min(Q * keys, max(c["median"], Q))
    return dict(bytes=S * hkv * distinct * 2 * c["dim"] * BYTES[c["cache"]] + T * c["hq"] * c["dim"] * 4 + T * hkv * c["k"] * 4,
                flops=4.0 * T * c["hq"] * keys * c["dim"])


# ------------------------------------------------------------------------------- 64 bits
def exact(c, seed):
    """The definitions in float64, request by request or row by row where that is quick."""
    st = prepare(c, seed)
    op = c["op"]
    f64 = torch.float64
    if op == "advance":  # whole numbers: replayed on the host, token by token
        table, ctx, q = st["block_table"].tolist(), st["seq_lens"].tolist(), st["query_lens"].tolist()
        free, head, B = st["free_blocks"].tolist(), int(st["free_head"]), st["B"]
        slots, positions, qsl = [], [], [0]
        for s in range(st["S"]):
            for p in range(ctx[s], ctx[s] + q[s]):
                if p % B == 0:
                    table[s][p // B] = free[head]
                    head += 1
                slots.append(table[s][p // B] * B + p % B)
                positions.append(p)
            qsl.append(len(slots))
        pad = st["T"] - len(slots)
        i32 = torch.int32
        return [torch.tensor(table, dtype=i32), torch.tensor([a + b for a, b in zip(ctx, q)], dtype=i32),
                torch.tensor([head], dtype=i32), torch.tensor(qsl, dtype=i32), torch.tensor(slots + [-1] * pad),
                torch.tensor(positions + [0] * pad, dtype=i32)]
    if op == "norm_rope":
        rot, half, T = c["rot"], c["rot"] // 2, c["tokens"]
        cos = torch.empty((T, half), dtype=f64, device=DEV)
        sin = torch.empty_like(cos)
        start = 0
        for a, n in enumerate(_sections(c)):  # each axis fills its pairs
            row = st["cos_sin"].double()[(st["positions"] if c["axes"] == 1 else st["positions"][a]).long()]
            cos[:, start: start + n], sin[:, start: start + n] = row[:, start: start + n], row[:, half + start: half + start + n]
            start += n
        rows = []
        for x, w in ((st["q"], st["q_weight"]), (st["k"], st["k_weight"])):
            y = x.double()
            if w is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / c["dim"] + st["eps"]).sqrt() * w.double()
            z = y.clone()
            lo = slice(0, rot, 2) if c["interleaved"] else slice(0, half)
            hi = slice(1, rot, 2) if c["interleaved"] else slice(half, rot)
            z[..., lo] = y[..., lo] * cos[:, None] - y[..., hi] * sin[:, None]
            z[..., hi] = y[..., hi] * cos[:, None] + y[..., lo] * sin[:, None]
            rows.append(z)
        live = st["slots"] >= 0
        out = [rows[0]]
        for x, cache, scale in ((rows[1], st["k_cache"], st["k_scale"]), (st["v"].double(), st["v_cache"], st["v_scale"])):
            z = torch.zeros(cache.shape, dtype=f64, device=DEV).view(-1, c["hkv"], c["dim"])
            y = x / scale
            z[st["slots"][live]] = (y.clamp(-448, 448).to(torch.float8_e4m3fn).double() if c["cache"] == E4M3 else y)[live]
            out.append(z.view(cache.shape))
        return out
    L, table = st["seq_lens"].tolist(), st["block_table"].long()
    B, Q, W = st["B"], st["Q"], st["W"]
    if op == "bounds":
        out = st["bounds"].double()
        for s in range(st["S"]):
            for b in range((L[s] - Q) // B, (L[s] - 1) // B + 1):
                k = st["k_cache"][table[s, b], : min(B, L[s] - b * B)].double()
                out[table[s, b], :, 0], out[table[s, b], :, 1] = k.min(0).values, k.max(0).values
        return out
    hkv = c["hkv"]
    if op == "select":
        return None  # whole numbers from given scores: the plain form's are exact
    G, D = c["hq"] // hkv, c["dim"]
    if op == "scores":
        out = torch.full(st["scores"].shape, -math.inf, dtype=f64, device=DEV)
        for s in range(st["S"]):
            lo, hi = st["bounds"][table[s]].double().unbind(2)  # [W, hkv, D]
            for t in range(Q):
                row = s * Q + t
                n = (L[s] - Q + t) // B + 1
                q = st["q"][row].double().view(hkv, G, 1, D)
                top = torch.maximum(q * lo[:n].transpose(0, 1)[:, None], q * hi[:n].transpose(0, 1)[:, None])
                out[row, :, :n] = top.sum(-1).amax(1)
        return out
    out = torch.zeros(st["out"].shape, dtype=f64, device=DEV)
    idx = st["block_idx"].tolist()
    for row in range(st["T"]):
        s, last = row // Q, L[row // Q] - Q + row % Q
        for h in range(hkv):
            listed_blocks = [b for b in idx[row][h] if b >= 0]
            b = torch.tensor(listed_blocks, device=DEV)
            k, v = st["k_cache"][table[s, b], :, h].double(), st["v_cache"][table[s, b], :, h].double()
            cut = (len(listed_blocks) - 1) * B + min(B, last - listed_blocks[-1] * B + 1)  # the last block may be partial
            k, v = k.reshape(-1, D)[:cut] * st["k_scale"], v.reshape(-1, D)[:cut] * st["v_scale"]
            q = st["q"][row, h * G: (h + 1) * G].double()
            out[row, h * G: (h + 1) * G] = torch.softmax(q @ k.T * st["scale"], -1) @ v
    return out
