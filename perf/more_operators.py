"""The operators of an integer-coded paged cache, as cases to measure.

A serving loop whose cache holds 4- or 8-bit integer codes runs

  store   quantise new key and value rows into the pages (a smallest value and a step for each token
          and KV head), and read the same rows back as the values their codes stand for
  read    a context's rows out of the pages, packed row after row, for the next chunk of its prompt
  decode  attention of one or a few new tokens over the pages
  packed  causal attention of whole prompts, or of chunks behind their contexts, over packed rows

With ``own`` false, ``run`` computes them in elementary torch operations; with ``own`` true it
calls the library.

The cache: uint8 [num_blocks, num_kv_heads, block_size * (head_dim * bits / 8 + 4)]; of a block and
head first the rows' codes (element 2 i in the low half of byte i when bits = 4), then for every
row the smallest value and the step, both bfloat16.
"""
import math

import torch

own = False

DEV = "cuda"
GQA = dict(hq=32, hkv=8, dim=128)  # the repository's grouped-query workloads
BF16, F32 = "bf16", "f32"
TORCH = {BF16: torch.bfloat16, F32: torch.float32}
BYTES = {BF16: 2, F32: 4}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # the rows of a decode step: 256 requests, one token each; latency counts
        dict(name="store decode 256 int4", op="store", seqs=256, query=1, median=1024, hkv=8, dim=128, block=16, bits=4,
             dtype=BF16, fused=True),
        # four prompts of 4096 tokens
        dict(name="store prompt 4x4096 int8", op="store", seqs=4, query=4096, median=4096, hkv=8, dim=128, block=16,
             bits=8, dtype=BF16, fused=True),
        # one short context ahead of a chunk
        dict(name="read 1x1900 int8", op="read", seqs=1, median=1900, spread=0.1, hkv=8, dim=128, block=16, bits=8,
             dtype=BF16),
        # the contexts of four chunks
        dict(name="read 4x8192 int4", op="read", seqs=4, median=8192, spread=0.1, hkv=8, dim=128, block=16, bits=4,
             dtype=BF16),
        # two requests verifying four drafted tokens each over long contexts: few rows, latency
        dict(name="decode draft 2x4 int4", op="decode", seqs=2, query=4, median=40000, spread=0.1, **GQA, block=16, bits=4),
        # the repository's decode batch: 256 requests of very different lengths
        dict(name="decode 256 int4", op="decode", seqs=256, query=1, median=1024, spread=1.0, **GQA, block=16, bits=4),
        # every query head with a key head of its own
        dict(name="decode 64 heads 32/32 int8", op="decode", seqs=64, query=1, median=1000, spread=0.5, hq=32, hkv=32,
             dim=128, block=16, bits=8),
        # long contexts
        dict(name="decode 64x32k int8", op="decode", seqs=64, query=1, median=32768, spread=0.1, **GQA, block=64, bits=8),
        # eight prompts of about 500 tokens
        dict(name="packed 8x500", op="packed", seqs=8, query=500, spread=0.6, context=0, **GQA, fused=True),
        # chunks of 512 tokens behind contexts of about 8192
        dict(name="packed chunk 4x512", op="packed", seqs=4, query=512, spread=0.0, context=8192, **GQA, fused=False),
        # one long prompt
        dict(name="packed 1x16384", op="packed", seqs=1, query=16384, spread=0.0, context=0, **GQA, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "read", "decode", "decode", "packed", "packed"])
    hq, hkv, dim = rng.choice([(32, 8, 128), (32, 32, 128), (32, 4, 128), (16, 2, 64), (8, 4, 64), (4, 1, 128), (8, 1, 128)])
    bits, block = rng.choice([4, 8]), rng.choice([8, 16, 16, 32, 64, 128])
    dtype = rng.choice([BF16, BF16, F32])
    if op == "store":
        query = rng.choice([1, _log(rng, 2, 3000)])
        return dict(op=op, seqs=_log(rng, 1, 600 if query == 1 else 5), query=query, median=max(query, _log(rng, 1, 3000)),
                    hkv=min(hkv, 8), dim=dim, block=block, bits=bits, dtype=dtype, fused=rng.random() < 0.5)
    if op == "read":
        return dict(op=op, seqs=_log(rng, 1, 16), median=_log(rng, 1, 2000), spread=rng.choice([0.1, 0.6]),
                    hkv=min(hkv, 8), dim=dim, block=block, bits=bits, dtype=dtype)
    if op == "decode":
        query = rng.choice([1, 1, 1, rng.randint(2, 8)])
        spread = rng.choice([0.1, 0.5, 1.0])
        seqs = _log(rng, 1, 200 if query == 1 else 8)
        return dict(op=op, seqs=seqs, query=query, median=_log(rng, 1, min(20000, 160000 // seqs)), spread=spread, hq=hq,
                    hkv=hkv, dim=dim, block=block, bits=bits)
    seqs = _log(rng, 1, 12)
    query = _log(rng, 1, 9000 // seqs)
    return dict(op=op, seqs=seqs, query=query, spread=rng.choice([0.0, 0.4, 0.8]),
                context=rng.choice([0, 0, _log(rng, 1, 3000)]), hq=hq, hkv=hkv, dim=dim, fused=rng.random() < 0.5)


# ------------------------------------------------------------------------------- codes
def _levels(bits):
    return 2 ** bits - 1


def _down(x):
    """The largest bfloat16 not above x (float32), as float32."""
    u = x.view(torch.int32)
    t = u & -65536
    return torch.where((u < 0) & (t != u), t + 65536, t).view(torch.float32)


def _up(x):
    """The smallest bfloat16 not below x >= 0 (float32), as float32."""
    u = x.view(torch.int32)
    t = u & -65536
    return torch.where(t != u, t + 65536, t).view(torch.float32)


def _quantise(x, bits):
    """Codes (float32 whole numbers), smallest value and step of every row of x [..., D]."""
    x = x.float()
    lo = _down(x.amin(-1))
    spread = x.amax(-1) - lo
    step = _up(spread / torch.full_like(spread, _levels(bits))).clamp(min=2.0 ** -126)
    inv = torch.ones_like(step) / step
    codes = ((x - lo[..., None]).double() * inv[..., None].double()).round()  # 64 bits: products next to a half
    return codes, lo, step


def _pack(codes, lo, step, bits):
    """Cache content [num_blocks, num_kv_heads, bytes] of codes [num_blocks, num_kv_heads, block, D]."""
    c = codes.to(torch.uint8)
    if bits == 4:
        c = c[..., 0::2] | (c[..., 1::2] << 4)
    p = torch.stack([lo, step], -1).to(torch.bfloat16).view(torch.uint8)
    return torch.cat([c.flatten(2), p.flatten(2)], 2)


def _unpack(cache, dim, bits):
    """Codes, smallest values and steps of blocks: cache [..., bytes] -> [..., block, D], [..., block] twice, float32."""
    row = dim * bits // 8
    B = cache.shape[-1] // (row + 4)
    c = cache[..., : B * row].unflatten(-1, (B, row))
    if bits == 4:
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    p = cache[..., B * row:].contiguous().view(torch.bfloat16).unflatten(-1, (B, 2)).float()
    return c.float(), p[..., 0], p[..., 1]


def _values(cache, dim, bits):
    c, lo, step = _unpack(cache, dim, bits)
    return lo[..., None] + step[..., None] * c


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _spread(n, s, top, g):
    """Factors exp(s z) over the normal's quantiles z (z s from -1.7 s to `top`), in an order of the seed's."""
    z = torch.special.ndtri((torch.arange(n, device=DEV, dtype=torch.float64) + 0.5) / n)
    return z.mul(s).clamp(-1.7 * s, top).exp()[torch.randperm(n, generator=g, device=DEV)]


def _lens(c, seqs, g):
    """Lengths: lognormal around the median, at most 8 times it (the spread 0.1: a quarter of an octave)."""
    s = c.get("spread", 0.1)
    return _spread(seqs, s, 2.08 * s, g).mul(c["median"]).round().clamp_(min=1).to(torch.int32)


def _longest(c):
    return int(math.ceil(c["median"] * math.exp(2.08 * c.get("spread", 0.1)))) + 1


def _table(c, S, longest, g):
    W = -(-longest // c["block"])
    NB = S * W + 3
    return W, NB, torch.randperm(NB, generator=g, device=DEV)[: S * W].to(torch.int32).view(S, W)


def _rows(shape, g):
    """Projected rows: channels of different spread and offset."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.rand(shape[-1], generator=g, device=DEV).mul_(1.5).add_(0.25)
    return x.add_(torch.randn(shape[-1], generator=g, device=DEV).mul_(0.2))


def _cache(c, NB, g):
    """A cache full of quantised rows, made a piece of the blocks at a time."""
    B, H, D = c["block"], c["hkv"], c["dim"]
    out = torch.empty((NB, H, B * (D * c["bits"] // 8 + 4)), dtype=torch.uint8, device=DEV)
    piece = max(1, (1 << 27) // (B * H * D))
    for b in range(0, NB, piece):
        n = min(piece, NB - b)
        out[b: b + n] = _pack(*_quantise(_rows((n, H, B, D), g).to(torch.bfloat16), c["bits"]), c["bits"])
    return out


def prepare(c, seed):
    g = _gen(seed)
    op, D = c["op"], c["dim"]
    i32 = dict(dtype=torch.int32, device=DEV)
    if op == "packed":
        S, Hq, Hkv = c["seqs"], c["hq"], c["hkv"]
        ql = _spread(S, c["spread"], 1.0, g).mul(c["query"]).round().clamp_(min=1).to(torch.int32)
        ctx = torch.linspace(0.75, 1.0, S, device=DEV, dtype=torch.float64).mul(c["context"]).round().to(torch.int32)
        ctx = ctx[torch.randperm(S, generator=g, device=DEV)]
        qs = torch.nn.functional.pad(ql.cumsum(0), (1, 0)).to(torch.int32)
        ks = torch.nn.functional.pad((ql + ctx).cumsum(0), (1, 0)).to(torch.int32)
        Tq, Tk = int(qs[-1]), int(ks[-1])
        if c["fused"] and c["context"] == 0:  # slices of one projection's rows
            qkv = torch.cat([torch.randn((Tq, Hq, D), generator=g, device=DEV), _rows((Tq, 2 * Hkv, D), g)], 1)
            q, k, v = qkv.to(torch.bfloat16).split([Hq, Hkv, Hkv], 1)
        else:
            q = torch.randn((Tq, Hq, D), generator=g, device=DEV).to(torch.bfloat16)
            k, v = (_rows((Tk, Hkv, D), g).to(torch.bfloat16) for _ in range(2))
        return dict(c=c, q=q, k=k, v=v, q_start_loc=qs, k_start_loc=ks, max_query_len=int(ql.max()), scale=D ** -0.5,
                    q_host=qs.tolist(), k_host=ks.tolist(), out=torch.empty((Tq, Hq, D), dtype=torch.bfloat16, device=DEV))
    S, B, Hkv = c["seqs"], c["block"], c["hkv"]
    Q = c.get("query", 0)
    lens = _lens(c, S, g).clamp_(min=max(Q, 1))
    W, NB, table = _table(c, S, max(_longest(c), Q), g)
    st = dict(c=c, S=S, B=B, W=W, NB=NB, seq_lens=lens, block_table=table, max_seq_len=W * B)
    if op == "store":
        T, dt = S * Q, TORCH[c["dtype"]]
        if c["fused"]:
            k, v = _rows((T, 2 * Hkv, D), g).to(dt).split([Hkv, Hkv], 1)
        else:
            k, v = (_rows((T, Hkv, D), g).to(dt) for _ in range(2))
        pos = lens.long()[:, None] - Q + torch.arange(Q, device=DEV)
        slots = (table.long().gather(1, pos // B) * B + pos % B).view(-1)
        shape = (NB, Hkv, B * (D * c["bits"] // 8 + 4))
        caches = [torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2)]
        outs = [torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        return dict(st, k=k, v=v, slots=slots, k_cache=caches[0], v_cache=caches[1], k_out=outs[0], v_out=outs[1],
                    start=lens - Q, row_start_loc=torch.arange(S + 1, **i32) * Q)
    st["k_cache"], st["v_cache"] = _cache(c, NB, g), _cache(c, NB, g)
    if op == "read":
        st["row_start_loc"] = torch.nn.functional.pad(lens.cumsum(0), (1, 0)).to(torch.int32)
        rows = int(st["row_start_loc"][-1])
        st["k_out"], st["v_out"] = (torch.empty((rows, Hkv, D), dtype=TORCH[c["dtype"]], device=DEV) for _ in range(2))
        return st
    q = torch.randn((S * Q, c["hq"], D), generator=g, device=DEV).to(torch.bfloat16)
    st.update(q=q, out=torch.empty_like(q), query_start_loc=torch.arange(S + 1, **i32) * Q, scale=D ** -0.5)
    if own:
        import paged_kv_cache_161_gb300 as pa

        n = pa.attention_int_workspace_size(S, S * Q, c["hq"], Hkv, D)
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------------- one pass
def run(st):
    op = st["c"]["op"]
    if own:
        return _own(op, st)
    return {"store": _store, "read": _read, "decode": _decode, "packed": _packed}[op](st)


def _own(op, st):
    import paged_kv_cache_161_gb300 as pa

    if op == "packed":
        pa.attention_packed(st["out"], st["q"], st["k"], st["v"], st["q_start_loc"], st["k_start_loc"],
                            max_query_len=st["max_query_len"], scale=st["scale"])
        return st["out"]
    bits = st["c"]["bits"]
    if op == "decode":
        pa.attention_int(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_table"], st["seq_lens"],
                         st["query_start_loc"], bits=bits, max_query_len=st["c"]["query"], max_seq_len=st["max_seq_len"],
                         scale=st["scale"], workspace=st["workspace"])
        return st["out"]
    start = None
    if op == "store":
        pa.kv_write_int(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"], bits=bits)
        start = st["start"]
    pa.kv_read_int(st["k_out"], st["v_out"], st["k_cache"], st["v_cache"], st["block_table"], start, st["seq_lens"],
                   st["row_start_loc"], bits=bits)
    return [st["k_out"], st["v_out"]]


def _store(st):
    c, B, D, bits = st["c"], st["B"], st["c"]["dim"], st["c"]["bits"]
    row = D * bits // 8
    blk, off = st["slots"] // B, st["slots"] % B
    out = []
    for x, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
        one = _pack(*(y[:, :, None] for y in _quantise(x, bits)), bits)  # blocks of one row: [T, Hkv, row + 4]
        codes = cache[:, :, : B * row].unflatten(2, (B, row))  # views of the cache
        params = cache[:, :, B * row:].unflatten(2, (B, 4))
        codes[blk, :, off] = one[:, :, :row]
        params[blk, :, off] = one[:, :, row:]
        back = torch.cat([codes[blk, :, off], params[blk, :, off]], 2)
        out.append(_values(back, D, bits)[:, :, 0].to(torch.bfloat16))
    return out


def _read(st):
    c = st["c"]
    L, B = st["seq_lens"].long(), st["B"]
    s = torch.repeat_interleave(torch.arange(st["S"], device=DEV), L, output_size=st["k_out"].shape[0])
    pos = torch.arange(st["k_out"].shape[0], device=DEV) - st["row_start_loc"].long()[s]
    blk, off = st["block_table"].long()[s, pos // B], pos % B
    row = c["dim"] * c["bits"] // 8
    out = []
    for cache in (st["k_cache"], st["v_cache"]):
        codes = cache[:, :, : B * row].unflatten(2, (B, row))[blk, :, off]
        params = cache[:, :, B * row:].unflatten(2, (B, 4))[blk, :, off]
        out.append(_values(torch.cat([codes, params], 2), c["dim"], c["bits"])[:, :, 0].to(st["k_out"].dtype))
    return out


def _decode(st):
    c, S, W, B, Q = st["c"], st["S"], st["W"], st["B"], st["c"]["query"]
    Hkv, G, D, bits = c["hkv"], c["hq"] // c["hkv"], c["dim"], c["bits"]
    out = []
    step = max(1, (1 << 31) // (W * B * Hkv * D))  # requests at a time: a few of these in float32 fit the card
    for s in range(0, S, step):
        t = st["block_table"][s: s + step].long()
        n = t.shape[0]
        k = _values(st["k_cache"][t], D, bits).transpose(1, 2).reshape(n, Hkv, W * B, D)
        v = _values(st["v_cache"][t], D, bits).transpose(1, 2).reshape(n, Hkv, W * B, D)
        q = st["q"][s * Q: (s + n) * Q].float().view(n, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(n, Hkv, Q * G, D)
        x = torch.matmul(q, k.transpose(2, 3)).mul_(st["scale"]).view(n, Hkv, Q, G, W * B)
        p = st["seq_lens"][s: s + n].long()[:, None] - Q + torch.arange(Q, device=DEV)
        hidden = torch.arange(W * B, device=DEV) > p[:, None, :, None, None]
        x = x.masked_fill_(hidden, -math.inf)
        x = (x - x.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(x.view(n, Hkv, Q * G, W * B), v).view(n, Hkv, Q, G, D) / x.sum(-1, keepdim=True)
        out.append(o.permute(0, 2, 1, 3, 4).reshape(n * Q, Hkv * G, D).to(torch.bfloat16))
    return torch.cat(out)


def _packed(st):
    c = st["c"]
    Hkv, G, D = c["hkv"], c["hq"] // c["hkv"], c["dim"]
    out = torch.empty_like(st["out"])
    for s in range(c["seqs"]):
        q0, q1, k0, k1 = st["q_host"][s], st["q_host"][s + 1], st["k_host"][s], st["k_host"][s + 1]
        Q, K = q1 - q0, k1 - k0
        hidden = torch.arange(K, device=DEV) > torch.arange(K - Q, K, device=DEV)[:, None]
        step = max(1, min(Hkv, (1 << 31) // (G * Q * K)))  # KV heads at a time
        for h in range(0, Hkv, step):
            n = min(step, Hkv - h)
            q = st["q"][q0: q1, h * G: (h + n) * G].float().view(Q, n, G, D).permute(1, 2, 0, 3)
            k = st["k"][k0: k1, h: h + n].float().permute(1, 2, 0)[:, None]
            v = st["v"][k0: k1, h: h + n].float().transpose(0, 1)[:, None]
            x = torch.matmul(q, k).mul_(st["scale"]).masked_fill_(hidden, -math.inf)
            x = x.sub_(x.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
            out[q0: q1, h * G: (h + n) * G] = o.permute(2, 0, 1, 3).reshape(Q, n * G, D).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------------------- what a pass needs
def work(c):
    D = c["dim"]
    if c["op"] == "packed":
        T = c["seqs"] * c["query"]
        K = T + c["seqs"] * c["context"] * 7 / 8
        seen = T * (c["query"] / 2 * math.exp(c["spread"] ** 2) + c["context"] * 7 / 8)  # key rows of all query rows
        return dict(bytes=4 * T * c["hq"] * D + 4 * K * c["hkv"] * D, flops=4.0 * c["hq"] * D * seen)
    row = c["hkv"] * (D * c["bits"] // 8 + 4) * 2  # a token's codes
    if c["op"] == "store":
        T = c["seqs"] * c["query"]
        return dict(bytes=T * (2 * c["hkv"] * D * (BYTES[c["dtype"]] + 2) + row + 8), flops=6.0 * T * 2 * c["hkv"] * D)
    L = c["seqs"] * c["median"] * math.exp(c["spread"] ** 2 / 2)
    if c["op"] == "read":
        return dict(bytes=L * (2 * c["hkv"] * D * BYTES[c["dtype"]] + row), flops=2.0 * L * 2 * c["hkv"] * D)
    T = c["seqs"] * c["query"]
    return dict(bytes=L * row + 4 * T * c["hq"] * D, flops=4.0 * L * c["query"] * c["hq"] * D)


# ------------------------------------------------------------------------------- 64 bits
def _exact_rows(cache, blocks, D, bits):
    """Values in float64 of the rows of `blocks` (one request's, in order): [positions, Hkv, D]."""
    raw = cache[blocks]
    n, H, size = raw.shape
    row = D * bits // 8
    B = size // (row + 4)
    codes = raw[:, :, : B * row].reshape(n, H, B, row)
    if bits == 4:
        full = torch.empty((n, H, B, D), dtype=torch.uint8, device=DEV)
        full[..., 0::2], full[..., 1::2] = codes % 16, codes // 16
        codes = full
    par = raw[:, :, B * row:].reshape(n, H, B, 4).contiguous().view(torch.bfloat16).double()
    val = par[..., :1] + par[..., 1:] * codes.double()
    return val.permute(0, 2, 1, 3).reshape(n * B, H, D)


def _exact_stored(x, bits):
    """What a row reads back as, from the definition: float64, the two bfloat16 parameters by search."""
    y = x.double()
    low, high = y.min(-1).values, y.max(-1).values
    lo = low.float().bfloat16()
    lo = torch.where(lo.double() > low, torch.nextafter(lo, torch.full_like(lo, -math.inf)), lo)
    want = ((high - lo.double()).float().double() / _levels(bits)).float()
    step = want.bfloat16()
    step = torch.where(step.float() < want, torch.nextafter(step, torch.full_like(step, math.inf)), step)
    step = step.double().clamp(min=2.0 ** -126)
    inv = (1.0 / step).float().double()[..., None]
    code = torch.round((y - lo.double()[..., None]).float().double() * inv)
    return lo.double()[..., None] + step[..., None] * code


def _exact_attention(q, k, v, first, scale):
    """q [Q, Hq, D], k and v [K, Hkv, D] in float64; row j sees keys 0 .. first + j."""
    Q, Hq, D = q.shape
    K, Hkv = k.shape[:2]
    G = Hq // Hkv
    out = torch.empty((Q, Hq, D), dtype=torch.float64, device=DEV)
    piece = max(1, (1 << 28) // K)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        for j in range(0, Q, piece):
            n = min(piece, Q - j)
            last = first + j + n  # keys the piece can see
            x = q[j: j + n, h] @ kh[:last].T * scale
            seen = torch.arange(last, device=DEV)[None] <= first + j + torch.arange(n, device=DEV)[:, None]
            out[j: j + n, h] = torch.softmax(x.where(seen, torch.tensor(-math.inf, dtype=x.dtype, device=DEV)), 1) @ vh[:last]
    return out


def exact(c, seed):
    """The definitions in float64, request by request."""
    st = prepare(c, seed)
    D = c["dim"]
    if c["op"] == "packed":
        qs, ks = st["q_host"], st["k_host"]
        return torch.cat([_exact_attention(st["q"][a:b].double(), st["k"][e:f].double(), st["v"][e:f].double(),
                                           (f - e) - (b - a), st["scale"])
                          for a, b, e, f in zip(qs, qs[1:], ks, ks[1:])])
    if c["op"] == "store":
        return [_exact_stored(st["k"], c["bits"]), _exact_stored(st["v"], c["bits"])]
    lens = st["seq_lens"].tolist()
    table = st["block_table"].long()

    def rows(s, cache):
        return _exact_rows(cache, table[s, : -(-lens[s] // c["block"])], D, c["bits"])[: lens[s]]

    if c["op"] == "read":
        return [torch.cat([rows(s, cache) for s in range(c["seqs"])]) for cache in (st["k_cache"], st["v_cache"])]
    Q = c["query"]
    return torch.cat([_exact_attention(st["q"][s * Q: (s + 1) * Q].double(), rows(s, st["k_cache"]),
                                       rows(s, st["v_cache"]), lens[s] - Q, st["scale"]) for s in range(c["seqs"])])
