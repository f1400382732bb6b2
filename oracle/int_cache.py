"""Integer-coded caches and packed prompts, stated in NumPy.

A row x of one token and KV head is held as codes c in 0 .. 2^bits - 1 with a smallest value lo and
a step (both bfloat16): x ~ lo + step c. The definition's binary32 roundings (the spread, its part,
the reciprocal, the difference) are stated as such; everything else is float64. The cache is
uint8 [num_blocks, num_kv_heads, block_size * (D * bits / 8 + 4)]: the rows' codes, then their lo and
step. No counterpart in the pages beyond the blocks, slots and tables they describe.
"""
import numpy as np

MIN_STEP = 2.0 ** -126


def _grid(x):
    """The spacing of bfloat16 values around x (8 significant bits, none below 2^-133)."""
    _, e = np.frexp(np.where(x == 0, 1.0, x))
    return np.where(x == 0, 1.0, np.maximum(np.ldexp(1.0, e - 8), 2.0 ** -133))


def bf16_down(x):
    x = np.asarray(x, np.float64)
    return np.floor(x / _grid(x)) * _grid(x)


def bf16_up(x):
    x = np.asarray(x, np.float64)
    return np.ceil(x / _grid(x)) * _grid(x)


def quantise(x, bits):
    """x [..., D], values of float32: (codes [..., D] int, lo [...], step [...]); NaN lo and step where the
    row holds something that is not finite, or spreads past the largest float32."""
    x = np.asarray(x, np.float64)
    n = 2 ** bits - 1
    with np.errstate(all="ignore"):
        lo = bf16_down(x.min(-1))
        spread = np.float32(x.max(-1) - lo)
        step = np.maximum(bf16_up(np.float32(spread / np.float32(n))), MIN_STEP)
        inv = np.float32(1.0 / step)
        top = float(np.finfo(np.float32).max)
        bad = ~np.isfinite(x).all(-1) | (np.abs(lo) > top) | ~np.isfinite(spread) | (step > top)
        codes = np.rint(np.float32(x - lo[..., None]).astype(np.float64) * inv[..., None].astype(np.float64))
    codes = np.where(bad[..., None], 0, codes).astype(np.int64)
    return codes, np.where(bad, np.nan, lo), np.where(bad, np.nan, step)


def value(codes, lo, step):
    return lo[..., None] + step[..., None] * codes


def _bf16_bits(x):
    with np.errstate(all="ignore"):
        f = np.asarray(x, np.float64).astype(np.float32)
    return np.where(np.isnan(f), 0x7FC0, f.view(np.uint32) >> 16).astype(np.uint16)


def row_bytes(D, bits):
    return D * bits // 8


def block_size_of(cache, D, bits):
    return cache.shape[2] // (row_bytes(D, bits) + 4)


def write(cache, x, slots, bits):
    """The cache (a copy) with row x[t] (t-th token, [Hkv, D]) in slot slots[t]; negative: nowhere."""
    cache = cache.copy()
    T, H, D = x.shape
    B, row = block_size_of(cache, D, bits), row_bytes(D, bits)
    codes, lo, step = quantise(x, bits)
    if bits == 4:
        data = (codes[..., 0::2] + 16 * codes[..., 1::2]).astype(np.uint8)
    else:
        data = codes.astype(np.uint8)
    params = np.stack([_bf16_bits(lo), _bf16_bits(step)], -1).view(np.uint8)  # little-endian
    for t in range(T):
        if slots[t] >= 0:
            b, o = divmod(int(slots[t]), B)
            cache[b, :, o * row:(o + 1) * row] = data[t]
            cache[b, :, B * row + 4 * o: B * row + 4 * o + 4] = params[t]
    return cache


def rows(cache, table, length, D, bits):
    """(values, lo, step) of positions 0 .. length - 1 of one request: [length, Hkv, D], [length, Hkv] twice."""
    B, row = block_size_of(cache, D, bits), row_bytes(D, bits)
    pos = np.arange(length)
    blk, off = np.asarray(table)[pos // B].astype(np.int64), pos % B
    H = cache.shape[1]
    data = cache[blk][:, :, : B * row].reshape(length, H, B, row)[pos, :, off]
    if bits == 4:
        codes = np.empty((length, H, D), np.int64)
        codes[..., 0::2], codes[..., 1::2] = data & 15, data >> 4
    else:
        codes = data.astype(np.int64)
    par = cache[blk][:, :, B * row:].reshape(length, H, B, 4)[pos, :, off].astype(np.uint32)
    lo = ((par[..., 0] | par[..., 1] << 8) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
    step = ((par[..., 2] | par[..., 3] << 8) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
    return value(codes, lo, step), lo, step


def attend(q, k, v, first, scale):
    """q [Q, Hq, D], k and v [K, Hkv, D]; row j sees keys 0 .. first + j. Returns (out, the weights' mean of
    |v|, the largest scale sum_d |q_d k_d|, sigma = sqrt(sum w^2 v^2) + |out| sqrt(sum w^2)); rows that see
    nothing are zero."""
    Q, Hq, D = q.shape
    K, G = k.shape[0], Hq // k.shape[1]
    out, mag, sigma = (np.zeros(q.shape) for _ in range(3))
    size = np.zeros((Q, Hq, 1))
    hidden = np.arange(K)[None] > first + np.arange(Q)[:, None]
    if K == 0:
        return out, mag, size, sigma
    none = hidden.all(1)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        x = scale * (q[:, h] @ kh.T)
        x[hidden] = -np.inf
        x[none] = 0.0
        w = np.exp(x - x.max(1, keepdims=True))
        w[hidden] = 0.0
        total = w.sum(1, keepdims=True)
        w /= np.where(total > 0, total, 1.0)
        out[:, h], mag[:, h] = w @ vh, w @ np.abs(vh)
        size[:, h, 0] = (scale * (np.abs(q[:, h]) @ np.abs(kh).T)).max(1)
        sigma[:, h] = np.sqrt((w * w) @ (vh * vh)) + np.abs(out[:, h]) * np.sqrt((w * w).sum(1, keepdims=True))
    return out, mag, size, sigma


def packed(q, k, v, q_start, k_start, scale):
    """attend() of every request of packed rows; NaN in the rows of no request."""
    res = [np.full(q.shape, np.nan), np.full(q.shape, np.nan), np.full(q.shape[:2] + (1,), np.nan),
           np.full(q.shape, np.nan)]
    for a, b, c, d in zip(q_start, q_start[1:], k_start, k_start[1:]):
        for to, got in zip(res, attend(q[a:b], k[c:d], v[c:d], (d - c) - (b - a), scale)):
            to[a:b] = got
    return res
