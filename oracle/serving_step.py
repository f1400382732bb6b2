"""Oracle serving-step operators in float64: batch metadata from lengths, norm + rotary +
cache write, and block-sparse attention (bounds, scores, selection, attention).

Test infrastructure (see the package docstring). Arrays are float64 values (a cache is
[num_blocks, B, Hkv, D] of the values its elements stand for); written as loops over
requests, tokens and heads, straight from the definitions.

Sources and readings:
- advance_ref: vLLM 0.10.0 flow page, 3.3 / 3.5 (block_table, slot_mapping,
  query_start_loc) and the docs page's algorithm flow: blocks are taken lazily, in request
  order, from the head of the free list. A step that does not fit changes nothing.
- the norm, the rotation and block-sparse attention have no counterpart in the pages: the
  definitions are the header's.
"""
from __future__ import annotations

import numpy as np


def advance_ref(table, seq_lens, query_lens, free, head, num_tokens, B, num_blocks):
    """Returns (table, seq_lens, head, query_start_loc, slots, positions)."""
    S, W = table.shape
    slots, positions = [-1] * num_tokens, [0] * num_tokens
    need = [-(-(c + n) // B) - -(-c // B) for c, n in zip(seq_lens, query_lens)]
    if (min([*seq_lens, *query_lens, 0]) < 0 or any(c + n > W * B for c, n in zip(seq_lens, query_lens))
            or sum(query_lens) > num_tokens or head < 0 or head + sum(need) > len(free)):
        return table.copy(), list(seq_lens), head, [0] * (S + 1), slots, positions
    table, qsl, t = table.copy(), [0], 0
    for s in range(S):
        for p in range(seq_lens[s], seq_lens[s] + query_lens[s]):
            if p % B == 0:
                table[s, p // B] = free[head]
                head += 1
            b = int(table[s, p // B])
            slots[t] = b * B + p % B if 0 <= b < num_blocks else -1
            positions[t] = p
            t += 1
        qsl.append(t)
    return table, [c + n for c, n in zip(seq_lens, query_lens)], head, qsl, slots, positions


def norm_rope_ref(x, weight, eps, cos, sin, interleaved):
    """One head row x [D]: its norm, and the norm rotated by cos, sin [rot / 2]."""
    y = x if weight is None else x / np.sqrt(np.mean(x * x) + eps) * weight
    z = y.copy()
    half = len(cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        z[a] = y[a] * cos[i] - y[b] * sin[i]
        z[b] = y[b] * cos[i] + y[a] * sin[i]
    return y, z


def angles_of(cos_sin, positions, sections, t):
    """cos, sin [rot / 2] of token t: pair i turns with the position of its axis."""
    half = cos_sin.shape[1] // 2
    axis = np.repeat(np.arange(len(sections)), sections)
    rows = [positions[a][t] for a in axis]
    return (np.array([cos_sin[r, i] for i, r in enumerate(rows)]),
            np.array([cos_sin[r, half + i] for i, r in enumerate(rows)]))


def rows_of(seq_lens, query_start_loc):
    """(token, request, position) of every query token."""
    for s, L in enumerate(seq_lens):
        a, b = query_start_loc[s], query_start_loc[s + 1]
        for t in range(a, b):
            yield t, s, L - (b - a) + t - a


def bounds_ref(bounds, k, table, seq_lens, query_start_loc):
    """bounds [num_blocks, Hkv, 2, D] with the touched blocks' entries replaced."""
    bounds, B = bounds.copy(), k.shape[1]
    for _, s, p in rows_of(seq_lens, query_start_loc):
        id_ = table[s][p // B]
        keys = k[id_, : min(B, seq_lens[s] - p // B * B)]
        bounds[id_, :, 0], bounds[id_, :, 1] = keys.min(0), keys.max(0)
    return bounds


def scores_ref(q, bounds, table, seq_lens, query_start_loc, B, width):
    """(scores [T, Hkv, width], the sums of the terms' magnitudes); rows of no request are NaN."""
    T, Hq, _ = q.shape
    Hkv = bounds.shape[1]
    G = Hq // Hkv
    out, size = np.full((T, Hkv, width), np.nan), np.zeros((T, Hkv, width))
    for t, s, p in rows_of(seq_lens, query_start_loc):
        out[t] = -np.inf
        for b in range(p // B + 1):
            lo, hi = bounds[table[s][b], :, 0], bounds[table[s][b], :, 1]
            for g in range(Hkv):
                heads = q[t, g * G:(g + 1) * G]
                terms = np.maximum(heads * lo[g], heads * hi[g])
                out[t, g, b] = terms.sum(-1).max()
                both = np.abs(heads * lo[g]) + np.abs(heads * hi[g])
                size[t, g, b] = both.sum(-1).max()
    return out, size


def select_ref(scores, seq_lens, query_start_loc, B, k, init, local):
    """block lists [T, Hkv, k]; rows of no request are -2."""
    T, Hkv, _ = scores.shape
    out = np.full((T, Hkv, k), -2, np.int32)
    for t, _, p in rows_of(seq_lens, query_start_loc):
        last = p // B
        for g in range(Hkv):
            forced = [b for b in range(last + 1) if b < init or b > last - local]
            rest = [b for b in range(last + 1) if b not in forced and scores[t, g, b] > -np.inf]
            rest.sort(key=lambda b: (-scores[t, g, b], b))
            chosen = sorted(forced + rest[: k - len(forced)])
            out[t, g] = chosen + [-1] * (k - len(chosen))
    return out


def attention_sparse_ref(q, k, v, table, seq_lens, query_start_loc, block_idx, scale):
    """(out [T, Hq, D], sum_j w_j |v_j|, max_j scale sum_d |q_d k_jd|); rows of no request are NaN."""
    T, Hq, D = q.shape
    B, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out, mag, logit = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros((T, Hq, 1))
    for t, s, p in rows_of(seq_lens, query_start_loc):
        out[t] = 0.0
        for g in range(Hkv):
            at = [(table[s][b], i) for b in block_idx[t, g] if b >= 0 for i in range(B) if b * B + i <= p]
            if not at:
                continue
            ids, offs = np.array(at).T
            K, V = k[ids, offs, g], v[ids, offs, g]
            for h in range(g * G, (g + 1) * G):
                x = scale * (K @ q[t, h])
                w = np.exp(x - x.max())
                w /= w.sum()
                out[t, h], mag[t, h] = w @ V, w @ np.abs(V)
                logit[t, h] = scale * (np.abs(K) @ np.abs(q[t, h])).max()
    return out, mag, logit
