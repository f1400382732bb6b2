"""Pins of the serving-step oracle: each function against something other than itself."""
import numpy as np
import pytest

from oracle import BlockAllocator, dense_causal_ref
from oracle import serving_step as ss


@pytest.mark.parametrize("seed", range(8))
def test_advance_equals_the_block_allocator(seed):
    """Request by request appends on the block manager give the same tables and slots."""
    rng = np.random.default_rng(seed)
    B, S, NB = int(rng.choice([1, 4, 16])), 7, 400
    order = rng.permutation(NB).astype(np.int32)
    ref = BlockAllocator(NB, B, order)
    for s in range(S):
        ref.add_seq(s)
    W = 60 // B + 2
    table, lens, head = np.full((S, W), -1), [0] * S, 0
    for _ in range(4):
        q = rng.integers(0, 12, S).tolist()
        want = [x for s in range(S) for x in ref.append(s, q[s])]
        table, lens, head, qsl, slots, pos = ss.advance_ref(table, lens, q, order, head, sum(q) + 3, B, NB)
        assert slots == want + [-1] * 3
        assert lens == [ref.seq_len(s) for s in range(S)] and qsl[-1] == sum(q)
        for s in range(S):
            n = len(ref.block_table(s))
            assert table[s, :n].tolist() == ref.block_table(s)
            assert pos[qsl[s]:qsl[s + 1]] == list(range(lens[s] - q[s], lens[s]))


def test_advance_changes_nothing_when_the_step_does_not_fit():
    table = np.array([[3, -1], [5, 7]])
    for lens, q, free, tokens in [([2, 6], [3, 1], [1], 0), ([2, 6], [4, 1], [], 9), ([4, 8], [1, 1], [1, 2], 9),
                                  ([-1, 6], [1, 1], [1], 9), ([2, 6], [-1, 1], [1], 9)]:
        t, ln, head, qsl, slots, _ = ss.advance_ref(table, lens, q, free, 0, tokens, 4, 8)
        assert np.array_equal(t, table) and ln == lens and head == 0 and qsl == [0, 0, 0] and set(slots) <= {-1}


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation(interleaved):
    """As complex numbers: pair (a, b) times exp(i angle); norms of pairs kept; unit RMS norm."""
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal(64), rng.uniform(0.5, 2, 64)
    ang = rng.uniform(0, 6, 16)
    y, z = ss.norm_rope_ref(x, w, 0.0, np.cos(ang), np.sin(ang), interleaved)
    np.testing.assert_allclose(np.mean((y / w) ** 2), 1.0)
    a, b = (slice(0, 32, 2), slice(1, 32, 2)) if interleaved else (slice(0, 16), slice(16, 32))
    np.testing.assert_allclose(z[a] + 1j * z[b], (y[a] + 1j * y[b]) * np.exp(1j * ang))
    assert np.array_equal(z[32:], y[32:])


def test_scores_bound_every_logit_and_bounds_hold_every_key():
    rng = np.random.default_rng(4)
    B, Hkv, G, D, L = 4, 2, 2, 8, 19
    k = rng.standard_normal((8, B, Hkv, D))
    table, lens, qsl = [[6, 1, 3, 0, 5]], [L], [0, L]
    bounds = ss.bounds_ref(np.zeros((8, Hkv, 2, D)), k, table, lens, qsl)
    q = rng.standard_normal((L, Hkv * G, D))
    scores, _ = ss.scores_ref(q, bounds, table, lens, qsl, B, 6)
    for t in range(L):
        for g in range(Hkv):
            for b in range(6):
                keys = [k[table[0][b], i, g] for i in range(B) if b * B + i < L] if b * B <= t else []
                logits = [q[t, g * G + h] @ key for key in keys for h in range(G)]
                assert (scores[t, g, b] >= max(logits)) if logits else scores[t, g, b] == -np.inf
    # one key a block: the bound is the logit
    one = ss.bounds_ref(np.zeros((8, Hkv, 2, D)), k[:, :1], [[6, 1]], [2], [0, 2])
    s, _ = ss.scores_ref(q[:2], one, [[6, 1]], [2], [0, 2], 1, 2)
    np.testing.assert_allclose(s[1, 0, 1], (q[1, :G] @ k[1, 0, 0]).max())


def test_selection_is_the_top_of_a_stable_sort():
    rng = np.random.default_rng(5)
    s = np.round(rng.standard_normal((1, 3, 40)) * 2)
    out = ss.select_ref(s, [160], [0, 1], 4, 9, 0, 0)
    for g in range(3):
        order = np.argsort(-s[0, g], kind="stable")[:9]
        assert out[0, g].tolist() == sorted(order.tolist())
    s[0, 0, 5:] = -np.inf
    assert ss.select_ref(s, [160], [0, 1], 4, 9, 1, 2)[0, 0].tolist() == [0, 1, 2, 3, 4, 38, 39, -1, -1]


def test_sparse_attention_over_all_blocks_is_dense_attention():
    rng = np.random.default_rng(6)
    B, Hkv, G, D, L, n = 4, 2, 2, 8, 15, 5
    k, v = (rng.standard_normal((6, B, Hkv, D)) for _ in range(2))
    table = [[2, 4, 0, 5]]
    q = rng.standard_normal((n, Hkv * G, D))
    idx = np.tile(np.array([3, 0, 2, 1, -1]), (n, Hkv, 1))
    out, mag, _ = ss.attention_sparse_ref(q, k, v, table, [L], [0, n], idx, 0.4)
    K, V = (x[table[0]].reshape(-1, Hkv, D)[:L] for x in (k, v))
    np.testing.assert_allclose(out, dense_causal_ref(q, K, V, 0.4), rtol=1e-12)
    assert (mag >= np.abs(out)).all()
    empty, _, _ = ss.attention_sparse_ref(q, k, v, table, [L], [0, n], np.full((n, Hkv, 2), -1), 0.4)
    assert not empty.any()
