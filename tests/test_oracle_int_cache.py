"""Pins of the integer-coded cache's oracle: its roundings against torch's bfloat16, the codes against
their definition row by row, the layout byte by byte, attention against torch's own."""
import numpy as np
import pytest
import torch

from oracle import int_cache as ic


def _f32(*shape, seed=0, size=1.0):
    return (np.random.default_rng(seed).standard_normal(shape) * size).astype(np.float32)


def test_directed_roundings_bracket_the_value_with_neighbours():
    x = np.concatenate([_f32(4000, seed=1), _f32(500, seed=2, size=1e30), _f32(500, seed=3, size=1e-38), [0.0, 1.0, -2.5]])
    x = x.astype(np.float32).astype(np.float64)
    down, up = ic.bf16_down(x), ic.bf16_up(x)
    assert (down <= x).all() and (x <= up).all()
    for y in (down, up):
        t = torch.tensor(y, dtype=torch.float64)
        assert torch.equal(t.to(torch.bfloat16).double(), t)  # bfloat16 values
    exact = torch.tensor(x).to(torch.bfloat16).double().numpy() == x
    assert np.array_equal(down == up, exact)
    a, b = (torch.tensor(y).to(torch.bfloat16) for y in (down, up))
    nxt = torch.nextafter(a, torch.full_like(a, float("inf")))
    assert torch.equal(torch.where(torch.tensor(exact), a, nxt), b)  # nothing lies between


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("size,shift", [(1.0, 0.0), (1e-3, 5.0), (1e30, 0.0), (1e-38, 0.0)])
def test_codes_stay_in_range_and_values_within_half_a_step(bits, size, shift):
    x = (_f32(300, 64, seed=bits, size=size) + np.float32(shift)).astype(np.float64)
    c, lo, step = ic.quantise(x, bits)
    assert c.min() >= 0 and c.max() <= 2 ** bits - 1
    # three binary32 roundings of y, inv and their product move a border by 2^-22 of the code
    assert (np.abs(ic.value(c, lo, step) - x) <= step[:, None] * (0.5 + 2.0 ** -22 * 2 ** bits)).all()
    assert (lo <= x.min(1)).all()


def test_rows_of_one_value_bfloat16_minimum_and_bad_rows():
    x = np.zeros((6, 8))
    x[1] = -3.25
    x[2] = np.arange(8)
    x[3, 4] = np.nan
    x[4, 0] = np.inf
    x[5, :2] = 3e38, -3e38
    c, lo, step = ic.quantise(x, 8)
    assert (c[:2] == 0).all() and lo[0] == 0 and lo[1] == -3.25 and (step[:2] == ic.MIN_STEP).all()
    assert lo[2] == 0 and np.abs(ic.value(c, lo, step)[2] - x[2]).max() <= step[2] / 2
    assert np.isnan(lo[3:]).all() and np.isnan(step[3:]).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_layout(bits):
    B, H, D = 4, 2, 64
    row = D * bits // 8
    cache = np.full((3, H, B * (row + 4)), 0xAA, np.uint8)
    x = _f32(3, H, D, seed=5).astype(np.float64)
    out = ic.write(cache, x, [9, -1, 2], bits)
    c, lo, step = ic.quantise(x, bits)
    for t, (b, o) in ((0, (2, 1)), (2, (0, 2))):
        for h in range(H):
            got = out[b, h, o * row:(o + 1) * row]
            want = c[t, h] if bits == 8 else [c[t, h, 2 * i] | c[t, h, 2 * i + 1] << 4 for i in range(D // 2)]
            assert got.tolist() == list(want)
            par = torch.tensor(out[b, h, B * row + 4 * o: B * row + 4 * o + 4].copy()).view(torch.bfloat16).double()
            assert par.tolist() == [lo[t, h], step[t, h]]
    same = out == cache
    assert same[1].all() and (~same).sum() <= 2 * H * (row + 4)  # nothing else was written
    values, l2, s2 = ic.rows(out, [2, 1, 0], 11, D, bits)
    assert np.array_equal(values[1], ic.value(c, lo, step)[0]) and np.array_equal(values[10], ic.value(c, lo, step)[2])
    assert np.array_equal(l2[1], lo[0]) and np.array_equal(s2[10], step[2])


@pytest.mark.parametrize("Q,K,Hq,Hkv", [(5, 5, 4, 2), (3, 9, 4, 1), (1, 7, 2, 2), (6, 4, 2, 1), (2, 0, 2, 1)])
def test_attend_equals_torch(Q, K, Hq, Hkv):
    g = torch.Generator().manual_seed(Q)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((Q, Hq, 16), (K, Hkv, 16), (K, Hkv, 16)))
    out = ic.attend(q.numpy(), k.numpy(), v.numpy(), K - Q, 0.3)[0]
    seen = torch.arange(K)[None] <= K - Q + torch.arange(Q)[:, None]
    live = seen.any(1).numpy()
    assert (out[~live] == 0).all()
    if K:
        kk, vv = (x.repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for x in (k, v))
        ref = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk, vv, attn_mask=seen, scale=0.3)
        assert np.abs(out - ref.transpose(0, 1).numpy())[live].max() < 1e-12


def test_packed_is_attend_per_request():
    g = np.random.default_rng(3)
    q, k, v = g.standard_normal((7, 2, 8)), g.standard_normal((9, 1, 8)), g.standard_normal((9, 1, 8))
    out = ic.packed(q, k, v, [0, 2, 2, 6], [0, 5, 5, 9], 0.5)[0]
    assert np.isnan(out[6]).all()
    assert np.array_equal(out[2:6], ic.attend(q[2:6], k[5:9], v[5:9], 0, 0.5)[0])
    assert np.array_equal(out[:2], ic.attend(q[:2], k[:5], v[:5], 3, 0.5)[0])
