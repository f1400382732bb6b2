"""Refusals of the serving-step entry points: every bad argument is answered on the host,
before any CUDA call (so all of this runs on a machine without a GPU)."""
import ctypes

import pytest
import torch

import paged_kv_cache_161_gb300 as pa

OK, INVALID, UNSUPPORTED = 0, 1, 2
L = pa.lib


def _at(n):
    """A distinct, aligned address (never dereferenced: the calls below are all refused)."""
    return 0x10000000 * n


def _check(fn, good, changes):
    for i, val, want in changes:
        a = list(good)
        a[i] = val
        assert getattr(L, fn)(*a) == want, (fn, i, val)


def test_advance_batch():
    #       table  W  lens   qlens  free   F  head   lens'  head'  qsl    slots  pos    S  T   B   NB
    good = [_at(1), 8, _at(2), _at(3), _at(4), 9, _at(5), _at(6), _at(7), _at(8), _at(9), _at(10), 4, 20, 16, 64, None]
    _check("pa_advance_batch", good, [
        (0, None, INVALID), (0, _at(1) + 2, INVALID), (1, 0, INVALID), (1, 1 << 30, INVALID), (2, None, INVALID),
        (3, None, INVALID), (4, None, INVALID), (5, -1, INVALID), (6, None, INVALID), (7, None, INVALID),
        (8, None, INVALID), (9, None, INVALID), (10, None, INVALID), (10, _at(9) + 4, INVALID), (11, None, INVALID),
        (12, -1, INVALID), (13, -1, INVALID), (14, 0, INVALID), (15, 0, INVALID), (12, 2**31 - 1, UNSUPPORTED),
        (13, 2**31 - 1, UNSUPPORTED),
        # outputs over inputs or one another; seq_lens_out / free_head_out beside, not on, their inputs
        (7, _at(2) + 4, INVALID), (7, _at(3), INVALID), (8, _at(4), INVALID), (9, _at(2), INVALID),
        (10, _at(1), INVALID), (11, _at(9) + 8, INVALID), (11, _at(5), INVALID), (9, _at(6) - 4, INVALID),
    ])


def test_norm_rope_write():
    sec = (ctypes.c_int * 3)(16, 24, 24)
    bad_sum, neg = (ctypes.c_int * 3)(16, 24, 25), (ctypes.c_int * 3)(-1, 40, 25)
    good = [_at(1), _at(2), _at(3), _at(4), 4096, 1024, 1024, _at(5), _at(6), 1e-6, _at(7), 100, 128, 0, _at(8), 3, sec,
            _at(9), _at(10), _at(11), 5, 64, 16, 32, 8, 128, 1, 1, 1.0, 1.0, None]
    inf, nan = float("inf"), float("nan")
    _check("pa_norm_rope_write", good, [
        (0, None, INVALID), (1, None, INVALID), (2, None, INVALID), (3, None, INVALID), (10, None, INVALID),
        (14, None, INVALID), (17, None, INVALID), (18, None, INVALID), (19, None, INVALID),
        (1, _at(2) + 2, INVALID), (7, _at(5) + 8, INVALID), (10, _at(7) + 4, INVALID), (14, _at(8) + 2, INVALID),
        (17, _at(9) + 4, INVALID), (4, 4095, INVALID), (4, 4090, INVALID), (5, 1023, INVALID), (6, 1016, INVALID),
        (4, 4100, INVALID), (9, -1.0, INVALID), (9, nan, INVALID), (9, inf, INVALID), (11, 0, INVALID),
        (12, 0, INVALID), (12, 144, UNSUPPORTED), (12, 120, UNSUPPORTED), (15, 0, INVALID), (15, 5, INVALID),
        (16, None, INVALID), (16, bad_sum, INVALID), (16, neg, INVALID), (20, -1, INVALID), (21, 0, INVALID),
        (22, 0, INVALID), (23, 0, INVALID), (24, 0, INVALID), (25, 96, UNSUPPORTED), (26, 2, INVALID), (26, 7, INVALID),
        (27, 0, INVALID), (27, 9, INVALID), (28, 0.0, INVALID), (28, inf, INVALID), (29, nan, INVALID),
        (0, _at(2) + 16, INVALID), (0, _at(3), INVALID), (0, _at(4) - 16, INVALID),
        (20, 0, OK), (20, 1 << 40, UNSUPPORTED),
    ])
    a = list(good)
    a[4], a[0] = 6144, _at(2)  # q_out on a q whose tokens lie apart
    assert L.pa_norm_rope_write(*a) == INVALID


def test_block_bounds():
    good = [_at(1), _at(2), _at(3), 8, _at(4), _at(5), 4, 9, 3, 100, 8, 128, 16, 64, 1, None]
    _check("pa_block_bounds", good, [
        (0, None, INVALID), (0, _at(1) + 8, INVALID), (1, None, INVALID), (1, _at(2) + 8, INVALID), (2, None, INVALID),
        (2, _at(3) + 2, INVALID), (3, 0, INVALID), (3, 6, INVALID), (3, 1 << 30, INVALID), (4, None, INVALID),
        (5, None, INVALID), (6, -1, INVALID), (6, 0, OK), (7, -1, INVALID), (7, 0, OK), (8, -1, INVALID), (8, 0, OK),
        (8, 101, INVALID), (9, -1, INVALID), (9, 129, INVALID), (10, 0, INVALID), (11, 96, UNSUPPORTED),
        (12, 0, INVALID), (12, 8, UNSUPPORTED), (12, 24, UNSUPPORTED), (13, 0, INVALID), (14, 0, UNSUPPORTED),
        (14, 5, INVALID), (10, 1 << 29, UNSUPPORTED),
    ])


def test_block_scores():
    good = [_at(1), 7, _at(2), _at(3), _at(4), 8, _at(5), _at(6), 4, 9, 3, 100, 32, 8, 128, 16, 64, None]
    _check("pa_block_scores", good, [
        (0, None, INVALID), (0, _at(1) + 2, INVALID), (1, 6, INVALID), (1, 0, INVALID), (2, None, INVALID),
        (2, _at(2) + 8, INVALID), (3, None, INVALID), (3, _at(3) + 8, INVALID), (4, None, INVALID), (5, 6, INVALID),
        (6, None, INVALID), (7, None, INVALID), (8, -1, INVALID), (8, 0, OK), (9, -1, INVALID), (9, 0, OK),
        (10, 101, INVALID), (11, -1, INVALID), (12, 12, INVALID), (12, 24, UNSUPPORTED), (12, 128, UNSUPPORTED),
        (12, 0, INVALID), (13, 0, INVALID), (14, 32, UNSUPPORTED), (15, 8, UNSUPPORTED), (16, 0, INVALID),
    ])


def test_select_blocks():
    good = [_at(1), 8, _at(2), 100, _at(3), _at(4), 4, 9, 8, 16, 1, 2, None]
    _check("pa_select_blocks", good, [
        (0, None, INVALID), (0, _at(1) + 2, INVALID), (1, 0, INVALID), (1, 2, INVALID), (2, None, INVALID),
        (3, 0, INVALID), (3, 1 << 30, INVALID), (4, None, INVALID), (5, None, INVALID), (5, _at(4) + 2, INVALID),
        (6, -1, INVALID), (6, 0, OK), (7, 0, OK), (7, -1, INVALID), (8, 0, INVALID), (9, 0, INVALID),
        (9, 20, UNSUPPORTED), (10, -1, INVALID), (11, -1, INVALID), (11, 8, INVALID), (8, 1 << 30, UNSUPPORTED),
    ])


def test_attention_sparse():
    good = [_at(1), _at(2), _at(3), _at(4), _at(5), 8, _at(6), _at(7), _at(8), 4, 4, 9, 100, 32, 8, 128, 16, 64, 0.1, 1,
            1.0, 1.0, None]
    inf, nan = float("inf"), float("nan")
    _check("pa_attention_sparse", good, [
        (0, None, INVALID), (0, _at(1) + 8, INVALID), (1, None, INVALID), (1, _at(2) + 8, INVALID), (2, None, INVALID),
        (3, None, INVALID), (3, _at(4) + 8, INVALID), (4, None, INVALID), (5, 6, INVALID), (6, None, INVALID),
        (7, None, INVALID), (8, None, INVALID), (8, _at(8) + 2, INVALID), (9, 0, INVALID), (9, 1 << 30, UNSUPPORTED),
        (10, -1, INVALID), (10, 0, OK), (11, -1, INVALID), (11, 0, OK), (11, 1 << 29, UNSUPPORTED), (12, 129, INVALID),
        (13, 24, UNSUPPORTED), (13, 12, INVALID), (14, 0, INVALID), (15, 96, UNSUPPORTED), (16, 8, UNSUPPORTED),
        (17, 0, INVALID), (18, 0.0, INVALID), (18, nan, INVALID), (18, inf, INVALID), (19, 0, UNSUPPORTED),
        (19, 6, INVALID), (20, 2.0, INVALID), (21, 0.5, INVALID), (20, 0.0, INVALID), (21, inf, INVALID),
    ])


def test_the_binding_refuses_host_tensors():
    z = torch.zeros
    with pytest.raises(ValueError):
        pa.advance_batch(*[z(1, 1, dtype=torch.int32)] * 10, block_size=16, num_blocks=4)
    with pytest.raises(ValueError):
        pa.select_blocks(z(1, 1, 1, dtype=torch.int32), z(1, 1, 1), z(1, dtype=torch.int32), z(2, dtype=torch.int32),
                         block_size=16)
    with pytest.raises(ValueError):
        pa.block_bounds(z(1, 1, 2, 64), z(1, 16, 1, 64), z(1, 1, dtype=torch.int32), z(1, dtype=torch.int32),
                        z(2, dtype=torch.int32), max_query_len=1, max_seq_len=1)
