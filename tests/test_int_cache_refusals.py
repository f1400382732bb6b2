"""Refusals of the integer-coded cache's calls and of packed attention: every bad argument is answered on
the host, before any CUDA call (so all of this runs on a machine without a GPU)."""
import pytest
import torch

import paged_kv_cache_161_gb300 as pa

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
L = pa.lib


def _at(n):
    """A distinct, aligned address (never dereferenced: the calls below are all refused)."""
    return 0x100000000 * n


def _check(fn, good, changes):
    for i, val, want in changes:
        a = list(good)
        a[i] = val
        assert getattr(L, fn)(*a) == want, (fn, i, val)


def test_kv_write_int():
    #       k       v       ks    vs    dt kc      vc      slots  T  NB  B   H  D    bits
    good = [_at(1), _at(2), 1024, 2048, 1, _at(3), _at(4), _at(5), 7, 64, 16, 8, 128, 4, None]
    _check("pa_kv_write_int", good, [
        (0, None, INVALID), (1, None, INVALID), (0, _at(1) + 8, INVALID), (2, 1016, INVALID), (2, 1025, INVALID),
        (3, 1023, INVALID), (4, 2, INVALID), (4, 9, INVALID), (5, None, INVALID), (6, None, INVALID),
        (5, _at(3) + 8, INVALID), (7, None, INVALID), (7, _at(5) + 4, INVALID), (8, -1, INVALID), (9, 0, INVALID),
        (10, 0, INVALID), (10, 6, UNSUPPORTED), (10, 1, UNSUPPORTED), (10, 1 << 21, UNSUPPORTED), (11, 0, INVALID),
        (11, 1 << 17, UNSUPPORTED), (12, 0, INVALID), (12, 96, UNSUPPORTED), (12, 256, UNSUPPORTED), (13, 2, UNSUPPORTED),
        (13, 0, UNSUPPORTED), (13, 16, UNSUPPORTED), (9, 1 << 40, UNSUPPORTED), (8, 1 << 40, UNSUPPORTED), (8, 0, OK),
    ])


def test_kv_read_int():
    #       ko      vo      dt kc      vc      table   W  start   lens    rows    S  R    NB  B   H  D    bits
    good = [_at(1), _at(2), 1, _at(3), _at(4), _at(5), 8, _at(6), _at(7), _at(8), 4, 100, 64, 16, 8, 128, 8, None]
    _check("pa_kv_read_int", good, [
        (0, None, INVALID), (1, None, INVALID), (0, _at(1) + 4, INVALID), (2, 2, INVALID), (3, None, INVALID),
        (4, None, INVALID), (5, None, INVALID), (5, _at(5) + 2, INVALID), (6, 0, INVALID), (6, 1 << 28, INVALID),
        (7, _at(6) + 1, INVALID), (8, None, INVALID), (9, None, INVALID), (10, -1, INVALID), (11, -1, INVALID),
        (12, 0, INVALID), (13, 2, UNSUPPORTED), (15, 32, UNSUPPORTED), (16, 5, UNSUPPORTED), (11, 1 << 40, UNSUPPORTED),
        (1, _at(1) + 128, INVALID), (0, _at(3) + 4096, INVALID), (1, _at(4), INVALID), (10, 0, OK), (11, 0, OK),
    ])


def test_attention_int():
    #       out     q       kc      vc      table   W  lens    qsl     S  T  mq ms  Hq  Hkv D    B   NB  scale bits ws     bytes
    good = [_at(1), _at(2), _at(3), _at(4), _at(5), 8, _at(6), _at(7), 4, 9, 3, 100, 32, 8, 128, 16, 64, 0.1, 4, _at(8), 1 << 30,
            None]
    inf, nan = float("inf"), float("nan")
    _check("pa_attention_int", good, [
        (0, None, INVALID), (1, None, INVALID), (0, _at(1) + 8, INVALID), (2, None, INVALID), (3, None, INVALID),
        (4, None, INVALID), (5, 0, INVALID), (5, 6, INVALID), (6, None, INVALID), (7, None, INVALID), (8, -1, INVALID),
        (9, -1, INVALID), (10, -1, INVALID), (10, 101, INVALID), (11, -1, INVALID), (12, 0, INVALID), (12, 30, INVALID),
        (13, 0, INVALID), (14, 32, UNSUPPORTED), (15, 18, UNSUPPORTED), (16, 0, INVALID), (17, 0.0, INVALID),
        (17, -1.0, INVALID), (17, inf, INVALID), (17, nan, INVALID), (18, 6, UNSUPPORTED), (19, None, WORKSPACE),
        (19, _at(8) + 8, WORKSPACE), (0, _at(2) + 4096, INVALID), (8, 4097, UNSUPPORTED), (9, 2**31 - 1, UNSUPPORTED),
        (8, 0, OK), (9, 0, OK),
    ])
    a = list(good)
    a[10] = a[11] = 0  # no queries announced
    assert L.pa_attention_int(*a) == OK


def test_attention_int_workspace_size():
    import ctypes

    out = ctypes.c_size_t(0)
    ref = ctypes.byref(out)
    f = L.pa_attention_int_workspace_size
    for args, want in (((-1, 4, 8, 2, 128, ref), INVALID), ((4, -1, 8, 2, 128, ref), INVALID), ((4, 4, 0, 2, 128, ref), INVALID),
                       ((4, 4, 8, 0, 128, ref), INVALID), ((4, 4, 8, 3, 128, ref), INVALID), ((4, 4, 8, 2, 96, ref), UNSUPPORTED),
                       ((4, 4, 8, 2, 128, None), INVALID)):
        assert f(*args) == want


def test_attention_packed():
    #       out     q       k       v       qs    ks    vs    qsl     ksl     S  T    K    mq Hq  Hkv D    scale dt
    good = [_at(1), _at(2), _at(3), _at(4), 4096, 1024, 1024, _at(5), _at(6), 4, 100, 120, 9, 32, 8, 128, 0.1, 1, None]
    _check("pa_attention_packed", good, [
        (0, None, INVALID), (1, None, INVALID), (2, None, INVALID), (3, None, INVALID), (0, _at(1) + 8, INVALID),
        (1, _at(2) + 2, INVALID), (4, 4095, INVALID), (4, 4088, INVALID), (5, 1023, INVALID), (6, 512, INVALID),
        (7, None, INVALID), (8, None, INVALID), (7, _at(5) + 2, INVALID), (9, -1, INVALID), (10, -1, INVALID),
        (11, -1, INVALID), (12, -1, INVALID), (13, 0, INVALID), (13, 33, INVALID), (13, 24, UNSUPPORTED),
        (13, 128, UNSUPPORTED), (14, 0, INVALID), (15, 96, UNSUPPORTED), (16, 0.0, INVALID), (16, float("nan"), INVALID),
        (17, 0, UNSUPPORTED), (17, 2, UNSUPPORTED), (17, 7, INVALID), (9, 4097, UNSUPPORTED), (10, 2**31 - 1, UNSUPPORTED),
        (11, 2**31 - 1, UNSUPPORTED), (12, 2**31 - 1, UNSUPPORTED), (4, 1 << 40, UNSUPPORTED), (0, _at(2) + 4096, INVALID),
        (0, _at(3) - 16, INVALID), (0, _at(4), INVALID), (9, 0, OK), (10, 0, OK), (12, 0, OK),
    ])


def test_tensors_off_the_gpu_are_refused():
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16 * 36, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pa.kv_write_int(k, k, cache, cache, torch.zeros(3, dtype=torch.int64), bits=4)
    with pytest.raises(ValueError):
        pa.kv_read_int(k, k, cache, cache, torch.zeros(1, 4, dtype=torch.int32), None, torch.zeros(1, dtype=torch.int32),
                       torch.zeros(2, dtype=torch.int32), bits=4)
    with pytest.raises(ValueError):
        pa.attention_packed(k, k, k, k, torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), max_query_len=3,
                            scale=1.0)
    with pytest.raises(TypeError):
        pa.attention_int(k, k, cache, cache)
    with pytest.raises(ValueError):  # pools of two geometries
        pa.swap_blocks(cache, cache, cache[:, :1].contiguous(), cache[:, :1].contiguous(), torch.zeros(0, 2, dtype=torch.int64))
    with pytest.raises(ValueError):
        pa.copy_blocks(cache, cache[:2], torch.zeros(0, 2, dtype=torch.int64))
