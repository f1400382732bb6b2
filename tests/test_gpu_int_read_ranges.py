"""pa_kv_read_int reports every request whose positions do not fit, with or without rows of its own."""
import pytest
import torch

from test_gpu_int_cache import I32, _cache, pa  # noqa: F401

pytestmark = pytest.mark.gpu


def _read(pa, lens, starts, rsl, R, W=8, B=16, H=2, D=64):  # noqa: F811
    cache = torch.zeros_like(_cache(8, H, B, D, 8))
    table = torch.arange(8, dtype=I32).repeat(len(lens), 1)[:, :W].contiguous().cuda()
    i32 = lambda v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    out = [torch.full((R, H, D), 7.0, device="cuda") for _ in range(2)]
    pa.kv_read_int(*out, cache, cache, table, None if starts is None else i32(starts), i32(lens), i32(rsl), bits=8)
    torch.cuda.synchronize()
    assert torch.equal(*out)
    return pa.read_device_errors(), (out[0] == 0).all(-1).all(-1).tolist()


def test_rows_past_the_buffer(pa):  # noqa: F811
    err, done = _read(pa, [5, 60], None, [0, 5, 65], 40)  # the second starts inside and runs past
    assert err == 0x4 and done == [True] * 5 + [False] * 35
    err, done = _read(pa, [5, 60], None, [0, 40, 100], 40)  # starts behind
    assert err == 0x4 and done == [True] * 5 + [False] * 35
    err, done = _read(pa, [5, 6], None, [0, 20, 50], 40)  # room past the buffer that no position needs
    assert err == 0 and done == [True] * 5 + [False] * 15 + [True] * 6 + [False] * 14


def test_positions_without_rows(pa):  # noqa: F811
    for S, at in ((3, 1), (700, 650), (300, 0), (513, 512)):
        lens, rsl = [0] * S, [0] * (S + 1)
        lens[at] = 9
        err, done = _read(pa, lens, None, rsl, 4)
        assert err == 0x4 and not any(done)
        lens[at] = 0
        assert _read(pa, lens, None, rsl, 4)[0] == 0
        starts = [0] * S
        starts[at] = -1
        assert _read(pa, lens, starts, rsl, 4)[0] == 0x4
        starts[at], lens[at] = 3, 3  # nothing asked for
        assert _read(pa, lens, starts, rsl, 4)[0] == 0
        starts[at], lens[at] = 200, 200  # longer than its table
        assert _read(pa, lens, starts, rsl, 4)[0] == 0x4


def test_an_empty_request_with_rows_elsewhere(pa):  # noqa: F811
    """Padding entries of a batch: no positions, rows behind the buffer or none."""
    err, done = _read(pa, [4, 0, 0, 0], [0, 0, 0, 0], [1, 5, 5, 70, 90], 10)
    assert err == 0 and done == [False] + [True] * 4 + [False] * 5
    err, done = _read(pa, [4, 2, 3], None, [0, 4, 3, 6], 10)  # row_start_loc decreases: two rows asked of -1
    assert err == 0x4
