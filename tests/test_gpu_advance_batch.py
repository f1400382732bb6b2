"""pa_advance_batch on the GPU against its oracle: whole numbers, so equality everywhere."""
import numpy as np
import pytest
import torch

from oracle import serving_step as ss

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_161_gb300 as m

    m.read_device_errors(clear=True)
    return m


def _state(lens, q, free, head, T, B, NB, W, seed=0, alias=False):
    rng = np.random.default_rng(seed)
    S = len(lens)
    table = np.full((S, W), -7, np.int32)
    for s, c in enumerate(lens):
        n = max(0, min(-(-c // B), W))
        table[s, :n] = rng.integers(0, NB, n)
    dev = lambda x, dt=I32: torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    st = dict(table=dev(table), lens=dev(lens), q=dev(q), free=dev(free), head=dev([head]),
              qsl=torch.full((S + 1,), -9, dtype=I32, device="cuda"),
              slots=torch.full((T,), -9, dtype=torch.int64, device="cuda"),
              pos=torch.full((T,), -9, dtype=I32, device="cuda"))
    st["lens_out"] = st["lens"] if alias else torch.full_like(st["lens"], -9)
    st["head_out"] = st["head"] if alias else torch.full_like(st["head"], -9)
    return table, st


def _run(pa, st, B, NB, stream=None):
    pa.advance_batch(st["table"], st["lens"], st["q"], st["free"], st["head"], st["lens_out"], st["head_out"], st["qsl"],
                     st["slots"], st["pos"], block_size=B, num_blocks=NB, stream=stream)


def _compare(st, want):
    table, lens, head, qsl, slots, pos = want
    got = {n: st[n].cpu().numpy().tolist() for n in ("lens_out", "head_out", "qsl", "slots", "pos")}
    assert np.array_equal(st["table"].cpu().numpy(), table)
    assert got["qsl"] == list(qsl)
    assert got["slots"] == list(slots)
    assert got["pos"] == list(pos)
    assert got["lens_out"] == list(lens) and got["head_out"] == [head]


CASES = [  # requests, block size, chunk length, share of chunks / requests without tokens, padding
    ("one_token", 1, 16, 1, 0.0, 0.0, 0),
    ("one_long", 1, 16, 9001, 1.0, 0.0, 5),
    ("decode_256", 256, 16, 1, 0.0, 0.0, 0),
    ("with_empty", 300, 4, 7, 0.3, 0.4, 11),
    ("all_empty", 5, 16, 1, 0.0, 1.0, 3),
    ("tile_edge", 1024, 16, 3, 0.1, 0.2, 1),
    ("two_tiles", 1025, 8, 5, 0.5, 0.1, 0),
    ("many_tiles", 3500, 16, 20, 0.2, 0.3, 77),
    ("sixteen_ctas", 90, 16, 1000, 0.5, 0.1, 40),
    ("block_1", 40, 1, 33, 0.5, 0.1, 2),
    ("wide_block", 70, 128, 500, 0.5, 0.1, 0),
]


@pytest.mark.parametrize("alias", [False, True], ids=["out", "in_place"])
@pytest.mark.parametrize("name,S,B,chunk,long,empty,pad", CASES, ids=[c[0] for c in CASES])
def test_equals_the_oracle(pa, name, S, B, chunk, long, empty, pad, alias):
    rng = np.random.default_rng(len(name) * 7 + S)
    kind = rng.random(S)
    q = np.where(kind < empty, 0, np.where(kind < empty + long, chunk, 1)).tolist()
    if name == "one_long":
        q = [chunk]
    lens = rng.integers(0, 5 * B, S).tolist()
    lens[0] = 0
    W = 5 + -(-chunk // B) + 1
    free = rng.permutation(S * W + 3).astype(np.int32)
    T = sum(q) + pad
    table, st = _state(lens, q, free, 2, T, B, len(free), W, seed=S, alias=alias)
    want = ss.advance_ref(table, lens, q, free, 2, T, B, len(free))
    _run(pa, st, B, len(free))
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    _compare(st, want)


def test_full_list_and_last_table_entry(pa):
    """The step takes the free list's last block and fills its row's last entry."""
    table, st = _state([15, 0], [17, 16], [4, 9], 0, 33, 16, 10, 2)
    want = ss.advance_ref(table, [15, 0], [17, 16], [4, 9], 0, 33, 16, 10)
    assert want[2] == 2 and want[1] == [32, 16]
    _run(pa, st, 16, 10)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    _compare(st, want)


@pytest.mark.parametrize("alias", [False, True], ids=["out", "in_place"])
@pytest.mark.parametrize("lens,q,free,head,T,flag", [
    ([3, 8], [2, 1], [1], 0, 9, "no_blocks"),          # two blocks wanted
    ([3, 8], [2, 1], [1, 2, 3], 2, 9, "no_blocks"),    # the list is used up but for one
    ([3, 8], [2, 1], [1, 2, 3], -1, 9, "no_blocks"),
    ([3, 8], [2, 1], [1, 2, 3], 2**31 - 1, 9, "no_blocks"),
    ([3, 8], [2, 1], [1, 2, 3], 0, 2, "seq_range"),    # more tokens than slots
    ([3, 15], [2, 2], [1, 2, 3], 0, 9, "seq_range"),   # longer than the table row
    ([3, -1], [2, 1], [1, 2, 3], 0, 9, "seq_range"),
    ([3, 8], [2, -1], [1, 2, 3], 0, 9, "seq_range"),
    ([2**31 - 1, 8], [1, 1], [1, 2, 3], 0, 9, "seq_range"),
    ([3, 8], [2**31 - 1, 1], [1, 2, 3], 0, 9, "seq_range"),
])
def test_a_step_that_does_not_fit_changes_nothing(pa, lens, q, free, head, T, flag, alias):
    table, st = _state(lens, q, free, head, T, 4, 8, 4, alias=alias)
    _run(pa, st, 4, 8)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == pa.PA_DEVERR[flag]
    _compare(st, (table, lens, head, [0, 0, 0], [-1] * T, [0] * T))


def test_bad_block_ids_give_padding_slots(pa):
    """A table or free-list id outside the pool: its tokens get slot -1, the others theirs."""
    table, st = _state([2, 4], [2, 2], [99, 3], 0, 4, 4, 8, 2)
    st["table"][0, 0] = -5
    table[0, 0] = -5
    _run(pa, st, 4, 8)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == pa.PA_DEVERR["block_range"]
    want = ss.advance_ref(table, [2, 4], [2, 2], [99, 3], 0, 4, 4, 8)
    assert want[4] == [-1, -1, -1, -1]
    _compare(st, want)


def test_nothing_but_padding(pa):
    """No requests (every slot is padding), and no tokens at all."""
    for S, T in [(0, 6), (3, 0), (0, 0)]:
        table, st = _state([4] * S, [0] * S, [1, 2], 1, T, 4, 8, 2)
        _run(pa, st, 4, 8)
        torch.cuda.synchronize()
        assert pa.read_device_errors() == 0
        _compare(st, (table, [4] * S, 1, [0] * (S + 1), [-1] * T, [0] * T))


def test_a_captured_step_replays_a_whole_generation(pa):
    """One captured call, lengths and list head in place: 40 replays equal 40 oracle steps."""
    S, B, W = 37, 4, 14
    lens = np.random.default_rng(1).integers(0, 9, S).tolist()
    q = [1] * S
    free = np.random.default_rng(2).permutation(S * W).astype(np.int32)
    table, st = _state(lens, q, free, 0, S, B, S * W, W, alias=True)
    head = 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(pa, st, B, S * W)
    for _ in range(40):
        g.replay()
        table, lens, head, qsl, slots, pos = ss.advance_ref(table, lens, q, free, head, S, B, S * W)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    _compare(st, (table, lens, head, qsl, slots, pos))


def test_two_streams_at_once(pa):
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    states = [_state([5] * 500, [3] * 500, np.arange(4000), i, 1500, 4, 4000, 6, seed=i) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for (table, st), s in zip(states, streams):
            _run(pa, st, 4, 4000, stream=s)
    torch.cuda.synchronize()
    for i, (table, st) in enumerate(states):
        _compare(st, ss.advance_ref(table, [5] * 500, [3] * 500, np.arange(4000), i, 1500, 4, 4000))
        outs.append(st)
    assert pa.read_device_errors() == 0


def test_the_binding_refuses(pa):
    table, st = _state([1], [1], [1], 0, 1, 4, 8, 2)
    good = dict(st)
    for name, bad in [("lens", st["lens"].long()), ("q", torch.zeros(2, dtype=I32, device="cuda")),
                      ("slots", st["slots"].int()), ("qsl", torch.zeros(1, dtype=I32, device="cuda")),
                      ("free", torch.zeros(8, dtype=I32, device="cuda")[::2]), ("head", torch.zeros(1, dtype=I32))]:
        with pytest.raises((TypeError, ValueError)):
            _run(pa, {**good, name: bad}, 4, 8)
    with pytest.raises(pa.PAError):
        _run(pa, {**good, "lens_out": st["q"]}, 4, 8)
