"""pa_attention_int over tables with block ids that are not there: their positions are skipped, whatever the
launch before left in shared memory."""
import numpy as np
import pytest
import torch

import introws
from test_gpu_int_cache import Batch, _f64, pa  # noqa: F401

pytestmark = pytest.mark.gpu


def _check(b, gone):
    assert b.pa.read_device_errors() == 0x2
    kc, vc, q, out = b.kc.cpu().numpy(), b.vc.cpu().numpy(), _f64(b.q), _f64(b.out)
    for s, L in enumerate(b.lens):
        a, e = b.qsl[s], b.qsl[s + 1]
        ref, tol = introws.attention(q[a:e], kc, vc, b.table[s].tolist(), L, b.scale, b.bits, gone.get(s, ()))
        err = np.abs(out[a:e] - ref)
        assert (err <= tol).all(), (s, L, float(err.max()))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B", [4, 12, 16, 32, 64, 128])
@pytest.mark.parametrize("qlens", [[1, 1, 1, 1, 1], [4, 1, 3, 2, 1]])
def test_their_positions_are_skipped(pa, bits, B, qlens):  # noqa: F811
    lens = [700, 33, 260, 129, 5000]
    b = Batch(pa, lens, qlens, 4, 1, 128, B, bits, seed=B)
    blocks = [-(-n // B) for n in lens]
    gone = {0: [0, 1, blocks[0] // 2], 2: [blocks[2] - 1], 3: list(range(blocks[3])),
            4: sorted({3, blocks[4] // 3, blocks[4] // 3 + 1, blocks[4] - 2})}
    for s, ids in gone.items():
        for i, x in enumerate(ids):
            b.table[s, x] = (-1, b.NB, 10 ** 6)[i % 3]
    got = []
    for seed in (1, 2):  # other contents of the shared memory that the call finds
        Batch(pa, [3000, 4000], [1, 2], 4, 1, 128, B, bits, seed=seed, size=3.0, vsize=9.0).run()
        assert pa.read_device_errors() == 0
        b.out.fill_(7.0)
        b.run()
        _check(b, gone)
        got.append(b.out.clone())
    assert torch.equal(*got)
    a = b.qsl[3]
    assert (b.out[a:b.qsl[4]] == 0).all()  # a request without any block


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("group", [4, 16])
def test_a_call_whose_first_keys_are_gone(pa, bits, group):  # noqa: F811
    """The first units of a run, and a whole warp's run: nothing that this launch wrote lies in the ring."""
    b = Batch(pa, [20000], [1], group, 1, 64, 16, bits, seed=7)
    gone = list(range(0, 300)) + list(range(700, 764))
    b.table[0, gone] = -7
    b.run()
    _check(b, {0: gone})
