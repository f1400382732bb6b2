"""pa_attention_int over keys, queries and value rows of extreme sizes whose logits and outputs are ordinary."""
import numpy as np
import pytest
import torch

import introws
from test_gpu_int_cache import BF16, Batch, _f64, pa  # noqa: F401

pytestmark = pytest.mark.gpu


def _check(b):
    assert b.pa.read_device_errors() == 0
    kc, vc, q, out = b.kc.cpu().numpy(), b.vc.cpu().numpy(), _f64(b.q), _f64(b.out)
    for s, L in enumerate(b.lens):
        a, e = b.qsl[s], b.qsl[s + 1]
        ref, tol = introws.attention(q[a:e], kc, vc, b.table[s].tolist(), L, b.scale, b.bits)
        err = np.abs(out[a:e] - ref)
        assert (err <= tol).all(), (s, L, float(np.nanmax(err / tol)))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("qlens", [[1, 1], [4, 3]])
@pytest.mark.parametrize("size", [1e31, 1e33, 1e37])
def test_large_keys(pa, bits, qlens, size):  # noqa: F811
    """Queries as small as the keys are large: the logits are those of unit sizes."""
    b = Batch(pa, [300, 40], qlens, 4, 1, 128, 16, bits, seed=41, size=size)
    b.q.div_(size)
    b.run()
    _check(b)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("qlens", [[1, 1], [4, 3]])
def test_queries_below_the_smallest_normal_number(pa, bits, qlens):  # noqa: F811
    b = Batch(pa, [300, 40], qlens, 4, 1, 128, 16, bits, seed=42, size=1e37)
    b.q.copy_((b.q.float() * 2.0 ** -131).to(BF16))
    assert 0 < float(b.q.float().abs().max()) < 2.0 ** -126
    b.scale = 16.0
    b.run()
    _check(b)
