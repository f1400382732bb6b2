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


def _rewrite(b, s, pos, k, v):
    """Rows of positions `pos` of request s, written anew."""
    pos = torch.tensor(pos)
    slots = b.table[s, pos // b.B].long() * b.B + pos % b.B
    b.pa.kv_write_int(k.to(BF16).cuda(), v.to(BF16).cuda(), b.kc, b.vc, slots.cuda(), bits=b.bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("qlens", [[1, 1], [4, 2]])
@pytest.mark.parametrize("power", [20, 32, 60])
def test_large_value_rows_without_weight(pa, bits, qlens, power):  # noqa: F811
    """A few value rows 2^power times the others, whose logits leave them no weight: no accuracy is lost."""
    Hkv, D = 2, 128
    for at in ([0], [63, 64], [150], [699], list(range(0, 700, 50))):
        b = Batch(pa, [700, 90], qlens, 8, Hkv, D, 16, bits, seed=43)
        b.q.add_(0.5)
        g = torch.Generator().manual_seed(power)
        k = torch.full((len(at), Hkv, D), -10.0)  # logits of about -56
        _rewrite(b, 0, at, k, torch.randn((len(at), Hkv, D), generator=g) * 2.0 ** power)
        b.run()
        _check(b)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("power", [32, 60])
def test_large_value_rows_that_later_keys_outweigh(pa, bits, power):  # noqa: F811
    """The context's first rows carry all weight until much larger logits come."""
    for qlens, L in (([1], 200), ([4], 200), ([1], 3000)):
        b = Batch(pa, [L], qlens, 4, 1, 128, 16, bits, seed=44)
        b.q.add_(0.5)
        g = torch.Generator().manual_seed(power)
        k = torch.full((90, 1, 128), -18.0)  # logits of about -100
        _rewrite(b, 0, list(range(90)), k, torch.randn((90, 1, 128), generator=g) * 2.0 ** power)
        b.run()
        _check(b)


@pytest.mark.parametrize("bits", [4, 8])
def test_a_large_value_row_for_one_query_head(pa, bits):  # noqa: F811
    """A row that one query head of a tile attends to alone, and the others not at all; and one that only the last
    of the drafted tokens sees."""
    for qlens in ([1], [4]):
        b = Batch(pa, [500], qlens, 4, 1, 128, 16, bits, seed=45)
        b.q.sub_(0.5)
        b.q[:, 1].add_(1.0)
        k = torch.full((2, 1, 128), 10.0)  # logits of about 56 for the second head, -56 for the others
        v = torch.randn((2, 1, 128), generator=torch.Generator().manual_seed(1)) * 2.0 ** 32
        _rewrite(b, 0, [70, 499], k, v)
        b.run()
        _check(b)


@pytest.mark.parametrize("bits", [4, 8])
def test_value_rows_from_the_largest_to_the_smallest(pa, bits):  # noqa: F811
    """The first rows huge, until logits a thousand powers of two larger come, of tiny rows."""
    b = Batch(pa, [260], [1], 4, 1, 128, 16, bits, seed=46, vsize=2.0 ** -100)
    b.q.add_(0.5)
    k = torch.full((90, 1, 128), -130.0)
    _rewrite(b, 0, list(range(90)), k, torch.randn((90, 1, 128), generator=torch.Generator().manual_seed(2)) * 2.0 ** 100)
    b.run()
    _check(b)
