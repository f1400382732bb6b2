"""pa_attention_int where its running maximum keeps moving, and with many requests of a call."""
import numpy as np
import pytest
import torch

from test_gpu_int_cache import BF16, Batch, pa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("qlens", [[1, 2], [4, 3]])
def test_large_logits(pa, bits, qlens):  # noqa: F811
    for size, scale in ((6.0, 1.0), (6.0, 0.2), (3.0, 0.25)):
        b = Batch(pa, [700, 300], qlens, 4, 1, 128, 16, bits, seed=11, size=size)
        b.scale = scale
        b.run().check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens,qlens", [([700], [1]), ([700], [4]), ([6000, 50], [1, 1]), ([6000], [4])])
def test_ever_larger_logits(pa, bits, lens, qlens):  # noqa: F811
    """The keys' mean grows along the context: unit after unit moves the maximum, in every warp's run."""
    b = Batch(pa, lens, qlens, 4, 1, 128, 16, bits, seed=14)
    n = lens[0]
    b.q.add_(0.5)
    pos = torch.arange(n)
    slots = (b.table[0, pos // 16].long() * 16 + pos % 16).cuda()
    k = torch.randn((n, 1, 128), generator=torch.Generator().manual_seed(3)) * 0.5
    v = torch.randn((n, 1, 128), generator=torch.Generator().manual_seed(4))
    ramp = torch.linspace(-n / 90, n / 90, n).view(n, 1, 1)  # 13 powers of two in 64 keys
    for up in (1.0, -1.0):  # and ever smaller ones
        b.pa.kv_write_int((k + up * ramp).to(BF16).cuda(), v.to(BF16).cuda(), b.kc, b.vc, slots, bits=bits)
        b.run().check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("S,qlen", [(385, 1), (1000, 1), (4096, 1), (257, 3), (4096, 3)])
def test_many_requests(pa, bits, S, qlen):  # noqa: F811
    g = np.random.default_rng(S)
    lens = [int(x) for x in g.integers(qlen, 60, S)]
    lens[S // 2] = 2000
    qlens = [qlen if g.random() < 0.9 else 0 for _ in range(S)]
    qlens[S // 2] = qlen
    b = Batch(pa, lens, qlens, 4, 1, 64, 16, bits, seed=S, pad=3)
    b.run().check([0, 1, S // 2] + [int(x) for x in g.integers(0, S, 40)] + list(range(S - 10, S)))
