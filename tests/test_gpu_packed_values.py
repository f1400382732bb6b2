"""pa_attention_packed: what a value row that is not finite reaches."""
import pytest
import torch

from test_gpu_attention_packed import Case, pa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq,Hkv,D,Q,K,key", [(1, 1, 128, 128, 228, 220), (4, 4, 64, 300, 300, 140), (4, 1, 128, 100, 133, 80),
                                              (8, 1, 64, 90, 1000, 999), (2, 1, 128, 200, 200, 0), (2, 2, 64, 40, 45, 44)])
def test_queries_before_its_tile_keep_their_bits(pa, bad, Hq, Hkv, D, Q, K, key):  # noqa: F811
    """Tiles of 128 / (Hq / Hkv) tokens from the request's first on: those that hold no query that sees the
    row keep their bits, and so does another request."""
    c = Case([Q, 50], [K, 50], Hq, Hkv, D, seed=21).run(pa).check(pa)
    clean = c.out.clone()
    c.v[key] = bad
    c.out.fill_(7.0)
    c.run(pa)
    assert pa.read_device_errors() == 0
    tokens, first = 128 * Hkv // Hq, max(0, key - (K - Q))  # the first query that sees the row
    kept = first // tokens * tokens
    assert torch.equal(c.out[:kept], clean[:kept]) and torch.equal(c.out[Q:], clean[Q:])
    assert not c.out[first:Q].isfinite().any()
