"""pa_attention_packed over one very long context: its time is no fault."""
import pytest
import torch

from test_gpu_attention_packed import BF16, I32, pa  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_tile_of_many_steps(pa):  # noqa: F811
    """One query over 120 million keys, all in one tile, which takes longer than a pipeline wait may."""
    K, D = 120_000_000, 64
    k, v = (torch.zeros((K, 1, D), dtype=BF16, device="cuda") for _ in range(2))
    q, out = torch.ones((1, 1, D), dtype=BF16, device="cuda"), torch.full((1, 1, D), 7.0, dtype=BF16, device="cuda")
    k[12345] = k[K - 7] = 2.0  # two logits of 128 among zeros, whose numerators all fall under 2^-100 of theirs
    v[12345], v[K - 7] = 1.0, 3.0
    i32 = lambda *x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    pa.attention_packed(out, q, k, v, i32(0, 1), i32(0, K), max_query_len=1, scale=1.0)
    torch.cuda.synchronize()
    del k, v
    torch.cuda.empty_cache()
    assert pa.read_device_errors() == 0
    assert (out == 2.0).all()
