"""A chunk of a prompt over an integer-coded cache as its definition gives it: the context read back ahead of the
chunk's own rows, which stay exact, then packed attention over both."""
import numpy as np
import pytest
import torch

from errmodel import diag_failures, northstar_failures
from oracle import int_cache as ic
from test_gpu_int_cache import BF16, I32, _cache, _f64, _rows, pa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64)])
def test_context_from_codes_own_rows_exact(pa, bits, Hq, Hkv, D):  # noqa: F811
    ctx, chunk, B = [130, 0, 17, 400, 33], [70, 40, 1, 128, 0], 16
    S, T, g = len(ctx), sum(chunk), torch.Generator().manual_seed(bits)
    W = -(-max(c + t for c, t in zip(ctx, chunk)) // B)
    NB = S * W
    table = torch.randperm(NB, generator=g)[: S * W].view(S, W).to(I32)
    kc, vc = _cache(NB, Hkv, B, D, bits, 0), _cache(NB, Hkv, B, D, bits, 0)
    slot = lambda s, p: int(table[s, p // B]) * B + p % B  # noqa: E731
    old = [slot(s, p) for s in range(S) for p in range(ctx[s])]
    k, v = _rows(len(old), Hkv, D, BF16, 5, False)
    pa.kv_write_int(k, v, kc, vc, torch.tensor(old).cuda(), bits=bits)

    k, v = _rows(T, Hkv, D, BF16, 6, True)
    q = torch.randn((T, Hq, D), generator=g).to(BF16).cuda()
    new = [slot(s, p) for s in range(S) for p in range(ctx[s], ctx[s] + chunk[s])]
    pa.kv_write_int(k, v, kc, vc, torch.tensor(new).cuda(), bits=bits)
    qs, ks = np.cumsum([0] + chunk), np.cumsum([0] + [c + t for c, t in zip(ctx, chunk)])
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=I32, device="cuda")  # noqa: E731
    kb, vb = (torch.full((int(ks[-1]), Hkv, D), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    pa.kv_read_int(kb, vb, kc, vc, table.cuda(), None, i32(ctx), i32(ks), bits=bits)
    own = torch.cat([torch.arange(ks[s] + ctx[s], ks[s + 1]) for s in range(S)]).cuda()
    assert (kb[own] == 7).all() and (vb[own] == 7).all()  # the room for the chunk's rows
    kb[own], vb[own] = k, v
    out = torch.empty_like(q)
    pa.attention_packed(out, q, kb, vb, i32(qs), i32(ks), max_query_len=max(chunk), scale=D ** -0.5)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0

    K, V = np.zeros((ks[-1], Hkv, D)), np.zeros((ks[-1], Hkv, D))
    for s in range(S):
        for to, cache, rows in ((K, kc, k), (V, vc, v)):
            codes = ic.rows(cache.cpu().numpy(), table[s].tolist(), ctx[s], D, bits)[0]
            to[ks[s]: ks[s] + ctx[s]] = _f64(torch.tensor(codes).float().to(BF16))
            to[ks[s] + ctx[s]: ks[s + 1]] = _f64(rows[qs[s]: qs[s + 1]])
    ref, _, _, sigma = ic.packed(_f64(q), K, V, qs.tolist(), ks.tolist(), D ** -0.5)
    assert not northstar_failures(_f64(out), ref).any() and not diag_failures(_f64(out), ref, sigma).any()
