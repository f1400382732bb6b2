"""pa_attention_packed on the GPU against the float64 oracle.

Bounds. The kernel rounds what the tensor-core prefill kernel of the pages rounds: numerators to
bf16, sums in fp32, the result to bf16 once; so both of errmodel's bars hold (the pass bar, and the diagnostic
bound |err| <= 2^-8 (1 + 2^-7) |ref| + 4 2^-8 sigma + 1e-5, sigma = sqrt(sum w^2 v^2) + |ref| sqrt(sum w^2)),
for inputs of unit size.
"""
import numpy as np
import pytest
import torch

from errmodel import diag_failures, northstar_failures
from oracle import int_cache as ic

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_161_gb300 as m

    m.read_device_errors(clear=True)
    return m


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _starts(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


class Case:
    def __init__(self, qlens, klens, Hq, Hkv, D, seed=0, fused=False, first=0, behind=0, size=1.0):
        g = torch.Generator().manual_seed(seed)
        self.qs, self.ks = _starts(qlens, first), _starts(klens, first)
        T, K = self.qs[-1] + behind, self.ks[-1] + behind
        if fused:
            qkv = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * size).to(BF16).cuda()
            self.q, self.k, self.v = qkv.split([Hq, Hkv, Hkv], 1)
        else:
            self.q = (torch.randn((T, Hq, D), generator=g) * size).to(BF16).cuda()
            self.k, self.v = (torch.randn((K, Hkv, D), generator=g).to(BF16).cuda() for _ in range(2))
        self.out = torch.full((T, Hq, D), 7.0, dtype=BF16, device="cuda")
        self.scale, self.max_q = D ** -0.5, max(qlens)
        self.i32 = [torch.tensor(x, dtype=I32, device="cuda") for x in (self.qs, self.ks)]

    def run(self, pa, **kw):
        kw = dict(dict(max_query_len=self.max_q, scale=self.scale), **kw)
        assert pa.attention_packed(self.out, self.q, self.k, self.v, *self.i32, **kw) is self.out
        torch.cuda.synchronize()
        return self

    def check(self, pa):
        assert pa.read_device_errors() == 0
        ref, _, _, sigma = ic.packed(_f64(self.q), _f64(self.k), _f64(self.v), self.qs, self.ks, self.scale)
        got, own = _f64(self.out), ~np.isnan(ref)
        assert (got[~own] == 7).all()
        assert not northstar_failures(got[own], ref[own]).any()
        bad = diag_failures(got[own], ref[own], sigma[own])
        assert not bad.any(), f"{bad.sum()} of {bad.size} elements outside the diagnostic bound"
        return self


HEADS = [(4, 1, 128), (8, 1, 128), (2, 2, 128), (4, 2, 64), (8, 1, 64), (1, 1, 64)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_one_prompt(pa, Hq, Hkv, D):
    for n in (1, 2, 31, 32, 33, 127, 128, 129, 255, 300, 777):
        Case([n], [n], Hq, Hkv, D, seed=n).run(pa).check(pa)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_packed_prompts_of_different_lengths(pa, Hq, Hkv, D):
    lens = [5, 400, 1, 0, 129, 33, 256, 64, 1, 700]
    Case(lens, lens, Hq, Hkv, D, seed=1, fused=True).run(pa).check(pa)
    Case(lens, lens, Hq, Hkv, D, seed=2, first=3, behind=40).run(pa).check(pa)  # rows of no request on both sides


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_chunks_behind_contexts(pa, Hq, Hkv, D):
    q = [64, 1, 130, 17, 0, 5]
    k = [64 + 300, 1000, 130 + 1, 17 + 128, 9, 5 + 2000]
    Case(q, k, Hq, Hkv, D, seed=3).run(pa).check(pa)


def test_queries_that_see_no_key_are_zero(pa):
    c = Case([10, 200, 3, 40], [4, 130, 0, 40], 4, 1, 128, seed=4).run(pa).check(pa)
    assert (c.out[:6] == 0).all() and (c.out[10: 10 + 70] == 0).all() and (c.out[210:213] == 0).all()
    c = Case([5, 6], [0, 0], 4, 2, 64, seed=5)  # no key rows at all
    c.run(pa)
    assert pa.read_device_errors() == 0 and (c.out == 0).all()


def test_more_tiles_than_sms(pa):
    g = np.random.default_rng(1)
    lens = [int(x) for x in np.clip(np.exp(g.normal(4.0, 1.2, 90)), 1, 900)]
    c = Case(lens, lens, 8, 4, 128, seed=6).run(pa).check(pa)
    first = c.out.clone()
    for _ in range(3):
        c.out.fill_(7.0)
        c.run(pa)
        assert torch.equal(first, c.out)


def test_many_requests(pa):
    n = 4096  # the most of a call; their order is the batch's beyond 512 with queries
    lens = [1 + i % 3 for i in range(n)]
    Case(lens, lens, 2, 1, 64, seed=7).run(pa).check(pa)
    lens = [0] * n
    lens[17], lens[4000] = 200, 70
    Case(lens, lens, 4, 1, 128, seed=8).run(pa).check(pa)


def test_more_tiles_than_ctas(pa):
    """Requests of one token each: a tile a request and KV head, far more than the rows would fill."""
    Case([1] * 700, [40] * 700, 8, 4, 64, seed=18).run(pa).check(pa)
    lens = [0, 1, 33, 0, 2, 1] * 300  # and tiles of several sizes among requests without queries
    Case(lens, [n + 5 if n else 9 for n in lens], 16, 2, 64, seed=19).run(pa).check(pa)


def test_large_logits_move_the_maximum(pa):
    for scale in (0.5, 1.0):
        c = Case([600, 90], [600, 900], 4, 2, 128, seed=9, size=2.0)
        c.scale = scale
        c.run(pa).check(pa)
    c = Case([400], [400], 4, 1, 64, seed=10)  # ever larger keys: every step moves it
    c.k.mul_(torch.linspace(0.1, 12, 400, device="cuda").view(-1, 1, 1).to(BF16))
    c.run(pa).check(pa)


def test_other_requests_rows_do_not_matter(pa):
    """NaN and infinities in neighbours' rows and in rows of no request: the same bits."""
    q, k = [70, 33, 150], [70, 200, 150]
    c = Case(q, k, 4, 1, 128, seed=11, first=5, behind=30).run(pa).check(pa)
    clean = c.out.clone()
    for bad in (float("nan"), float("inf")):
        for x, at in ((c.q, c.qs), (c.k, c.ks), (c.v, c.ks)):
            x[: at[0]] = bad
            x[at[1]: at[2]] = bad  # the second request
            x[at[3]:] = bad
        c.out.fill_(7.0)
        c.run(pa)
        a, b = c.qs[1], c.qs[2]
        assert torch.equal(c.out[:a], clean[:a]) and torch.equal(c.out[b:], clean[b:]) and c.out[a:b].isnan().all()


def test_a_nan_key_reaches_those_that_see_it_only(pa):
    c = Case([300], [300], 4, 1, 128, seed=12).run(pa)
    clean = c.out.clone()
    c.k[140] = float("nan")
    c.run(pa)
    assert torch.equal(c.out[:140], clean[:140]) and c.out[140:].isnan().all()


def test_malformed_requests_are_reported_and_leave_their_rows(pa):
    c = Case([20, 30, 40], [20, 30, 40], 4, 1, 64, seed=13)
    good = c.run(pa).out.clone()
    c.out.fill_(7.0)
    c.run(pa, max_query_len=35)
    assert pa.read_device_errors() == 0x4
    assert (c.out[50:] == 7).all() and torch.equal(c.out[:50], good[:50])
    c.i32[1][3] = 2000  # keys past the rows
    c.out.fill_(7.0)
    c.run(pa)
    assert pa.read_device_errors() == 0x4 and (c.out[50:] == 7).all() and torch.equal(c.out[:50], good[:50])
    c.i32[0][1] = -5
    c.out.fill_(7.0)
    c.run(pa)
    assert pa.read_device_errors() == 0x4


def test_unaligned_output_and_strides(pa):
    """out at 16 bytes past a 32-byte boundary; q, k and v out of wider rows."""
    c = Case([150, 40], [150, 40], 4, 1, 128, seed=14).run(pa).check(pa)
    flat = torch.full((c.out.numel() + 8,), 7.0, dtype=BF16, device="cuda")
    wide = torch.zeros((190, 12, 128), dtype=BF16, device="cuda")
    wide[:, 2:6], wide[:, 7:8], wide[:, 9:10] = c.q, c.k, c.v
    out = flat[8:].view(c.out.shape)
    pa.attention_packed(out, wide[:, 2:6], wide[:, 7:8], wide[:, 9:10], *c.i32, max_query_len=150, scale=c.scale)
    torch.cuda.synchronize()
    assert torch.equal(out, c.out) and (flat[:8] == 7).all()


def test_two_streams_and_a_captured_graph(pa):
    cases = [Case([500, 90], [500, 90], 8, 2, 128, seed=15), Case([200] * 6, [300] * 6, 4, 1, 64, seed=16)]
    want = [c.run(pa).check(pa).out.clone() for c in cases]
    streams, graphs = [torch.cuda.Stream() for _ in cases], []
    for c, s in zip(cases, streams):
        c.out.fill_(7.0)
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pa.attention_packed(c.out, c.q, c.k, c.v, *c.i32, max_query_len=c.max_q, scale=c.scale)
        graphs.append(g)
    for _ in range(3):
        for c in cases:
            c.out.fill_(7.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c.out, w)
    assert pa.read_device_errors() == 0


def test_equals_attention_through_pages(pa):
    """The same prompts through pa_attention's pages: within both calls' bar."""
    lens, B = [300, 129, 64], 16
    c = Case(lens, lens, 8, 2, 128, seed=17).run(pa)
    W = -(-max(lens) // B)
    kc = torch.zeros((3 * W, B, 2, 128), dtype=BF16, device="cuda")
    vc, table = torch.zeros_like(kc), torch.arange(3 * W, dtype=I32, device="cuda").view(3, W)
    slots = torch.cat([torch.arange(n) + s * W * B for s, n in enumerate(lens)]).cuda()
    pa.kv_write(c.k, c.v, kc, vc, slots)
    out = pa.attention(torch.empty_like(c.out), c.q, kc, vc, table, torch.tensor(lens, dtype=I32, device="cuda"), c.i32[0],
                       max_query_len=300, max_seq_len=W * B, scale=c.scale)
    a, b = _f64(c.out), _f64(out)
    assert (np.abs(a - b) <= 2 * (1.5e-2 + 1e-2 * np.abs(b))).all() and np.abs(a - b).mean() < 2e-3
