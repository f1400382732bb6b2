"""The integer-coded cache as a serving loop runs it: prompts, a chunk behind its context, decode steps and
drafts, each advance -> norm + rotary -> quantising write -> attention (packed over a prompt's own rows or
over a context read back, from the codes for decode), on one stream, eagerly and as captured graphs.

Every step is checked against the oracle from the kernels' own inputs of that step: the cache's bytes equal,
the rows read back equal, the outputs within each attention's bound.
"""
import numpy as np
import pytest
import torch

import intmodel
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


class Loop:
    def __init__(self, pa, S, T, bits, B=16, Hq=8, Hkv=2, D=128, W=24, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.pa, self.S, self.T, self.bits, self.B, self.Hq, self.Hkv, self.D, self.W = pa, S, T, bits, B, Hq, Hkv, D, W
        self.NB, self.limit = S * W + 3, W * B
        i32 = dict(dtype=I32, device="cuda")
        self.table = torch.full((S, W), -1, **i32)
        self.lens, self.qlens, self.ctx = (torch.zeros(S, **i32) for _ in range(3))
        self.free, self.head = torch.randperm(self.NB, generator=g).to(I32).cuda(), torch.zeros(1, **i32)
        self.qsl, self.pos = torch.zeros(S + 1, **i32), torch.zeros(T, **i32)
        self.slots, self.own = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.arange(T, device="cuda")
        self.qkv = torch.zeros((T, Hq + 2 * Hkv, D), dtype=BF16, device="cuda")
        ang = torch.arange(self.limit).double()[:, None] * 10000.0 ** (-torch.arange(0, D, 2).double() / D)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        self.w = [(1 + 0.2 * torch.randn(D, generator=g)).to(BF16).cuda() for _ in range(2)]
        self.k, self.v = (torch.zeros((T, Hkv, D), dtype=BF16, device="cuda") for _ in range(2))
        self.kc, self.vc = (torch.zeros((self.NB, Hkv, B * (D * bits // 8 + 4)), dtype=torch.uint8, device="cuda")
                            for _ in range(2))
        self.q = torch.zeros((T, Hq, D), dtype=BF16, device="cuda")
        self.out = torch.full((T, Hq, D), 7.0, dtype=BF16, device="cuda")
        self.kbuf, self.vbuf = (torch.full((S * self.limit, Hkv, D), 7.0, dtype=BF16, device="cuda") for _ in range(2))
        self.ksl = torch.zeros(S + 1, **i32)
        self.ws = torch.empty(pa.attention_int_workspace_size(S, T, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        self.scale = D ** -0.5

    def rows(self):
        pa = self.pa
        pa.advance_batch(self.table, self.lens, self.qlens, self.free, self.head, self.lens, self.head, self.qsl,
                         self.slots, self.pos, block_size=self.B, num_blocks=self.NB)
        q, k, v = self.qkv.split([self.Hq, self.Hkv, self.Hkv], 1)
        shape = (self.T, 1, self.Hkv, self.D)  # the rotated rows themselves: a cache of one-token blocks, in order
        pa.norm_rope_write(self.q, q, k, v, *self.w, self.cos_sin, self.pos, self.own, self.k.view(shape), self.v.view(shape))
        pa.kv_write_int(self.k, self.v, self.kc, self.vc, self.slots, bits=self.bits)

    def prompt(self, max_q):
        self.rows()
        self.pa.attention_packed(self.out, self.q, self.k, self.v, self.qsl, self.qsl, max_query_len=max_q, scale=self.scale)

    def chunk(self, max_q):
        self.rows()
        self.ksl[1:] = self.lens.cumsum(0)
        self.pa.kv_read_int(self.kbuf, self.vbuf, self.kc, self.vc, self.table, None, self.lens, self.ksl, bits=self.bits)
        self.pa.attention_packed(self.out, self.q, self.kbuf, self.vbuf, self.qsl, self.ksl, max_query_len=max_q,
                                 scale=self.scale)

    def decode(self, max_q):
        self.rows()
        self.pa.attention_int(self.out, self.q, self.kc, self.vc, self.table, self.lens, self.qsl, bits=self.bits,
                              max_query_len=max_q, max_seq_len=self.limit, scale=self.scale, workspace=self.ws)

    def check(self, kind, before):
        torch.cuda.synchronize()
        assert self.pa.read_device_errors() == 0
        lens, qsl, table = self.lens.tolist(), self.qsl.tolist(), self.table.cpu().numpy()
        n = qsl[-1]
        k, v, q, out = (_f64(t) for t in (self.k, self.v, self.q, self.out))
        kc, vc = self.kc.cpu().numpy(), self.vc.cpu().numpy()
        slots = self.slots.tolist()
        for got, old, x in ((kc, before[0], k), (vc, before[1], v)):
            assert np.array_equal(got, ic.write(old, x, slots, self.bits))
        assert (out[n:] == 7).all()
        for s in range(self.S):
            a, b, L = qsl[s], qsl[s + 1], lens[s]
            if a == b:
                continue
            if kind == "decode":
                ref, tol = intmodel.attention(q[a:b], kc, vc, table[s], L, self.scale, self.bits)
                assert (np.abs(out[a:b] - ref) <= tol).all()
                continue
            K, V = k[a:b], v[a:b]
            if kind == "chunk":
                c = self.ksl[s].item()
                K, V = _f64(self.kbuf[c:c + L]), _f64(self.vbuf[c:c + L])
                for got, cache in ((K, kc), (V, vc)):
                    want = torch.tensor(ic.rows(cache, table[s], L, self.D, self.bits)[0]).float().to(BF16)
                    assert np.array_equal(got, _f64(want))
            ref, _, _, sigma = ic.attend(q[a:b], K, V, K.shape[0] - (b - a), self.scale)
            assert not northstar_failures(out[a:b], ref).any() and not diag_failures(out[a:b], ref, sigma).any()
        return kc, vc


@pytest.mark.parametrize("bits", [4, 8])
def test_prompts_chunks_decodes_and_drafts(pa, bits):
    loop = Loop(pa, 5, 300, bits, seed=bits)
    before = loop.kc.cpu().numpy(), loop.vc.cpu().numpy()
    g = torch.Generator(device="cuda").manual_seed(1)
    for kind, qlens in (("prompt", [90, 17, 150, 1, 33]), ("chunk", [1, 60, 100, 0, 64]), ("decode", [1] * 5),
                        ("decode", [1, 0, 4, 8, 1]), ("chunk", [3, 0, 0, 40, 0]), ("decode", [1] * 5)):
        loop.qkv.normal_(generator=g)
        loop.qlens.copy_(torch.tensor(qlens))
        loop.out.fill_(7.0)
        getattr(loop, kind)(max(qlens))
        before = loop.check(kind, before)


def test_two_captured_loops_replayed_together(pa):
    """Two loops' decode steps captured as two graphs, replayed on two streams at once: each as if alone."""
    def start(i, bits):
        loop = Loop(pa, 7, 120, bits, seed=10 + i)
        loop.qkv.normal_(generator=torch.Generator(device="cuda").manual_seed(i))
        loop.qlens.copy_(torch.tensor([40, 1, 0, 17, 3, 33, 16]))
        loop.prompt(40)
        loop.qlens.fill_(1)
        torch.cuda.synchronize()
        return loop

    want = []
    for i, bits in enumerate((4, 8)):
        loop = start(i, bits)
        for _ in range(5):
            loop.decode(1)
        torch.cuda.synchronize()
        want.append((loop.out.clone(), loop.kc.clone(), loop.lens.clone()))
    loops, streams, graphs = [start(i, bits) for i, bits in enumerate((4, 8))], [torch.cuda.Stream() for _ in range(2)], []
    for loop, s in zip(loops, streams):
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            loop.decode(1)
        graphs.append(graph)
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    for loop, (out, kc, lens) in zip(loops, want):
        assert torch.equal(loop.out, out) and torch.equal(loop.kc, kc) and torch.equal(loop.lens, lens)


def test_copy_on_write_of_a_coded_block(pa):
    """A forked request's shared last block is copied before its writer goes on; the other's rows stay."""
    loop = Loop(pa, 2, 64, 4, seed=3)
    bm = pa.BlockManager(loop.NB, loop.B, range(loop.NB))
    bm.add_seq(0)
    slots = torch.tensor(bm.append(0, 20)).cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randn((22, loop.Hkv, loop.D), generator=g, device="cuda").to(BF16)
    pa.kv_write_int(rows[:20], rows[:20], loop.kc, loop.vc, slots, bits=4)
    bm.fork(0, 1)
    new = [torch.tensor(bm.append(s, 1)).cuda() for s in (0, 1)]
    pairs = torch.tensor(bm.take_copies()).cuda()
    assert pairs.shape == (1, 2)
    pa.copy_blocks(loop.kc, loop.vc, pairs)
    for i in range(2):
        pa.kv_write_int(rows[20 + i: 21 + i], rows[20 + i: 21 + i], loop.kc, loop.vc, new[i], bits=4)
    torch.cuda.synchronize()
    values = ic.value(*ic.quantise(_f64(rows), 4))
    for i in range(2):
        got = ic.rows(loop.kc.cpu().numpy(), bm.block_table(i), 21, loop.D, 4)[0]
        assert np.array_equal(got, np.concatenate([values[:20], values[20 + i: 21 + i]]))
