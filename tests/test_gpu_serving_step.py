"""The serving-step operators together, as a serving loop runs them: a prompt chunk, then decode
steps, each advance -> norm + rotary + cache write -> bounds -> scores -> selection -> sparse
attention, on one stream, eagerly and as one captured graph that advances its own lengths.

Checked after every step against the oracle chained in float64 from the kernel's own cache and
lists (each link's rounding is then that link's alone): lengths, slots and positions equal;
the cache's new rows and the queries within the norm + rotary bound; bounds exact; every
selected list exactly the oracle's selection from the kernel's scores; outputs within the
attention bound. With every block selected the outputs equal pa_attention's within its bar.
"""
import numpy as np
import pytest
import torch

from oracle import serving_step as ss

pytestmark = pytest.mark.gpu
BF16, E4M3, I32 = torch.bfloat16, torch.float8_e4m3fn, torch.int32


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_161_gb300 as m

    m.read_device_errors(clear=True)
    return m


def _f64(t):
    return t.detach().float().cpu().double().numpy()


class Loop:
    """The buffers of a serving loop with room for T tokens a step."""

    def __init__(self, pa, S, T, cache, k, B=16, Hq=8, Hkv=2, D=128, W=24, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.pa, self.S, self.T, self.B, self.Hq, self.Hkv, self.D, self.W, self.k = pa, S, T, B, Hq, Hkv, D, W, k
        self.NB = S * W + 7
        i32 = dict(dtype=I32, device="cuda")
        self.table = torch.full((S, W), -1, **i32)
        self.lens, self.qlens = torch.zeros(S, **i32), torch.zeros(S, **i32)
        self.free = torch.randperm(self.NB, generator=g).to(I32).cuda()
        self.head = torch.zeros(1, **i32)
        self.qsl, self.pos = torch.zeros(S + 1, **i32), torch.zeros(T, **i32)
        self.slots = torch.zeros(T, dtype=torch.int64, device="cuda")
        self.qkv = torch.zeros((T, Hq + 2 * Hkv, D), dtype=BF16, device="cuda")
        self.w = [(1 + 0.2 * torch.randn(D, generator=g)).to(BF16).cuda() for _ in range(2)]
        ang = torch.arange(W * B).double()[:, None] * 10000.0 ** (-torch.arange(0, D, 2).double() / D)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        self.kc = torch.zeros((self.NB, B, Hkv, D), device="cuda").to(cache)
        self.vc = torch.zeros_like(self.kc)
        self.scales = (2.0 ** -4, 2.0 ** -4) if cache == E4M3 else (1.0, 1.0)
        self.q = torch.zeros((T, Hq, D), dtype=BF16, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.bounds = torch.zeros((self.NB, Hkv, 2, D), dtype=BF16, device="cuda")
        self.scores = torch.zeros((T, Hkv, W), device="cuda")
        self.idx = torch.full((T, Hkv, k), -1, **i32)
        self.scale = D ** -0.5

    def step(self, max_q):
        pa, limit = self.pa, self.W * self.B
        pa.advance_batch(self.table, self.lens, self.qlens, self.free, self.head, self.lens, self.head, self.qsl,
                         self.slots, self.pos, block_size=self.B, num_blocks=self.NB)
        q, k, v = self.qkv.split([self.Hq, self.Hkv, self.Hkv], 1)
        pa.norm_rope_write(self.q, q, k, v, *self.w, self.cos_sin, self.pos, self.slots, self.kc, self.vc,
                           k_scale=self.scales[0], v_scale=self.scales[1])
        meta = (self.table, self.lens, self.qsl)
        pa.block_bounds(self.bounds, self.kc, *meta, max_query_len=max_q, max_seq_len=limit, num_tokens=self.T)
        pa.block_scores(self.scores, self.q, self.bounds, *meta, block_size=self.B, max_query_len=max_q, max_seq_len=limit)
        pa.select_blocks(self.idx, self.scores, *meta[1:], block_size=self.B, init_blocks=1, local_blocks=1)
        pa.attention_sparse(self.out, self.q, self.kc, self.vc, *meta, self.idx, max_seq_len=limit, scale=self.scale,
                            k_scale=self.scales[0], v_scale=self.scales[1])

    def check(self, before):
        """The step that led from the host state `before` (table, lens, head), returning the next."""
        torch.cuda.synchronize()
        assert self.pa.read_device_errors() == 0
        table, lens, head = before
        free, qlens = self.free.tolist(), self.qlens.tolist()
        table, lens, head, qsl, slots, pos = ss.advance_ref(table, lens, qlens, free, head, self.T, self.B, self.NB)
        assert np.array_equal(self.table.cpu().numpy(), table)
        for got, want in ((self.lens, lens), (self.head, [head]), (self.qsl, qsl), (self.slots, slots), (self.pos, pos)):
            assert got.tolist() == list(want)
        x, w, cs = _f64(self.qkv), [_f64(t) for t in self.w], _f64(self.cos_sin)
        half, q = self.D // 2, _f64(self.q)
        kc, vc = (_f64(c) * s for c, s in zip((self.kc, self.vc), self.scales))
        k_rows, v_rows = (c.reshape(-1, self.Hkv, self.D) for c in (kc, vc))
        e4m3 = self.kc.dtype == E4M3
        for t in range(0, qsl[-1], max(1, qsl[-1] // 40)):
            for h in range(self.Hq + self.Hkv):
                y, z = ss.norm_rope_ref(x[t, h], w[h >= self.Hq], 1e-6, cs[pos[t], :half], cs[pos[t], half:], False)
                slack = 2.0 ** -19 * (np.abs(y) + np.abs(np.roll(y, half)))
                got, rnd = (q[t, h], 2.0 ** -8) if h < self.Hq else (k_rows[slots[t], h - self.Hq], 2.0 ** -4 if e4m3 else 2.0 ** -8)
                low = 2.0 ** -10 * self.scales[0] if e4m3 and h >= self.Hq else 0.0
                assert (np.abs(got - z) <= np.maximum(rnd * (np.abs(z) + slack), low) + slack).all()
            v = x[t, self.Hq + self.Hkv:]
            assert (np.abs(v_rows[slots[t]] - v) <= (2.0 ** -4 * np.abs(v) + 2.0 ** -10 * self.scales[1] if e4m3 else 0)).all()
        want = ss.bounds_ref(_f64(self.bounds), _f64(self.kc), table, lens, qsl)
        assert np.array_equal(_f64(self.bounds), want)
        s = self.scores.cpu().numpy()
        ref, size = ss.scores_ref(q, want, table, lens, qsl, self.B, self.W)
        n = qsl[-1]
        fin = np.isfinite(ref[:n])
        assert (np.abs(s[:n][fin] - ref[:n][fin]) <= 2 * self.D * 2.0 ** -23 * size[:n][fin]).all()
        idx = self.idx.cpu().numpy()
        assert np.array_equal(idx[:n], ss.select_ref(s[:n], lens, qsl, self.B, self.k, 1, 1))
        o, mag, logit = ss.attention_sparse_ref(q, kc, vc, table, lens, qsl, idx, self.scale)
        p = 2.0 ** -11 + 2.0 ** -25 if e4m3 else 2.0 ** -8
        tol = (p + 2 * self.D * 2.0 ** -23 * logit + 2.0 ** -18) * mag
        tol = tol + 2.0 ** -8 * (np.abs(o) + tol)
        assert (np.abs(_f64(self.out)[:n] - o[:n]) <= tol[:n]).all()
        return table, lens, head


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("k", [4, 24])
def test_prompts_then_decode_steps(pa, cache, k):
    S, T = 5, 300
    loop = Loop(pa, S, T, cache, k, seed=k)
    state = (np.full((S, loop.W), -1), [0] * S, 0)
    g = torch.Generator(device="cuda").manual_seed(1)
    for qlens in ([90, 17, 150, 1, 33], [1, 1, 100, 0, 64], [1] * 5, [1, 0, 1, 4, 1], [1] * 5):
        loop.qkv.normal_(generator=g)
        loop.qlens.copy_(torch.tensor(qlens))
        pad = loop.out[sum(qlens):].clone()
        loop.step(max(qlens))
        state = loop.check(state)
        assert torch.equal(loop.out[sum(qlens):], pad)  # rows behind the last request stay as they were
    if k == loop.W:  # every block selected: attention over everything
        ref = torch.empty_like(loop.out[:5])
        args = (ref, loop.q[:5].contiguous(), loop.kc, loop.vc, loop.table, loop.lens, loop.qsl)
        kw = dict(max_query_len=1, max_seq_len=loop.W * loop.B, scale=loop.scale)
        if cache == BF16:
            pa.attention(*args, **kw)
        else:
            pa.attention_fp8(*args, **kw, k_scale=loop.scales[0], v_scale=loop.scales[1])
        torch.cuda.synchronize()
        a, b = _f64(loop.out[:5]), _f64(ref)
        assert (np.abs(a - b) <= 2 * (1.5e-2 + 1e-2 * np.abs(b))).all()


def test_two_captured_loops_replayed_together(pa):
    """Two loops' steps captured as two graphs and replayed on two streams at once: nothing is
    shared between them; each replay advances its own lengths."""
    loops = [Loop(pa, 9, 9, cache, 5, seed=i) for i, cache in enumerate((BF16, E4M3))]
    streams, graphs, states = [torch.cuda.Stream() for _ in loops], [], []
    for loop in loops:
        loop.qlens.fill_(1)
        loop.qkv.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
        state = (np.full((9, loop.W), -1), [0] * 9, 0)
        loop.step(1)  # once eagerly: what a first call sets up is set up before the capture
        states.append(loop.check(state))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            loop.step(1)
        graphs.append(g)
    for _ in range(20):
        for stream, g in zip(streams, graphs):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for loop, state in zip(loops, states):
        for _ in range(19):  # the same replays on the host's side
            table, lens, head, _, _, _ = ss.advance_ref(*state[:2], [1] * 9, loop.free.tolist(), state[2], 9, loop.B, loop.NB)
            state = (table, lens, head)
        loop.check(state)


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_a_captured_step_of_chunks_and_decodes(pa, cache):
    """Both score kernels in one graph, behind the kernels that write their queries and bounds; new rows
    before each replay, which advances the lengths."""
    loop = Loop(pa, 5, 100, cache, 6, seed=3)
    loop.qlens.copy_(torch.tensor([33, 1, 40, 0, 20]))
    state = (np.full((5, loop.W), -1), [0] * 5, 0)
    g = torch.Generator(device="cuda").manual_seed(8)
    loop.qkv.normal_(generator=g)
    loop.step(40)
    state = loop.check(state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step(40)
    for _ in range(6):
        loop.qkv.normal_(generator=g)
        graph.replay()
        state = loop.check(state)


FIRST = """
import sys, torch
sys.path.insert(0, "tests")
import paged_kv_cache_161_gb300 as pa
from test_gpu_block_sparse import BF16, E4M3, I32, Batch

def everything(b, k):
    bounds = b.bounds(pa)
    s = b.scores(pa, bounds)
    idx = b.select(pa, s, k, 1, 1)
    return bounds, s, idx, b.attend(pa, idx)

def advance(S, q):
    i = lambda *shape: torch.ones(shape, dtype=I32, device="cuda")
    free = torch.arange(S * 2000, dtype=I32, device="cuda")
    lens, head, qsl, pos = i(S), i(1), i(S + 1), i(S * q)
    slots = torch.ones(S * q, dtype=torch.int64, device="cuda")
    table = i(S, 2000)
    pa.advance_batch(table, i(S), i(S) * q, free, i(1), lens, head, qsl, slots, pos, block_size=16, num_blocks=S * 2000)
    return table, lens, head, qsl, slots, pos

def norm(T, cache):
    x = torch.arange(T * 12 * 128, device="cuda").sin().view(T, 12, 128).to(BF16)
    kc = torch.zeros((T // 16 + 1, 16, 2, 128), device="cuda").to(cache)
    vc, out = torch.zeros_like(kc), torch.empty((T, 8, 128), dtype=BF16, device="cuda")
    cs = torch.arange(64 * 128, device="cuda").cos().view(64, 128)
    pa.norm_rope_write(out, x[:, :8], x[:, 8:10], x[:, 10:], None, None, cs, torch.zeros(T, dtype=I32, device="cuda"),
                       torch.arange(T, device="cuda"), kc, vc)
    return out, kc.float(), vc.float()

batches = [Batch(lens=[300, 90], qs=[1, 1], cache=c, **s) for c in (BF16, E4M3) for s in (dict(D=64), dict())]
batches += [Batch(lens=[300, 90], qs=[100, 30], cache=c, Hq=16, Hkv=8, D=D) for c in (BF16, E4M3) for D in (64, 128)]
calls = [lambda b=b: everything(b, 4) for b in batches]
calls += [lambda: advance(3, 1), lambda: advance(3, 1000), lambda: advance(3, 12000), lambda: norm(5, BF16),
          lambda: norm(5, E4M3), lambda: norm(14000, BF16), lambda: norm(14000, E4M3)]
for i, call in enumerate(calls):
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    torch.cuda.synchronize()
    want = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), i
assert pa.read_device_errors() == 0
print("fine")
"""


def test_the_first_call_of_each_kernel_may_be_captured():
    """What a kernel's first call sets up does not disturb a capture under way."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout + r.stderr
