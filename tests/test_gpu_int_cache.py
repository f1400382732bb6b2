"""Integer-coded caches on the GPU: the cache's bytes and what is read back equal the oracle's bit for bit
(the definition names every rounding); attention over the codes against
float64, within intmodel's tolerance.
"""
import numpy as np
import pytest
import torch

import intmodel
from oracle import int_cache as ic

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_161_gb300 as m

    m.read_device_errors(clear=True)
    return m


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _cache(NB, H, B, D, bits, fill=None):
    shape = (NB, H, B * (D * bits // 8 + 4))
    if fill is not None:
        return torch.full(shape, fill, dtype=torch.uint8, device="cuda")
    return torch.randint(0, 256, shape, dtype=torch.uint8, generator=torch.Generator().manual_seed(NB)).cuda()


def _rows(T, H, D, dtype, seed, fused):
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn((T, 2 * H, D), generator=g) * (torch.rand(D, generator=g) * 1.5 + 0.1) + torch.randn(D, generator=g) * 0.3
    kv = kv.to(dtype).cuda()
    k, v = kv.split([H, H], 1)
    return (k, v) if fused else (k.contiguous(), v.contiguous())


# ------------------------------------------------------------------------------- write and read
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,H,D,B,fused", [(1, 1, 64, 4, False), (3, 2, 128, 16, True), (37, 8, 128, 16, False),
                                           (61, 3, 64, 12, True), (700, 8, 128, 32, True), (900, 4, 64, 128, False)])
def test_cache_bytes_equal_the_oracle(pa, dtype, bits, T, H, D, B, fused):
    k, v = _rows(T, H, D, dtype, T, fused)
    NB = -(-T // B) + 2
    slots = torch.randperm(NB * B, generator=torch.Generator().manual_seed(1))[:T]
    slots[T // 2: T // 2 + T // 9] = -1
    kc, vc = _cache(NB, H, B, D, bits), _cache(NB, H, B, D, bits, fill=7)
    want = [ic.write(c.cpu().numpy(), _f64(x), slots.tolist(), bits) for c, x in ((kc, k), (vc, v))]
    assert pa.kv_write_int(k, v, kc, vc, slots.cuda(), bits=bits) is None
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    for got, ref in zip((kc, vc), want):
        assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_unusual_rows(pa, bits, dtype):
    """Constant rows, signed zeros, subnormals, the largest floats, ties, NaN and infinities."""
    D, B = 64, 16
    x = torch.zeros((12, 1, D))
    x[1] = -3.25
    x[2, 0, ::2] = -0.0
    x[3] = torch.linspace(-1e-39, 2e-39, D)
    x[4] = torch.linspace(-1.6e38, 1.6e38, D)
    x[5, 0, :2] = torch.tensor([3e38, -3e38])
    x[6, 0, 5] = float("nan")
    x[7, 0, 63] = float("inf")
    x[8, 0, 0] = -float("inf")
    x[9] = torch.arange(D) * 0.5  # half-integer codes: ties to even
    x[10, 0, 3] = 1e-30
    x[11] = 7 + torch.arange(D) * 2.0 ** -18
    x = x.to(dtype).cuda()
    kc, vc = _cache(1, 1, B, D, bits), _cache(1, 1, B, D, bits)
    slots = torch.arange(12)
    want = [ic.write(c.cpu().numpy(), _f64(x), slots.tolist(), bits) for c in (kc, vc)]
    pa.kv_write_int(x, x, kc, vc, slots.cuda(), bits=bits)
    out = torch.zeros((2, 12, 1, D), device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    pa.kv_read_int(out[0], out[1], kc, vc, torch.zeros((1, 1), dtype=I32, device="cuda"), None, i32(12), i32(0, 12), bits=bits)
    torch.cuda.synchronize()
    for got, ref in zip((kc, vc), want):
        assert np.array_equal(got.cpu().numpy(), ref)
    values = ic.rows(want[0], [0], 12, D, bits)[0]
    assert np.isnan(values[5:9]).all() and np.isfinite(values[:5]).all()
    assert np.array_equal(out[0].cpu().numpy(), values.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,D,B,lens,starts", [
    (1, 64, 4, [1], None), (8, 128, 16, [40, 0, 1, 333, 16], None), (3, 128, 64, [100, 64, 65], [0, 64, 1]),
    (4, 64, 12, [7, 150, 0, 0, 25], [6, 3, 0, 0, 25]), (2, 128, 128, [1000], [999])])
def test_read_back(pa, bits, dtype, H, D, B, lens, starts):
    """Values in their rows; rows behind a request's positions, and of no request, stay as they were."""
    g = torch.Generator().manual_seed(B)
    S = len(lens)
    W = max(1, -(-max(lens) // B))
    NB = S * W + 2
    table = torch.randperm(NB, generator=g)[: S * W].view(S, W).to(I32)
    kc, vc = _cache(NB, H, B, D, bits, 0), _cache(NB, H, B, D, bits, 0)
    slots = torch.arange(NB * B)
    k, v = _rows(NB * B, H, D, BF16, 3, False)
    pa.kv_write_int(k, v, kc, vc, slots.cuda(), bits=bits)
    first = starts or [0] * S
    room = [max(0, L - s) + (i % 3) for i, (L, s) in enumerate(zip(lens, first))]
    rsl = [2]
    for n in room:
        rsl.append(rsl[-1] + n)
    R = rsl[-1] + 3
    out = [torch.full((R, H, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    i32 = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    pa.kv_read_int(out[0], out[1], kc, vc, table.cuda(), None if starts is None else i32(starts), i32(lens), i32(rsl), bits=bits)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    for got, c in zip(out, (kc, vc)):
        want = np.full((R, H, D), 7.0)
        for s in range(S):
            n = lens[s] - first[s]
            if n > 0:
                want[rsl[s]: rsl[s] + n] = ic.rows(c.cpu().numpy(), table[s].tolist(), lens[s], D, bits)[0][first[s]:]
        want = torch.tensor(want).float().to(dtype)  # two roundings of an exact sum of few bits: fp32, then the output's
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,D,B,S", [(2603, 8, 128, 16, 9), (5001, 5, 64, 4, 700)])
def test_many_rows(pa, bits, dtype, T, H, D, B, S):
    """Sizes at which a lane takes more of the work, with unusual rows and padding among the others."""
    g = torch.Generator().manual_seed(T)
    k, v = _rows(T, H, D, dtype, T, True)
    for x in (k, v):
        x[5::97, H - 1, 3] = float("nan")
        x[7::89, 0, D - 1] = -float("inf")
        x[11::83] = 2.75
        x[13::79, :, ::2] = -0.0
    cuts = torch.cat([torch.zeros(1), torch.randint(0, T + 1, (S - 1,), generator=g).sort().values, torch.tensor([T])]).to(I32)
    lens = cuts.diff()
    W = max(1, -(-int(lens.max()) // B))
    NB = int((-(-lens // B)).sum()) + 3
    table, ids = torch.full((S, W), -1, dtype=I32), torch.randperm(NB, generator=g).to(I32)
    slots = torch.empty(T, dtype=torch.int64)
    for s in range(S):
        n, ids = -(-int(lens[s]) // B), ids[-(-int(lens[s - 1]) // B) if s else 0:]
        table[s, :n] = ids[:n]
        at = torch.arange(int(lens[s]))
        slots[cuts[s]: cuts[s + 1]] = table[s, at // B].long() * B + at % B
    slots[T // 2: T // 2 + 20] = -1
    kc, vc = _cache(NB, H, B, D, bits), _cache(NB, H, B, D, bits, fill=0)
    want = [ic.write(c.cpu().numpy(), _f64(x), slots.tolist(), bits) for c, x in ((kc, k), (vc, v))]
    pa.kv_write_int(k, v, kc, vc, slots.cuda(), bits=bits)
    out = [torch.empty((T, H, D), dtype=dtype, device="cuda") for _ in range(2)]
    pa.kv_read_int(out[0], out[1], kc, vc, table.cuda(), None, lens.cuda(), cuts.cuda(), bits=bits)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    for got, c, w in zip(out, (kc, vc), want):
        assert np.array_equal(c.cpu().numpy(), w)
        rows = np.concatenate([ic.rows(w, table[s].tolist(), int(lens[s]), D, bits)[0] for s in range(S)])
        assert torch.equal(got.cpu().nan_to_num(nan=1e30), torch.tensor(rows).float().to(dtype).nan_to_num(nan=1e30))


def test_read_takes_what_fits_only(pa):
    """Positions past the rows or the table, negative ones and bad blocks are reported and leave their rows."""
    H, D, B = 1, 64, 16
    kc = _cache(4, H, B, D, 8)
    table = torch.tensor([[0, 1], [2, 9], [3, 0], [1, 2]], dtype=I32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=I32, device="cuda")  # noqa: E731
    out = [torch.full((120, H, D), 7.0, device="cuda") for _ in range(2)]
    pa.kv_read_int(*out, kc, kc, table, i32(0, 0, 0, -1), i32(40, 20, 32, 5), i32(0, 40, 60, 91, 120), bits=8)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0x6
    a = out[0].cpu()
    assert (a[:40] == 7).all() and (a[56:] == 7).all() and not (a[40:56] == 7).all()
    out[0].fill_(7.0)
    pa.kv_read_int(*out, kc, kc, table[:1], None, i32(20), i32(5, 24), bits=8)  # 20 positions, 19 rows
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0x4 and (out[0] == 7).all()


def test_write_skips_slots_outside(pa):
    k, v = _rows(3, 2, 64, BF16, 0, False)
    kc, vc = _cache(2, 2, 16, 64, 4), _cache(2, 2, 16, 64, 4)
    want = ic.write(kc.cpu().numpy(), _f64(k), [5, -1, -7], 4)
    pa.kv_write_int(k, v, kc, vc, torch.tensor([5, 32, -7], device="cuda"), bits=4)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0x1
    assert np.array_equal(kc.cpu().numpy(), want)


def test_blocks_are_copied_and_swapped_whole(pa):
    kc, vc = _cache(6, 2, 16, 64, 4), _cache(6, 2, 16, 64, 4, fill=3)
    before = kc.clone()
    pa.copy_blocks(kc, vc, torch.tensor([[1, 4], [0, 2]], device="cuda"))
    host = [torch.zeros((3,) + tuple(kc.shape[1:]), dtype=torch.uint8).pin_memory() for _ in range(2)]
    pa.swap_blocks(kc, vc, host[0], host[1], torch.tensor([[4, 0], [5, 2]], device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(kc[4], before[1]) and torch.equal(kc[2], before[0]) and torch.equal(kc[5], before[5])
    assert torch.equal(host[0][0], before[1].cpu()) and torch.equal(host[0][2], before[5].cpu()) and (host[1][0] == 3).all()


# ------------------------------------------------------------------------------- attention
class Batch:
    """Requests over a pool whose every slot was written; `tail` fills what lies behind the contexts."""

    def __init__(self, pa, lens, qlens, Hq, Hkv, D, B, bits, seed=0, pad=0, size=1.0, vsize=1.0, spread=None):
        g = torch.Generator().manual_seed(seed)
        self.pa, self.lens, self.qlens, self.bits, self.B, self.D = pa, lens, qlens, bits, B, D
        S = len(lens)
        self.W = max(1, -(-max(lens) // B)) + 1
        self.NB = S * self.W + 1
        self.table = torch.randperm(self.NB, generator=g)[: S * self.W].view(S, self.W).to(I32)
        n = self.NB * B
        k = torch.randn((n, Hkv, D), generator=g) * (torch.rand(D, generator=g) + 0.3) * size + torch.randn(D, generator=g) * 0.2
        v = torch.randn((n, Hkv, D), generator=g) * vsize + 0.1 * vsize
        if spread:  # value rows of very different sizes
            v = v * torch.exp2(torch.randint(-spread, spread + 1, (n, Hkv, 1), generator=g).float())
        self.kc, self.vc = (_cache(self.NB, Hkv, B, D, bits, 0) for _ in range(2))
        pa.kv_write_int(k.to(BF16).cuda(), v.to(BF16).cuda(), self.kc, self.vc, torch.arange(n).cuda(), bits=bits)
        self.qsl = [0]
        for x in qlens:
            self.qsl.append(self.qsl[-1] + x)
        T = self.qsl[-1] + pad
        self.q = torch.randn((T, Hq, D), generator=g).to(BF16).cuda()
        self.out = torch.full((T, Hq, D), 7.0, dtype=BF16, device="cuda")
        self.scale = D ** -0.5
        self.ws = torch.randint(0, 256, (pa.attention_int_workspace_size(S, T, Hq, Hkv, D),), dtype=torch.uint8,
                                device="cuda")  # no contents needed

    def i32(self, x):
        return torch.tensor(x, dtype=I32, device="cuda")

    def run(self, max_q=None, **kw):
        self.args = (self.out, self.q, self.kc, self.vc, self.table.cuda(), self.i32(self.lens), self.i32(self.qsl))
        kw = dict(dict(bits=self.bits, max_query_len=max(self.qlens) if max_q is None else max_q,
                       max_seq_len=max(max(self.lens), 1), scale=self.scale, workspace=self.ws), **kw)
        self.kw = kw
        got = self.pa.attention_int(*self.args, **kw)
        torch.cuda.synchronize()
        assert got is self.out
        return self

    def check(self, requests=None):
        assert self.pa.read_device_errors() == 0
        kc, vc, q, out = self.kc.cpu().numpy(), self.vc.cpu().numpy(), _f64(self.q), _f64(self.out)
        for s in range(len(self.lens)) if requests is None else requests:
            a, b, L = self.qsl[s], self.qsl[s + 1], self.lens[s]
            if a == b:
                continue
            ref, tol = intmodel.attention(q[a:b], kc, vc, self.table[s].tolist(), L, self.scale, self.bits)
            err = np.abs(out[a:b] - ref)
            assert (err <= tol).all(), (s, L, float((err / tol).max()))
        n = self.qsl[-1]
        assert (self.out[n:] == 7).all()  # rows of no request
        return self


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (8, 2, 64), (3, 3, 128), (8, 1, 64), (16, 1, 128), (6, 2, 128), (5, 5, 64)])
@pytest.mark.parametrize("B", [4, 16, 64])
def test_decode(pa, bits, Hq, Hkv, D, B):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 64, 100, 257, 1000]
    Batch(pa, lens, [1] * len(lens), Hq, Hkv, D, B, bits, seed=B, pad=2).run().check()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("qlens,B", [([3, 1, 8, 2], 16), ([0, 5, 1, 0, 2], 8), ([40, 1], 128), ([17, 33], 12)])
def test_drafts_and_chunks(pa, bits, qlens, B):
    lens = [q + x for q, x in zip(qlens, (90, 0, 300, 31, 1))]
    for Hq, Hkv, D in ((4, 1, 128), (8, 1, 64), (2, 2, 128)):
        Batch(pa, lens, qlens, Hq, Hkv, D, B, bits, seed=len(qlens), pad=1).run().check()


@pytest.mark.parametrize("bits", [4, 8])
def test_one_long_request_cut_over_the_grid(pa, bits):
    Batch(pa, [30011], [1], 4, 1, 128, 16, bits, seed=5).run().check()
    Batch(pa, [9001, 5], [4, 1], 8, 2, 64, 32, bits, seed=6).run().check()


@pytest.mark.parametrize("bits", [4, 8])
def test_uneven_lengths_cut_between_warps_and_ctas(pa, bits):
    g = np.random.default_rng(bits)
    lens = [int(x) for x in np.clip(np.exp(g.normal(5, 1.5, 70)), 1, 6000)]
    b = Batch(pa, lens, [1] * 70, 8, 2, 128, 16, bits, seed=9).run().check(range(0, 70, 3))
    first = b.out.clone()
    b.run()  # the same bits again, over what the first run left in the workspace
    assert torch.equal(first, b.out)


@pytest.mark.parametrize("bits", [4, 8])
def test_large_logits_and_value_rows_of_many_sizes(pa, bits):
    Batch(pa, [700, 300], [1, 2], 4, 1, 128, 16, bits, seed=11, size=6.0).run(scale=1.0)  # the maximum moves often
    b = Batch(pa, [700, 300], [1, 2], 4, 1, 128, 16, bits, seed=11, size=2.0, spread=12)
    b.scale = 0.5
    b.run().check()
    for vsize in (1e-30, 1e30):
        Batch(pa, [333], [1], 4, 2, 64, 16, bits, seed=12, vsize=vsize).run().check()


@pytest.mark.parametrize("bits", [4, 8])
def test_queries_of_any_size(pa, bits):
    for size in (1e-30, 1e30):
        b = Batch(pa, [200], [1], 4, 1, 128, 16, bits, seed=13)
        b.q.mul_(size)
        b.scale = float(D_SCALE / size)
        b.run().check()
    b = Batch(pa, [200], [1], 4, 1, 128, 16, bits, seed=13)
    b.q.zero_()
    b.run().check()


D_SCALE = 128 ** -0.5


@pytest.mark.parametrize("bits", [4, 8])
def test_what_lies_behind_a_request_does_not_matter(pa, bits):
    """NaN rows behind every context, in its last block: the outputs keep their bits; a NaN row inside
    reaches the tokens that see it and no other."""
    lens, qlens, B, D = [33, 50, 17], [1, 4, 2], 16, 128
    b = Batch(pa, lens, qlens, 4, 1, D, B, bits, seed=21).run().check()
    clean = b.out.clone()
    row = D * bits // 8

    def poison(cache, s, pos):
        blk, o = int(b.table[s, pos // B]), pos % B
        cache[blk, :, B * row + 4 * o: B * row + 4 * o + 4] = torch.tensor([0xC0, 0x7F] * 2, dtype=torch.uint8, device="cuda")
        cache[blk, :, o * row:(o + 1) * row] = 0xFF

    for s in range(3):
        for pos in range(lens[s], -(-lens[s] // B) * B):
            poison(b.kc, s, pos)
            poison(b.vc, s, pos)
    b.run()
    assert torch.equal(b.out, clean)
    for cache in (b.kc, b.vc):
        saved = cache.clone()
        poison(cache, 1, 47)  # positions 46 .. 49 ask: the first does not see it
        b.run()
        cache.copy_(saved)
        a = b.qsl[1]
        assert torch.equal(b.out[: a + 1], clean[: a + 1]) and torch.equal(b.out[b.qsl[2]:], clean[b.qsl[2]:])
        assert b.out[a + 1: a + 4].isnan().all()


def test_malformed_requests_are_reported_and_leave_their_rows(pa):
    b = Batch(pa, [40, 3, 60, 20], [1, 4, 2, 1], 4, 1, 64, 16, 4, seed=31)  # the second has more queries than keys
    b.run()
    assert pa.read_device_errors() == 0x4
    out = _f64(b.out)
    assert (out[1:5] == 7).all() and not (out[5:7] == 7).any() and not (out[0] == 7).any()
    b.out.fill_(7.0)
    b.lens[1] = 10
    b.run(max_q=3)  # 4 queries where 3 were announced
    assert pa.read_device_errors() == 0x4 and (b.out[1:5] == 7).all()
    b.out.fill_(7.0)
    b.run(max_seq_len=50)  # a request of 60 keys
    assert pa.read_device_errors() == 0x4 and (b.out[5:7] == 7).all() and not (b.out[1:5] == 7).any()
    b.table[0, 1] = 10 ** 6  # a block that is not there: reported, the others' rows are right
    b.out.fill_(7.0)
    b.run()
    assert pa.read_device_errors() == 0x2
    b.check(range(1, 4))
    with pytest.raises(pa.PAError) as e:
        b.run(workspace=b.ws[:-256].clone())
    assert e.value.status == 3


def test_requests_that_lie_over_one_another(pa):
    """More work than 32 bits count, which only a decreasing query_start_loc can ask for: reported, not run."""
    T, H, D, W, S = 65536, 8, 64, 65536, 64
    cache = torch.zeros((1, H, 16 * (D // 2 + 4)), dtype=torch.uint8, device="cuda")
    table = torch.zeros((S, W), dtype=torch.int32, device="cuda")
    lens = torch.full((S,), 16 * W, dtype=torch.int32, device="cuda")
    qsl = torch.tensor([0, T] * (S // 2) + [0], dtype=torch.int32, device="cuda")
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = torch.empty(pa.attention_int_workspace_size(S, T, H, H, D), dtype=torch.uint8, device="cuda")
    pa.attention_int(out, q, cache, cache, table, lens, qsl, bits=4, max_query_len=T, max_seq_len=16 * W, scale=1.0,
                     workspace=ws)
    torch.cuda.synchronize()
    assert pa.read_device_errors(clear=True) == pa.PA_DEVERR["seq_range"]
    assert (out == 7).all()


def test_argument_checks_of_the_binding(pa):
    b = Batch(pa, [40], [1], 4, 1, 64, 16, 4)
    for kw, err in ((dict(bits=5), ValueError), (dict(bits=8), ValueError), (dict(bits=0), ValueError), (dict(scale=0.0), pa.PAError),
                    (dict(workspace=b.ws.int()), TypeError), (dict(workspace=b.ws.cpu()), ValueError),
                    (dict(max_query_len=2 ** 40), ValueError)):
        with pytest.raises(err):
            b.run(**kw)
    with pytest.raises(TypeError):
        pa.attention_int(b.out.float(), *b.args[1:], **b.kw)
    with pytest.raises(ValueError):
        pa.attention_int(b.out, b.q, b.kc, b.vc[:1], *b.args[4:], **b.kw)
    k = torch.zeros((2, 1, 64), dtype=BF16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        pa.kv_write_int(k.half(), k.half(), b.kc, b.vc, slots, bits=4)
    with pytest.raises(ValueError):
        pa.kv_write_int(k, k, b.kc, b.vc, slots[:1], bits=4)
    with pytest.raises(ValueError):
        pa.kv_write_int(k.expand(2, 2, 64), k.expand(2, 2, 64), b.kc, b.vc, slots, bits=4)
    with pytest.raises(ValueError):
        pa.kv_write_int(k[..., ::2], k[..., ::2], b.kc, b.vc, slots, bits=4)


def test_another_stream_and_offsets_past_32_bits(pa):
    """A pool of more than 2^32 bytes, its last blocks used, on a stream of the caller's."""
    H, D, B, bits = 1, 128, 128, 8
    rec = B * (D + 4)
    NB = (1 << 32) // rec + 40
    kc, vc = (torch.zeros((NB, H, rec), dtype=torch.uint8, device="cuda") for _ in range(2))
    n = 3 * B - 5
    k, v = _rows(n, H, D, BF16, 1, False)
    table = torch.tensor([[NB - 1, NB - 2, 5]], dtype=I32, device="cuda")
    pos = torch.arange(n)
    slots = (table.cpu().long()[0][pos // B] * B + pos % B).cuda()
    q = torch.randn((1, 4, D), device="cuda").to(BF16)
    out, back = torch.zeros_like(q), [torch.zeros((n, H, D), dtype=F32, device="cuda") for _ in range(2)]
    ws = torch.empty(pa.attention_int_workspace_size(1, 1, 4, H, D), dtype=torch.uint8, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    lens, qsl, rsl = i32(n), i32(0, 1), i32(0, n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pa.kv_write_int(k, v, kc, vc, slots, bits=bits, stream=s)
    pa.kv_read_int(*back, kc, vc, table, None, lens, rsl, bits=bits, stream=s)
    pa.attention_int(out, q, kc, vc, table, lens, qsl, bits=bits, max_query_len=1, max_seq_len=n, scale=0.1, workspace=ws, stream=s)
    s.synchronize()
    assert pa.read_device_errors() == 0
    ref = [ic.value(*ic.quantise(_f64(x), bits)) for x in (k, v)]
    for got, want in zip(back, ref):
        assert np.array_equal(got.cpu().numpy(), want.astype(np.float32))
    o = ic.attend(_f64(q), ref[0], ref[1], n - 1, 0.1)[0]
    assert np.abs(_f64(out) - o).max() < 2.0 ** -7 * np.abs(o).max() + 2e-3
