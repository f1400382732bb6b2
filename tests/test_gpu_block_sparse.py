"""Block-sparse attention on the GPU (bounds, scores, selection, attention) against its
float64 oracle.

Tolerances, derived. Bounds and selection: none (minimum, maximum and whole numbers).
Scores: products of bf16 values are exact in fp32; a sum of 2 D terms, each addition off by at
most 2^-23 of the terms' magnitudes (the tensor core truncates), so 2 D 2^-23 sum |term|.
Attention: each logit off by at most D 2^-23 scale sum |q_d k_d| (call it e, natural units;
+ 2^-21 for the exponential); numerators rounded to bf16 (2^-8) or, over E4M3 caches, f16
(2^-11, and at most 2^-25 of the largest absolutely); the sum runs over the unrounded ones:
(p + 2 e + 2^-18) sum w |v| with p the numerators' rounding, and the result once to bf16.
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


class Batch:
    """Requests of given lengths and query lengths over a shuffled pool; everything the pool
    holds outside the requests' keys is NaN."""

    def __init__(self, lens, qs, B=16, Hq=32, Hkv=8, D=128, cache=BF16, seed=0, pad=0, wide=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.qs, self.B, self.Hq, self.Hkv, self.D, self.cache = lens, qs, B, Hq, Hkv, D, cache
        S = len(lens)
        n = [-(-x // B) for x in lens]
        self.W = max(n) + wide
        self.NB = sum(n) + 5
        perm = torch.randperm(self.NB, generator=g).tolist()
        self.table = np.full((S, self.W), 1 << 30, np.int32)  # entries past a request's blocks are never read
        self.k = torch.full((self.NB, B, Hkv, D), float("nan"))
        self.v = self.k.clone()
        for s in range(S):
            for b in range(n[s]):
                self.table[s, b] = perm.pop()
                rows = min(B, lens[s] - b * B)
                spread = 0.25 + 1.5 * torch.rand(D, generator=g)
                self.k[self.table[s, b], :rows] = torch.randn((rows, Hkv, D), generator=g) * spread
                self.v[self.table[s, b], :rows] = torch.randn((rows, Hkv, D), generator=g)
        self.scales = (1.0, 1.0)
        if cache == E4M3:
            self.scales = (2.0 ** -5, 0.0173)
            self.k, self.v = self.k / self.scales[0], self.v / self.scales[1]
            self.k, self.v = self.k.clamp(-448, 448), self.v.clamp(-448, 448)
        self.k, self.v = self.k.to(cache).cuda(), self.v.to(cache).cuda()
        self.qsl = np.concatenate([[0], np.cumsum(qs)]).astype(int).tolist()
        self.T = self.qsl[-1] + pad
        self.q = torch.randn((self.T, Hq, D), generator=g).to(BF16).cuda()
        dev = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
        self.meta = (dev(self.table), dev(lens), dev(self.qsl))
        self.max_seq, self.max_q = max(lens), max(qs)
        self.scale = D ** -0.5

    def values(self):
        return _f64(self.k) * self.scales[0], _f64(self.v) * self.scales[1]

    def bounds(self, pa):
        out = torch.full((self.NB, self.Hkv, 2, self.D), 5.0, dtype=BF16, device="cuda")
        return pa.block_bounds(out, self.k, *self.meta, max_query_len=self.max_q, max_seq_len=self.max_seq)

    def scores(self, pa, bounds, width=None):
        out = torch.full((self.T, self.Hkv, width or self.W), float("nan"), device="cuda")
        return pa.block_scores(out, self.q, bounds, *self.meta, block_size=self.B, max_query_len=self.max_q,
                               max_seq_len=self.max_seq)

    def select(self, pa, scores, k, init=0, local=0):
        out = torch.full((self.T, self.Hkv, k), -2, dtype=I32, device="cuda")
        return pa.select_blocks(out, scores, *self.meta[1:], block_size=self.B, init_blocks=init, local_blocks=local)

    def attend(self, pa, idx, out=None, **kw):
        out = torch.full((self.T, self.Hq, self.D), float("nan"), dtype=BF16, device="cuda") if out is None else out
        args = dict(max_seq_len=self.max_seq, scale=self.scale, k_scale=self.scales[0], v_scale=self.scales[1])
        return pa.attention_sparse(out, self.q, self.k, self.v, *self.meta, idx, **{**args, **kw})

    def check_attention(self, got, idx, pos_table=None):
        k, v = self.values()
        ref, mag, logit = ss.attention_sparse_ref(_f64(self.q), k, v, self.table, self.lens, self.qsl, idx.cpu().numpy(),
                                                  self.scale)
        p = 2.0 ** -11 + 2.0 ** -25 if self.cache == E4M3 else 2.0 ** -8
        e = self.D * 2.0 ** -23 * logit
        tol = (p + 2 * e + 2.0 ** -18) * mag
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        got = _f64(got)
        live = ~np.isnan(ref)
        assert np.array_equal(live, ~np.isnan(got)), "rows of no request were touched, or others not"
        bad = np.abs(got - ref)[live] > tol[live]
        assert not bad.any(), (int(bad.sum()), np.abs(got - ref)[live].max(), tol[live].max())
        return ref


BATCHES = {
    "one_token": dict(lens=[1], qs=[1]),
    "decode": dict(lens=[15, 16, 17, 300, 1, 64], qs=[1] * 6),
    "decode_padded": dict(lens=[70, 33], qs=[1, 1], pad=3, wide=3),
    "some_without_queries": dict(lens=[70, 33, 90, 5], qs=[1, 0, 3, 0]),
    "chunk": dict(lens=[40, 100], qs=[40, 37], Hq=8, Hkv=2),
    "mixed": dict(lens=[200, 31, 77, 9], qs=[50, 1, 30, 9], Hq=4, Hkv=1),
    "draft": dict(lens=[500, 259], qs=[4, 3]),
    "mha": dict(lens=[50, 120], qs=[1, 6], Hq=6, Hkv=6),
    "g2_d64": dict(lens=[50, 120, 33], qs=[1, 20, 1], Hq=6, Hkv=3, D=64),
    "g8": dict(lens=[50, 333], qs=[1, 5], Hq=16, Hkv=2),
    "b32": dict(lens=[31, 33, 200], qs=[1, 33, 2], B=32, Hq=8, Hkv=4),
    "b128_d64": dict(lens=[129, 700], qs=[5, 1], B=128, Hq=8, Hkv=1, D=64),
    "b48": dict(lens=[95, 97], qs=[3, 1], B=48, Hq=4, Hkv=2),
    "many_short": dict(lens=list(range(1, 81)), qs=[1] * 80, Hq=8, Hkv=4),
    "e4m3_decode": dict(lens=[15, 16, 17, 300, 1], qs=[1] * 5, cache=E4M3),
    "e4m3_chunk_d64": dict(lens=[100, 40], qs=[60, 1], cache=E4M3, Hq=8, Hkv=2, D=64),
    "e4m3_b64_g8": dict(lens=[100, 640], qs=[1, 3], cache=E4M3, B=64, Hq=8, Hkv=1),
}


def _batch(name):
    return Batch(**BATCHES[name], seed=len(name))


@pytest.mark.parametrize("name", BATCHES)
def test_bounds(pa, name):
    b = _batch(name)
    got = b.bounds(pa)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    ref = ss.bounds_ref(np.full(got.shape, 5.0), _f64(b.k), b.table, b.lens, b.qsl)
    assert np.array_equal(_f64(got), ref)  # untouched blocks keep their 5.0; NaN rows past the length are not read


def _full_bounds(pa, b):
    """Every block's bounds, by a call whose queries cover all positions."""
    full = Batch.__new__(Batch)
    full.__dict__.update(b.__dict__)
    S = len(b.lens)
    full.qsl = [0, *np.cumsum(b.lens).tolist()]
    full.max_q = b.max_seq
    full.meta = (b.meta[0], b.meta[1], torch.tensor(full.qsl, dtype=I32, device="cuda"))
    assert S == len(full.meta[1])
    return full.bounds(pa)


@pytest.mark.parametrize("name", BATCHES)
def test_scores(pa, name):
    b = _batch(name)
    bounds = _full_bounds(pa, b)
    got = _f64(b.scores(pa, bounds))
    assert pa.read_device_errors() == 0
    ref, size = ss.scores_ref(_f64(b.q), _f64(bounds), b.table, b.lens, b.qsl, b.B, b.W)
    assert np.array_equal(np.isnan(ref), np.isnan(got))  # padding rows keep their NaN
    assert np.array_equal(ref == -np.inf, got == -np.inf)
    fin = np.isfinite(ref)
    assert (np.abs(got[fin] - ref[fin]) <= 2 * b.D * 2.0 ** -23 * size[fin]).all()


CHUNKS = {  # several column tiles, several block tiles, both kernels in one call
    "long_g4": dict(lens=[4500, 700], qs=[70, 150], Hq=8, Hkv=2),
    "g1_d64": dict(lens=[600, 40], qs=[300, 1], Hq=2, Hkv=2, D=64),
    "g2": dict(lens=[2100], qs=[129], Hq=4, Hkv=2),
    "g8_mixed": dict(lens=[300, 50, 2300, 9], qs=[100, 4, 33, 9], Hq=8, Hkv=1),
    "g8_d64": dict(lens=[500], qs=[64], Hq=16, Hkv=2, D=64),
    "edge_32_and_33_columns": dict(lens=[200, 200, 200], qs=[8, 9, 16], Hq=4, Hkv=1),
    "padded_wide": dict(lens=[90, 77], qs=[64, 65], Hq=4, Hkv=1, pad=5, wide=140),
}


@pytest.mark.parametrize("name", CHUNKS)
def test_scores_of_chunks(pa, name):
    b = Batch(**CHUNKS[name], seed=len(name))
    bounds = _full_bounds(pa, b)
    for _ in range(2):
        got = _f64(b.scores(pa, bounds))
        assert pa.read_device_errors() == 0
        ref, size = ss.scores_ref(_f64(b.q), _f64(bounds), b.table, b.lens, b.qsl, b.B, b.W)
        assert np.array_equal(np.isnan(ref), np.isnan(got))
        assert np.array_equal(ref == -np.inf, got == -np.inf)
        fin = np.isfinite(ref)
        assert (np.abs(got[fin] - ref[fin]) <= 2 * b.D * 2.0 ** -23 * size[fin]).all()


@pytest.mark.parametrize("G,D", [(1, 64), (2, 128), (4, 64), (8, 128)])
def test_scores_of_chunks_among_decodes(pa, G, D):
    """Few long requests between many short and empty ones: the chunks' places in the grid."""
    few = 32 // G
    qs = [1] * 90 + [few + 1] + [0, 2, few] * 15 + [3 * few + 5, 0, 256 // G + 1] + [1] * 40 + [few + 2] * 9
    lens = [q + 7 * i % 150 for i, q in enumerate(qs)]
    b = Batch(lens, qs, Hq=2 * G, Hkv=2, D=D, seed=G)
    bounds = _full_bounds(pa, b)
    got = _f64(b.scores(pa, bounds))
    assert pa.read_device_errors() == 0
    ref, size = ss.scores_ref(_f64(b.q), _f64(bounds), b.table, b.lens, b.qsl, b.B, b.W)
    assert np.array_equal(np.isnan(ref), np.isnan(got))
    assert np.array_equal(ref == -np.inf, got == -np.inf)
    fin = np.isfinite(ref)
    assert (np.abs(got[fin] - ref[fin]) <= 2 * b.D * 2.0 ** -23 * size[fin]).all()


def test_scores_of_fewer_tokens_than_the_longest_request_announced(pa):
    b = Batch([50, 90], [1, 2], Hq=8, Hkv=2)
    bounds = _full_bounds(pa, b)
    expect = b.scores(pa, bounds)
    b.max_q = 80  # at most the longest context
    assert torch.equal(expect, b.scores(pa, bounds))
    assert pa.read_device_errors() == 0


def test_scores_of_chunks_with_bad_blocks(pa):
    b = Batch([400, 300], [100, 20], Hq=8, Hkv=2)
    bounds = _full_bounds(pa, b)
    b.meta[0][0, 7], b.meta[0][1, 2] = b.NB, -1
    s = b.scores(pa, bounds)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == pa.PA_DEVERR["block_range"]
    assert (s[:100, :, 7] == -float("inf")).all() and (s[100:, :, 2] == -float("inf")).all()
    assert torch.isfinite(s[:100, :, 8]).all() and torch.isfinite(s[100:, :, 3]).all()


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("name", BATCHES)
def test_select(pa, name, ties):
    b = _batch(name)
    rng = np.random.default_rng(3)
    s = rng.standard_normal((b.T, b.Hkv, b.W)).astype(np.float32) * 3
    s = np.round(s) if ties else s
    s[:, :, ::7] = -np.inf
    dev = torch.tensor(s, device="cuda")
    for k, init, local in [(1, 0, 0), (3, 1, 1), (8, 0, 2), (b.W + 4, 1, 3)]:
        got = b.select(pa, dev, k, init, local).cpu().numpy()
        assert np.array_equal(got, ss.select_ref(s, b.lens, b.qsl, b.B, k, init, local)), (k, init, local)
    assert pa.read_device_errors() == 0


@pytest.mark.parametrize("n", [1, 31, 32, 33, 1000, 1024, 1025, 4096, 4097, 16385, 32768, 32800, 70000])
@pytest.mark.parametrize("kind", ["normal", "ties", "one_value", "huge_range", "infinities", "zeros_and_subnormals",
                                  "flat_and_infinite", "far_apart"])
def test_select_widths(pa, n, kind):
    """Every width's variant, at its edges: one query token over n blocks."""
    rng = np.random.default_rng(n)
    x = rng.standard_normal((1, 2, n)).astype(np.float32)
    if kind == "ties":
        x = np.round(x * 4) / 4
    if kind == "one_value":
        x[:] = -2.5
    if kind == "huge_range":
        x = (np.sign(x) * 10.0 ** np.clip(x * 12, -44, 38)).astype(np.float32)
    if kind == "infinities":
        x[x > 1.5], x[x < -1], x[np.abs(x) < 0.05] = np.inf, -np.inf, np.nan
        x[0, 0, :3] = [0.0, -0.0, 0.0][: min(3, n)]
    if kind == "flat_and_infinite":  # one value and infinities
        x = rng.choice(np.array([1.5, 1.5, 1.5, np.inf, -np.inf], np.float32), (1, 2, n))
    if kind == "far_apart":  # two close groups of huge values: no linear range separates them
        x = (rng.choice(np.array([3e38, -3e38]), (1, 2, n)) * (1 + 1e-3 * rng.random((1, 2, n)))).astype(np.float32)
        x[0, 1] = 1e30 + rng.integers(0, 3, n) * 2.0 ** 77
        x[0, :, ::5] = np.inf
    if kind == "zeros_and_subnormals":
        x = rng.choice(np.array([0.0, -0.0, 1e-45, -1e-45, 3e-45, -3e-45, 1e-38], np.float32), (1, 2, n))
    lens = torch.tensor([n * 16], dtype=I32, device="cuda")
    qsl = torch.tensor([0, 1], dtype=I32, device="cuda")
    dev = torch.tensor(x, device="cuda")
    for k, init, local in [(64, 1, 2), (max(1, n // 3), 0, 0), (5, 5, 0)]:
        out = torch.full((1, 2, k), -2, dtype=I32, device="cuda")
        pa.select_blocks(out, dev, lens, qsl, block_size=16, init_blocks=init, local_blocks=local)
        for g in range(2):
            y = x[0, g].astype(np.float64)
            idx = np.arange(n)
            forced = (idx < init) | (idx > n - 1 - local)
            y = np.where(forced, np.inf, np.where(np.isnan(y), -np.inf, y))
            order = np.lexsort((idx, -y, ~forced))
            want = np.sort(order[y[order] > -np.inf][:k])
            got = out[0, g].cpu().numpy()
            assert np.array_equal(got[: len(want)], want) and (got[len(want):] == -1).all(), (k, init, local)
    assert pa.read_device_errors() == 0


def _random_lists(b, k, seed=1):
    """Lists in any order with holes, repeats and blocks behind the context."""
    rng = np.random.default_rng(seed)
    idx = np.full((b.T, b.Hkv, k), -1, np.int32)
    for t, s, p in ss.rows_of(b.lens, b.qsl):
        for g in range(b.Hkv):
            n = p // b.B + 1
            picks = rng.integers(0, n, k)
            picks[rng.random(k) < 0.3] = -1
            if k > 2:
                picks[rng.integers(k)] = min(n, b.W - 1)  # behind the context (or the last block again)
                picks[rng.integers(k)] = n - 1
            idx[t, g] = picks
    idx[b.qsl[-1]:] = 1 << 29
    return torch.tensor(idx, device="cuda")


@pytest.mark.parametrize("k", [1, 2, 7, 40])
@pytest.mark.parametrize("name", BATCHES)
def test_attention(pa, name, k):
    b = _batch(name)
    idx = _random_lists(b, k)
    got = b.attend(pa, idx)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    b.check_attention(got, idx)


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_attention_over_every_block_is_attention(pa, cache):
    """All blocks listed: pa_attention's result, within both kernels' rounding."""
    b = Batch([700, 33, 1, 256], [1, 1, 1, 1], cache=cache)
    idx = torch.arange(b.W, device="cuda", dtype=I32).expand(b.T, b.Hkv, b.W).contiguous()
    got = b.attend(pa, idx)
    ref = b.check_attention(got, idx)
    out = torch.empty_like(got)
    if cache == BF16:
        pa.attention(out, b.q, b.k, b.v, *b.meta, max_query_len=1, max_seq_len=b.max_seq, scale=b.scale)
    else:
        pa.attention_fp8(out, b.q, b.k, b.v, *b.meta, max_query_len=1, max_seq_len=b.max_seq, scale=b.scale,
                         k_scale=b.scales[0], v_scale=b.scales[1])
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    assert (np.abs(_f64(out) - ref) <= 1.5e-2 + 1e-2 * np.abs(ref)).all()


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("lens,qs,k,Hkv", [([3000], [1], 187, 2), ([9000, 50], [1, 1], 300, 2), ([1500] * 40, [1] * 40, 60, 2),
                                           ([90] * 41, [1] * 41, 3, 8), ([300, 40] * 30, [2, 9] * 30, 17, 1)])
def test_split_and_unsplit_units(pa, lens, qs, k, Hkv, cache):
    """Lists long enough for clusters of 8 CTAs, units of one CTA each, and units of one warp each."""
    b = Batch(lens, qs, Hq=8, Hkv=Hkv, cache=cache)
    idx = _random_lists(b, k)
    got = b.attend(pa, idx)
    again = b.attend(pa, idx)
    torch.cuda.synchronize()
    assert torch.equal(got, again)  # a fixed merge order
    assert pa.read_device_errors() == 0
    b.check_attention(got, idx)


def test_empty_lists_give_zeros(pa):
    b = Batch([300, 20], [1, 2])
    idx = torch.full((b.T, b.Hkv, 33), -1, dtype=I32, device="cuda")
    idx[1] = 5  # behind request 1's context: nothing either
    got = b.attend(pa, idx)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0 and not got.any()


def test_sharp_softmax(pa):
    b = Batch([900, 400], [1, 3])
    b.scale = 1.0
    idx = _random_lists(b, 24)
    b.check_attention(b.attend(pa, idx), idx)
    assert pa.read_device_errors() == 0


def test_bad_indices_are_skipped_and_flagged(pa):
    b = Batch([200, 90], [1, 1])
    idx = torch.tensor([0, 3, 5], dtype=I32, device="cuda").expand(2, b.Hkv, 3).contiguous()
    clean = b.attend(pa, idx).clone()
    more = torch.cat([idx, torch.full_like(idx[:, :, :1], b.W), torch.full_like(idx[:, :, :1], 2 ** 31 - 1)], 2).contiguous()
    got = b.attend(pa, more)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == pa.PA_DEVERR["block_range"]
    assert torch.allclose(got.float(), clean.float(), atol=2e-2, rtol=2e-2)
    for bad in (-3, b.NB, 2 ** 31 - 1):  # a bad physical block: attention, scores and bounds skip it
        b.meta[0][0, 3] = bad
        b.attend(pa, idx)
        torch.cuda.synchronize()
        assert pa.read_device_errors() == pa.PA_DEVERR["block_range"]
        bounds = torch.zeros((b.NB, b.Hkv, 2, b.D), dtype=BF16, device="cuda")
        s = b.scores(pa, bounds)
        torch.cuda.synchronize()
        assert pa.read_device_errors() == pa.PA_DEVERR["block_range"]
        assert (s[0, :, 3] == -float("inf")).all() and torch.isfinite(s[0, :, 2]).all()
        _full_bounds(pa, b)
        torch.cuda.synchronize()
        assert pa.read_device_errors() == pa.PA_DEVERR["block_range"]


def test_lengths_that_do_not_fit_leave_rows_alone(pa):
    """q_len > seq_len, and a request longer than its table row."""
    b = Batch([40, 90], [1, 1], Hq=8, Hkv=2)
    for lens in ([0, 90], [b.W * b.B + 1, 90]):
        b.meta = (b.meta[0], torch.tensor(lens, dtype=I32, device="cuda"), b.meta[2])
        flag = pa.PA_DEVERR["seq_range"]
        bounds = torch.full((b.NB, b.Hkv, 2, b.D), 5.0, dtype=BF16, device="cuda")
        s = b.scores(pa, bounds)
        torch.cuda.synchronize()
        assert pa.read_device_errors() == flag and torch.isnan(s[0]).all() and not torch.isnan(s[1]).any()
        idx = b.select(pa, torch.zeros_like(s), 3)
        torch.cuda.synchronize()
        assert pa.read_device_errors() == flag and (idx[0] == -2).all() and (idx[1] == torch.arange(3, device="cuda")).all()
        out = b.attend(pa, idx)
        torch.cuda.synchronize()
        assert pa.read_device_errors() == flag and torch.isnan(out[0]).all() and not torch.isnan(out[1]).any()
        b.bounds(pa)
        torch.cuda.synchronize()
        assert pa.read_device_errors() == flag


def test_nan_and_infinite_scores_and_queries_stay_in_their_rows(pa):
    b = Batch([200, 90], [1, 1])
    bounds = _full_bounds(pa, b)
    b.q[0, 3] = float("nan")
    b.q[0, 30] = float("inf")
    s = b.scores(pa, bounds)
    idx = b.select(pa, s, 4, 1, 1)
    out = b.attend(pa, idx)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    assert torch.isnan(out[0, 3]).all() and torch.isfinite(out[1]).all()
    assert ((idx >= -1) & (idx < b.W)).all() and (idx[0, :, 0] == 0).all()


def test_relabelled_blocks_give_the_same_bits(pa):
    b = Batch([300, 140], [2, 1])
    idx = _random_lists(b, 9)
    a = b.attend(pa, idx)
    perm = torch.randperm(b.NB, generator=torch.Generator().manual_seed(5)).cuda()
    k, v = torch.empty_like(b.k), torch.empty_like(b.v)
    k[perm], v[perm] = b.k, b.v
    b.k, b.v = k, v
    t = b.meta[0].long()
    b.meta = (torch.where(t < b.NB, perm[t.clamp(max=b.NB - 1)], t).to(I32), *b.meta[1:])
    assert torch.equal(a, b.attend(pa, idx))
    assert pa.read_device_errors() == 0


def test_offsets_past_32_bits(pa):
    """The same requests in the last blocks of a pool of 2.3e9 elements (4.6 GB) a cache."""
    b = Batch([300, 140, 33], [2, 40, 1])
    idx = _random_lists(b, 9)
    far = Batch.__new__(Batch)
    far.__dict__.update(b.__dict__)
    far.NB = 140000
    far.k, far.v = (torch.empty((far.NB, *x.shape[1:]), dtype=BF16, device="cuda") for x in (b.k, b.v))
    far.k[-b.NB:], far.v[-b.NB:] = b.k, b.v
    t = b.meta[0]
    far.meta = (torch.where(t < b.NB, t + (far.NB - b.NB), t), *b.meta[1:])
    assert torch.equal(b.attend(pa, idx), far.attend(pa, idx))
    near_bounds, far_bounds = _full_bounds(pa, b), _full_bounds(pa, far)
    assert torch.equal(near_bounds[b.meta[0][0, :19].long()], far_bounds[far.meta[0][0, :19].long()])
    assert torch.equal(b.scores(pa, near_bounds), far.scores(pa, far_bounds))
    # a cache write there, beside the same write in a small pool
    q, slots = torch.randn((9, 12, 128), device="cuda").to(BF16), torch.tensor([5, 100, -1, 3, 70, 9, 20, 21, 22], device="cuda")
    cs = torch.rand((50, 128), device="cuda")
    pos = torch.arange(9, dtype=I32, device="cuda")
    outs = []
    for k, v, off in ((b.k, b.v, 0), (far.k, far.v, (far.NB - b.NB) * 16)):
        out = torch.empty((9, 4, 128), dtype=BF16, device="cuda")
        q8 = torch.cat([q[:, :4]] * 4, 1)
        pa.norm_rope_write(out, q[:, :4], q8[:, :8], q8[:, 8:], None, None, cs, pos, torch.where(slots < 0, slots, slots + off),
                           k, v)
        outs.append((out, k[-b.NB:].clone(), v[-b.NB:].clone()))
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    for x, y in zip(*outs):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_more_queries_than_announced_are_flagged(pa):
    """max_query_len is an upper bound; a batch beyond it is reported, not answered silently."""
    b = Batch([300, 64], [50, 1], Hq=8, Hkv=2)
    b.max_q = 1
    bounds = torch.zeros((b.NB, b.Hkv, 2, b.D), dtype=BF16, device="cuda")
    b.scores(pa, bounds)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == pa.PA_DEVERR["seq_range"]
    b.bounds(pa)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == pa.PA_DEVERR["seq_range"]


def test_the_bindings_refuse(pa):
    b = Batch([40], [1])
    bounds = b.bounds(pa)
    s = b.scores(pa, bounds)
    idx = b.select(pa, s, 2)
    with pytest.raises(TypeError):
        pa.attention_sparse(torch.empty_like(b.q), b.q.float(), b.k, b.v, *b.meta, idx, max_seq_len=40, scale=0.1)
    with pytest.raises(ValueError):
        b.attend(pa, idx[:, :4])
    with pytest.raises(ValueError):
        b.attend(pa, idx, out=torch.empty((2, b.Hq, b.D), dtype=BF16, device="cuda"))
    with pytest.raises(TypeError):
        b.attend(pa, idx.long())
    with pytest.raises(pa.PAError):
        b.attend(pa, idx, scale=0.0)
    with pytest.raises(pa.PAError):
        b.attend(pa, idx, k_scale=2.0)  # a bf16 cache has no scale
    with pytest.raises(pa.PAError):
        b.select(pa, s, 2, 2, 1)
    with pytest.raises(pa.PAError):
        b.scores(pa, bounds, width=2)  # three blocks
    with pytest.raises(ValueError):
        pa.block_bounds(bounds[:, :4], b.k, *b.meta, max_query_len=1, max_seq_len=40)
    with pytest.raises(pa.PAError):
        pa.block_bounds(bounds, b.k.float(), *b.meta, max_query_len=1, max_seq_len=40)


def _check_numerators(pa, lens, qs, k, G, Hkv, D, cache):
    b = Batch(lens, qs, Hq=G * Hkv, Hkv=Hkv, D=D, cache=cache, seed=k)
    v = b.v.float()
    v[:, 1::2] = -v[:, 0::2]
    b.v = v.to(cache)
    b.q = (b.q * 0.05).to(BF16)
    idx = np.full((b.T, b.Hkv, k), -1, np.int32)
    rng = np.random.default_rng(k)
    for t, _, p in ss.rows_of(b.lens, b.qsl):
        whole = (p + 1) // b.B  # blocks without a token behind the causal limit
        for g in range(b.Hkv):
            idx[t, g] = rng.choice(whole, k, replace=False)
    idx = torch.tensor(idx, device="cuda")
    got = _f64(b.attend(pa, idx))
    assert pa.read_device_errors() == 0
    kv = b.values()
    ref, mag, logit = ss.attention_sparse_ref(_f64(b.q), *kv, b.table, b.lens, b.qsl, idx.cpu().numpy(), b.scale)
    assert np.median(np.abs(ref)) < 0.1 * np.median(mag)
    p = 2.0 ** -22 if cache == E4M3 else 2.0 ** -16
    tol = (p + 2 * b.D * 2.0 ** -23 * logit + 2.0 ** -17) * mag
    tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), (np.abs(got - ref) / tol).max())


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("lens,qs,k,Hkv,D", [([640, 320], [1, 3], 1, 8, 128), ([640, 320], [1, 3], 12, 2, 64),
                                             ([320] * 45, [1] * 45, 6, 8, 128)])
def test_numerators_keep_fp32_precision(pa, lens, qs, k, Hkv, D, cache):
    """Tokens in pairs v, -v under almost flat weights: the sums cancel to about 1 / 30 of their
    terms, so what the numerators lose before the second product shows beside the output's own
    rounding. A numerator is carried in two 16-bit parts: of bf16 within 2^-16 relative, of f16 within
    2^-22. The fp32 sums: up to 2 k MMAs of a warp, four warps or CTAs merged, each addition
    2^-23 of the magnitudes; 2^-21 for the exponential: together at most 2^-17 up to k = 12.
    The logits as above (2 e)."""
    _check_numerators(pa, lens, qs, k, 4, Hkv, D, cache)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,Hkv,T", [(1, 8, 45), (2, 8, 3), (8, 8, 45), (8, 2, 2)])
def test_numerators_of_other_groups(pa, G, Hkv, T, D, cache):
    """The same with one, two and eight query heads a KV head, units of a warp and of a cluster."""
    _check_numerators(pa, [320] * T, [1] * T, 6, G, Hkv, D, cache)


@pytest.mark.parametrize("S,q,flagged", [(100, 8, True), (100, 3, True), (1, 300, True), (100, 2, False), (100, 0, False)])
def test_more_tokens_than_the_bounds_grid_was_sized_for_are_flagged(pa, S, q, flagged):
    """num_tokens (S * max_query_len unless given) sizes the grid of pa_block_bounds: a batch with more
    query tokens is reported, since some of its blocks have no place there."""
    b = Batch([max(q, 1) + 20] * S, [q] * S, Hq=2, Hkv=2, D=64)
    out = torch.full((b.NB, b.Hkv, 2, b.D), 5.0, dtype=BF16, device="cuda")
    pa.block_bounds(out, b.k, *b.meta, max_query_len=2, max_seq_len=b.max_seq)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == (pa.PA_DEVERR["seq_range"] if flagged else 0)
    pa.block_bounds(out, b.k, *b.meta, max_query_len=max(q, 2), max_seq_len=b.max_seq, num_tokens=max(S * q, 1))
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    ref = ss.bounds_ref(np.full(out.shape, 5.0), _f64(b.k), b.table, b.lens, b.qsl)
    assert np.array_equal(_f64(out), ref)


def _check_scores(b, bounds, got):
    """Scores of every token against float64, on the GPU: value, -inf behind the context, rows of no request."""
    lo, hi = bounds.double().unbind(2)
    G = b.Hq // b.Hkv
    seen = torch.zeros(b.T, dtype=torch.bool)
    for t, s, p in ss.rows_of(b.lens, b.qsl):
        n = p // b.B + 1
        ids = b.meta[0][s, :n].long()
        q = b.q[t].double().view(b.Hkv, G, 1, b.D)
        x, y = q * lo[ids].transpose(0, 1)[:, None], q * hi[ids].transpose(0, 1)[:, None]
        want, size = torch.maximum(x, y).sum(-1).amax(1), (x.abs() + y.abs()).sum(-1).amax(1)
        row = got[t]
        assert (row[:, n:] == -float("inf")).all(), (t, n)
        assert ((row[:, :n].double() - want).abs() <= 2 * b.D * 2.0 ** -23 * size).all(), (t, n)
        seen[t] = True
    assert torch.isnan(got[~seen.cuda()]).all()


RUNS = {  # CTAs of the chunks' kernel that take three to six tiles of blocks, one after another
    "g4": dict(lens=[8200, 8193, 600, 8199], qs=[512, 500, 512, 64], Hq=32, Hkv=8),  # one context ends inside a run
    "g4_d64": dict(lens=[8200, 2049, 600, 8199], qs=[512, 512, 511, 512], Hq=32, Hkv=8, D=64),
    "g1": dict(lens=[8200, 8193, 600, 8199], qs=[512, 33, 600, 512], Hq=8, Hkv=8),
    "g8_d64_wide": dict(lens=[8200, 8210, 1, 7000], qs=[300, 9, 1, 512], Hq=32, Hkv=4, D=64, wide=200, pad=3),
    "g2_b48": dict(lens=[24600, 300], qs=[700, 300], Hq=16, Hkv=8, B=48),
}


@pytest.mark.parametrize("name", RUNS)
def test_scores_of_chunks_over_runs_of_tiles(pa, name):
    b = Batch(**RUNS[name], seed=len(name))
    bounds = _full_bounds(pa, b)
    got = b.scores(pa, bounds)
    again = b.scores(pa, bounds)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    assert torch.equal(got.nan_to_num(nan=7.0), again.nan_to_num(nan=7.0))
    _check_scores(b, bounds, got)


@pytest.mark.parametrize("Hkv", [1, 2, 3, 8])
@pytest.mark.parametrize("G,D,qs", [(4, 128, [1, 4, 2, 1]), (8, 64, [1, 4, 1, 3]), (1, 128, [1, 31, 9, 1])])
def test_scores_of_long_contexts(pa, Hkv, G, D, qs):
    """Decodes and drafts over more tiles than a warp's ring has stages, and more than a CTA takes."""
    b = Batch([5000, 9001, 33, 16400], qs, Hq=G * Hkv, Hkv=Hkv, D=D, seed=Hkv, wide=5)
    bounds = _full_bounds(pa, b)
    got = b.scores(pa, bounds)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    _check_scores(b, bounds, got)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("lens,qs,k,spec", [
    # 1216 units: a warp each, over 33, 64 and 70 chunks
    ([1300] * 4, [38] * 4, 33, dict(Hq=8, Hkv=8, D=64)),
    ([1300, 1001, 900, 1290], [38] * 4, 64, dict(Hq=16, Hkv=8, D=128)),
    ([1300, 1001, 900, 1290], [38] * 4, 70, dict(Hq=8, Hkv=8, D=64)),
    ([2600, 2001], [76] * 2, 18, dict(Hq=16, Hkv=8, D=64, B=64)),
    # 160 units: a CTA each, over 140 and 33 x 4 chunks
    ([2500, 2301], [10, 10], 140, dict(Hq=16, Hkv=8, D=128)),
    ([2500, 2301], [10, 10], 33, dict(Hq=8, Hkv=8, D=64, B=64)),
    # clusters of 8 CTAs, 1100 chunks
    ([18000], [1], 1100, dict(Hq=8, Hkv=2, D=64)),
    ([18000], [2], 1100, dict(Hq=4, Hkv=1, D=128)),
])
def test_lists_longer_than_a_window(pa, lens, qs, k, spec, cache):
    """Lists of which a warp takes more than 32 chunks: its second and third window of look-ups."""
    b = Batch(lens, qs, cache=cache, seed=k, **spec)
    idx = _random_lists(b, k)
    got = b.attend(pa, idx)
    again = b.attend(pa, idx)
    torch.cuda.synchronize()
    assert torch.equal(got, again) and pa.read_device_errors() == 0
    b.check_attention(got, idx)
