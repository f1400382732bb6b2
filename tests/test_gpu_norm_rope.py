"""pa_norm_rope_write on the GPU against its float64 oracle.

Tolerance, derived from the arithmetic. fp32 with 2^-24 a rounding: the sum of 128 squares is
8 in order, then a tree of 4 shuffles (12 additions and the products: at most 13 roundings,
halved by the root), rsqrt 2 units, two products: the normed value is within 2^-20 relative.
The rotation of (a, b) has three roundings of terms bounded by |a| + |b|. Together at most
2^-19 (|a| + |b|), before one rounding to the output: half a step, 2^-8 relative for bf16,
2^-24 for fp32; E4M3 codes of x / scale: 2^-4 relative, or 2^-10 (half the smallest step).
"""
import numpy as np
import pytest
import torch

from oracle import serving_step as ss

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_161_gb300 as m

    m.read_device_errors(clear=True)
    return m


def _f64(t):
    return t.detach().float().cpu().double().numpy()


class Case:
    def __init__(self, T, Hq, Hkv, D, dtype=BF16, cache=None, rot=None, axes=1, interleaved=False, norm=(True, True),
                 fused=False, seed=0, limit=1000, size=2.0, sections=None):
        g = torch.Generator().manual_seed(seed)
        cache = cache or dtype
        self.T, self.Hq, self.Hkv, self.D, self.B = T, Hq, Hkv, D, 4
        self.rot, self.interleaved, self.eps = rot or D, interleaved, 1e-5
        qkv = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * size).to(dtype).cuda()
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() if n else None for n in norm]
        ang = torch.arange(limit).double()[:, None] * 10000.0 ** (-torch.arange(0, self.rot, 2).double() / self.rot)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        half = self.rot // 2
        self.sections = sections or (None if axes == 1 else tuple([half - (axes - 1) * (half // 4)] + [half // 4] * (axes - 1)))
        shape = (T,) if self.sections is None else (len(self.sections), T)
        self.pos = torch.randint(0, limit, shape, generator=g, dtype=torch.int32).cuda()
        NB = T // self.B + 3
        self.slots = torch.randperm(NB * self.B, generator=g)[:T].cuda()
        self.kc = torch.zeros((NB, self.B, Hkv, D), device="cuda").to(cache)
        self.vc = torch.zeros_like(self.kc)
        self.out = torch.full((T, Hq, D), 7.0, dtype=dtype, device="cuda")
        self.scales = (2.0 ** -5, 0.0173) if cache == E4M3 else (1.0, 1.0)

    def run(self, pa, **kw):
        args = dict(eps=self.eps, interleaved=self.interleaved, sections=self.sections, k_scale=self.scales[0],
                    v_scale=self.scales[1])
        args.update(kw)
        return pa.norm_rope_write(self.out, self.q, self.k, self.v, *self.w, self.cos_sin, self.pos, self.slots, self.kc,
                                  self.vc, **args)

    def check(self, skip=(), tokens=None):
        table = _f64(self.cos_sin)
        pos = self.pos.cpu().numpy().reshape(-1, self.T)
        sections = self.sections or (self.rot // 2,)
        slots = self.slots.tolist()
        rows = self.kc.shape[0] * self.B
        kc, vc = (_f64(x).reshape(rows, self.Hkv, self.D) for x in (self.kc, self.vc))
        out, v = _f64(self.out), _f64(self.v)
        w = [None if x is None else _f64(x) for x in self.w]
        unit = 2.0 ** -8 if self.out.dtype == BF16 else 2.0 ** -24
        written = set() if tokens is None else {x for x in slots if 0 <= x < rows}
        for t in range(self.T) if tokens is None else tokens:
            if t in skip:
                assert (out[t] == 7.0).all()
                continue
            cos, sin = ss.angles_of(table, pos, sections, t)
            for x, wt, got, scale in ((_f64(self.q[t]), w[0], out[t], None),
                                      (_f64(self.k[t]), w[1], kc[slots[t]] if 0 <= slots[t] < rows else None, self.scales[0])):
                if got is None:
                    continue
                for h in range(x.shape[0]):
                    y, z = ss.norm_rope_ref(x[h], wt, self.eps, cos, sin, self.interleaved)
                    mate = y.copy()
                    half = self.rot // 2
                    a, b = (slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.interleaved else \
                        (slice(0, half), slice(half, self.rot))
                    mate[a], mate[b] = y[b], y[a]
                    slack = 2.0 ** -19 * (np.abs(y) + np.abs(mate))
                    self._near(got[h], z, slack, scale if self.kc.dtype == E4M3 else None, unit)
            if 0 <= slots[t] < rows:
                written.add(slots[t])
                if self.vc.dtype == E4M3:
                    self._near(vc[slots[t]], v[t], 2.0 ** -23 * np.abs(v[t]), self.scales[1], unit)
                else:
                    assert np.array_equal(vc[slots[t]], v[t])
        others = [r for r in range(rows) if r not in written]
        assert not kc[others].any() and not vc[others].any()

    @staticmethod
    def _near(got, want, slack, scale, unit):
        if scale is None:
            tol = (np.abs(want) + slack) * unit + slack
        else:
            x = np.clip(want / scale, -448, 448)
            want, tol = x, np.maximum((np.abs(x) + slack / scale) * 2.0 ** -4, 2.0 ** -10) + slack / scale
        bad = np.abs(got - want) > tol
        assert not bad.any(), (np.abs(got - want)[bad].max(), tol[bad].max())


CASES = {
    "one_token": dict(T=1, Hq=32, Hkv=8, D=128),
    "fused_gqa": dict(T=37, Hq=32, Hkv=8, D=128, fused=True),
    "mha_f32": dict(T=9, Hq=8, Hkv=8, D=128, dtype=F32),
    "f32_d64_fused": dict(T=33, Hq=5, Hkv=1, D=64, dtype=F32, fused=True),
    "odd_heads": dict(T=13, Hq=9, Hkv=3, D=64, fused=True),
    "interleaved": dict(T=21, Hq=4, Hkv=2, D=128, interleaved=True),
    "interleaved_partial_d64": dict(T=21, Hq=4, Hkv=2, D=64, rot=16, interleaved=True, fused=True),
    "partial_rot": dict(T=11, Hq=4, Hkv=1, D=128, rot=48),
    "partial_rot_16": dict(T=11, Hq=4, Hkv=1, D=64, rot=16, dtype=F32),
    "three_axes": dict(T=40, Hq=8, Hkv=2, D=128, axes=3, fused=True),
    "three_axes_interleaved": dict(T=40, Hq=8, Hkv=2, D=64, axes=3, interleaved=True),
    "four_axes_odd_sections": dict(T=19, Hq=2, Hkv=2, D=128, sections=(3, 0, 50, 11)),
    "odd_sections_interleaved": dict(T=19, Hq=2, Hkv=2, D=128, sections=(1, 30, 33), interleaved=True),
    "one_section": dict(T=5, Hq=2, Hkv=2, D=64, sections=(32,)),
    "no_norm": dict(T=15, Hq=8, Hkv=4, D=128, norm=(False, False)),
    "q_norm_only": dict(T=15, Hq=8, Hkv=4, D=128, norm=(True, False)),
    "k_norm_only_f32": dict(T=15, Hq=8, Hkv=4, D=64, norm=(False, True), dtype=F32),
    "e4m3": dict(T=29, Hq=32, Hkv=8, D=128, cache=E4M3, fused=True),
    "e4m3_f32_d64": dict(T=29, Hq=4, Hkv=2, D=64, dtype=F32, cache=E4M3, interleaved=True),
    "e4m3_saturates": dict(T=9, Hq=4, Hkv=2, D=128, cache=E4M3, size=30.0, norm=(True, False)),
    "small_values": dict(T=9, Hq=4, Hkv=2, D=128, size=1e-4),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_the_oracle(pa, name):
    c = Case(**CASES[name], seed=len(name))
    assert c.run(pa) is c.out
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    c.check()


LONG = {  # enough tokens for the streaming kernel; checked on a sample of tokens and every untouched slot
    "fused_gqa": dict(Hq=32, Hkv=8, D=128, fused=True),
    "three_axes": dict(Hq=8, Hkv=2, D=128, axes=3, fused=True),
    "odd_heads_d64": dict(Hq=7, Hkv=3, D=64),
    "odd_sections_interleaved": dict(Hq=4, Hkv=1, D=128, sections=(1, 30, 0, 33), interleaved=True),
    "partial_rot_f32": dict(Hq=4, Hkv=2, D=128, rot=32, dtype=F32),
    "e4m3": dict(Hq=8, Hkv=4, D=128, cache=E4M3, axes=2),
    "e4m3_f32_d64_no_norm": dict(Hq=3, Hkv=1, D=64, dtype=F32, cache=E4M3, norm=(False, False)),
    "wide_mha_f32": dict(Hq=24, Hkv=24, D=128, dtype=F32),  # a token too large for the ring: the other kernel
}


@pytest.mark.parametrize("name", LONG)
def test_long_prompts_match_the_oracle(pa, name):
    spec = LONG[name]
    row = spec["D"] * (4 if spec.get("dtype") == F32 else 2)
    T = (40 << 20) // ((spec["Hq"] + 2 * spec["Hkv"]) * row) + 77  # 40 MB of rows: where the stream begins
    c = Case(T=T, **spec, seed=len(name))
    c.slots[11] = -1
    c.slots[T - 1] = -7
    c.pos.view(-1, T)[0, T // 2] = 1000  # out of range: skipped
    c.run(pa)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == pa.PA_DEVERR["position"]
    c.slots[T // 2] = -1
    c.check(skip=(T // 2,), tokens=sorted({0, 1, 11, 455, 456, T // 2, T - 2, T - 1, *range(5, T, T // 25)}))


def test_long_prompt_in_place_and_by_parts(pa):
    """The streaming kernel on 14000 tokens, in place, equals calls on 500 at a time (the other one)."""
    c, d = (Case(14000, 8, 2, 128, fused=False, axes=2, seed=4) for _ in range(2))
    c.out = c.q
    c.run(pa)
    whole = (d.q, d.k, d.v, d.pos, d.slots, d.out)
    for i in range(0, 14000, 500):
        d.q, d.k, d.v, d.slots, d.out = (x[i:i + 500] for x in (whole[0], whole[1], whole[2], whole[4], whole[5]))
        d.pos = whole[3][:, i:i + 500].contiguous()
        d.run(pa)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    assert torch.equal(c.q, whole[5]) and torch.equal(c.kc, d.kc) and torch.equal(c.vc, d.vc)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_in_place_equals_out_of_place(pa, dtype):
    c = Case(50, 8, 2, 128, dtype=dtype, axes=2)
    c.run(pa)
    want, kc = c.out.clone(), c.kc.clone()
    c.out = c.q
    c.kc.zero_()
    c.run(pa)
    torch.cuda.synchronize()
    assert torch.equal(c.q, want) and torch.equal(c.kc, kc)


def test_padding_and_slots_out_of_range(pa):
    """Negative slots write nothing, slots past the pool nothing and a flag; queries always."""
    c = Case(12, 4, 2, 128)
    c.slots[3] = -1
    c.slots[7] = -(2 ** 40)
    c.run(pa)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0
    c.check()
    c.kc.zero_(), c.vc.zero_()
    c.slots[5] = c.kc.shape[0] * c.B
    c.slots[6] = 2 ** 40
    c.run(pa)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == pa.PA_DEVERR["slot_range"]
    c.check()


@pytest.mark.parametrize("axes", [1, 3])
def test_positions_out_of_range_skip_their_token(pa, axes):
    c = Case(10, 4, 2, 64, axes=axes)
    flat = c.pos.view(-1, 10)
    flat[-1, 2], flat[0, 8] = 1000, -1
    c.run(pa)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == pa.PA_DEVERR["position"]
    for t in (2, 8):
        c.slots[t] = -1
    c.pos.clamp_(0, 999)
    c.check(skip=(2, 8))


def test_zero_rows_and_no_tokens(pa):
    c = Case(4, 2, 1, 128)
    c.q.zero_(), c.k.zero_()
    c.run(pa)
    torch.cuda.synchronize()
    assert not c.out.any() and not c.kc.any() and pa.read_device_errors() == 0
    e = Case(0, 2, 1, 128)
    e.run(pa)
    torch.cuda.synchronize()
    assert pa.read_device_errors() == 0


@pytest.mark.parametrize("T", [5, 41000])
def test_not_a_number_stays_with_its_pair(pa, T):
    """Without a norm a NaN or infinity spoils its own pair, or (not rotated) only itself."""
    c = Case(T, 2, 1, 128, rot=32, norm=(False, False))
    c.q[2, 1, 3], c.q[2, 1, 60], c.q[2, 0, 100] = float("nan"), float("inf"), float("nan")
    c.run(pa)
    torch.cuda.synchronize()
    bad = torch.nonzero(~torch.isfinite(c.out)).tolist()
    assert bad == [[2, 0, 100], [2, 1, 3], [2, 1, 19], [2, 1, 60]]


def test_angles_of_far_positions_come_from_the_table(pa):
    """Position 2^20 - 1: the table's float64 angles, not fp32 products."""
    c = Case(3, 2, 1, 128, limit=1 << 20)
    c.pos[:] = torch.tensor([(1 << 20) - 1, 0, 777777])
    c.run(pa)
    torch.cuda.synchronize()
    c.check()


def test_captured_and_on_another_stream(pa):
    c = Case(64, 8, 2, 128, fused=True)
    c.run(pa)
    torch.cuda.synchronize()
    want = (c.out.clone(), c.kc.clone(), c.vc.clone())
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    c.out.zero_(), c.kc.zero_(), c.vc.zero_()
    torch.cuda.synchronize()
    c.run(pa, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (c.out, c.kc, c.vc)))
    with torch.cuda.graph(g):
        c.run(pa)
    for _ in range(2):
        c.out.zero_(), c.kc.zero_(), c.vc.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (c.out, c.kc, c.vc)))


def test_the_binding_refuses(pa):
    c = Case(6, 4, 2, 128)
    for name, bad in [("q", c.q.float()), ("k", c.k[:, :1]), ("q", c.q.transpose(0, 1).contiguous().transpose(0, 1)),
                      ("pos", c.pos.long()), ("slots", c.slots.int()), ("out", c.out[:3]), ("cos_sin", c.cos_sin.double()),
                      ("v", c.v.cpu()), ("w", [c.w[0].float(), c.w[1]]), ("sections", (10, 54)), ("vc", c.vc.float())]:
        d = Case(6, 4, 2, 128)
        setattr(d, name, bad)
        with pytest.raises((TypeError, ValueError)):
            d.run(pa)
    d = Case(6, 4, 2, 128)
    d.q = torch.zeros(6 * 4 * 128 + 1, dtype=BF16, device="cuda")[1:].view(6, 4, 128)  # 2-byte aligned
    with pytest.raises(pa.PAError):
        d.run(pa)
    with pytest.raises(pa.PAError):
        c.run(pa, k_scale=0.0)
