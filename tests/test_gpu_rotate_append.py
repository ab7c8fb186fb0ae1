"""Norms, rotation and append of new tokens in one call, against the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_kv_decode_host_gb300 as pkd

pytestmark = pytest.mark.gpu


def table(lens, page, seed=0, spare=3):
    counts = [-(-n // page) for n in lens]
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    pool = int(indptr[-1]) + spare
    where = np.random.default_rng(seed).permutation(pool)[: indptr[-1]].astype(np.int32)
    last = np.array([n - page * (c - 1) for n, c in zip(lens, counts)], np.int32)
    return indptr, where, last, pool


def freqs(rotary, theta=10_000.0):
    return [theta ** (-2.0 * i / rotary) for i in range(rotary // 2)]


def rotated(x, at, freq, axes, pairs, scale):
    """x [n, H, D] in 64 bits; at [n, axes]."""
    half = len(freq)
    angle = at.double()[:, axes] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    cos, sin = scale * torch.cos(angle)[:, None], scale * torch.sin(angle)[:, None]
    lo = torch.arange(half) * (2 if pairs else 1)
    hi = lo + (1 if pairs else half)
    y = x.clone()
    y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
    y[..., hi] = x[..., hi] * cos + x[..., lo] * sin
    return y


class Case:
    def __init__(self, hq=8, hkv=2, D=128, page=16, layout="NHD", kv="bf16", old=(21, 0, 7), new=(3, 16, 1), rotary=128,
                 pairs=False, axes=1, norms=None, scale=1.0, seed=0, far=0, contiguous=False):
        self.__dict__.update(hq=hq, hkv=hkv, D=D, page=page, layout=layout, kvd=kv, pairs=pairs)
        lens = [a + b for a, b in zip(old, new)]
        self.indptr, self.indices, self.last, self.pool = table(lens, page, seed)
        self.n = n = sum(new)
        g = torch.Generator("cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
        shape = (self.pool, 2, page, hkv, D) if layout == "NHD" else (self.pool, 2, hkv, page, D)
        self.cache = rnd(*shape).to(torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16)
        self.k_scale, self.v_scale = (0.02, 0.013) if kv == "e4m3" else (1.0, 1.0)
        both = rnd(n, hq + 2 * hkv, D).bfloat16()
        self.q, self.k, self.v = both[:, :hq], both[:, hq:hq + hkv], both[:, hq + hkv:]
        if contiguous:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.rows = torch.cat([torch.full((c,), b) for b, c in enumerate(new)]).int().cuda()
        self.places = torch.cat([torch.arange(o, o + c) for o, c in zip(old, new)]).int().cuda()
        self.at = torch.randint(-far, far + 1, (n, axes), generator=g, device="cuda", dtype=torch.int32) if far else \
            torch.stack([self.places] * axes, 1).contiguous() * 3 + torch.arange(axes, device="cuda", dtype=torch.int32)
        self.freq, self.scale = freqs(rotary), scale
        self.axes = [i % axes for i in range(rotary // 2)]
        self.rope = pkd.RotaryPositions(self.freq, interleaved=pairs, axes=self.axes, scale=scale) if rotary else None
        w = lambda: None if norms is None else (1 + 0.3 * rnd(D)).to(norms)
        self.q_norm, self.k_norm = w(), w()
        self.tables = [torch.from_numpy(x).cuda() for x in (self.indptr, self.indices, self.last)]

    def run(self, **kw):
        return pkd.rotate_append_kv(self.q, self.k, self.v, self.rope, self.rows, self.places, *self.tables, self.cache,
                                    rope_positions=self.at, q_norm=self.q_norm, k_norm=self.k_norm, eps=1e-5,
                                    k_scale=self.k_scale, v_scale=self.v_scale, kv_layout=self.layout, **kw)

    def formula(self, x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w.double()
        return x if self.rope is None else rotated(x, self.at, self.freq, self.axes, self.pairs, self.scale), x.abs().max()

    def check(self, **kw):
        before = self.cache.clone()
        q_in = self.q.clone()
        expect_q, top_q = self.formula(q_in, self.q_norm)
        expect_k, top_k = self.formula(self.k, self.k_norm)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out, cache = self.run(err=err, **kw)
        assert err.item() == 0 and cache is self.cache
        # fp32 throughout (sines off by under 2^-20, norms and products by under 2^-20 of a value), then
        # one rounding: bf16 by 2^-8 of the result, e4m3 by 2^-4 of it or half its smallest step, 2^-10
        slack = abs(self.scale) * 2.0 ** -18
        assert ((q_out.double() - expect_q).abs() <= 2.0 ** -8 * expect_q.abs() + slack * top_q).all()
        rows = lambda c: c if self.layout == "NHD" else c.transpose(2, 3)
        host = before.float().double()
        got = self.cache.float().double()
        page = torch.tensor([self.indices[self.indptr[b] + t // self.page]
                             for b, t in zip(self.rows.tolist(), self.places.tolist())]).cuda()
        place = self.places.long() % self.page
        new_k, new_v = rows(got)[page, 0, place], rows(got)[page, 1, place]
        if self.kvd == "bf16":
            assert ((new_k - expect_k).abs() <= 2.0 ** -8 * expect_k.abs() + slack * top_k).all()
            assert torch.equal(new_v, self.v.double())
        else:
            for new, x, c, top in ((new_k, expect_k, self.k_scale, top_k), (new_v, self.v.double(), self.v_scale, 0.0)):
                x = (x / c).clamp(-448, 448)
                assert ((new - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 + (slack * top) / c + 2.0 ** -20 * x.abs()).all()
        rows(host)[page, 0, place], rows(host)[page, 1, place] = new_k, new_v
        assert torch.equal(host, got)   # and nothing else was written
        return q_out


@pytest.mark.parametrize("D,rotary", [(64, 64), (64, 32), (128, 128), (128, 96), (128, 16), (256, 256), (256, 64), (128, 0)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norms", [None, torch.bfloat16, torch.float32])
def test_forms(D, rotary, pairs, norms):
    Case(D=D, rotary=rotary, pairs=pairs, norms=norms, seed=rotary).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (6, 3), (8, 8), (32, 8), (64, 8), (5, 2)])
@pytest.mark.parametrize("layout,page,kv", [("NHD", 1, "bf16"), ("HND", 5, "e4m3"), ("NHD", 16, "e4m3"), ("HND", 64, "bf16")])
def test_heads_and_caches(hq, hkv, layout, page, kv):
    Case(hq=hq, hkv=hkv, layout=layout, page=page, kv=kv, norms=torch.bfloat16, seed=hq).check()


@pytest.mark.parametrize("new", [(1,), (1, 1, 1), (700, 3), (4001,)])
def test_token_counts(new):
    Case(old=(5,) * len(new), new=new, hq=32, hkv=8, seed=1).check()


@pytest.mark.parametrize("axes", [2, 3, 4])
def test_several_axes(axes):
    Case(axes=axes, seed=axes, norms=torch.bfloat16).check()


@pytest.mark.parametrize("far", [200_000, 2 ** 31 - 1])
@pytest.mark.parametrize("pairs", [False, True])
def test_far_positions(far, pairs):
    """Angles of up to 2^31 radians, of either sign (the oracle's own angles, in doubles, are then off
    by up to 2^31 * 2^-53 * 2 = 2^-21)."""
    Case(far=far, axes=2, pairs=pairs, seed=2, scale=1.25).check()


def test_in_place_and_given_outputs():
    c = Case(norms=torch.bfloat16)
    want = c.run()[0].clone()
    out = torch.empty(c.n, c.D, c.hq, dtype=torch.bfloat16, device="cuda").transpose(1, 2).contiguous()
    assert c.run(q_out=out)[0] is out and torch.equal(out, want)
    wide = torch.zeros(c.n, c.hq + 3, c.D, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(c.run(q_out=wide[:, 1:1 + c.hq])[0], want)
    assert (wide[:, 0] == 0).all() and (wide[:, 1 + c.hq:] == 0).all()
    k, v = c.k.clone(), c.v.clone()
    assert torch.equal(c.run(q_out=c.q)[0], want)     # in place, in the projection's output
    assert torch.equal(c.k, k) and torch.equal(c.v, v)


def test_without_queries_and_without_tokens():
    c = Case()
    c.q = None
    cache = c.cache.clone()
    q_out, _ = c.run()
    assert q_out is None
    d = Case()
    assert not torch.equal(c.cache, cache) and torch.equal(c.cache, d.run()[1])
    e = Case()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    q_out, _ = pkd.rotate_append_kv(e.q[:0], e.k[:0], e.v[:0], e.rope, none, none, *e.tables, e.cache)
    assert q_out.shape == (0, 8, 128) and torch.equal(e.cache, cache)


def test_positions_by_default_are_the_places():
    c, d = Case(), Case()
    c.at = None
    d.at = d.places
    assert torch.equal(c.run()[0], d.run()[0]) and torch.equal(c.cache, d.cache)


def test_tokens_without_a_slot():
    c, d = Case(norms=torch.bfloat16), Case(norms=torch.bfloat16)
    keep = c.run()[0]
    d.rows[1], d.rows[4] = -1, 3
    d.places[7], d.places[19] = -1, 8     # (the last request has 8 tokens)
    d.tables[1][int(d.indptr[1])] = d.pool  # a page outside the pool
    before = d.cache.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(d.run(err=err)[0], keep)
    assert err.item() == 2
    page = int(d.indices[int(d.indptr[0]) + 1])   # request 0: places 21, 22, 23
    assert torch.equal(d.cache[page, :, 6], before[page, :, 6])
    assert torch.equal(d.cache[page, :, 5], c.cache[page, :, 5])
    first = int(d.indices[int(d.indptr[1])])
    assert torch.equal(d.cache[first], before[first])
    assert torch.equal(d.cache[int(d.indices[-1])], before[int(d.indices[-1])])
    d.tables[1] = d.tables[1][:-1]                # an index list that is too short
    err.zero_()
    d.run(err=err)
    assert err.item() == 2 and torch.equal(d.cache[int(d.indices[-1])], before[int(d.indices[-1])])


def test_values_that_are_not_finite():
    c = Case(kv="e4m3", rotary=64)
    c.v[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e30]).bfloat16()
    c.q[0, 0, 100] = float("inf")     # behind the rotated dims: passes
    c.k[1, 1, 64:66] = torch.tensor([1e30, -1e30]).bfloat16()
    q_out, cache = c.run()
    page, place = int(c.indices[int(c.indptr[0]) + 21 // 16]), 21 % 16
    got = cache.float()[page, 1, place, 0, :4]
    assert got[0] == 448 and got[1] == -448 and torch.isnan(got[2]) and got[3] == 448
    assert cache.float()[page, 0, place + 1, 1, 64] == 448 and cache.float()[page, 0, place + 1, 1, 65] == -448
    assert q_out[0, 0, 100] == float("inf") and torch.isfinite(q_out[0, 0, 101:].float()).all()
    d = Case()
    d.v[2, 0, :2] = torch.tensor([float("nan"), float("inf")]).bfloat16()
    d.run()
    place = 23 % 16
    assert torch.equal(d.cache[page, 1, place].view(torch.int16), d.v[2].contiguous().view(torch.int16))


def test_streams_and_graphs():
    c, d = Case(norms=torch.bfloat16), Case(norms=torch.bfloat16)
    want = c.run()[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = d.run(stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(c.cache, d.cache)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        d.run(q_out=out)
    d.cache.zero_(), d.q.mul_(2.0), d.v.mul_(2.0)
    graph.replay()
    c.q.mul_(2.0), c.v.mul_(2.0)
    c.cache.zero_()
    assert torch.equal(out, c.run()[0]) and torch.equal(c.cache, d.cache)


def test_queued_behind_kernels_that_release_it_early():
    """The call reads what the kernel before it writes."""
    c = Case(old=(0,), new=(2000,), hq=32, hkv=8)
    src = c.q.clone()
    want = c.run()[0]
    for _ in range(5):
        c.q.zero_()
        c.q.copy_(src)
        assert torch.equal(c.run()[0], want)


def test_refusals():
    c = Case()
    bad = lambda **kw: pytest.raises((ValueError, TypeError, pkd.PkdError))
    q, k, v = c.q, c.k, c.v
    for args in ((q.float(), k, v), (q[:-1], k, v), (q, k[:, :1], v), (q, k, v[..., :64]), (q.cpu(), k, v),
                 (q[..., ::2], k, v)):
        with bad():
            pkd.rotate_append_kv(*args, c.rope, c.rows, c.places, *c.tables, c.cache)
    odd = torch.zeros(c.n, 8 * 128 + 4, dtype=torch.bfloat16, device="cuda")[:, :1024].view(c.n, 8, 128)
    go = lambda **kw: pkd.rotate_append_kv(kw.pop("q", q), k, v, kw.pop("rope", c.rope), c.rows, c.places, *c.tables,
                                           kw.pop("cache", c.cache), **kw)
    for kw in (dict(q=odd), dict(rope_positions=c.at.long()), dict(rope_positions=c.at[:-1]),
               dict(q_norm=torch.ones(64, device="cuda")), dict(q_norm=torch.ones(128, device="cuda").half()),
               dict(q_norm=torch.ones(128, device="cuda"), k_norm=torch.ones(128, device="cuda").bfloat16()),
               dict(q_out=torch.zeros(1, device="cuda")), dict(k_scale=2.0), dict(v_scale=0.5), dict(eps=-1.0),
               dict(eps=float("nan")), dict(cache=c.cache.float()), dict(cache=c.cache[:, :1]), dict(kv_layout="x"),
               dict(q_out=q.contiguous()[:, :, :64]), dict(err=torch.zeros(1, device="cuda")),
               dict(rope=pkd.RotaryPositions(freqs(256))),
               dict(rope=pkd.RotaryPositions(freqs(128), axes=[1] * 64))):
        with bad():
            go(**kw)
    e = Case(kv="e4m3")
    for s in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        e.k_scale = s
        with bad():
            e.run()
    for args in (([],), ([1.0] * 3,), ([float("nan")] * 8,), ([1.0] * 136,)):
        with pytest.raises(ValueError):
            pkd.RotaryPositions(*args)
    for kw in (dict(axes=[0] * 7), dict(axes=[4] * 8), dict(axes=[-1] * 8), dict(scale=float("inf"))):
        with pytest.raises(ValueError):
            pkd.RotaryPositions([1.0] * 8, **kw)


@pytest.mark.parametrize("scale", [0.03, 1.0 / 90.0, 0.7, 3.0, 1e-6, 2.0 ** 20, 3e-39, 3.3e38])
@pytest.mark.parametrize("norms", [None, torch.bfloat16])
def test_e4m3_codes_of_every_value(scale, norms):
    """Every bf16 value as a value, and as a key that is not turned: the code next to the fp32
    quotient."""
    c = Case(hq=1, hkv=8, kv="e4m3", old=(5,), new=(64,), rotary=0, norms=norms, layout="HND")
    values = torch.arange(-2 ** 15, 2 ** 15, device="cuda").to(torch.int16).view(torch.bfloat16).view(64, 8, 128)
    c.v = values
    if norms is None:
        c.k, c.k_scale = values.flip(0).contiguous(), scale
    c.v_scale = scale
    _, cache = c.run()
    page = torch.from_numpy(c.indices).cuda().long()[c.places.long() // c.page]
    got = cache.view(torch.uint8).transpose(2, 3)[page, :, c.places.long() % c.page]

    def code(x):   # (numpy's: torch on the GPU multiplies by 1 / scale instead)
        with np.errstate(all="ignore"):
            y = np.clip(x.float().cpu().numpy() / np.float32(scale), np.float32(-448), np.float32(448))
        return torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).cuda()

    for at, x in ((1, values),) + (((0, c.k),) if norms is None else ()):
        number = ~x.isnan()
        assert torch.equal(got[:, at][number], code(x)[number]) and ((got[:, at][~number] & 0x7f) == 0x7f).all()
