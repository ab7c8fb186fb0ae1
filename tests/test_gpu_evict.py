"""Accumulated attention weights and eviction by them, against the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_kv_decode_host_gb300 as pkd
from test_gpu_latent import table

gpu = pytest.mark.gpu
D = 128


def kv_shape(pages, page, hkv, layout):
    return (pages, 2, page, hkv, D) if layout == "NHD" else (pages, 2, hkv, page, D)


def keys_of(kv, layout, pages):
    """[tokens, Hkv, D] in 64 bits of the listed pages."""
    k = kv.view(torch.uint8)[pages, 0].view(kv.dtype) if kv.element_size() == 1 else kv[pages, 0]
    k = k.double() if layout == "NHD" else k.double().transpose(1, 2)
    return k.reshape(-1, k.shape[2], D)


class Step:
    """One decode step's plan, inputs and lse."""

    def __init__(self, hkv, g, lens, page, dtype="bf16", layout="NHD", seed=0, **kw):
        self.hkv, self.g, self.lens, self.page, self.layout = hkv, g, lens, page, layout
        self.t = table(lens, page, seed)
        pages = self.t[3]
        gen = torch.Generator("cuda").manual_seed(seed)
        self.q = torch.randn(len(lens), hkv * g, D, generator=gen, device="cuda").bfloat16()
        x = torch.randn(kv_shape(pages, page, hkv, layout), generator=gen, device="cuda")
        self.ks = 1.0
        if dtype == "e4m3":
            self.ks = 1 / 100
            self.kv = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            self.kv = x.bfloat16()
        self.dec = pkd.BatchDecodeWithPagedKVCache(
            hkv * g, hkv, D, page, max_batch=len(lens), max_num_pages=len(self.t[1]),
            num_pages=pages, kv_dtype=dtype, kv_layout=layout, **kw)
        self.dec.plan(*self.t[:3])
        _, self.lse = self.dec.run(self.q, self.kv, k_scale=self.ks)
        self.per_slot = (pages, hkv, page)
        self.weights = torch.rand(self.per_slot, generator=gen, device="cuda")

    def pages_of(self, i):
        return torch.from_numpy(self.t[1][self.t[0][i]:self.t[0][i + 1]]).long().cuda()

    def expected(self, weights, new):
        """The sums after the step, and the sum over heads of |x| + |lse| bounds."""
        w = weights.double()
        for i, n in enumerate(self.lens):
            pg = self.pages_of(i)
            k = keys_of(self.kv, self.layout, pg)[:n]
            q = self.q[i].double().view(self.hkv, self.g, D)
            x = torch.einsum("hgd,thd->hgt", q, k) * (self.ks / math.sqrt(D))
            add = torch.exp(x - self.lse[i].double().view(self.hkv, self.g, 1)).sum(1)
            was = w[pg].transpose(0, 1).reshape(self.hkv, -1)
            was[:, max(0, n - new[i]):n] = 0
            was[:, :n] += add
            w[pg] = was.view(self.hkv, -1, self.page).transpose(0, 1)
        return w


def near(got, want):
    """exp of an fp32 exponent: scores and lse of magnitude under 24 (in bits of the exponent)
    carry 2^-24 x 24 x ~3 roundings, under 5e-6, and the 128-term product sums as much again;
    the sums of at most 9 such terms stay relative.  2e-5 covers both."""
    assert ((got.double() - want).abs() <= 2e-5 * want.abs() + 1e-12).all()


@gpu
@pytest.mark.parametrize("hkv,g", [(8, 4), (1, 1), (8, 8), (3, 2), (5, 1), (7, 4)])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("dtype,layout", [("bf16", "NHD"), ("bf16", "HND"), ("e4m3", "NHD"),
                                          ("e4m3", "HND")])
def test_accumulate(hkv, g, page, dtype, layout):
    lens = [1, 2, 15, 16, 17, 33, 300, 1200]
    s = Step(hkv, g, lens, page, dtype, layout, seed=hkv * g + page)
    new = [1, 0, 15, 3, 99, -4, 2, 1]
    seen = [n + 10 for n in lens]
    positions = torch.full(s.per_slot, -7, dtype=torch.int32, device="cuda")
    want = s.expected(s.weights, [max(0, x) for x in new])
    want_pos = positions.clone()
    for i, n in enumerate(lens):
        pg, flat = s.pages_of(i), None
        flat = want_pos[pg].transpose(0, 1).reshape(hkv, -1)
        for t in range(max(0, n - max(0, new[i])), n):
            flat[:, t] = 10 + t
        want_pos[pg] = flat.view(hkv, -1, page).transpose(0, 1)
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    once = s.weights.clone()
    s.dec.accumulate_weights(s.q, s.kv, s.lse, s.weights, positions=positions, new_tokens=d(new),
                             seen=d(seen), k_scale=s.ks)
    near(s.weights, want)
    assert torch.equal(positions, want_pos)
    s.dec.accumulate_weights(s.q, s.kv, s.lse, once, new_tokens=d(new), k_scale=s.ks)
    assert torch.equal(once, s.weights) and s.dec.device_error() == 0


@gpu
def test_accumulate_sums_to_the_heads():
    """Every query head hands out one unit of weight in all."""
    s = Step(8, 4, [1, 777, 4000], 16, seed=3)
    w = torch.zeros(s.per_slot, device="cuda")
    s.dec.accumulate_weights(s.q, s.kv, s.lse, w)
    for i in range(3):
        assert (w[s.pages_of(i)].sum((0, 2)) - 4).abs().max() <= 4 * 2e-5


@gpu
def test_accumulate_empty_state_nan_and_stale_slots():
    s = Step(2, 4, [20, 7], 16, seed=4)
    clean = s.expected(s.weights, [0, 0])
    for i, n in enumerate(s.lens):   # behind the end: NaN rows that are not to be read
        pg = int(s.pages_of(i)[-1])
        s.kv[pg, :, (n - 1) % 16 + 1:] = float("nan")
    w = s.weights.clone()
    s.dec.accumulate_weights(s.q, s.kv, s.lse, w)
    near(w, clean)
    s.lse[0] = -float("inf")
    w2 = s.weights.clone()
    s.dec.accumulate_weights(s.q, s.kv, s.lse, w2)
    assert torch.equal(w2[s.pages_of(0)], s.weights[s.pages_of(0)])
    assert torch.equal(w2[s.pages_of(1)], w[s.pages_of(1)])


@gpu
def test_accumulate_refusals():
    s = Step(2, 2, [20, 7], 16, seed=5)
    args = (s.q, s.kv, s.lse)
    with pytest.raises(ValueError):
        s.dec.accumulate_weights(*args, s.weights[:, :1].contiguous())
    with pytest.raises(ValueError):
        s.dec.accumulate_weights(*args, s.weights, positions=s.weights.int())
    with pytest.raises(ValueError):
        s.dec.accumulate_weights(s.q, s.kv, None, s.weights)
    twice = s.t[1].copy()
    twice[1] = twice[0]
    s.dec.plan(s.t[0], twice, s.t[2])
    with pytest.raises(pkd.PkdError, match="BAD_TABLE"):
        s.dec.accumulate_weights(*args, s.weights)
    epoch = s.dec.plan(*s.t[:3])
    with pytest.raises(pkd.PkdError, match="STALE"):
        s.dec.accumulate_weights(*args, s.weights, expect_epoch=epoch - 1)
    s.dec.accumulate_weights(*args, s.weights, expect_epoch=epoch)
    shared = pkd.BatchDecodeWithPagedKVCache(4, 2, D, 16, max_batch=2, max_num_pages=3,
                                             num_pages=s.t[3], shared_prefix=True)
    shared.plan_shared(np.array([0, 2], np.int32), s.t[0][:2], s.t[1], s.t[2][:1])
    with pytest.raises(pkd.PkdError, match="INVALID"):
        shared.accumulate_weights(*args, s.weights)


def evict_reference(kvs, weights, positions, t, lens, seen, budget, page, layout, sinks, recent,
                    per_head):
    """The definition, in place on CPU copies: rows as bytes."""
    for kv, w, p in zip(kvs, weights, positions):
        view = kv if layout == "NHD" else kv.swapaxes(2, 3)
        heads = w.shape[1]
        for i, n in enumerate(lens):
            if n <= budget:
                continue
            at = np.arange(n)
            pg, sl = t[1][t[0][i] + at // page], at % page
            moves = []
            for h in range(heads if per_head else 1):
                x = w[pg, h, sl].astype(np.float64)
                for k in range(1, 1 if per_head else heads):
                    with np.errstate(invalid="ignore"):   # inf - inf: a NaN weight
                        x = x + w[pg, k, sl].astype(np.float64)
                x = x.astype(np.float32).astype(np.float64)
                nan = np.isnan(x)
                x[nan] = -np.inf
                a = p[pg, h, sl]
                safe = (a < sinks) | (a >= seen[i] - recent)
                best = np.lexsort((at, nan, -x, ~safe))[:budget]
                kept = np.zeros(n, bool)
                kept[best] = True
                to, src = np.nonzero(~kept[:budget])[0], budget + np.nonzero(kept[budget:])[0]
                for hh in [h] if per_head else range(heads):
                    moves.append((hh, to, src))
            for hh, to, src in moves:
                view[pg[to], :, sl[to], hh] = view[pg[src], :, sl[src], hh]
                w[pg[to], hh, sl[to]] = w[pg[src], hh, sl[src]]
                p[pg[to], hh, sl[to]] = p[pg[src], hh, sl[src]]


def evict_case(hkv, page, lens, budget, *, layers=1, dtype=torch.bfloat16, layout="NHD", d=D, seed=0,
               kind="mixed"):
    t = table(lens, page, seed)
    pages = t[3]
    r = np.random.default_rng(seed)
    raw = np.int16 if dtype == torch.bfloat16 else np.uint8
    shape = (pages, 2, page, hkv, d) if layout == "NHD" else (pages, 2, hkv, page, d)
    kvs = [r.integers(0, 200, shape).astype(raw) for _ in range(layers)]
    ws, ps = [], []
    for _ in range(layers):
        w = r.exponential(size=(pages, hkv, page)).astype(np.float32)
        if kind == "mixed":
            w = np.where(r.random(w.shape) < 0.4, np.floor(w * 4) / 4, w).astype(np.float32)
        elif kind == "equal":
            w[:] = 0.25
        elif kind == "odd":
            pick = r.integers(0, 7, w.shape)
            for k, v in enumerate([np.nan, np.inf, -np.inf, 0.0, -0.0, -1.0]):
                w[pick == k] = v
        ws.append(w)
        p = np.full((pages, hkv, page), -1, np.int32)
        for i, n in enumerate(lens):
            at = np.arange(n)
            order = np.sort(r.choice(2 * n, n, replace=False))
            half = n // 2
            order[:half] = r.permutation(order[:half])
            p[t[1][t[0][i] + at // page], :, at % page] = order[:, None]
        ps.append(p)
    return t, kvs, ws, ps, [2 * n for n in lens]


def to_gpu(kv, dtype):
    return torch.from_numpy(kv).cuda().view(dtype)


def run_evict(t, kvs, ws, ps, seen, budget, dtype, **kw):
    g = ([to_gpu(x, dtype) for x in kvs], [torch.from_numpy(x).cuda() for x in ws],
         [torch.from_numpy(x).cuda() for x in ps])
    d = [torch.from_numpy(x).cuda() for x in t[:3]]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkd.evict_kv(*g, *d, torch.tensor(seen, dtype=torch.int32, device="cuda"), budget, err=err, **kw)
    raw = torch.int16 if dtype == torch.bfloat16 else torch.uint8
    return [x.view(raw).cpu().numpy() for x in g[0]], [x.cpu().numpy() for x in g[1]], \
        [x.cpu().numpy() for x in g[2]], err.item()


def same(got, want):
    for a, b in zip(got[:3], want):
        for x, y in zip(a, b):
            if x.dtype == np.float32:
                x, y = x.view(np.int32), y.view(np.int32)
            differ = int((x != y).sum())
            assert differ == 0


@gpu
@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("kind", ["mixed", "equal", "odd"])
@pytest.mark.parametrize("hkv,page,layout", [(8, 16, "NHD"), (3, 1, "HND"), (1, 5, "NHD"),
                                             (4, 64, "HND")])
def test_evict(per_head, kind, hkv, page, layout):
    lens = [1, 31, 32, 33, 34, 65, 100, 700, 2500]
    for budget, sinks, recent in ((32, 4, 8), (33, 0, 0), (33, 0, 33), (1, 0, 1), (699, 2, 100)):
        t, kvs, ws, ps, seen = evict_case(hkv, page, lens, budget, layout=layout, seed=budget, kind=kind)
        got = run_evict(t, kvs, ws, ps, seen, budget, torch.bfloat16, max_len=2500, sinks=sinks,
                        recent=recent, per_head=per_head, kv_layout=layout)
        evict_reference(kvs, ws, ps, t, lens, seen, budget, page, layout, sinks, recent, per_head)
        same(got, (kvs, ws, ps))
        assert got[3] == 0


@gpu
@pytest.mark.parametrize("per_head,hkv,lens,budget", [
    (True, 2, [40_000], 12_345), (False, 4, [70_001, 50], 35_000), (True, 1, [262_144], 131_072),
    (True, 8, [1025] * 40, 1024)])
def test_evict_long(per_head, hkv, lens, budget):
    t, kvs, ws, ps, seen = evict_case(hkv, 16, lens, budget, d=16, dtype=torch.uint8, seed=9)
    got = run_evict(t, kvs, ws, ps, seen, budget, torch.uint8, max_len=max(lens), sinks=4,
                    recent=64, per_head=per_head)
    evict_reference(kvs, ws, ps, t, lens, seen, budget, 16, "NHD", 4, 64, per_head)
    same(got, (kvs, ws, ps))


@gpu
def test_evict_layers_and_e4m3():
    lens, budget = [500, 90, 513], 256
    t, kvs, ws, ps, seen = evict_case(8, 16, lens, budget, layers=5, dtype=torch.float8_e4m3fn, seed=2)
    got = run_evict(t, kvs, ws, ps, seen, budget, torch.float8_e4m3fn, max_len=513, sinks=1, recent=9)
    evict_reference(kvs, ws, ps, t, lens, seen, budget, 16, "NHD", 1, 9, True)
    same(got, (kvs, ws, ps))


@gpu
def test_evict_wrong_tables_are_left_alone():
    lens, budget = [100, 80, 60], 40
    t, kvs, ws, ps, seen = evict_case(2, 16, lens, budget, seed=1)
    bad = t[1].copy()
    bad[1] = t[3]                                   # a page outside the pool, in request 0
    last = t[2].copy()
    last[1] = 17                                    # more than a page, in request 1
    for table_, max_len, alone in (((t[0], bad, last), 100, [0, 0, 60]), (t[:3], 79, [0, 0, 60]),
                                   ((t[0], bad, t[2]), 100, [0, 80, 60])):
        want = [[x.copy() for x in y] for y in (kvs, ws, ps)]
        got = run_evict(table_, kvs, ws, ps, seen, budget, torch.bfloat16, max_len=max_len)
        evict_reference(*want, table_, alone, seen, budget, 16, "NHD", 0, 0, True)
        same(got, want)
        assert got[3] == pkd.DEV_ERR_BOUNDS


@gpu
@pytest.mark.parametrize("lens,budget", [([1600, 2000, 1700], 901), ([20_000, 9000], 4000)])
def test_evict_wrong_pages_of_long_requests(lens, budget):
    """As above where the moves are a kernel of their own: nothing of the request with the wrong page."""
    t, kvs, ws, ps, seen = evict_case(2, 16, lens, budget, seed=4)
    bad = t[1].copy()
    bad[t[0][1] - 1] = t[3]                         # request 0's last page
    want = [[x.copy() for x in y] for y in (kvs, ws, ps)]
    got = run_evict((t[0], bad, t[2]), kvs, ws, ps, seen, budget, torch.bfloat16, max_len=max(lens))
    evict_reference(*want, t, [0] + lens[1:], seen, budget, 16, "NHD", 0, 0, True)
    same(got, want)
    assert got[3] == pkd.DEV_ERR_BOUNDS


@gpu
def test_evict_refusals():
    lens = [100]
    t, kvs, ws, ps, seen = evict_case(2, 16, lens, 40, layers=2)
    call = lambda budget=40, **kw: run_evict(t, kvs, ws, ps, seen, budget, torch.bfloat16,
                                             **dict(dict(max_len=100), **kw))
    for kw in (dict(budget=0), dict(sinks=30, recent=11), dict(sinks=-1), dict(max_len=-1)):
        with pytest.raises(pkd.PkdError, match="INVALID"):
            call(**kw)
    with pytest.raises(pkd.PkdError, match="CAPACITY"):
        call(max_len=262_145)
    with pytest.raises(ValueError):
        call(kv_layout="HND")
    kv, w, p = to_gpu(kvs[0], torch.bfloat16), torch.from_numpy(ws[0]).cuda(), torch.from_numpy(ps[0]).cuda()
    d = [torch.from_numpy(x).cuda() for x in t[:3]] + [torch.tensor(seen, dtype=torch.int32, device="cuda")]
    with pytest.raises(pkd.PkdError, match="INVALID"):
        pkd.evict_kv([kv, kv], [w, w.clone()], [p, p.clone()], *d, 40, max_len=100)
    with pytest.raises(ValueError):
        pkd.evict_kv([kv], [w], [p.float()], *d, 40, max_len=100)


@gpu
def test_evict_indices_shorter_than_the_table():
    lens, budget = [100, 80], 40
    t, kvs, ws, ps, seen = evict_case(2, 16, lens, budget, seed=6)
    want = [[x.copy() for x in y] for y in (kvs, ws, ps)]
    got = run_evict((t[0], t[1][:9], t[2]), kvs, ws, ps, seen, budget, torch.bfloat16, max_len=100)
    evict_reference(*want, t, [100, 0], seen, budget, 16, "NHD", 0, 0, True)
    same(got, want)
    assert got[3] == pkd.DEV_ERR_BOUNDS


@gpu
def test_offsets_past_32_bits():
    """A pool of 5 GB whose last pages hold the requests."""
    page, hkv, pages, lens, budget = 16, 8, 80_000, [100, 700], 60
    kv = torch.empty(kv_shape(pages, page, hkv, "NHD"), dtype=torch.bfloat16, device="cuda")
    assert kv.numel() * 2 > 1 << 32
    counts = [7, 44]
    indptr = np.array([0, 7, 51], np.int32)
    ids = (pages - 1 - np.random.default_rng(0).permutation(51)).astype(np.int32)
    last = np.array([4, 12], np.int32)
    at = torch.from_numpy(ids).long().cuda()
    kv[at] = torch.randn(51, 2, page, hkv, D, device="cuda").bfloat16()
    w = torch.zeros(pages, hkv, page, device="cuda")
    p = torch.zeros(pages, hkv, page, dtype=torch.int32, device="cuda")
    dec = pkd.BatchDecodeWithPagedKVCache(hkv, hkv, D, page, max_batch=2, max_num_pages=51, num_pages=pages)
    dec.plan(indptr, ids, last)
    q = torch.randn(2, hkv, D, device="cuda").bfloat16()
    _, lse = dec.run(q, kv)
    d = [torch.from_numpy(x).cuda() for x in (indptr, ids, last)]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dec.accumulate_weights(q, kv, lse, w, positions=p, new_tokens=n, seen=n)
    for i in range(2):
        k = keys_of(kv, "NHD", at[indptr[i]:indptr[i + 1]])[:lens[i]]
        x = torch.einsum("hd,thd->ht", q[i].double(), k) / math.sqrt(D)
        got = w[at[indptr[i]:indptr[i + 1]]].transpose(0, 1).reshape(hkv, -1)[:, :lens[i]]
        near(got, torch.exp(x - lse[i].double()[:, None]))
    raw = kv[at].view(torch.int16).cpu().numpy()
    small = [[raw], [w[at].cpu().numpy()], [p[at].cpu().numpy()]]
    pkd.evict_kv([kv], [w], [p], *d, n, budget, max_len=700, sinks=2, recent=10)
    local = (indptr, np.arange(51, dtype=np.int32), last)
    evict_reference(*small, local, lens, lens, budget, page, "NHD", 2, 10, True)
    same(([kv[at].view(torch.int16).cpu().numpy()], [w[at].cpu().numpy()], [p[at].cpu().numpy()]), small)


@gpu
@pytest.mark.parametrize("n,budget", [(300, 295), (3000, 1500)])
def test_accumulate_and_evict_in_a_graph(n, budget):
    """Captured once, replayed on new inputs, against eager calls; on two streams at once."""
    def state(seed):
        s = Step(2, 4, [n, 40], 16, seed=seed)
        s.pos = torch.full(s.per_slot, -1, dtype=torch.int32, device="cuda")
        at = np.arange(n)
        s.pos[s.t[1][s.t[0][0] + at // 16], :, at % 16] = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
        s.d = [torch.from_numpy(x).cuda() for x in s.t[:3]]
        s.seen = torch.tensor([n, 40], dtype=torch.int32, device="cuda")
        s.new = torch.ones(2, dtype=torch.int32, device="cuda")
        return s

    def step(s, **kw):
        s.dec.accumulate_weights(s.q, s.kv, s.lse, s.weights, positions=s.pos, new_tokens=s.new, seen=s.seen)
        pkd.evict_kv([s.kv], [s.weights], [s.pos], *s.d, s.seen, budget, max_len=n, sinks=2, recent=20)

    a, b, c = state(1), state(1), state(1)
    step(b)                                  # warms up, too
    g = torch.cuda.CUDAGraph()
    keep = [x.clone() for x in (a.kv, a.weights, a.pos)]
    with torch.cuda.graph(g):
        step(a)
    for x, y in zip((a.kv, a.weights, a.pos), keep):
        x.copy_(y)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    g.replay()
    with torch.cuda.stream(other):
        step(c)
    torch.cuda.synchronize()
    for x in (a, c):
        assert torch.equal(x.kv, b.kv) and torch.equal(x.weights, b.weights) and torch.equal(x.pos, b.pos)


def test_evicted_table():
    t = table([100, 16, 40, 33], 16, 3)
    indptr, indices, last, freed = pkd.evicted_table(*t[:3], 16, 33)
    assert indptr.tolist() == [0, 3, 4, 7, 10] and last.tolist() == [1, 16, 1, 1]
    assert indices.tolist() == [*t[1][0:3], *t[1][7:8], *t[1][8:11], *t[1][11:14]]
    assert freed.tolist() == t[1][3:7].tolist()
    twice = t[1].copy()
    twice[0] = twice[5]
    for bad in ((t[0], twice, t[2]), (t[0] + 1, t[1], t[2]), (t[0], t[1][:5], t[2]),
                (t[0], t[1], t[2] + 16)):
        with pytest.raises(pkd.PkdError, match="BAD_TABLE"):
            pkd.evicted_table(*bad, 16, 33)
    with pytest.raises(ValueError):
        pkd.evicted_table(*t[:3], 16, 0)


@gpu
def test_serving_loop_with_a_budget():
    """append -> plan -> run -> accumulate -> evict over many steps: the cache stays at its
    budget, and each step's result is the attention over the tokens that stayed."""
    page, hkv, g, budget, sinks, recent, B, steps = 16, 2, 4, 48, 2, 8, 3, 80
    per = -(-(budget + 1) // page)
    pool = B * per
    ids = np.random.default_rng(0).permutation(pool).astype(np.int32).reshape(B, per)
    kv = torch.zeros(kv_shape(pool, page, hkv, "NHD"), dtype=torch.bfloat16, device="cuda")
    w = torch.rand(pool, hkv, page, device="cuda")
    p = torch.zeros(pool, hkv, page, dtype=torch.int32, device="cuda")
    dec = pkd.BatchDecodeWithPagedKVCache(hkv * g, hkv, D, page, max_batch=B, max_num_pages=B * per,
                                          num_pages=pool)
    lens = [0] * B
    # by (request, head): position -> (k, v, weight sum), the model of the cache
    model = [[{} for _ in range(hkv)] for _ in range(B)]
    gen = torch.Generator("cuda").manual_seed(1)
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for step in range(steps):
        lens = [n + 1 for n in lens]
        counts = [-(-n // page) for n in lens]
        indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        indices = np.concatenate([ids[i, :c] for i, c in enumerate(counts)])
        last = np.array([n - page * (c - 1) for n, c in zip(lens, counts)], np.int32)
        dt = [torch.from_numpy(x).cuda() for x in (indptr, indices, last)]
        k = torch.randn(B, hkv, D, generator=gen, device="cuda").bfloat16()
        v = torch.randn(B, hkv, D, generator=gen, device="cuda").bfloat16()
        q = torch.randn(B, hkv * g, D, generator=gen, device="cuda").bfloat16()
        pkd.append_kv(k, v, d(list(range(B))), d([n - 1 for n in lens]), *dt, kv)
        dec.plan(indptr, indices, last)
        out, lse = dec.run(q, kv)
        dec.accumulate_weights(q, kv, lse, w, positions=p, new_tokens=d([1] * B), seen=d([step + 1] * B))
        pkd.evict_kv([kv], [w], [p], *dt, d([step + 1] * B), budget, max_len=max(lens), sinks=sinks,
                     recent=recent)
        wc, pc = w.cpu(), p.cpu()
        for i in range(B):
            for h in range(hkv):
                m = model[i][h]
                m[step] = [k[i, h].double().cpu(), v[i, h].double().cpu(), 0.0]
                pos = sorted(m)
                K = torch.stack([m[x][0] for x in pos])
                V = torch.stack([m[x][1] for x in pos])
                x = q[i, h * g:(h + 1) * g].double().cpu() @ K.T / math.sqrt(D)
                a = torch.softmax(x, 1)
                ref = a @ V
                # P and the result are rounded to bf16: 2^-8 of max |v| and of |out|
                top = V.abs().max() + ref.abs().max()
                assert (out[i, h * g:(h + 1) * g].double().cpu() - ref).abs().max() <= 1.01 * 2 ** -8 * top
                for j, s in enumerate(pos):
                    m[s][2] += float(a[:, j].sum())
                # the kernel's own choice, held to the model's sums
                n = lens[i]
                at = np.arange(min(n, budget))
                stay = set(pc[ids[i][at // page], h, at % page].tolist())
                assert len(stay) == min(n, budget) and stay <= set(pos)
                gone = set(pos) - stay
                for s in gone:
                    assert sinks <= s < step + 1 - recent
                    free = [m[x][2] for x in stay if sinks <= x < step + 1 - recent]
                    assert m[s][2] <= min(free) * (1 + 1e-3)
                    del m[s]
                got = {int(a_): float(b_) for a_, b_ in zip(pc[ids[i][at // page], h, at % page],
                                                            wc[ids[i][at // page], h, at % page])}
                for s in stay:
                    assert abs(got[s] - m[s][2]) <= 1e-3 * m[s][2] + 1e-6
        lens = [min(n, budget) for n in lens]
    assert dec.device_error() == 0


@gpu
def test_evict_workspace_belongs_to_the_calls_stream(monkeypatch):
    """The bitmaps' memory comes from the stream that writes them: a block of the current
    stream's may still be in use there."""
    t, kvs, ws, ps, seen = evict_case(2, 16, [3000], 1500)
    side, taken, empty = torch.cuda.Stream(), [], torch.empty

    def spy(*a, **kw):
        taken.append(torch.cuda.current_stream() == side)
        return empty(*a, **kw)

    gpu_state = ([to_gpu(x, torch.bfloat16) for x in kvs], [torch.from_numpy(x).cuda() for x in ws],
                 [torch.from_numpy(x).cuda() for x in ps])
    d = [torch.from_numpy(x).cuda() for x in t[:3]] + [torch.tensor(seen, dtype=torch.int32, device="cuda")]
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", spy)
    pkd.evict_kv(*gpu_state, *d, 1500, max_len=3000, stream=side)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert taken == [True]
    evict_reference(kvs, ws, ps, t, [3000], seen, 1500, 16, "NHD", 0, 0, True)
    same(([x.view(torch.int16).cpu().numpy() for x in gpu_state[0]],
          *[[x.cpu().numpy() for x in y] for y in gpu_state[1:]]), (kvs, ws, ps))


def late(target, right, cycles=400_000):
    """A kernel that writes `right` over `target`, a while after the calls that follow were launched."""
    wrong = torch.full_like(target, float("nan")) if target.is_floating_point() else torch.zeros_like(target)
    target.copy_(wrong)
    torch.cuda.synchronize()
    torch.cuda._sleep(cycles)
    torch.mul(right, 1, out=target)


@gpu
def test_calls_wait_for_the_kernel_before():
    """Weight sums, evictions and latent appends are launched early: what they read and write is the
    kernel's before them until it has ended."""
    n, budget = 3000, 1500
    s = Step(2, 4, [n, 40], 16, seed=11)
    lse, start = s.lse.clone(), s.weights.clone()
    want = s.expected(start, [0, 0])
    late(s.lse, lse)
    near(s.dec.accumulate_weights(s.q, s.kv, s.lse, s.weights), want)
    s.weights.copy_(start)
    late(s.weights, start)
    near(s.dec.accumulate_weights(s.q, s.kv, s.lse, s.weights), want)

    t, kvs, ws, ps, seen = evict_case(2, 16, [n], budget, seed=5)
    for few in (n - 3, budget):                    # one kernel, and two
        g = [to_gpu(kvs[0], torch.bfloat16)], [torch.from_numpy(ws[0]).cuda()], [torch.from_numpy(ps[0]).cuda()]
        d = [torch.from_numpy(x).cuda() for x in t[:3]] + [torch.tensor(seen, dtype=torch.int32, device="cuda")]
        for target in (g[1][0], g[2][0], d[0]):
            late(target, target.clone())
            pkd.evict_kv(*g, *d, few, max_len=n)
            ref = [[x.copy() for x in y] for y in (kvs, ws, ps)]
            evict_reference(*ref, t, [n], seen, few, 16, "NHD", 0, 0, True)
            same(([x.view(torch.int16).cpu().numpy() for x in g[0]],
                  *[[x.cpu().numpy() for x in y] for y in g[1:]]), ref)
            for x, y in zip((g[0][0].view(torch.int16), g[1][0], g[2][0]), (kvs[0], ws[0], ps[0])):
                x.copy_(torch.from_numpy(y))

    cache = torch.zeros(t[3], 16, 576, device="cuda").bfloat16()
    new = torch.randn(1, 576, device="cuda").bfloat16()
    row, at = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), n - 1, dtype=torch.int32, device="cuda")
    slot = int(t[1][(n - 1) // 16]), (n - 1) % 16
    for target in (new, at, cache):
        late(target, target.clone())
        pkd.append_latent(new[:, :512], new[:, 512:], row, at, *d[:3], cache)
        assert torch.equal(cache[slot], new[0]) and cache.count_nonzero() == new.count_nonzero()
        cache.zero_()
