"""Accepted drafts moved into place in every layer, and a whole step with drafts."""
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


class Case:
    def __init__(self, lens=(37, 16, 5), drafted=(9, 16, 5), paths=((1, 4, 7), (0, 1, 2, 3), ()), page=16, hkv=2, D=128,
                 layout="NHD", kv="bf16", layers=3, width=None, seed=0):
        self.__dict__.update(lens=lens, drafted=drafted, paths=paths, page=page, layout=layout)
        self.indptr, self.indices, self.last, self.pool = table(lens, page, seed)
        g = torch.Generator("cuda").manual_seed(seed)
        shape = (self.pool, 2, page, hkv, D) if layout == "NHD" else (self.pool, 2, hkv, page, D)
        dt = torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16
        self.kvs = [torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(layers)]
        width = max([len(p) for p in paths] + [1]) if width is None else width
        self.accepted = torch.tensor([list(p) + [-1] * (width - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        self.d_drafted = torch.tensor(drafted, dtype=torch.int32, device="cuda")
        self.tables = [torch.from_numpy(x).cuda() for x in (self.indptr, self.indices, self.last)]

    def run(self, **kw):
        return pkd.accept_kv(self.kvs, self.accepted, self.d_drafted, *self.tables, kv_layout=self.layout, **kw)

    def expected(self, skip=()):
        got = []
        for kv in self.kvs:
            new = kv.view(torch.uint8).cpu().clone()
            rows = new if self.layout == "NHD" else new.transpose(2, 3)
            old = rows.clone()
            for b, path in enumerate(self.paths):
                at = lambda t: (int(self.indices[self.indptr[b] + t // self.page]), t % self.page)
                ctx = self.lens[b] - self.drafted[b]
                for i, a in enumerate(path if b not in skip else ()):
                    (pt, st), (pf, sf) = at(ctx + i), at(ctx + a)
                    rows[pt, :, st] = old[pf, :, sf]
            got.append(new)
        return got

    def check(self, skip=()):
        want = self.expected(skip)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert self.run(err=err) is self.kvs
        assert err.item() == (2 if skip else 0)
        for kv, w in zip(self.kvs, want):
            assert torch.equal(kv.view(torch.uint8).cpu(), w)


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("page,kv,hkv,D", [(16, "bf16", 2, 128), (1, "bf16", 8, 128), (5, "e4m3", 3, 128),
                                           (64, "e4m3", 1, 16), (7, "bf16", 8, 256), (16, "bf16", 1, 8)])
def test_caches(layout, page, kv, hkv, D):
    Case(page=page, kv=kv, hkv=hkv, D=D, layout=layout).check()


@pytest.mark.parametrize("layers", [1, 2, 128])
def test_layers(layers):
    Case(layers=layers, hkv=1).check()


@pytest.mark.parametrize("n,path", [(1, (0,)), (1, ()), (40, tuple(range(40))), (40, tuple(range(1, 40))),
                                    (40, (39,)), (300, tuple(range(0, 300, 2))), (300, tuple(range(3, 300))),
                                    (1024, tuple(range(1024)))])
def test_paths(n, path):
    Case(lens=(n + 21,), drafted=(n,), paths=(path,)).check()
    Case(lens=(n,), drafted=(n,), paths=(path,), width=1024).check()


def test_rows_that_are_wrong_are_left_as_they_are():
    paths = ((1, 4, 7), (0, 2, 2), (3, 2), (0, 9), (2, 5), (1, 0, 3, 2, 5, 4, 7, 6), (1, 2))
    c = Case(lens=(37, 30, 20, 33, 40, 8, 12), drafted=(9, 9, 9, 9, 9, 9, 3), paths=paths)
    c.drafted = (9, 9, 9, 9, 9, 8, 3)
    c.d_drafted[5] = 2       # more accepted than drafted, not increasing
    c.check(skip=(1, 2, 3, 5))
    d = Case(lens=(37, 30, 20), drafted=(9, 9, 9), paths=((1, 4), (1, 4), (1, 4)))
    d.d_drafted[0], d.d_drafted[1] = 38, -1
    d.check(skip=(0, 1))
    e = Case(lens=(37, 30), drafted=(9, 9), paths=((1, 4), (1, 4)))
    e.tables[1][int(e.indptr[2]) - 1] = e.pool     # the page that request 1's drafts lie in
    e.check(skip=(1,))
    f = Case(lens=(37, 30), drafted=(9, 9), paths=((1, 4), (1, 4)))
    f.tables[1] = f.tables[1][:-1]
    f.check(skip=(1,))
    g = Case(lens=(37, 30), drafted=(9, 9), paths=((1, 4), (1, 4)))
    g.tables[2][0] = 17
    g.check(skip=(0,))


def test_entries_behind_the_first_negative_one_do_not_count():
    c = Case(lens=(37,), drafted=(9,), paths=((1, 4, -1, 6, 100),))
    c.paths = ((1, 4),)
    c.check()


def test_streams_and_graphs():
    c, d = Case(), Case()
    c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    d.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(c.kvs, d.kvs))
    e = Case()
    keep = [kv.clone() for kv in e.kvs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.run()
    for kv, k in zip(e.kvs, keep):
        kv.copy_(k)
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(c.kvs, e.kvs))


def test_refusals():
    c = Case()
    for kw in (dict(kvs=[]), dict(kvs=c.kvs * 50), dict(kvs=[c.kvs[0], c.kvs[0]]), dict(kvs=[c.kvs[0], c.kvs[1][:-1]]),
               dict(kvs=[c.kvs[0].float()]), dict(accepted=c.accepted.long()), dict(accepted=c.accepted[:2]),
               dict(accepted=torch.zeros(3, 1025, dtype=torch.int32, device="cuda")), dict(d_drafted=c.d_drafted[:2]),
               dict(layout="x")):
        d = Case()
        d.__dict__.update(kw)
        with pytest.raises((ValueError, TypeError, pkd.PkdError)):
            d.run()


def attention(q, k, v, scale):
    """[H, D] over [t, Hkv, D], in 64 bits."""
    hkv = k.shape[1]
    x = torch.einsum("hgd,thd->hgt", q.view(hkv, -1, q.shape[-1]), k) * scale
    return torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v).reshape(q.shape)


@pytest.mark.parametrize("path", ["tensors", "addresses", "ctypes"])
def test_three_steps_with_drafts(path, monkeypatch):
    """Rotate and append trees of drafts, attend, accept a path, and go on: every step's results and
    the cache are those of the accepted tokens alone."""
    from paged_kv_decode_host_gb300 import drafts as calls
    if path != "tensors":
        monkeypatch.setattr(calls, "_step", lambda: None)
    else:
        assert calls._step() is not None
    if path == "ctypes":
        monkeypatch.setattr(calls, "_fast", lambda: None)
    hq, hkv, D, page, batch, layers = 8, 2, 128, 16, 3, 2
    g = torch.Generator("cuda").manual_seed(7)
    r = np.random.default_rng(7)
    rope = pkd.RotaryPositions([10_000.0 ** (-i / 64) for i in range(64)])
    freq = torch.tensor([10_000.0 ** (-i / 64) for i in range(64)], dtype=torch.float64, device="cuda")
    pool, pages = 60, 20
    ids = [list(map(int, x)) for x in r.permutation(pool).reshape(batch, pages)]
    kvs = [torch.full((pool, 2, page, hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    dec = pkd.BatchTreeDecodeWithPagedKVCache(hq, hkv, D, page, max_tokens=200, max_num_pages=batch * pages, num_pages=pool)
    kept = [[[] for _ in range(batch)] for _ in range(layers)]   # accepted tokens' (k, v), rotated, in 64 bits
    w = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16()

    def turn(x, at):
        x = x.double() / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6) * w.double()
        a = at.double()[:, None, None] * freq
        lo, hi = x[..., :64], x[..., 64:]
        return torch.cat([lo * torch.cos(a) - hi * torch.sin(a), hi * torch.cos(a) + lo * torch.sin(a)], -1)

    for step, drafts in enumerate(((40, 17, 1), (9, 12, 6), (1, 30, 8))):
        ctx = [len(kept[0][b]) for b in range(batch)]
        lens = [a + n for a, n in zip(ctx, drafts)]
        counts = [-(-n // page) for n in lens]
        indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        indices = np.concatenate([ids[b][:counts[b]] for b in range(batch)]).astype(np.int32)
        last = np.array([n - page * (c - 1) for n, c in zip(lens, counts)], np.int32)
        tables = [torch.from_numpy(x).cuda() for x in (indptr, indices, last)]
        q_indptr = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        parents = np.concatenate([[j - 1 if step == 0 else int(r.integers(-1, j)) for j in range(n)]
                                  for n in drafts]).astype(np.int32)   # first the prompts: chains
        mask, depths = pkd.tree_mask(q_indptr, parents)
        n = int(q_indptr[-1])
        rows = torch.from_numpy(np.repeat(np.arange(batch), drafts)).int().cuda()
        places = torch.from_numpy(np.concatenate([np.arange(a, b) for a, b in zip(ctx, lens)])).int().cuda()
        at = torch.from_numpy(np.repeat(ctx, drafts) + depths).int().cuda()
        d_mask, d_depths = torch.from_numpy(mask).cuda(), torch.from_numpy(depths).cuda()
        dec.plan(q_indptr, indptr, indices, last)
        turned = []
        for l in range(layers):
            both = torch.randn(n, hq + 2 * hkv, D, generator=g, device="cuda").bfloat16()
            q, k, v = both[:, :hq], both[:, hq:hq + hkv], both[:, hq + hkv:]
            q_out, _ = pkd.rotate_append_kv(q, k, v, rope, rows, places, *tables, kvs[l], rope_positions=at,
                                            q_norm=w, k_norm=w)
            out, _ = dec.run(q_out, kvs[l], mask=d_mask, depths=d_depths)
            eq, ek, ev = turn(q, at), turn(k, at), v.double()
            turned.append((ek, ev))
            for b in range(batch):
                for i in range(drafts[b]):
                    row = int(q_indptr[b]) + i
                    own, j = [], i
                    while j >= 0:
                        own.append(j)
                        j = int(parents[q_indptr[b] + j])
                    own = [int(q_indptr[b]) + j for j in sorted(own)]
                    ks = torch.stack([x for x, _ in kept[l][b]] + [ek[j] for j in own])
                    vs = torch.stack([x for _, x in kept[l][b]] + [ev[j] for j in own])
                    ref = attention(eq[row], ks, vs, D ** -0.5)
                    # q and k rounded to bf16 (2^-8 each): a score moves by at most 2 * 2^-8 * 128 * 2^0
                    # of |q||k| scale in the worst case; of random signs, a few per cent of a weight
                    assert (out[row].double() - ref).abs().max() <= 0.06
        paths = []
        for b in range(batch):
            i = int(r.integers(0, drafts[b])) if step else drafts[b] - 1
            path = []
            while i >= 0:
                path.append(i)
                i = int(parents[q_indptr[b] + i])
            paths.append(sorted(path))
        wide = max(map(len, paths))
        accepted = torch.tensor([p + [-1] * (wide - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        drafted = torch.tensor(drafts, dtype=torch.int32, device="cuda")
        pkd.accept_kv(kvs, accepted, drafted, *tables)
        for l in range(layers):
            for b, path in enumerate(paths):
                kept[l][b] += [(turned[l][0][int(q_indptr[b]) + i], turned[l][1][int(q_indptr[b]) + i]) for i in path]
        table2 = pkd.accepted_table(indptr, indices, last, page, np.array(drafts, np.int32),
                                    np.array([len(p) for p in paths], np.int32))
        for b in range(batch):
            mine = table2[1][table2[0][b]:table2[0][b + 1]]
            length = page * (len(mine) - 1) + int(table2[2][b])
            assert length == len(kept[0][b]) and list(mine) == ids[b][:len(mine)]
            for l in range(layers):
                got = kvs[l][torch.from_numpy(mine).long().cuda()].double().transpose(0, 1).reshape(2, -1, hkv, D)[:, :length]
                ks, vs = torch.stack([x for x, _ in kept[l][b]]), torch.stack([x for _, x in kept[l][b]])
                assert torch.equal(got[1], vs)
                assert ((got[0] - ks).abs() <= 2.0 ** -8 * ks.abs() + 2.0 ** -18 * 8).all()
        assert dec.device_error() == 0


def test_two_steps_over_an_e4m3_cache():
    """Prompts appended to an E4M3 cache, trees of drafts over it, the accepted moved, and one more token:
    every result is the attention over what the cache holds, and the cache holds the accepted rows."""
    hq, hkv, D, page, pool = 8, 2, 128, 32, 12
    g = torch.Generator("cuda").manual_seed(11)
    rope = pkd.RotaryPositions([10_000.0 ** (-i / 64) for i in range(64)])
    ids = [[7, 2, 9, 4], [0, 11, 5, 3]]
    kv = torch.zeros(pool, 2, hkv, page, D, dtype=torch.float8_e4m3fn, device="cuda")
    scales = dict(k_scale=2 ** -5, v_scale=2 ** -6)
    dec = pkd.BatchTreeDecodeWithPagedKVCache(hq, hkv, D, page, max_tokens=100, max_num_pages=8, num_pages=pool,
                                              kv_dtype="e4m3", kv_layout="HND")

    def held(b, n):
        x = kv.view(torch.uint8)[torch.tensor(ids[b], device="cuda")].view(torch.float8_e4m3fn).double()
        x = x.transpose(2, 3).transpose(0, 1).reshape(2, -1, hkv, D)[:, :n]
        return x[0] * scales["k_scale"], x[1] * scales["v_scale"]

    def step(ctx, counts, parents):
        lens = [a + n for a, n in zip(ctx, counts)]
        pages = [-(-n // page) for n in lens]
        indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        indices = np.concatenate([ids[b][:pages[b]] for b in range(2)]).astype(np.int32)
        last = np.array([n - page * (c - 1) for n, c in zip(lens, pages)], np.int32)
        tables = [torch.from_numpy(x).cuda() for x in (indptr, indices, last)]
        q_indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        mask, depths = (None, None) if parents is None else pkd.tree_mask(q_indptr, parents)
        n = int(q_indptr[-1])
        deep = np.concatenate([np.arange(c) for c in counts]) if parents is None else depths
        rows = torch.from_numpy(np.repeat([0, 1], counts)).int().cuda()
        places = torch.from_numpy(np.concatenate([np.arange(a, b) for a, b in zip(ctx, lens)])).int().cuda()
        at = torch.from_numpy(np.repeat(ctx, counts) + deep).int().cuda()
        both = torch.randn(n, hq + 2 * hkv, D, generator=g, device="cuda").bfloat16()
        q, _ = pkd.rotate_append_kv(both[:, :hq], both[:, hq:hq + hkv], both[:, hq + hkv:], rope, rows, places, *tables,
                                    kv, rope_positions=at, kv_layout="HND", **scales)
        dec.plan(q_indptr, indptr, indices, last, causal=parents is None)
        d_mask = None if mask is None else torch.from_numpy(mask).cuda()
        out, lse = dec.run(q, kv, mask=d_mask, **scales)
        for b in range(2):
            k, v = (x.repeat_interleave(hq // hkv, 1) for x in held(b, lens[b]))
            for i in range(counts[b]):
                row = int(q_indptr[b]) + i
                sees = [t < ctx[b] or (t - ctx[b] <= i if parents is None else
                                       bool(int(mask[row, 0]) >> (t - ctx[b]) & 1)) for t in range(lens[b])]
                x = torch.einsum("hd,thd->ht", q[row].double(), k[sees]) * D ** -0.5
                ref = torch.einsum("ht,thd->hd", x.softmax(-1), v[sees])
                # (P and the output in bf16, values up to 6)
                assert (out[row].double() - ref).abs().max() <= 1.1 * 2 ** -8 * 12
                assert (lse[row].double() - x.logsumexp(-1)).abs().max() <= 2e-4
        assert dec.device_error() == 0
        return tables, lens

    step([0, 0], [50, 33], None)
    drafts = [6, 9]
    tables, lens = step([50, 33], drafts, np.array([-1, 0, 0, 2, 3, -1] + [-1, 0, 1, 0, 3, 4, 5, 6, -1], np.int32))
    before = [held(b, lens[b]) for b in range(2)]
    paths = [[0, 2, 3], [0, 3, 4, 6]]
    pkd.accept_kv([kv], torch.tensor([paths[0] + [-1], paths[1]], dtype=torch.int32, device="cuda"),
                  torch.tensor(drafts, dtype=torch.int32, device="cuda"), *tables, kv_layout="HND")
    for b, ctx in enumerate((50, 33)):
        now, rows = held(b, ctx + len(paths[b])), list(range(ctx)) + [ctx + j for j in paths[b]]
        assert all(torch.equal(x, y[rows]) for x, y in zip(now, before[b]))
    step([53, 37], [1, 1], None)


def test_caches_beside_one_another_and_overlapping():
    c = Case(layers=4)
    pool = torch.stack(c.kvs)          # the layers of one allocation, one behind the other
    c.kvs = list(pool)
    c.check()
    c.kvs = [pool[2], pool[0], pool[3]]
    c.check()
    flat = pool.flatten(0, 1)
    c.kvs = [flat[:c.pool], flat[c.pool - 1:2 * c.pool - 1]]
    keep = flat.clone()
    with pytest.raises(pkd.PkdError, match="INVALID"):
        c.run()
    assert torch.equal(flat, keep)


@pytest.mark.parametrize("ctas", [0, 8])
@pytest.mark.parametrize("fp8", [False, True])
def test_queued_directly_behind_a_tree_run(ctas, fp8):
    """The tree kernel and its merge let the next launch start early: the moves and appends that follow
    on the same cache, with nothing between them, touch none of it before the run has read it, nor each
    other's rows.  With 8 CTAs nothing is split (the tree kernel itself comes before the moves) and most
    of the GPU is free for what starts early."""
    hq, hkv, D, page, n, batch = 32, 8, 128, 16, 24, 6
    lens = [4000 + 37 * b for b in range(batch)]
    indptr, indices, last, pool = table(lens, page)
    q_indptr = (np.arange(batch + 1) * n).astype(np.int32)
    g = torch.Generator("cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    parents = np.random.default_rng(3).integers(-1, np.tile(np.maximum(np.arange(n), 0), batch)).astype(np.int32)
    mask, depths = (torch.from_numpy(x).cuda() for x in pkd.tree_mask(q_indptr, parents))
    dec = pkd.BatchTreeDecodeWithPagedKVCache(hq, hkv, D, page, max_tokens=batch * n, max_num_pages=len(indices),
                                              num_pages=pool, num_ctas=ctas, kv_dtype="e4m3" if fp8 else "bf16")
    dec.plan(q_indptr, indptr, indices, last)
    assert (dec.plan_info()["num_units"] == 0) == (ctas == 8)
    start = rnd(pool, 2, page, hkv, D)
    start = start.to(torch.float8_e4m3fn) if fp8 else start
    kv = torch.empty_like(start)
    tables = [torch.from_numpy(x).cuda() for x in (indptr, indices, last)]
    accepted = torch.tensor([[1, 2, 5, 9, 10, 17, 20, 23]] * batch, dtype=torch.int32, device="cuda")
    drafted = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    rope = pkd.RotaryPositions([10_000.0 ** (-i / 64) for i in range(64)])
    q, both = rnd(batch * n, hq, D), rnd(batch * n, hq + 2 * hkv, D)
    rows = torch.arange(batch, device="cuda", dtype=torch.int32).repeat_interleave(n)
    places = torch.tensor([x - n + i for x in lens for i in range(n)], dtype=torch.int32, device="cuda")
    # new tokens take the places behind the 8 that stay, and the last 4 of those
    m = torch.arange(batch * n, device="cuda").view(batch, n)[:, 4:].reshape(-1)
    both, rows, places = both[m], rows[m].contiguous(), places[m].contiguous()

    def step(wait):
        kv.view(torch.uint8).copy_(start.view(torch.uint8))
        wait()
        out, lse = dec.run(q, kv, mask=mask, depths=depths)
        wait()
        pkd.accept_kv([kv], accepted, drafted, *tables)
        wait()
        turned, _ = pkd.rotate_append_kv(both[:, :hq], both[:, hq:hq + hkv], both[:, hq + hkv:], rope, rows, places,
                                         *tables, kv)
        wait()
        return out, lse, turned, kv.view(torch.uint8).clone()

    want = step(torch.cuda.synchronize)
    for _ in range(25):
        got = step(lambda: None)
        for x, y in zip(want, got):
            assert torch.equal(x, y)
    assert dec.device_error() == 0
