"""Decode over the latent cache and its append, against the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_kv_decode_host_gb300 as pkd

gpu = pytest.mark.gpu
ROW, DIM = 576, 512
SCALE = 1.0 / math.sqrt(192.0)


def table(lens, page, seed=0, spare=3):
    """(indptr, indices, last, pool pages): pages scattered over the pool."""
    counts = [-(-n // page) for n in lens]
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    pool = int(indptr[-1]) + spare
    where = np.random.default_rng(seed).permutation(pool)[: indptr[-1]].astype(np.int32)
    last = np.array([n - page * (c - 1) for n, c in zip(lens, counts)], np.int32)
    return indptr, where, last, pool


def reference(q, cache, lens, t, page, scale=SCALE):
    indptr, indices = t[0], t[1]
    outs, lses = [], []
    for i, n in enumerate(lens):
        mine = torch.from_numpy(indices[indptr[i]:indptr[i + 1]]).long().to(cache.device)
        c = cache[mine].reshape(-1, ROW)[:n].double()
        x = q[i].double() @ c.T * scale
        lse = torch.logsumexp(x, 1)
        outs.append(torch.exp(x - lse[:, None]) @ c[:, :DIM])
        lses.append(lse)
    return torch.stack(outs), torch.stack(lses)


def make(heads, lens, page, seed=0, **kw):
    t = table(lens, page, seed)
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randn(len(lens), heads, ROW, generator=g, device="cuda").bfloat16()
    cache = torch.randn(t[3], page, ROW, generator=g, device="cuda").bfloat16()
    dec = pkd.BatchLatentDecodeWithPagedCache(heads, DIM, 64, page, scale=SCALE,
                                              max_batch=max(1, len(lens)),
                                              max_num_pages=len(t[1]), num_pages=t[3], **kw)
    return t, q, cache, dec


def close(got, ref, top):
    """P and the result are rounded to bf16 (half a step: 2^-8 relative).  A result is a weighted
    mean of cached values of magnitude at most `top`: the rounding of P moves it by at most 2^-8
    top, its own by 2^-8 |out|; the fp32 sums (2^-24 per step, under 2^14 steps) by under 2^-10 of
    that, which 1 % covers.  lse: fp32 sums of 576 products, each at most 6 x 6 x scale < 2.6 in
    these inputs: 576 x 2^-24 x 576 x 2.6 would be the worst case, rounding errors of random sign
    grow with the root, under 2^-24 x 24 x 24 x 2.6 < 1e-4."""
    (out, lse), (ro, rl) = got, ref
    assert (out.double() - ro).abs().max() <= 1.01 * 2 ** -8 * (top + ro.abs().max())
    assert (lse.double() - rl).abs().max() <= 2e-4


@gpu
@pytest.mark.parametrize("heads", [1, 5, 16, 17, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("page", [16, 64])
def test_heads_and_lengths(heads, page):
    lens = [1, 15, 16, 17, 63, 64, 65, 111, 112, 113, 127, 128, 129, 250, 700]
    t, q, cache, dec = make(heads, lens, page, seed=heads)
    dec.plan(*t[:3])
    out, lse = dec.run(q, cache)
    close((out, lse), reference(q, cache, lens, t, page), cache.abs().max().double())
    assert dec.device_error() == 0


@gpu
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(num_ctas=3), dict(num_ctas=1)])
def test_split_requests(heads, kw):
    lens = [9001, 3, 1500]
    t, q, cache, dec = make(heads, lens, 16, seed=1, **kw)
    dec.plan(*t[:3])
    out, lse = dec.run(q, cache)
    close((out, lse), reference(q, cache, lens, t, 16), cache.abs().max().double())
    out2, lse2 = dec.run(q, cache)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert dec.device_error() == 0


@gpu
def test_rising_scores_rescale():
    """Scores that grow along the sequence raise the softmax base in every tile."""
    lens = [1000]
    t, q, cache, dec = make(64, lens, 16, seed=2, min_chunk_tokens=4096)
    ramp = torch.linspace(0.0, 8.0, 1008, device="cuda")
    at = torch.from_numpy(t[1]).long().cuda()
    flat = cache[at].reshape(-1, ROW)
    flat[:, 512:] = ramp[:, None].bfloat16()
    cache[at] = flat.view(-1, 16, ROW)
    q[:, :, 512:] = 1.0 / 4
    dec.plan(*t[:3])
    out, lse = dec.run(q, cache)
    close((out, lse), reference(q, cache, lens, t, 16), cache.abs().max().double())


@gpu
def test_stale_slots_are_not_read():
    """NaN and infinities behind the last token, and in pages of the pool that are not the request's."""
    lens = [5, 130, 64]
    t, q, cache, dec = make(40, lens, 16, seed=3)
    ref = reference(q, cache, lens, t, 16)
    dirty = torch.full_like(cache, float("nan"))
    dirty[::2] = float("inf")
    for i, n in enumerate(lens):
        for k in range(n):
            pg, sl = int(t[1][t[0][i] + k // 16]), k % 16
            dirty[pg, sl] = cache[pg, sl]
    dec.plan(*t[:3])
    out, lse = dec.run(q, dirty)
    close((out, lse), ref, cache.abs().max().double())


@gpu
def test_infinite_scores_in_one_place():
    """A score of -inf weighs nothing; a head whose scores are all -inf is an empty state."""
    lens = [40]
    t, q, cache, dec = make(16, lens, 16, seed=4)
    cache[:, :, 575] = 0.0
    first = int(t[1][0])
    cache[first, 3, 575] = float("inf")
    q[:, :, 575] = -1.0
    dec.plan(*t[:3])
    out, lse = dec.run(q, cache)
    ref = reference(q, cache, lens, t, 16)
    close((out, lse), ref, 6.0)
    cache[:, :, 575] = float("inf")
    out, lse = dec.run(q, cache)
    assert (out == 0).all() and (lse == -float("inf")).all()


@gpu
def test_v_scale_and_no_lse():
    lens = [77, 200]
    t, q, cache, dec = make(20, lens, 16, seed=5)
    dec.plan(*t[:3])
    out = dec.run(q, cache, return_lse=False)
    assert torch.equal(out, dec.run(q, cache)[0])


@gpu
def test_append_then_decode_in_a_graph():
    """Two steps of a serving loop: append, plan, replayed decode, against the formulas."""
    page, lens, heads = 16, [31, 64, 1], 16
    t = table([n + 2 for n in lens], page, 7)
    cache = torch.randn(t[3], page, ROW, device="cuda").bfloat16()
    q = torch.empty(len(lens), heads, ROW, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(len(lens), heads, DIM, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(len(lens), heads, device="cuda")
    dec = pkd.BatchLatentDecodeWithPagedCache(heads, DIM, 64, page, scale=SCALE, max_batch=3,
                                              max_num_pages=len(t[1]), num_pages=t[3])
    graph = None
    for step in range(2):
        now = [n + step + 1 for n in lens]
        counts = [-(-n // page) for n in now]
        indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        indices = np.concatenate([t[1][t[0][i]:t[0][i] + c] for i, c in enumerate(counts)])
        last = np.array([n - page * (c - 1) for n, c in zip(now, counts)], np.int32)
        both = torch.randn(3, 600, device="cuda").bfloat16()
        before = cache.clone()
        pkd.append_latent(both[:, :512], both[:, 512:576], torch.arange(3, device="cuda").int(),
                          torch.tensor([n - 1 for n in now], device="cuda").int(),
                          torch.from_numpy(indptr).cuda(), torch.from_numpy(indices).cuda(),
                          torch.from_numpy(last).cuda(), cache)
        for i, n in enumerate(now):
            before[int(indices[indptr[i] + (n - 1) // page]), (n - 1) % page] = both[i, :576]
        assert torch.equal(before, cache)
        q.copy_(torch.randn_like(q))
        dec.plan(indptr, indices, last)
        if graph is None:
            graph = dec.capture([q], [cache], [out], [lse])
        graph.launch()
        ref = reference(q, cache, now, (indptr, indices), page)
        close((out, lse), ref, cache.abs().max().double())


@gpu
def test_append_skips_and_flags():
    page = 16
    t = table([20, 5], page)
    d = [torch.from_numpy(x).cuda() for x in t[:3]]
    cache = torch.zeros(t[3], page, ROW, dtype=torch.bfloat16, device="cuda")
    new = torch.ones(5, ROW, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 0, 1, 2, -1], device="cuda").int()
    at = torch.tensor([19, 20, 4, 0, 0], device="cuda").int()   # 20 and requests 2, -1: outside
    pkd.append_latent(new[:, :512], new[:, 512:], rows, at, *d, cache, err=err)
    assert err.item() == pkd.DEV_ERR_BOUNDS
    assert int((cache != 0).any(-1).sum()) == 2
    assert cache[int(t[1][1]), 3].all() and cache[int(t[1][2]), 4].all()
    err.zero_()
    short = d[1][:2].clone()   # request 1's page is past the indices' end
    pkd.append_latent(new[2:4, :512], new[2:4, 512:], rows[2:4], at[2:4], d[0], short, d[2],
                      torch.zeros_like(cache), err=err)
    assert err.item() == pkd.DEV_ERR_BOUNDS
    pkd.append_latent(new[:0, :512], new[:0, 512:], rows[:0], at[:0], *d, cache)


@gpu
@pytest.mark.parametrize("n", [1, 3, 31, 2431, 2432, 2433, 6003])
def test_append_many(n):
    """Tokens of several requests in any order, some outside the table."""
    page, lens = 16, [3000, 1, 4100]
    t = table(lens, page, n)
    d = [torch.from_numpy(x).cuda() for x in t[:3]]
    gen = np.random.default_rng(n)
    every = [(b, p) for b, m in enumerate(lens) for p in range(m)]
    pick = gen.permutation(len(every))[:n]
    rows = np.array([every[k][0] for k in pick], np.int32)
    at = np.array([every[k][1] for k in pick], np.int32)
    out = gen.random(n) < 0.1
    rows[out], at[out] = gen.integers(-2, 5, out.sum()), 5000   # past every request's end
    both = torch.randn(n, 584, device="cuda").bfloat16()
    cache = torch.randn(t[3], page, ROW, device="cuda").bfloat16()
    want = cache.clone()
    for i in np.nonzero(~out)[0]:
        want[int(t[1][t[0][rows[i]] + at[i] // page]), int(at[i] % page)] = both[i, 8:584]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkd.append_latent(both[:, 8:520], both[:, 520:584], torch.from_numpy(rows).cuda(),
                      torch.from_numpy(at).cuda(), *d, cache, err=err)
    assert torch.equal(cache, want)
    assert err.item() == (pkd.DEV_ERR_BOUNDS if out.any() else 0)


@gpu
def test_other_stream_and_refusals():
    lens = [100]
    t, q, cache, dec = make(16, lens, 16, seed=8)
    with pytest.raises(pkd.PkdError):
        dec.run(q, cache)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dec.plan(*t[:3])
        got = dec.run(q, cache)
    s.synchronize()
    close(got, reference(q, cache, lens, t, 16), cache.abs().max().double())
    for bad in (q.float(), q[:, :8], q[:, :, :512].contiguous()):
        with pytest.raises((TypeError, ValueError)):
            dec.run(bad, cache)
    with pytest.raises(ValueError):
        dec.run(q, cache[:, :, :512])
    with pytest.raises(pkd.PkdError):
        dec.plan_cascade(None, None, None)
    for kw in (dict(num_heads=129), dict(num_heads=0), dict(page_size=8), dict(latent_dim=256)):
        args = dict(num_heads=16, latent_dim=512, rope_dim=64, page_size=16)
        args.update(kw)
        with pytest.raises(pkd.PkdError):
            pkd.BatchLatentDecodeWithPagedCache(**args, scale=1.0, max_batch=1, max_num_pages=4,
                                                num_pages=4)
    with pytest.raises(ValueError):
        pkd.append_latent(q[0, :, :512].t(), q[0, :, 512:], *[torch.zeros(16, device="cuda").int()] * 4,
                          torch.zeros(15, device="cuda").int(), cache)


@gpu
def test_graph_follows_later_plans():
    """A step captured while no request was split replays under a plan that splits them, and back."""
    page, heads = 16, 40
    lens_a, lens_b = [100, 50, 7], [3000, 900, 5000]
    t = table(lens_b, page, 11)
    cache = torch.randn(t[3], page, ROW, device="cuda").bfloat16()
    q = torch.randn(3, heads, ROW, device="cuda").bfloat16()
    out = torch.zeros(3, heads, DIM, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(3, heads, device="cuda")
    dec = pkd.BatchLatentDecodeWithPagedCache(heads, DIM, 64, page, scale=SCALE, max_batch=4,
                                              max_num_pages=len(t[1]), num_pages=t[3])

    def tables(lens):
        counts = [-(-n // page) for n in lens]
        indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        ids = np.concatenate([t[1][t[0][i]:t[0][i] + c] for i, c in enumerate(counts)])
        return indptr, ids, np.array([n - page * (c - 1) for n, c in zip(lens, counts)], np.int32)

    dec.plan(*tables(lens_a))
    assert dec.plan_info()["num_units"] == 0
    graph = dec.capture([q], [cache], [out], [lse])
    for lens in (lens_a, lens_b, lens_a):
        dec.plan(*tables(lens))
        graph.launch()
        close((out, lse), reference(q, cache, lens, tables(lens), page), cache.abs().max().double())
    assert dec.device_error() == 0
    dec.plan(*[x[:k] for x, k in zip(tables(lens_a), (3, 99, 2))])
    with pytest.raises(pkd.PkdError, match="STALE"):   # the queries' map is of three requests
        graph.launch()


@gpu
def test_capture_with_host_buffers_and_torch_graph():
    lens, page, heads = [70, 300], 16, 16
    t, q, cache, dec = make(heads, lens, page, seed=12)
    dec.plan(*t[:3])
    ref = reference(q, cache, lens, t, page)
    top = cache.abs().max().double()
    out, lse = torch.empty(2, heads, DIM, dtype=torch.bfloat16, device="cuda"), torch.empty(2, heads, device="cuda")
    hq, ho, hl = q.cpu().pin_memory(), out.cpu().pin_memory(), lse.cpu().pin_memory()
    qd = torch.zeros_like(q)
    graph = dec.capture([qd], [cache], [out], [lse], host_qs=[hq], host_outs=[ho], host_lses=[hl])
    graph.launch()
    torch.cuda.synchronize()
    close((ho.cuda(), hl.cuda()), ref, top)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = dec.run(q, cache)
    g.replay()
    close(got, ref, top)


@gpu
def test_epoch_on_another_stream_and_empty_batch():
    lens, page = [500, 33], 16
    t, q, cache, dec = make(32, lens, page, seed=13)
    upload = torch.cuda.Stream()
    for _ in range(3):
        epoch = dec.plan(*t[:3], stream=upload)
        got = dec.run(q, cache, expect_epoch=epoch)   # waits for the schedule on the device
    close(got, reference(q, cache, lens, t, page), cache.abs().max().double())
    with pytest.raises(pkd.PkdError, match="STALE"):
        dec.run(q, cache, expect_epoch=epoch - 1)
    torch.cuda.synchronize()
    dec.plan(np.zeros(1, np.int32), np.zeros(0, np.int32), np.zeros(0, np.int32))
    out, lse = dec.run(q[:0], cache)
    assert out.shape == (0, 32, DIM) and lse.shape == (0, 32) and dec.device_error() == 0


@gpu
def test_offsets_past_32_bits():
    """A pool of 5 GB whose last pages hold the request, appended there and read back."""
    page, pages, heads, n = 64, 70_000, 16, 200
    cache = torch.empty(pages, page, ROW, dtype=torch.bfloat16, device="cuda")
    assert cache.numel() * 2 > 1 << 32
    ids = np.array([pages - 1, pages - 3, pages - 2, pages - 4], np.int32)
    t = (np.array([0, 4], np.int32), ids, np.array([n - 192], np.int32))
    rows = torch.randn(n, ROW, device="cuda").bfloat16()
    pkd.append_latent(rows[:, :512], rows[:, 512:], torch.zeros(n, device="cuda").int(),
                      torch.arange(n, device="cuda").int(), *[torch.from_numpy(x).cuda() for x in t], cache)
    assert torch.equal(cache[torch.from_numpy(ids).long().cuda()].reshape(-1, ROW)[:n], rows)
    dec = pkd.BatchLatentDecodeWithPagedCache(heads, DIM, 64, page, scale=SCALE, max_batch=1,
                                              max_num_pages=4, num_pages=pages)
    dec.plan(*t)
    q = torch.randn(1, heads, ROW, device="cuda").bfloat16()
    close(dec.run(q, cache), reference(q, cache, [n], t, page), rows.abs().max().double())


@gpu
def test_two_contexts_at_once():
    """Two contexts on two streams over one cache, many times over."""
    lens, page = [2000, 100, 5000], 16
    t, q, cache, a = make(64, lens, page, seed=14)
    b = pkd.BatchLatentDecodeWithPagedCache(64, DIM, 64, page, scale=SCALE, max_batch=3,
                                            max_num_pages=len(t[1]), num_pages=t[3], num_ctas=50)
    ref = reference(q, cache, lens, t, page)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a.plan(*t[:3])
    with torch.cuda.stream(s):
        b.plan(*t[:3])
    for _ in range(20):
        x = a.run(q, cache)
        with torch.cuda.stream(s):
            y = b.run(q, cache)
    torch.cuda.synchronize()
    for got in (x, y):
        close(got, ref, cache.abs().max().double())


@pytest.mark.parametrize("heads", [16, 64, 128])
@pytest.mark.parametrize("lens", [[1], [517], [4096] * 32, [100_000] + [300] * 8, list(range(1, 200)),
                                  [], [129, 128, 127, 255, 256, 257] * 7])
@pytest.mark.parametrize("n_cta,page", [(152, 16), (152, 64), (7, 16), (1, 16), (2, 128)])
def test_plan_covers_every_token_once(heads, lens, n_cta, page):
    """Host only: every (request, token, block of heads) in one item, slots as the reduction map
    has them, and no CTA's cost above the plan's."""
    t = table(lens, page) if lens else (np.zeros(1, np.int32), np.zeros(0, np.int32), np.zeros(0, np.int32), 1)
    cfg = pkd.make_config(heads, 1, DIM, page, max(1, len(lens)), max(1, len(t[1])), max(1, t[3]),
                          num_ctas=n_cta, flags=pkd.FLAG_LATENT)
    words, info, off = pkd.plan_host(cfg, *t[:3])
    s = pkd.decode_schedule(words, off, info)
    blocks = -(-heads // 64)
    seen = {}
    for (req, tb, te, dst, page0, n_req, stride), b in zip(s["items"], s["heads"]):
        assert n_req == 1 and 0 <= b < blocks and tb % page == 0 and te > tb
        assert page0 == t[0][req] + tb // page
        seen.setdefault((req, b), []).append((tb, te, dst))
    slots = {req: list(range(s["merge_indptr"][u], s["merge_indptr"][u + 1]))
             for u, (req, _) in enumerate(s["units"])}
    for i, n in enumerate(lens):
        for b in range(blocks):
            parts = sorted(seen.pop((i, b)))
            assert [p[0] for p in parts] == [0] + [p[1] for p in parts[:-1]] and parts[-1][1] == n
            assert [p[2] for p in parts] == (slots[i] if len(parts) > 1 else [-1])
    assert not seen and info["num_slots"] == sum(len(x) for x in slots.values())
    cost = [sum(128 + te - tb for _, tb, te, *_ in s["items"][a:z])
            for a, z in zip(s["cta_indptr"], s["cta_indptr"][1:])]
    assert max(cost, default=0) <= info["makespan"] * (blocks if n_cta < blocks else 1)
    even = (sum(lens) + 128 * len(lens)) / max(1, n_cta // blocks)
    assert info["makespan"] <= max(1.35 * even, even + 2 * (256 + page)) + 256
