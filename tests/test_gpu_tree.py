"""Attention of drafted tokens over a paged cache, against the formula in 64 bits."""
import math
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_decode_host_gb300 as pkd

pytestmark = pytest.mark.gpu
D = 128


def table(lens, page, seed=0, spare=3):
    counts = [-(-n // page) for n in lens]
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    pool = int(indptr[-1]) + spare
    where = np.random.default_rng(seed).permutation(pool)[: indptr[-1]].astype(np.int32)
    last = np.array([n - page * (c - 1) for n, c in zip(lens, counts)], np.int32)
    return indptr, where, last, pool


def trees(drafts, seed):
    """Random parents of every request's drafts."""
    r = np.random.default_rng(seed)
    return np.concatenate([[int(r.integers(max(-1, j // 3 - 2), j)) for j in range(n)] for n in drafts]
                          + [[]]).astype(np.int32)


KV_SCALES = torch.tensor([0.5, 0.25], dtype=torch.float64).view(1, 2, 1, 1, 1)


class Case:
    def __init__(self, hq=8, hkv=2, page=16, layout="NHD", lens=(37, 16, 5), drafts=(4, 3, 5), causal=False,
                 window=0, cap=0.0, slopes=False, seed=0, rows=None, depths=True, magnitude=1.0, scale=None, fp8=False, **kw):
        self.__dict__.update(hq=hq, hkv=hkv, page=page, layout=layout, lens=lens, drafts=drafts, causal=causal,
                             window=window, cap=cap, scale=scale, fp8=fp8)
        self.scales = dict(k_scale=0.5, v_scale=0.25) if fp8 else {}
        self.indptr, self.indices, self.last, self.pool = table(lens, page, seed)
        self.q_indptr = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        self.tokens = int(self.q_indptr[-1])
        g = torch.Generator("cuda").manual_seed(seed)
        shape = (self.pool, 2, page, hkv, D) if layout == "NHD" else (self.pool, 2, hkv, page, D)
        self.kv = torch.randn(shape, generator=g, device="cuda").bfloat16()
        if fp8:   # values of about 1 once scaled
            self.kv[:, 0] *= 2
            self.kv[:, 1] *= 4
            self.kv = self.kv.to(torch.float8_e4m3fn)
        self.q = (magnitude * torch.randn(self.tokens if rows is None else rows, hq, D, generator=g,
                                          device="cuda")).bfloat16()
        self.mask = self.depths = self.slopes = None
        if not causal:
            mask, depth = pkd.tree_mask(self.q_indptr, trees(drafts, seed))
            pad = len(self.q) - self.tokens
            self.mask = torch.from_numpy(np.concatenate([mask, np.zeros((pad, mask.shape[1]), np.int32)])).cuda()
            if depths:
                self.depths = torch.from_numpy(np.concatenate([depth, np.zeros(pad, np.int32)])).cuda()
        if slopes:
            self.slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], device="cuda")
        self.dec = pkd.BatchTreeDecodeWithPagedKVCache(
            hq, hkv, D, page, max_tokens=max(1, self.tokens, len(lens)), max_num_pages=len(self.indices),
            num_pages=self.pool, kv_layout=layout, kv_dtype="e4m3" if fp8 else "bf16", **kw)
        self.plan()

    def plan(self, **kw):
        return self.dec.plan(self.q_indptr, self.indptr, self.indices, self.last, causal=self.causal,
                             window=self.window, **kw)

    def run(self, **kw):
        return self.dec.run(self.q, self.kv, mask=self.mask, depths=self.depths, score_cap=self.cap,
                            slopes=self.slopes, scale=self.scale, **self.scales, **kw)

    def sees(self, b):
        """[n, l] which tokens every query token of request b sees, and how far away they are."""
        n, length, first = self.drafts[b], self.lens[b], int(self.q_indptr[b])
        ctx = length - n
        depth = np.arange(n) if self.depths is None else self.depths[first:first + n].cpu().numpy().astype(np.int64)
        depth = np.maximum(depth, 0)
        at = np.concatenate([np.arange(ctx), ctx + depth])
        away = (ctx + depth)[:, None] - at[None, :]
        see = np.ones((n, length), bool)
        if self.causal:
            see[:, ctx:] = np.tril(np.ones((n, n), bool))
        else:
            words = self.mask[first:first + n].cpu().numpy().view(np.uint32)
            for j in range(n):
                see[:, ctx + j] = (words[:, j // 32] >> np.uint32(j % 32)) & 1
        if self.window:
            see &= away < self.window
        return torch.from_numpy(see).cuda(), torch.from_numpy(away).cuda()

    def reference(self):
        outs, lses = [], []
        for b, (n, length) in enumerate(zip(self.drafts, self.lens)):
            if n == 0:
                continue
            mine = torch.from_numpy(self.indices[self.indptr[b]:self.indptr[b + 1]]).long().cuda()
            kv = (self.kv.view(torch.uint8)[mine].view(torch.float8_e4m3fn).double() * KV_SCALES.cuda() if self.fp8
                  else self.kv[mine].double())
            kv = kv if self.layout == "NHD" else kv.transpose(2, 3)
            k, v = (kv[:, c].reshape(-1, self.hkv, D)[:length] for c in (0, 1))
            first = int(self.q_indptr[b])
            q = self.q[first:first + n].double().view(n, self.hkv, -1, D)
            x = torch.einsum("nhgd,thd->hgnt", q, k) * (D ** -0.5 if self.scale is None else self.scale)
            see, away = self.sees(b)
            if self.cap:
                x = self.cap * torch.tanh(x / self.cap)
            if self.slopes is not None:
                x = x - self.slopes.double().view(self.hkv, -1, 1, 1) * away
            x = torch.where(see, x, -math.inf)
            lse = torch.logsumexp(x, -1)
            p = torch.where(see, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
            # what is not seen does not matter, whatever it holds
            out = torch.zeros(self.hkv, self.hq // self.hkv, n, D, dtype=torch.float64, device="cuda")
            for i in range(n):
                t = see[i].nonzero()[:, 0]
                out[:, :, i] = torch.einsum("hgt,thd->hgd", p[:, :, i, t], v[t])
            outs.append(out.permute(2, 0, 1, 3).reshape(n, -1, D))
            lses.append(lse.permute(2, 0, 1).reshape(n, -1))
        return torch.cat(outs), torch.cat(lses)

    def check(self, got=None):
        out, lse = self.run() if got is None else got
        ro, rl = self.reference()
        out, lse = out[:self.tokens], lse[:self.tokens]
        assert self.dec.device_error() == 0
        fine = torch.isfinite(rl)
        assert torch.equal(torch.isfinite(lse), fine) and (lse[~fine] == -math.inf).all()
        assert (out[~fine] == 0).all()
        # P is rounded to bf16 (half a step: 2^-8 of itself) and the row's sum is not: that moves a
        # weighted mean of values of magnitude at most top by at most 2^-8 top, its own rounding by
        # 2^-8 |out|; scores in fp32 (below) move the weights by under 2^-12 of themselves
        kv = self.kv.float() * (KV_SCALES.float().cuda() if self.fp8 else 1.0)
        top = float(kv[torch.isfinite(kv)].abs().max())
        assert (out.double() - ro).abs().max() <= 1.1 * 2 ** -8 * (top + float(ro.abs().max()))
        # lse: a score is an fp32 sum of 128 products, random errors of 2^-24 of its terms' partial
        # sums (under 2^-24 * 128 * 6 * scale of the queries' magnitude, < 1e-4); the cap's tanh is
        # off by under 2^-21 of the cap, a bias by 2^-24 of itself; sums of n weights by under 2^-24 n
        tol = 2e-4 + self.cap * 2 ** -20 + 2 ** -21 * float(rl[fine].abs().max() if fine.any() else 0)
        assert fine.sum() == 0 or (lse[fine].double() - rl[fine]).abs().max() <= tol


GROUPS = [(1, 1), (2, 1), (8, 1), (3, 3), (12, 3), (8, 2), (8, 8), (32, 8), (64, 8)]


@pytest.mark.parametrize("hq,hkv", GROUPS)
@pytest.mark.parametrize("layout,page", [("NHD", 16), ("HND", 48)])
def test_heads_and_layouts(hq, hkv, layout, page):
    Case(hq=hq, hkv=hkv, layout=layout, page=page, lens=(37, 16, 5, 300), drafts=(4, 3, 5, 9), seed=hq).check()


@pytest.mark.parametrize("lens,drafts", [
    ((1,), (1,)), ((2,), (2,)), ((16,), (16,)), ((17,), (1,)), ((127,), (3,)), ((128,), (3,)), ((129,), (3,)),
    ((130,), (130,)), ((191, 192, 193), (64, 64, 65)), ((255, 256, 257), (1, 1, 1)), ((640,), (33,)),
    ((40, 7, 90), (0, 7, 3)), ((40, 7), (0, 0)), ((500, 3), (70, 3)), ((64, 64, 64), (63, 1, 64))])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(lens, drafts, causal):
    c = Case(hq=8, hkv=2, lens=lens, drafts=drafts, causal=causal, seed=len(lens))
    if c.tokens:
        c.check()
    else:
        out, lse = c.run()
        assert out.numel() == 0 and c.dec.device_error() == 0


@pytest.mark.parametrize("kw", [dict(cap=30.0), dict(cap=2.0, magnitude=4.0), dict(slopes=True), dict(window=1),
                                dict(window=50), dict(window=200), dict(window=3, depths=False), dict(window=10**9),
                                dict(cap=50.0, window=130, slopes=True), dict(slopes=True, depths=False),
                                dict(magnitude=8.0)])
@pytest.mark.parametrize("causal", [False, True])
def test_score_shapes(kw, causal):
    if causal and "depths" in kw:
        kw = {k: v for k, v in kw.items() if k != "depths"}
    Case(hq=8, hkv=2, lens=(37, 400, 5, 260), drafts=(4, 40, 5, 1), causal=causal, seed=3, **kw).check()


@pytest.mark.parametrize("lens,drafts,causal", [((3000, 40, 1500), (12, 3, 40), False), ((5000,), (1,), False),
                                                ((20_000, 30), (8, 8), False), ((2500, 600), (200, 70), True)])
@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0, window=1300), dict(slopes=True)])
def test_split_requests(lens, drafts, causal, kw):
    c = Case(hq=16, hkv=4, lens=lens, drafts=drafts, causal=causal, seed=5, min_chunk_tokens=128, alpha=0, **kw)
    assert c.dec.plan_info()["num_units"] > 0
    c.check()
    few = Case(hq=16, hkv=4, lens=lens, drafts=drafts, causal=causal, seed=5, num_ctas=3, **kw)   # fewer CTAs than heads
    few.check()


def test_long_requests_with_many_parts():
    c = Case(hq=2, hkv=1, lens=(30_000, 77), drafts=(5, 2), min_chunk_tokens=128, alpha=0, page=64)
    assert c.dec.plan_info()["num_slots"] > 5 * 64   # past the merge's long units
    c.check()


@pytest.mark.parametrize("split", [False, True])
def test_rows_that_see_nothing(split):
    kw = dict(min_chunk_tokens=128, alpha=0) if split else dict(num_ctas=1)
    c = Case(hq=4, hkv=1, lens=(300, 9), drafts=(300, 9), **kw)
    assert (c.dec.plan_info()["num_units"] > 0) == split
    c.mask[1] = 0
    c.mask[303] = 0
    c.mask[7:11] = 0
    c.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("split", [False, True])
def test_what_is_masked_may_hold_anything(bad, split):
    kw = dict(min_chunk_tokens=128, alpha=0) if split else dict(num_ctas=1)
    c = Case(hq=8, hkv=2, lens=(400, 21), drafts=(150, 5), window=0, seed=9, **kw)
    used = set(c.indices.tolist())
    for page in range(c.pool):
        if page not in used:
            c.kv[page] = bad                              # pages of no request
    c.kv[int(c.indices[c.indptr[2] - 1]), :, c.last[1]:] = bad   # behind a request's end
    for draft in (3, 60, 149):                             # drafts that few rows see
        c.mask[:150, draft // 32] &= ~(1 << (draft % 32)) if draft % 32 != 31 else 0x7fffffff
        page, slot = divmod(250 + draft, 16)
        c.kv[int(c.indices[page]), :, slot] = bad
    c.check()


def test_values_that_are_seen_keep_what_they_hold():
    c = Case(hq=4, hkv=1, lens=(300,), drafts=(40,), seed=2)
    c.mask[:, :] = 0
    c.mask[5, 0] = 1 << 7
    page, slot = divmod(260 + 7, 16)
    c.kv[int(c.indices[page]), 1, slot, 0, 33] = float("nan")
    c.kv[int(c.indices[page]), 1, slot, 0, 70] = float("inf")
    out, lse = c.run()
    assert torch.isnan(out[5, :, 33]).all() and (out[5, :, 70] == float("inf")).all()
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[5, :, 33] = rest[5, :, 70] = False
    assert torch.isfinite(out[rest]).all() and torch.isfinite(lse).all()
    c.kv[int(c.indices[page]), 1, slot, 0, 33] = c.kv[int(c.indices[page]), 1, slot, 0, 70] = 0.0
    c.mask[5, 0] = 0   # (its other dims: as in the call where it sees the draft, within the bound)
    ref = c.reference()[0]
    keep = torch.ones(40, dtype=torch.bool)
    keep[5] = False
    good = out[keep].double()
    top = float(c.kv.float().abs().max())
    good[~torch.isfinite(good)] = 0
    assert (good - ref[keep]).abs().max() <= 1.1 * 2 ** -8 * (top + float(ref.abs().max()))


@pytest.mark.parametrize("kw", [dict(), dict(slopes=True), dict(cap=30.0), dict(window=120), dict(window=300, slopes=True)])
def test_odd_values_beside_masked_ones(kw):
    """A context token that all rows see, in a round with drafts and with a window's edge, shows; tokens
    before the window of every row, or of some, do not reach those that do not see them."""
    c = Case(hq=8, hkv=2, lens=(700, 90), drafts=(30, 5), seed=8, **kw)
    ctx, before = 670, c.reference()
    def v(t):
        page, slot = divmod(t, 16)
        return c.kv[int(c.indices[page]), 1, slot]
    edges = (3, ctx - c.window + 1, ctx - c.window + 2)   # before all rows' windows, or before deep rows' only
    keep = {t: v(t).clone() for t in (ctx - 3,) + edges * bool(c.window)}
    v(ctx - 3)[1, 17] = float("nan")
    v(ctx - 3)[0, 5] = -float("inf")
    out, lse = c.run()
    assert torch.isnan(out[:30, 4:, 17]).all() and (out[:30, :4, 5] == -float("inf")).all()
    out = out.clone()
    out[:30, 4:, 17] = out[:30, :4, 5] = 0
    assert torch.isfinite(out).all()
    before[0][:30, 4:, 17] = before[0][:30, :4, 5] = 0
    top = 6.0
    assert (out.double() - before[0]).abs().max() <= 1.1 * 2 ** -8 * (top + float(before[0].abs().max()))
    v(ctx - 3)[:] = keep[ctx - 3]
    if not c.window:
        return
    for t in edges:
        v(t)[:, :] = float("nan")
    see, _ = c.sees(0)
    bad = torch.stack([see[:, t] for t in edges]).any(0)
    assert bad.any() and not bad.all()
    out, lse = c.run()
    for i in range(30):
        assert torch.isnan(out[i]).all() if bad[i] else torch.isfinite(out[i]).all()
    good = torch.cat([~bad, torch.ones(5, dtype=torch.bool, device="cuda")])
    for t, x in keep.items():
        v(t)[:] = x
    assert (out[good].double() - c.reference()[0][good]).abs().max() <= 1.1 * 2 ** -8 * (top + 4.0)


def test_scores_that_rise_along_the_cache():
    """The base of the exponentials is raised in every round; the early tokens' weights vanish."""
    c = Case(hq=8, hkv=2, lens=(1500,), drafts=(6,), seed=4, num_ctas=2)
    c.q[:] = 1.0
    for t in range(1500):
        page, slot = divmod(t, 16)
        c.kv[int(c.indices[page]), 0, slot] = 0.02 * t
    c.check()
    c.kv[:, 0] = -c.kv[:, 0]
    c.check()


def test_rows_behind_the_last_query_are_left_alone():
    c = Case(lens=(300, 50), drafts=(7, 2), rows=20)
    out = torch.full((20, 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((20, 8), 7.0, device="cuda")
    c.check(c.run(out=out, lse=lse))
    assert (out[9:] == 7).all() and (lse[9:] == 7).all()
    assert c.run(return_lse=False).shape == out.shape


def test_same_bits_every_run_and_on_other_streams():
    c = Case(hq=16, hkv=4, lens=(4000, 700), drafts=(20, 9), min_chunk_tokens=128, alpha=0)
    out, lse = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o, l = c.run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_plan_on_another_stream_with_its_epoch():
    c = Case(hq=16, hkv=4, lens=(4000, 700), drafts=(20, 9), min_chunk_tokens=128, alpha=0)
    side = torch.cuda.Stream()
    for _ in range(4):
        epoch = c.plan(stream=side)
        c.check(c.run(expect_epoch=epoch))
    with pytest.raises(pkd.PkdError, match="STALE"):
        c.run(expect_epoch=epoch - 1)


def test_captured_step_under_later_plans():
    c = Case(hq=8, hkv=2, lens=(700, 90, 40), drafts=(12, 9, 4), min_chunk_tokens=128, alpha=0)
    out = torch.zeros(25, 8, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(25, 8, device="cuda")
    c.run(out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, lse=lse)
    out.zero_(), lse.zero_()
    graph.replay()
    c.check((out, lse))
    # fewer tokens, other lengths, no split
    full = c.lens, c.drafts, c.q_indptr, c.indptr, c.indices, c.last, c.tokens
    c.lens, c.drafts = (100, 5), (3, 5)
    c.indptr, c.indices, c.last = np.array([0, 7, 8], np.int32), c.indices[10:18].copy(), np.array([4, 5], np.int32)
    c.q_indptr, c.tokens = np.array([0, 3, 8], np.int32), 8
    mask, depth = pkd.tree_mask(c.q_indptr, trees(c.drafts, 1))
    c.mask[:8], c.depths[:8] = torch.from_numpy(mask).cuda(), torch.from_numpy(depth).cuda()
    c.plan()
    out.fill_(3.0)
    graph.replay()
    c.check((out, lse))
    assert (out[8:] == 3).all()
    # more tokens than the captured call has rows: no work, and the error word says so
    c.lens, c.drafts, c.q_indptr, c.indptr, c.indices, c.last, c.tokens = full
    q, o = c.q[:6].clone(), torch.zeros(6, 8, D, dtype=torch.bfloat16, device="cuda")
    c.dec.plan(np.array([0, 3, 6], np.int32), np.array([0, 3, 6], np.int32), c.indices[:6].copy(),
               np.array([8, 8], np.int32))
    graph2 = torch.cuda.CUDAGraph()
    mask6 = c.mask[:6].clone()
    c.dec.run(q, c.kv, mask=mask6, out=o)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph2):
        c.dec.run(q, c.kv, mask=mask6, out=o)
    c.plan()
    o.fill_(5.0)
    graph2.replay()
    torch.cuda.synchronize()
    assert (o == 5).all() and c.dec.device_error() == 2


def test_captured_under_an_empty_plan():
    # a step captured before any request has query tokens replays under later plans that have
    c = Case(lens=(60, 700), drafts=(5, 12), rows=20)
    none = np.zeros(3, np.int32)
    c.dec.plan(none, c.indptr, c.indices, c.last)
    out, lse = torch.zeros_like(c.q), torch.zeros(20, 8, device="cuda")
    bare, bare_lse = torch.zeros_like(c.q), torch.zeros(20, 8, device="cuda")
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, lse=lse)
    with torch.cuda.graph(graph2):   # (no mask: does for no tree)
        c.dec.run(c.q, c.kv, out=bare, lse=bare_lse)
    graph.replay()
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == 0).all() and c.dec.device_error() == 0
    c.plan()
    graph.replay()
    c.check((out, lse))
    assert (out[17:] == 0).all()
    graph2.replay()
    torch.cuda.synchronize()
    assert (bare == 0).all() and (bare_lse == 0).all()
    assert c.dec.device_error() == pkd.DEV_ERR_BOUNDS


@pytest.mark.parametrize("cap,scale,magnitude", [
    (1e6, None, 1.0), (1e6, None, 1e4), (1e4, 1e-2, 1.0), (1e4, 1e-3, 1e3), (2.0 ** 96, 1.0, 1.0),
    (2.0 ** 96, 2.0 ** -30, 2.0 ** 30), (2.0 ** -30, None, 1.0), (1e-3, 1e6, 1.0), (50.0, None, 40.0)])
@pytest.mark.parametrize("slopes", [False, True])
def test_caps_of_any_size(cap, scale, magnitude, slopes):
    c = Case(lens=(300, 40), drafts=(9, 5), cap=cap, scale=scale, magnitude=magnitude, slopes=slopes)
    out, lse = c.run()
    ro, rl = c.reference()
    assert c.dec.device_error() == 0
    # a score is an fp32 sum of 128 products and 6 more roundings, the cap's polynomial within 2^-23
    # of itself and past 0.4 of the cap within 2^-21 of the score (2^-22 of the cap at least); the
    # largest score is under cap and under 128 * 36 * scale * magnitude.  Sums: 300 * 2^-24.
    scale = 128 ** -0.5 if scale is None else scale
    most = min(cap, scale * float(torch.einsum("nhd,nhd->nh", c.q.double(), c.q.double()).max()) ** 0.5
               * float(c.kv[:, 0].double().pow(2).sum(-1).max()) ** 0.5)
    off = most * (128 * 2.0 ** -24 + 2.0 ** -20) + 300 * 2.0 ** -24 + 2.0 ** -23 * float(rl.abs().max())
    assert (lse.double() - rl).abs().max() <= off
    # weights move by e^(2 off), P by 2^-8
    top = float(c.kv.float().abs().max())
    assert (out.double() - ro).abs().max() <= 2 * top * (math.exp(min(2 * off, 20.0)) - 1) + \
        1.1 * 2 ** -8 * (top + float(ro.abs().max()))


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_steep_slopes(sign):
    # a bias that changes by more than fp32's exponents hold from one token of a round to the next
    # ones, scores against it, and drafts that see none of the newest tokens
    c = Case(hq=4, hkv=2, lens=(256 + 3, 700), drafts=(3, 5), slopes=True, magnitude=0.0)
    c.slopes = sign * torch.tensor([8.0, 2.0, 1.5, 40.0], device="cuda")
    c.mask[:3] = 0
    c.q[..., 0] = 30.0
    score = torch.where(torch.arange(16, device="cuda") == (0 if sign > 0 else 15), 40.0, -40.0)
    c.kv[:, 0, :, :, 0] = score[None, :, None]
    out, lse = c.run()
    ro, rl = c.reference()
    # scores of 106 and biases of up to 28,000: exponents off by 2^-23 of those
    off = 4 * 2.0 ** -24 * (106 + 40 * 700) + 2.0 ** -23 * float(rl.abs().max())
    assert c.dec.device_error() == 0 and torch.isfinite(lse).all()
    assert (lse.double() - rl).abs().max() <= off
    top = float(c.kv[:, 1].float().abs().max())
    assert (out.double() - ro).abs().max() <= 2 * top * (math.exp(2 * off) - 1) + \
        1.1 * 2 ** -8 * (top + float(ro.abs().max()))


@pytest.mark.parametrize("lens,drafts", [((300, 40), (9, 5)), ((3000,), (4,))])
def test_large_values_under_a_cap(lens, drafts):
    # scores at the cap and values near bf16's largest: a weighted mean of them is finite
    c = Case(lens=lens, drafts=drafts, cap=60.0, magnitude=60.0, seed=3)
    c.kv[:, 1] *= 2.0 ** 100
    out, lse = c.run()
    ro, rl = c.reference()
    assert c.dec.device_error() == 0 and torch.isfinite(out.float()).all()
    # scores off by 60 * (128 * 2^-24 + 2^-20): weights by 2 e-3 of themselves at most; P by 2^-8
    off = 60.0 * (128 * 2.0 ** -24 + 2.0 ** -20) + 3000 * 2.0 ** -24
    top = float(c.kv[:, 1].float().abs().max())
    assert (lse.double() - rl).abs().max() <= off
    assert (out.double() - ro).abs().max() <= 2 * top * (math.exp(2 * off) - 1) + \
        1.1 * 2 ** -8 * (top + float(ro.abs().max()))


@pytest.mark.parametrize("causal", [False, True])
def test_blocks_in_pieces(causal):
    # more than L2 holds, shared by a request's row blocks: cut alike, merged from many parts
    c = Case(hq=8, hkv=1, page=64, lens=(400_000, 70), drafts=(40, 3), causal=causal)
    info = c.dec.plan_info()
    assert info["num_units"] == 40 and info["num_slots"] > 40 * 8
    c.check()


@pytest.mark.parametrize("kw", [dict(), dict(cap=50.0), dict(slopes=True), dict(cap=50.0, slopes=True),
                                dict(cap=30.0, scale=1.0)])
def test_rows_of_one_token_are_its_value(kw):
    # one weight, 1: no rounding but the value's own
    c = Case(lens=(40, 700, 2), drafts=(4, 90, 1), window=1, causal=True, **kw)
    out, lse = c.run()
    mine = [torch.from_numpy(c.indices[c.indptr[b]:c.indptr[b + 1]]).long().cuda() for b in range(3)]
    v = torch.cat([c.kv[mine[b], 1].reshape(-1, 2, D)[c.lens[b] - c.drafts[b]:c.lens[b]] for b in range(3)])
    assert torch.equal(out, v.repeat_interleave(4, 1)) and c.dec.device_error() == 0
    c.check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (3, 3), (8, 2), (32, 8), (64, 8)])
@pytest.mark.parametrize("layout,page", [("NHD", 16), ("HND", 48), ("NHD", 256)])
def test_e4m3_heads_and_layouts(hq, hkv, layout, page):
    Case(hq=hq, hkv=hkv, layout=layout, page=page, lens=(37, 16, 5, 300, 900), drafts=(4, 3, 5, 9, 70), seed=hq,
         fp8=True).check()


@pytest.mark.parametrize("kw", [dict(), dict(cap=30.0), dict(slopes=True), dict(cap=30.0, slopes=True),
                                dict(window=1), dict(window=150), dict(cap=50.0, window=600)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,drafts", [((3000, 40, 1500), (12, 3, 40)), ((129, 2, 1, 640, 17), (1, 2, 1, 128, 16))])
def test_e4m3_scores(kw, causal, lens, drafts):
    Case(lens=lens, drafts=drafts, causal=causal, fp8=True, **kw).check()


def test_e4m3_many_rounds_and_items():
    Case(hq=32, hkv=8, lens=(20_000, 3, 9_000, 2_000), drafts=(70, 1, 33, 5), fp8=True).check()
    Case(hq=8, hkv=2, lens=(700,) * 40, drafts=(20,) * 40, fp8=True, num_ctas=4).check()


@pytest.mark.parametrize("split", [False, True])
def test_e4m3_what_is_masked_may_hold_anything(split):
    kw = dict(min_chunk_tokens=128, alpha=0) if split else {}
    c = Case(lens=(700, 60), drafts=(12, 5), fp8=True, window=300, **kw)
    see = [c.sees(b)[0].any(0).cpu() for b in range(2)]
    raw = c.kv.view(torch.uint8)
    for b in range(2):
        for t in (~see[b]).nonzero()[:, 0].tolist() + list(range(c.lens[b], 16 * (-(-c.lens[b] // 16)))):
            raw[int(c.indices[c.indptr[b] + t // 16]), :, t % 16] = 0x7F   # NaN
    # and a draft that only itself sees
    c.mask[3], c.mask[4:12, 0] = torch.tensor([8], device="cuda").int(), c.mask[4:12, 0] & ~8
    raw[int(c.indices[c.indptr[0] + 691 // 16]), :, 691 % 16] = 0xFF
    out, lse = c.run()
    mine = [i for i in range(17) if i != 3]
    ro, rl = c.reference()
    assert torch.isnan(out[3]).all() and torch.isnan(lse[3]).all()
    assert (out[mine].double() - ro[mine]).abs().max() <= 1.1 * 2 ** -8 * 8 and c.dec.device_error() == 0
    assert (lse[mine].double() - rl[mine]).abs().max() <= 2e-4


@pytest.mark.parametrize("kv_dtype", ["bf16", "e4m3"])
def test_first_context_of_a_process(kv_dtype):
    code = f"""
import paged_kv_decode_host_gb300 as pkd
d = pkd.BatchTreeDecodeWithPagedKVCache(8, 2, 128, 16, max_tokens=4, max_num_pages=4, num_pages=4, kv_dtype={kv_dtype!r})
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=120)


def test_e4m3_every_value():
    # a row of one token is that token's values, whatever they are
    c = Case(hq=2, hkv=2, lens=(4,), drafts=(4,), window=1, causal=True, fp8=True)
    raw = c.kv.view(torch.uint8)
    page = int(c.indices[0])
    raw[page, 0] = 0
    raw[page, 1, :4] = torch.arange(1024, device="cuda").fmod(256).to(torch.uint8).view(4, 2, D)
    out, lse = c.run()
    want = (c.kv[page, 1, :4].float() * 0.25).bfloat16()
    assert torch.equal(out.isnan(), want.isnan()) and int(want.isnan().sum()) == 8
    assert torch.equal(out.nan_to_num(), want.nan_to_num()) and c.dec.device_error() == 0


def test_e4m3_captured_and_as_bytes():
    c = Case(lens=(700, 90, 40), drafts=(12, 9, 4), fp8=True)
    want = c.run()
    c.kv = c.kv.view(torch.uint8)
    got = c.run()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, lse=lse)
    graph.replay()
    assert torch.equal(want[0], out) and torch.equal(want[1], lse)
    with pytest.raises(ValueError):
        c.dec.run(c.q, c.kv.bfloat16(), mask=c.mask)
    for bad in (dict(k_scale=0.0), dict(v_scale=float("inf")), dict(k_scale=float("nan")), dict(v_scale=-1.0)):
        with pytest.raises(pkd.PkdError, match="INVALID"):
            c.dec.run(c.q, c.kv, mask=c.mask, **bad)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(window=1), dict(slopes=True), dict(causal=True, window=130)])
def test_same_bits_whatever_ran_before(kw, fp8):
    # capped scores choose their way by their size: by those that count only, not by what other
    # launches, or tokens and rows that nobody sees, left behind
    c = Case(lens=(863, 21, 70), drafts=(40, 17, 5), cap=30.0, fp8=fp8, rows=70, **kw)
    other = [Case(lens=(500, 900), drafts=(30, 60), magnitude=m, seed=3) for m in (30.0, 1.0)]
    first = c.run()
    for k in range(6):
        other[k & 1].run()
        if k == 3:   # rows behind the plan's, slots behind the requests' ends
            c.q[62:] = 1e6
            raw = c.kv.view(torch.uint8)
            for b in range(3):
                for t in range(c.lens[b], 16 * -(-c.lens[b] // 16)):
                    raw[int(c.indices[c.indptr[b] + t // 16]), :, t % 16] = 0x7A   # 320, or 3e35
        again = c.run()
        assert torch.equal(first[0][:62], again[0][:62]) and torch.equal(first[1][:62], again[1][:62])
    assert c.dec.device_error() == 0


def test_two_contexts_at_once():
    # each on a stream of its own, one of them an E4M3 cache, with copies of the plans on the way
    cases = [Case(lens=(3000, 700, 90), drafts=(40, 9, 3), cap=30.0, seed=1),
             Case(lens=(2500, 60, 1200), drafts=(17, 5, 70), slopes=True, fp8=True, seed=2)]
    want = [[x.clone() for x in c.run()] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for k in range(12):
        for c, s, g in zip(cases, streams, got):
            with torch.cuda.stream(s):
                if k % 4 == 3:
                    c.plan()
                g.append(c.run())
    torch.cuda.synchronize()
    for c, w, g in zip(cases, want, got):
        assert all(torch.equal(x, y) for one in g for x, y in zip(one, w)) and c.dec.device_error() == 0


def test_pools_past_32_bits():
    """Pages whose elements lie past 2^31."""
    c = Case(hq=8, hkv=8, lens=(70, 40), drafts=(5, 3), window=60)
    far = 70_000
    kv = torch.zeros(far + c.pool, 2, 16, 8, D, dtype=torch.bfloat16, device="cuda")
    kv[far:] = c.kv
    dec = pkd.BatchTreeDecodeWithPagedKVCache(8, 8, D, 16, max_tokens=8, max_num_pages=len(c.indices),
                                              num_pages=far + c.pool)
    dec.plan(c.q_indptr, c.indptr, c.indices + far, c.last, window=60)
    c.check(dec.run(c.q, kv, mask=c.mask, depths=c.depths))
    assert dec.device_error() == 0


def test_depths_of_any_size():
    c = Case(lens=(300,), drafts=(6,), slopes=True, window=400, seed=6)
    c.depths[:] = torch.tensor([0, 90, -5, 150, 2000, 10], dtype=torch.int32)
    c.check()
    c = Case(lens=(300,), drafts=(3,), window=7, seed=6)
    c.depths[:] = torch.tensor([2 ** 31 - 1, 0, 3], dtype=torch.int32)
    c.check()


def test_refusals():
    c = Case()
    q, kv, mask = c.q, c.kv, c.mask
    for kw in (dict(mask=None), dict(mask=mask[:-1]), dict(mask=mask.float()), dict(mask=mask, depths=c.depths.long()),
               dict(mask=mask, slopes=torch.zeros(3, device="cuda")), dict(mask=mask, lse=torch.zeros(3, device="cuda")),
               dict(mask=mask[:, :0])):
        with pytest.raises((ValueError, pkd.PkdError)):
            c.dec.run(q, kv, **kw)
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(score_cap=-1.0), dict(score_cap=float("inf"))):
        with pytest.raises(pkd.PkdError, match="INVALID"):
            c.dec.run(q, kv, mask=mask, **kw)
    for args in ((q[:-1], kv), (q.float(), kv), (q, kv[:-1]), (q.transpose(0, 1), kv), (q.cpu(), kv)):
        with pytest.raises((ValueError, pkd.PkdError)):
            c.dec.run(*args, mask=mask)
    c.dec.plan(c.q_indptr, c.indptr, c.indices, c.last, causal=True)
    for kw in (dict(mask=mask), dict(depths=c.depths)):
        with pytest.raises(ValueError):
            c.dec.run(q, kv, **kw)
    for call in (c.dec.plan_shared, c.dec.plan_cascade, c.dec.accumulate_weights, c.dec.capture):
        with pytest.raises(pkd.PkdError):
            call()
    fresh = pkd.BatchTreeDecodeWithPagedKVCache(8, 2, D, 16, max_tokens=4, max_num_pages=4, num_pages=4)
    with pytest.raises(pkd.PkdError, match="NO_PLAN"):
        fresh.run(q, kv)
    with pytest.raises(pkd.PkdError):
        pkd.BatchTreeDecodeWithPagedKVCache(8, 2, 64, 16, max_tokens=4, max_num_pages=4, num_pages=4)
    with pytest.raises(pkd.PkdError):
        pkd.BatchTreeDecodeWithPagedKVCache(8, 2, D, 8, max_tokens=4, max_num_pages=4, num_pages=4)
    with pytest.raises(ValueError):
        pkd.BatchTreeDecodeWithPagedKVCache(8, 2, D, 16, max_tokens=4, max_num_pages=4, num_pages=4, kv_layout="x")
    assert c.dec.device_error() == 0


@pytest.mark.parametrize("kw", [dict(), dict(cap=30.0), dict(slopes=True), dict(window=1_900_000), dict(fp8=True)])
def test_recomputed_rows_outlast_no_wait(kw):
    # One CTA and two items, the first of 2,000,000 tokens: its rows that do not see a draft whose value is
    # not finite are summed again (1.3 us a token; 3.8 it was, 7.6 s) while the CTA's other warps are at the
    # next item already, in waits of 2 s
    n, page = 2_000_000, 4096
    c = Case(hq=8, hkv=1, page=page, lens=(n, 500), drafts=(8, 8), num_ctas=1, **kw)
    for w in range(16):
        c.mask[w] = 1 << (w % 8)
    c.kv[:, 1] = (c.kv[:, 1].float() + 8.0).to(c.kv.dtype)
    clean = [x.clone() for x in c.run()]
    assert c.dec.device_error() == 0
    for b in range(2):
        at, slot = divmod(c.lens[b] - 1, page)
        c.kv.view(torch.uint8)[int(c.indices[c.indptr[b] + at]), 1, slot] = 0x7F if c.fp8 else 0xFF   # NaN
    out, lse = c.run()
    assert c.dec.device_error() == 0 and torch.equal(lse, clean[1])
    top = 15.0 * (0.25 * 2 if c.fp8 else 1.0)
    for i in range(16):
        if i % 8 == 7:
            assert torch.isnan(out[i]).all()
        else:   # P in bf16 or in fp32, both results rounded to bf16
            assert (out[i].float() - clean[0][i].float()).abs().max() <= 1.1 * 2 ** -8 * 3 * top


def test_values_near_the_largest_that_is_finite():
    # weights that are not yet divided by their sum pass fp32's range, their mean does not
    c = Case(lens=(3000, 40), drafts=(5, 3), seed=4, num_ctas=1)
    c.kv[:, 1] = (c.kv[:, 1].float().sign() * 2.0 ** 127 * 1.9).bfloat16()
    c.kv[:, 1, ::2] *= 0.75
    out, lse = c.run()
    assert c.dec.device_error() == 0 and torch.isfinite(out.float()).all()
    ro, _ = c.reference()
    top = float(c.kv[:, 1].float().abs().max())
    assert (out.double() - ro).abs().max() <= 1.1 * 2 ** -8 * (top + float(ro.abs().max()))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("power", [-100, -60, 30])
def test_scales_of_values_of_any_size(power, fp8):
    # scores at their cap: sums of weights about 2^97, by which a small scale alone would vanish; powers
    # of two change no bit of the result but its exponent
    c = Case(lens=(3000, 500), drafts=(4, 3), cap=60.0, magnitude=60.0, seed=3, fp8=fp8, num_ctas=2)
    c.scales = dict(k_scale=1.0, v_scale=1.0)
    out, lse = (x.clone() for x in c.run())
    c.scales["v_scale"] = 2.0 ** power
    small, same = c.run()
    assert torch.equal(small.double(), out.double() * 2.0 ** power) and torch.equal(lse, same)
    assert out.double().abs().max() > 0.1 and c.dec.device_error() == 0


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 127, 128, 129, 300, 900])
@pytest.mark.parametrize("causal", [False, True])
def test_windows_within_long_pieces(window, causal):
    # rows whose window ends among the query tokens themselves, chains and trees of which depths say nothing
    Case(hq=4, hkv=2, lens=(900, 640, 70), drafts=(700, 640, 70), causal=causal, depths=False, window=window).check()


def test_results_on_the_queries_are_refused():
    # (a row that is summed again would read the results of its other dims as its query)
    c = Case(lens=(70, 40), drafts=(5, 3))
    both = torch.zeros(16, 8, D, dtype=torch.bfloat16, device="cuda")
    both[:8] = c.q
    want, lse = c.run()
    got, _ = c.dec.run(both[:8], c.kv, mask=c.mask, depths=c.depths, out=both[8:])   # (beside one another)
    assert torch.equal(got, want)
    for q, out in ((both[:8], both[:8]), (both[:8], both[1:9]), (both[8:], both[7:15])):
        with pytest.raises(pkd.PkdError, match="INVALID"):
            c.dec.run(q, c.kv, mask=c.mask, depths=c.depths, out=out)
    assert c.dec.device_error() == 0
