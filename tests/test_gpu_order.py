"""Calls whose kernels are launched while the kernel before still runs and has already let them:
what that one reads stays until it has read it, what it writes is waited for."""
import numpy as np
import pytest
import torch

import paged_kv_decode_host_gb300 as pkd
from test_gpu_evict import Step
from test_gpu_latent import DIM, ROW, SCALE, table

gpu = pytest.mark.gpu
TIMES = 25


def device_table(t):
    return [torch.from_numpy(x).cuda() for x in t[:3]]


@gpu
@pytest.mark.parametrize("heads,lens", [(16, [3000] * 64), (128, [5000] * 16), (40, [60_000, 30])])
def test_append_over_rows_that_a_latent_decode_reads(heads, lens):
    """Decode, then other rows for every request's last token and for one in its middle; again and again
    with nothing between the calls, against the same calls one at a time."""
    t, page = table(lens, 16), 16
    gen = torch.Generator("cuda").manual_seed(heads)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    q, cache = rand(len(lens), heads, ROW), rand(t[3], page, ROW)
    dec = pkd.BatchLatentDecodeWithPagedCache(heads, DIM, 64, page, scale=SCALE, max_batch=len(lens),
                                              max_num_pages=len(t[1]), num_pages=t[3])
    dec.plan(*t[:3])
    rows = torch.arange(len(lens), device="cuda").int().repeat(2)
    at = torch.tensor([n - 1 for n in lens] + [n // 2 for n in lens], device="cuda").int()
    new = [rand(2 * len(lens), ROW) * 3 for _ in range(TIMES)]
    outs = [torch.empty(len(lens), heads, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(TIMES)]
    lses = [torch.empty(len(lens), heads, device="cuda") for _ in range(TIMES)]
    d, first = device_table(t), cache.clone()

    def steps(wait):
        cache.copy_(first)
        torch.cuda.synchronize()
        if not wait:
            torch.cuda._sleep(20_000_000)   # all is launched before the first one runs
        for i in range(TIMES):
            dec.run(q, cache, out=outs[i], lse=lses[i])
            if wait:
                torch.cuda.synchronize()
            pkd.append_latent(new[i][:, :DIM], new[i][:, DIM:], rows, at, *d, cache)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [x.clone() for x in outs + lses + [cache]]

    want = steps(True)
    assert not torch.equal(want[0], want[1])
    for a, b in zip(steps(False), want):
        assert torch.equal(a, b)
    assert dec.device_error() == 0


@gpu
@pytest.mark.parametrize("lens,budget", [([3000] * 40, 1500), ([700] * 60, 697), ([40_000, 900], 20_000)])
def test_weights_and_evictions_behind_a_decode(lens, budget):
    """Decode, its weights, the eviction by them that moves the rows it read, and a decode of what
    stayed: with nothing between the calls, against one at a time."""
    s = Step(8, 4, lens, 16, seed=len(lens))
    d, n = device_table(s.t), torch.tensor(lens, dtype=torch.int32, device="cuda")
    after = table([min(x, budget) for x in lens], 16)
    kept = [s.t[1][s.t[0][i]:s.t[0][i] + c] for i, c in enumerate(np.diff(after[0]))]
    late = pkd.BatchDecodeWithPagedKVCache(32, 8, 128, 16, max_batch=len(lens), max_num_pages=len(s.t[1]),
                                           num_pages=s.t[3])
    late.plan(after[0], np.concatenate(kept).astype(np.int32), after[2])
    pos = torch.zeros(s.per_slot, dtype=torch.int32, device="cuda")
    first, zero = s.kv.clone(), torch.zeros_like(s.weights)
    keep = []

    def steps(wait):
        got = []
        gap = torch.cuda.synchronize if wait else lambda: None
        torch.cuda.synchronize()
        if not wait:
            torch.cuda._sleep(20_000_000)
        for _ in range(8):
            kv, w, p = first.clone(), zero.clone(), pos.clone()
            gap()
            out, lse = s.dec.run(s.q, kv)
            gap()
            s.dec.accumulate_weights(s.q, kv, lse, w, positions=p, new_tokens=n, seen=n)
            gap()
            pkd.evict_kv([kv], [w], [p], *d, n, budget, max_len=max(lens), sinks=2, recent=16)
            gap()
            out2, lse2 = late.run(s.q, kv)
            gap()
            got.append([out, lse, kv, w, p, out2, lse2])
        torch.cuda.synchronize()
        return got

    want = steps(True)[0]
    for got in steps(False):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert s.dec.device_error() == 0 and late.device_error() == 0
