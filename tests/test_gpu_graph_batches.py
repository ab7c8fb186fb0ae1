"""Calls that the caller captured, replayed under later plans of fewer and of more requests: what the
tensors of the captured call have no room for is refused on the device."""
import numpy as np
import pytest
import torch

import paged_kv_decode_host_gb300 as pkd
from test_gpu_evict import Step, near
from test_gpu_latent import DIM, ROW, SCALE, close, reference, table

gpu = pytest.mark.gpu


def captured(call):
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def first_of(t, n):
    return t[0][:n + 1], t[1][:t[0][n]], t[2][:n]


@gpu
@pytest.mark.parametrize("heads,lens", [(16, [100, 40, 7]), (128, [3000, 2000, 500])])
def test_latent_graph_under_plans_of_other_batches(heads, lens):
    page = 16
    t = table(lens + [90, 2500], page)
    q = torch.randn(3, heads, ROW, device="cuda").bfloat16()
    cache = torch.randn(t[3], page, ROW, device="cuda").bfloat16()
    out = torch.zeros(3, heads, DIM, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(3, heads, device="cuda")
    dec = pkd.BatchLatentDecodeWithPagedCache(heads, DIM, 64, page, scale=SCALE, max_batch=5,
                                              max_num_pages=len(t[1]), num_pages=t[3])
    dec.plan(*first_of(t, 3))
    g = captured(lambda: dec.run(q, cache, out=out, lse=lse))
    top = cache.abs().max().double()
    for n in (3, 5, 2, 4, 3):
        dec.plan(*first_of(t, n))
        out.zero_(), lse.zero_()
        g.replay()
        m = n if n <= 3 else 0
        assert dec.device_error() == (0 if m else pkd.DEV_ERR_BOUNDS)
        assert (out[m:] == 0).all() and (lse[m:] == 0).all()
        if m:
            close((out[:m], lse[:m]), reference(q[:m], cache, lens[:m], t, page), top)


@gpu
def test_weights_graph_under_plans_of_other_batches():
    lens = [40, 300, 9]
    s = Step(2, 4, lens + [77, 1000], 16, seed=1)
    q, lse = s.q[:3].clone(), s.lse[:3].clone()
    s.dec.plan(*first_of(s.t, 3))
    w = torch.zeros(s.per_slot, device="cuda")
    g = captured(lambda: s.dec.accumulate_weights(q, s.kv, lse, w))
    s.lens = lens
    want = s.expected(torch.zeros_like(w), [0] * 3)
    for n in (3, 5, 2, 4):
        s.dec.plan(*first_of(s.t, n))
        w.zero_()
        g.replay()
        m = n if n <= 3 else 0
        assert s.dec.device_error() == (0 if m else pkd.DEV_ERR_BOUNDS)
        for i in range(5):
            got = w[s.pages_of(i)]
            near(got, want[s.pages_of(i)] if i < m else torch.zeros_like(got, dtype=torch.double))
