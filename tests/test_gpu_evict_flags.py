"""What an eviction flags where nothing may be over the budget."""
import numpy as np
import pytest
import torch

import paged_kv_decode_host_gb300 as pkd
from test_gpu_evict import evict_case, run_evict, same

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("max_len,budget", [(30, 40), (40, 40), (5, 300)])
def test_wrong_rows_and_longer_requests_are_flagged_within_the_budget(max_len, budget):
    """max_len at most the budget: nothing is cut, and a request that is longer all the same, or
    whose row is wrong, is flagged as elsewhere."""
    def err(lens, last=None, indices=None):
        t, kvs, ws, ps, seen = evict_case(2, 16, lens, budget, layers=2, seed=3)
        row = (t[0], t[1] if indices is None else t[1][:indices], t[2] if last is None else np.array(last, np.int32))
        got = run_evict(row, kvs, ws, ps, seen, budget, torch.bfloat16, max_len=max_len)
        same(got, (kvs, ws, ps))
        return got[3]

    many = [min(max_len, 1 + k % 40) for k in range(300)]
    assert err([max_len, 1]) == 0 and err(many) == 0
    assert err([max_len + 1, 1]) == pkd.DEV_ERR_BOUNDS
    assert err(many[:-1] + [max_len + 1]) == pkd.DEV_ERR_BOUNDS
    assert err([1, 2], last=[1, 17]) == pkd.DEV_ERR_BOUNDS
    assert err([1, 2], last=[0, 2]) == pkd.DEV_ERR_BOUNDS
    assert err([1, 2], indices=1) == pkd.DEV_ERR_BOUNDS


@gpu
def test_flags_within_the_budget_wait_for_the_table():
    """The table may be the kernel's before the call."""
    t, kvs, ws, ps, seen = evict_case(1, 16, [50], 60)
    d = [torch.from_numpy(x).cuda() for x in t[:3]]
    g = [torch.from_numpy(kvs[0]).cuda().view(torch.bfloat16)], [torch.from_numpy(ws[0]).cuda()], [torch.from_numpy(ps[0]).cuda()]
    seen = torch.tensor(seen, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    right = d[2].clone()
    d[2].fill_(99)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000)
    torch.mul(right, 1, out=d[2])
    pkd.evict_kv(*g, *d, seen, 60, max_len=50, err=err)
    assert err.item() == 0
