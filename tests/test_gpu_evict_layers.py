"""Evictions of every layer of a model at once: thousands of jobs, with the moves in the choosing
kernel and in one of their own, for both cache types and layouts."""
import pytest
import torch

from test_gpu_evict import evict_case, evict_reference, run_evict, same

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("layers,hkv,lens,budget,dtype,layout,per_head", [
    (32, 8, [1300, 20, 1200, 700, 1299, 601, 600, 1100], 600, torch.float8_e4m3fn, "HND", True),
    (128, 2, [1300, 90, 1111], 640, torch.bfloat16, "NHD", False),
    (128, 8, [70, 64, 1, 90, 65], 64, torch.float8_e4m3fn, "NHD", True),
    (80, 1, [1025] * 12, 1020, torch.bfloat16, "HND", True),
])
def test_many_layers(layers, hkv, lens, budget, dtype, layout, per_head):
    t, kvs, ws, ps, seen = evict_case(hkv, 16, lens, budget, layers=layers, dtype=dtype, layout=layout, d=16,
                                      seed=layers + hkv)
    got = run_evict(t, kvs, ws, ps, seen, budget, dtype, max_len=max(lens), sinks=3, recent=17,
                    per_head=per_head, kv_layout=layout)
    evict_reference(kvs, ws, ps, t, lens, seen, budget, 16, layout, 3, 17, per_head)
    same(got, (kvs, ws, ps))
    assert got[3] == 0
