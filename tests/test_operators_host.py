"""Refusals of the latent, append, weight and eviction entry points, without a GPU."""
import ctypes

import pytest

import paged_kv_decode_host_gb300 as pkd

INVALID, SHAPE, SMALL, CAPACITY = -1, -3, -4, -7


@pytest.fixture(scope="module")
def lib():
    pkd.build()
    return pkd.load()


def layout_status(lib, **kw):
    args = dict(num_qo_heads=16, num_kv_heads=1, head_dim=512, page_size=16, max_batch=4,
                max_num_pages=16, num_pages=16, num_ctas=8, flags=pkd.FLAG_LATENT)
    args.update(kw)
    off = (ctypes.c_int64 * 6)()
    return lib.pkd_schedule_layout(ctypes.byref(pkd.make_config(**args)), off)


def test_latent_configurations(lib):
    for heads in (1, 16, 20, 64, 65, 127, 128):
        assert layout_status(lib, num_qo_heads=heads) == 0
    for kw in (dict(num_qo_heads=0), dict(num_qo_heads=129), dict(num_kv_heads=2), dict(head_dim=576),
               dict(head_dim=128), dict(page_size=8), dict(page_size=24), dict(page_size=1 << 21)):
        assert layout_status(lib, **kw) == SHAPE, kw
    for extra in (1, 2, 4, 8, 16, 32, 64, 128, 256):
        assert layout_status(lib, flags=pkd.FLAG_LATENT | extra) == INVALID, extra
    assert layout_status(lib, num_pages=0) == INVALID


def test_latent_plan_keeps_token_counts_in_32_bits():
    """A table that names one large page often: tokens past a request's end must count in 32 bits, too."""
    import numpy as np
    page = 1 << 20
    cfg = pkd.make_config(16, 1, 512, page, 1, 2048, 1, num_ctas=8, flags=pkd.FLAG_LATENT)
    table = lambda n, last: (np.array([0, n], np.int32), np.zeros(n, np.int32), np.array([last], np.int32))
    for n, last in ((2048, page), (2048, page - 1), (2048, page - 1023)):
        with pytest.raises(pkd.PkdError, match="CAPACITY"):
            pkd.plan_host(cfg, *table(n, last))
    pkd.plan_host(cfg, *table(2048, page - 1024 - 1))


def evict_status(lib, **kw):
    a = dict(layers=2, kv=[256, 512], weights=[1024, 1088], positions=[2048, 2112], indptr=64, indices=64,
             num_indices=4, last=64, seen=64, batch=1, max_len=100, budget=10, sinks=1, recent=2,
             per_head=1, num_pages=4, page_size=16, hkv=8, dim=128, flags=0, ws=None, ws_bytes=0,
             err=None)
    a.update(kw)
    n = len(a["kv"])
    arr = lambda x: (ctypes.c_void_p * n)(*x) if x is not None else None
    return lib.pkd_evict_kv(a["layers"], arr(a["kv"]), arr(a["weights"]), arr(a["positions"]),
                            a["indptr"], a["indices"], a["num_indices"], a["last"], a["seen"],
                            a["batch"], a["max_len"], a["budget"], a["sinks"], a["recent"],
                            a["per_head"], a["num_pages"], a["page_size"], a["hkv"], a["dim"],
                            a["flags"], a["ws"], a["ws_bytes"], a["err"], None)


def test_evict_refusals(lib):
    """Every call returns before it reaches the device (the addresses are none)."""
    for kw in (dict(layers=0), dict(layers=129), dict(batch=-1), dict(max_len=-1), dict(budget=0),
               dict(sinks=-1), dict(recent=-1), dict(sinks=5, recent=6), dict(per_head=2),
               dict(num_pages=0), dict(page_size=0), dict(hkv=0), dict(hkv=1025), dict(dim=0),
               dict(dim=12), dict(dim=128, hkv=256), dict(flags=1), dict(flags=pkd.FLAG_LATENT),
               dict(indptr=None), dict(indices=None), dict(last=None), dict(seen=None),
               dict(num_indices=-1), dict(err=2), dict(kv=[256, 256]), dict(kv=[256, 0]),
               dict(kv=[256, 520]), dict(weights=[1024, 1024]), dict(weights=[1024, 1090]),
               dict(positions=[2048, 2048]), dict(weights=[0, 1024]), dict(positions=[0, 2048])):
        assert evict_status(lib, **kw) == INVALID, kw
    assert evict_status(lib, max_len=262_145) == CAPACITY
    # nothing is over the budget, or no request: no launch
    assert evict_status(lib, max_len=10) == 0 and evict_status(lib, batch=0) == 0
    # long requests leave bitmaps in a workspace
    need = lib.pkd_evict_workspace_bytes(2, 1, 5000, 1000, 1, 8)
    assert need == 2 * 8 * ((5000 + 31) // 32) * 4
    assert evict_status(lib, max_len=5000, budget=1000) == INVALID
    assert evict_status(lib, max_len=5000, budget=1000, ws=256, ws_bytes=need - 1) == SMALL
    assert evict_status(lib, max_len=5000, budget=1000, ws=264, ws_bytes=need) == INVALID
    assert lib.pkd_evict_workspace_bytes(2, 1, 1025, 1024, 1, 8) == 0
    assert lib.pkd_evict_workspace_bytes(0, 1, 5000, 1000, 1, 8) == 0


def test_append_latent_refusals(lib):
    def status(latent=256, ls=512, rope=256, rs=64, rows=64, at=64, n=2, indptr=64, indices=64, nnz=1,
               last=64, batch=1, cache=256, pages=1, page=16, err=None):
        return lib.pkd_append_latent(latent, ls, rope, rs, rows, at, n, indptr, indices, nnz, last,
                                     batch, cache, pages, page, err, None)
    for kw in (dict(latent=None), dict(latent=258), dict(rope=None), dict(rope=264), dict(ls=511),
               dict(ls=516), dict(rs=63), dict(rs=68), dict(rows=None), dict(at=None), dict(n=-1),
               dict(indptr=None), dict(indices=None), dict(nnz=-1), dict(last=None), dict(batch=-1),
               dict(cache=None), dict(cache=264), dict(pages=0), dict(page=0), dict(err=2)):
        assert status(**kw) == INVALID, kw
    assert status(n=0, latent=None) == 0


def test_accumulate_without_context(lib):
    assert lib.pkd_accumulate_weights(None, 256, 256, 256, 256, None, None, None, 1.0, 0, None) == INVALID


def test_binding_refuses_before_the_library():
    import torch
    kv = torch.zeros(2, 2, 16, 1, 16, dtype=torch.bfloat16)
    w, p = torch.zeros(2, 1, 16), torch.zeros(2, 1, 16, dtype=torch.int32)
    t = [torch.zeros(2, dtype=torch.int32)] * 4
    with pytest.raises(TypeError):
        pkd.evict_kv([kv], [w], [p], *t, 4, max_len=8)          # not on the GPU
    with pytest.raises(ValueError):
        pkd.evict_kv([], [], [], *t, 4, max_len=8)
    with pytest.raises(TypeError):
        pkd.append_latent(w, w, *t, t[0], torch.zeros(1, 16, 576))
