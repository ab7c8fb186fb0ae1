"""What plans write, and what contexts upload, behind the page list."""
import ctypes

import numpy as np
import pytest

import paged_kv_decode_host_gb300 as pkd
from test_gpu_latent import table

gpu = pytest.mark.gpu
MARK = 0x5a5a5a5a


@pytest.mark.parametrize("flags,heads,kv_heads,dim", [
    (0, 32, 8, 128), (pkd.FLAG_KV_FP8, 8, 8, 128), (pkd.FLAG_LATENT, 40, 1, 512)])
@pytest.mark.parametrize("lens", [[], [1], [100, 17, 3000, 16], [5] * 30])
def test_host_plans_write_the_words_they_name(flags, heads, kv_heads, dim, lens):
    """schedule_words of them and no more, in a buffer of the page list's capacity."""
    lib = pkd.load()
    t = table(lens, 16) if lens else (np.zeros(1, np.int32), np.zeros(0, np.int32), np.zeros(0, np.int32), 1)
    cfg = pkd.make_config(heads, kv_heads, dim, 16, 40, 400, t[3], num_ctas=20, flags=flags)
    off = pkd.schedule_layout(cfg)
    assert off[5] == off[4] + 400
    words = np.full(off[5], MARK, np.int32)
    info = pkd.PlanInfo()
    p = lambda x: x.ctypes.data_as(ctypes.c_void_p)
    assert lib.pkd_plan_host(ctypes.byref(cfg), *[p(x) for x in t[:3]], len(lens), p(words), words.size,
                             ctypes.byref(info)) == 0
    assert info.schedule_words == off[4] + len(t[1])
    assert (words[info.schedule_words:] == MARK).all()
    assert (words[off[4]:info.schedule_words] == t[1]).all()


@gpu
@pytest.mark.parametrize("kind", ["shared", "dense", "cascade", "latent"])
def test_contexts_that_cannot_accumulate_upload_no_request_entries(kind):
    import torch
    lens = [40, 100]
    t = table(lens, 16)
    if kind == "latent":
        dec = pkd.BatchLatentDecodeWithPagedCache(16, 512, 64, 16, scale=1.0, max_batch=9,
                                                  max_num_pages=50, num_pages=t[3])
        plan = lambda: dec.plan(*t[:3])
    else:
        dec = pkd.BatchDecodeWithPagedKVCache(
            32, 8, 128, 16, max_batch=9, max_num_pages=50, num_pages=t[3],
            shared_prefix=kind != "cascade", dense_prefix=kind == "dense", cascade=kind == "cascade")
        groups = np.array([0, 3, 5], np.int32)
        suffix = table([7, 20, 16, 1, 33], 16)
        suffix = (suffix[0], suffix[1] % t[3], suffix[2])
        plan = (lambda: dec.plan_cascade(groups, t[:3], suffix)) if kind == "cascade" else \
            (lambda: dec.plan_shared(groups, *t[:3]))
    plan()
    info = dec.plan_info()
    end = pkd.schedule_layout(dec._layout_cfg(info))[4] + info["nnz"]
    behind = dec.workspace.view(torch.int32)[end:end + 40]
    behind[:50 - info["nnz"]] = MARK      # the page list's capacity, behind its words
    torch.cuda.synchronize()
    plan()
    torch.cuda.synchronize()
    assert (behind[:50 - info["nnz"]] == MARK).all()
