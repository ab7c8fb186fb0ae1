"""The latent workspace holds every plan's partial states, and little beside them."""
import ctypes

import numpy as np
import pytest

import paged_kv_decode_host_gb300 as pkd

STATE = 4 * 513   # bytes of a head's partial state: 512 sums and the lse


def config(heads, n_cta, max_batch, pages, page=16):
    return pkd.make_config(heads, 1, 512, page, max_batch, pages, pages, num_ctas=n_cta, flags=pkd.FLAG_LATENT)


@pytest.mark.parametrize("heads", [1, 16, 64, 65, 128])
@pytest.mark.parametrize("n_cta", [1, 2, 3, 152])
def test_slots_follow_the_cuts_of_a_plan(heads, n_cta):
    """At most two slots a cut, whatever the batch's capacity; the schedule beside them is 44 bytes an
    item (batch x blocks of heads, and 4 n_cta + 8 of any plan), 4 a page and two pages of rounding."""
    blocks = -(-heads // 64)
    cuts = max(1, n_cta // blocks) - 1
    for max_batch in (1, 64, 512):
        pages = 8 * max_batch
        need = pkd.load().pkd_workspace_bytes(ctypes.byref(config(heads, n_cta, max_batch, pages)))
        schedule = 44 * (blocks * max_batch + 4 * n_cta + 8) + 4 * (n_cta + pages) + 2048
        assert 2 * cuts * heads * STATE <= need <= 2 * cuts * heads * STATE + schedule


@pytest.mark.parametrize("heads", [16, 64, 128])
@pytest.mark.parametrize("n_cta", [1, 2, 3, 5, 152])
@pytest.mark.parametrize("floor", [-1, 1, 16])
def test_no_plan_runs_out_of_slots(heads, n_cta, floor):
    """Ragged, skewed and even batches at the batch's capacity, down to the finest split floor."""
    r = np.random.default_rng(heads + n_cta)
    shapes = [[40_000], [300] * 300, [20_000, 1, 20_000], [1] * 5, [2 * k + 1 for k in range(152)],
              [1700] * 152, [3000] * 75]
    shapes += [r.integers(1, int(10 ** r.uniform(1, 4.2)), int(10 ** r.uniform(0, 2.4))).tolist() for _ in range(60)]
    for lens in shapes:
        counts = np.array([-(-n // 16) for n in lens])
        indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        last = (np.array(lens) - 16 * (counts - 1)).astype(np.int32)
        cfg = config(heads, n_cta, len(lens), int(indptr[-1]))
        cfg.min_chunk_tokens = floor
        _, info, _ = pkd.plan_host(cfg, indptr, np.arange(indptr[-1], dtype=np.int32), last)
        assert info["num_slots"] <= 2 * (max(1, n_cta // (-(-heads // 64))) - 1)
