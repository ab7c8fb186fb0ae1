"""Latent decode where scores differ greatly along a request: tokens that a very low score masks,
from its start on; against the formulas in 64 bits."""
import pytest
import torch

from test_gpu_latent import DIM, ROW, SCALE, close, make, reference

gpu = pytest.mark.gpu
INF = float("inf")


def masked(heads, lens, page, low, where, seed, **kw):
    """A case in which token t of request 0 scores about `low` in every head if where(t): by the
    rotary key's last column, so the values stay as they are.  Elsewhere that column is 0."""
    t, q, cache, dec = make(heads, lens, page, seed=seed, **kw)
    cache[:, :, ROW - 1] = 0.0
    q[:, :, ROW - 1] = -1.0
    at = torch.arange(lens[0])
    at = at[where(at)]
    pages = torch.from_numpy(t[1][:t[0][1]]).long()
    cache[pages[at // page].cuda(), (at % page).cuda(), ROW - 1] = -low / SCALE
    dec.plan(*t[:3])
    return t, q, cache, dec


def check(t, q, cache, dec, lens, page):
    """Masked tokens weigh 2^-14,000 at most, that is nothing in either computation, and no score
    that weighs anything is larger than in close()'s own inputs: its tolerances hold as they are."""
    close(dec.run(q, cache), reference(q, cache, lens, t, page), cache[:, :, :DIM].abs().max().double())
    assert dec.device_error() == 0


@gpu
@pytest.mark.parametrize("low", [-INF, -1e30, -1e8, -1e6, -1e4])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_low_scores_first(heads, low):
    """Whole tiles of masked tokens before the others, parts of a tile, and all but one of a tile."""
    for lead in (63, 64, 65, 100, 128, 192):
        lens, page = [lead + 72, 40], 16
        check(*masked(heads, lens, page, low, lambda k: k < lead, lead), lens, page)


@gpu
@pytest.mark.parametrize("low", [-INF, -1e8])
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_low_scores_in_parts_of_a_split_request(heads, low):
    """Every other tile masked, and 4,000 tokens in a row: parts that begin with a masked tile, and
    parts that are empty states."""
    lens, page = [9001, 300], 16
    check(*masked(heads, lens, page, low, lambda k: (k // 64 % 2 == 0) | ((k >= 2000) & (k < 6000)), 7),
          lens, page)
    check(*masked(heads, lens, page, low, lambda k: k // 64 % 3 != 2, 8, num_ctas=3), lens, page)


@gpu
@pytest.mark.parametrize("heads", [16, 64])
def test_low_scores_of_some_heads(heads):
    """Heads of one block whose bases differ by 1e8, in the same tiles."""
    lens, page = [300], 16
    t, q, cache, dec = masked(heads, lens, page, -1e8, lambda k: k < 130, 9, num_ctas=1)
    q[:, 1::2, ROW - 1] = 0.0
    check(t, q, cache, dec, lens, page)
