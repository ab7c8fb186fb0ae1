"""How far latent results are from 64 bits, head by head, and a scale on the values."""
import ctypes
import math

import pytest
import torch

import paged_kv_decode_host_gb300 as pkd
from test_gpu_latent import DIM, ROW, SCALE, make, reference, table

gpu = pytest.mark.gpu


def step_of(x):
    """The step between bf16 values of each |x|: 2^-7 of the power of two below it."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -100)))) * 2.0 ** -7


def held(got, q, cache, lens, t, page, out_scale=1.0):
    """Squared distance of every (request, head)'s result, against what its roundings give.

    Output: rounded to bf16, so each element's error is uniform within half a step to either side:
    variance step^2 / 12, variance of the square step^4 / 180.  The sum over 512 elements is allowed 8
    standard deviations over its mean.
    P, above 32 heads: one bf16, so a token's weight is off by at most 2^-8 of itself (the sum that
    divides is not rounded); the errors of different tokens have random sign and rows of normal values
    stand nearly at right angles (a scalar product of two is within 6 / sqrt(512) of their lengths'), so
    the squared error is at most 2^-16 sum (p |c|)^2 and, for the angles, a quarter more.  Up to 32 heads P
    has 16 bits, an error 2^-8 of that, squared 2^-16.
    Scores and fp32 sums: 36 steps of 16 products that sum to 100 at most, each off by at most 2^-22 of
    the sum, times the scale: a weight is off by under 7e-5 of itself, 5e-9 squared, for which 1e-8 is
    room."""
    out, lse = got
    ro, rl = reference(q, cache, lens, t, page)
    assert (lse.double() - rl).abs().max() <= 2e-4
    ro = ro * out_scale
    err = (out.double() - ro).square().sum(-1)
    step = step_of(ro)
    allowed = (step ** 2).sum(-1) / 12 + 8 * ((step ** 4).sum(-1) / 180).sqrt()
    weighed = torch.empty_like(rl)
    for i, n in enumerate(lens):
        mine = torch.from_numpy(t[1][t[0][i]:t[0][i + 1]]).long().cuda()
        c = cache[mine].reshape(-1, ROW)[:n].double()
        p = torch.exp(q[i].double() @ c.T * SCALE - rl[i][:, None])
        weighed[i] = (p ** 2 @ (c[:, :DIM] ** 2).sum(-1)) * out_scale ** 2
    one = 2.0 ** -16 * 1.25
    allowed = allowed + weighed * ((one if q.shape[1] > 32 else one * 2.0 ** -16) + 1e-8)
    worst = (err / allowed).max()
    assert worst <= 1, worst


@gpu
@pytest.mark.parametrize("heads", [8, 16, 17, 32, 33, 40, 64, 65, 96, 128])
@pytest.mark.parametrize("lens,kw", [([9001, 1500, 3], {}), ([2000] * 9, {}), ([1, 2, 15, 16, 17, 64, 65, 700], {}),
                                     ([40_000], {}), ([9001, 300], dict(num_ctas=3))])
def test_every_head_is_within_its_roundings(heads, lens, kw):
    t, q, cache, dec = make(heads, lens, 16, seed=heads, **kw)
    dec.plan(*t[:3])
    held(dec.run(q, cache), q, cache, lens, t, 16)
    assert dec.device_error() == 0


@gpu
@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_parts_of_a_split_request_count_by_their_weight(heads):
    """Every 128 tokens hold one value, and the tokens' weights come from the rotary key alone: a result
    is the mean of a few hundred constants, weighed by their parts.  A dropped, doubled or misplaced
    part moves it by far more than two roundings (2^-8 each, all terms being positive) and 1 % of them
    for the fp32 sums."""
    n, page = 40_000, 16
    t, q, cache, dec = make(heads, [n], page, seed=3)
    q[:, :, :DIM] = 0.0
    at = torch.arange(n)
    pages = torch.from_numpy(t[1]).long()[at // page].cuda()
    value = 1.0 + ((at // 128) * 37 % 101).float()
    cache[pages, (at % page).cuda(), :DIM] = value.cuda().bfloat16()[:, None]
    dec.plan(*t[:3])
    assert dec.plan_info()["num_slots"] > 50
    out, lse = dec.run(q, cache)
    ro, rl = reference(q, cache, [n], t, page)
    assert ((out.double() - ro).abs() <= 2.02 * 2 ** -8 * ro).all()
    assert (lse.double() - rl).abs().max() <= 2e-4


@gpu
@pytest.mark.parametrize("heads", [8, 16, 17, 32, 64, 100, 128])
def test_rising_scores_rescale_every_tile(heads):
    """Scores that rise by some 13 bits a tile: every tile raises the bases by more than the 8 that are
    let be, and scales what was summed before, for every shape of block (P in one and in two parts).
    A tile rises by 64 x 1/4 x 8.7 x scale = 10 nats, ten of them and the last one's spread to 95, that is
    1,316 before the scale and under 1,450 with the latent columns' part.  An fp32 sum in 36 steps of 16
    products is off by at most 36 x 2^-22 x 1,450 = 0.0125, 9e-4 nats: the lse by as much and its own
    rounding (95 x 2^-23), a weight by 1e-3 of itself, a result by twice that (the sum that divides)."""
    lens = [640, 40, 640]
    t, q, cache, dec = make(heads, lens, 16, seed=2, min_chunk_tokens=4096, num_ctas=1)
    for i in (0, 2):
        at = torch.arange(lens[i])
        pages = torch.from_numpy(t[1][t[0][i]:t[0][i + 1]]).long()[at // 16].cuda()
        cache[pages, (at % 16).cuda(), DIM:] = (8.7 * (at // 64) + at % 64 / 16.0).cuda()[:, None].bfloat16()
    q[:, :, DIM:] = 1.0 / 4
    q[2] *= -1.0             # and falling ones: no raise after the first tile
    dec.plan(*t[:3])
    out, lse = dec.run(q, cache)
    ro, rl = reference(q, cache, lens, t, 16)
    top = cache[:, :, :DIM].abs().max().double()
    assert (lse.double() - rl).abs().max() <= 1e-3
    assert (out.double() - ro).abs().max() <= (1.01 * 2 ** -8 + 2e-3) * top + 2 ** -8 * ro.abs().max()


@gpu
@pytest.mark.parametrize("heads", [16, 40, 128])
@pytest.mark.parametrize("v_scale", [1.0, 0.375, -20.0, 0.0])
def test_values_are_scaled(heads, v_scale):
    """pkd_run_scaled's v_scale multiplies the results, of whole and of split requests."""
    lens = [5000, 77, 1]
    t, q, cache, dec = make(heads, lens, 16, seed=6)
    dec.plan(*t[:3])
    out = torch.empty(3, heads, DIM, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, heads, device="cuda")
    p = lambda x: ctypes.c_void_p(x.data_ptr())
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert pkd.load().pkd_run_scaled(dec._h, p(q), p(cache), p(out), p(lse), SCALE, v_scale, 0, stream) == 0
    held((out, lse), q, cache, lens, t, 16, out_scale=v_scale)


@gpu
def test_negative_and_zero_softmax_scales():
    lens, page, heads = [300, 64, 7], 16, 40
    t = table(lens, page)
    q = torch.randn(3, heads, ROW, device="cuda").bfloat16()
    cache = torch.randn(t[3], page, ROW, device="cuda").bfloat16()
    for scale in (-SCALE, 0.0):
        dec = pkd.BatchLatentDecodeWithPagedCache(heads, DIM, 64, page, scale=scale, max_batch=3,
                                                  max_num_pages=len(t[1]), num_pages=t[3])
        dec.plan(*t[:3])
        out, lse = dec.run(q, cache)
        ro, rl = reference(q, cache, lens, t, page, scale=scale)
        assert (lse.double() - rl).abs().max() <= 2e-4
        top = cache[:, :, :DIM].abs().max().double()
        assert (out.double() - ro).abs().max() <= 1.01 * 2 ** -8 * (top + ro.abs().max())
    assert math.isclose(float(lse[2, 0]), math.log(7), abs_tol=1e-6)
