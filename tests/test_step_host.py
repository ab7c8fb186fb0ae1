"""Tree plans, masks, tables and refusals of the calls around a step with drafts, without a GPU."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import paged_kv_decode_host_gb300 as pkd

INVALID, TABLE, SHAPE, CAPACITY = -1, -2, -3, -7


@pytest.fixture(scope="module")
def lib():
    pkd.build()
    return pkd.load()


def config(**kw):
    args = dict(num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, max_batch=64, max_num_pages=600,
                num_pages=600, num_ctas=8, flags=pkd.FLAG_TREE)
    args.update(kw)
    return pkd.make_config(**args)


def table(lens, page):
    counts = [-(-n // page) for n in lens]
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return indptr, np.arange(indptr[-1], dtype=np.int32)[::-1].copy(), \
        np.array([n - page * (c - 1) for n, c in zip(lens, counts)], np.int32)


def i32(*x):
    return np.array(x, np.int32)


def test_configurations(lib):
    off = (ctypes.c_int64 * 6)()
    status = lambda **kw: lib.pkd_schedule_layout(ctypes.byref(config(**kw)), off)
    for kw in (dict(), dict(num_qo_heads=64, num_kv_heads=8), dict(num_qo_heads=3, num_kv_heads=3),
               dict(flags=pkd.FLAG_TREE | pkd.FLAG_HND), dict(flags=pkd.FLAG_TREE | pkd.FLAG_KV_FP8),
               dict(flags=pkd.FLAG_TREE | pkd.FLAG_HND | pkd.FLAG_KV_FP8), dict(page_size=48), dict(max_batch=0), dict(num_ctas=1)):
        assert status(**kw) == 0, kw
    for kw in (dict(head_dim=64), dict(page_size=8), dict(num_qo_heads=6), dict(num_qo_heads=7),
               dict(num_qo_heads=18, num_kv_heads=9)):
        assert status(**kw) == SHAPE, kw
    for extra in (1, 2, 4, 16, 64, 128, 256, 1024):
        assert status(flags=pkd.FLAG_TREE | extra) == INVALID, extra


def check_plan(cfg, hq, hkv, page, lens, drafts, causal, window):
    batch, t = len(lens), table(lens, page)
    q_indptr = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
    w, info, off = pkd.plan_host_tree(cfg, q_indptr, *t, causal=causal, window=window)
    s = pkd.decode_schedule(w, off, info)
    rows = 128 // (hq // hkv)
    assert info["batch"] == sum(drafts) and s["cta_indptr"][-1] == info["num_items"]
    assert s["page_list"] == t[1].tolist()
    at = (off[4] + (info["nnz"] + 3) // 4 * 4) - 0
    entries = w[at:at + 4 * batch].reshape(batch, 4)
    if batch:
        assert entries.tolist() == [[int(q_indptr[b]), drafts[b], lens[b] - drafts[b], int(t[0][b])]
                                    for b in range(batch)]
    ranges, slots = {}, {}
    for it, head in zip(s["items"], s["heads"]):
        req, tb, te, dst, tokens, first, stride = it
        block = first // rows
        assert 0 <= req < batch and 0 <= head < hkv and tb < te <= lens[req] and tb % 16 == 0
        assert first % rows == 0 and tokens == min(rows, drafts[req] - first) > 0
        ranges.setdefault((req, block, head), []).append((tb, te, dst, stride))
    units = {}
    for u, (token, chunks) in enumerate(s["units"]):
        assert s["merge_indptr"][u + 1] - s["merge_indptr"][u] == chunks
        units[token] = (s["merge_indptr"][u], chunks)
    assert (s["merge_indptr"][-1] if units else 0) == info["num_slots"]
    for b, n in enumerate(drafts):
        for block in range(-(-n // rows)):
            ctx, r0, r1 = lens[b] - n, block * rows, min(n, block * rows + rows)
            least = ctx + (r0 if causal else 0)
            lo = max(0, least - window + 1) // 16 * 16 if window else 0
            hi = ctx + r1 if causal else lens[b]
            for head in range(hkv):
                parts = sorted(ranges.pop((b, block, head)))
                assert parts[0][0] == lo and parts[-1][1] == hi
                assert all(x[1] == y[0] and (x[1] - lo) % 128 == 0 for x, y in zip(parts, parts[1:]))
                for i in range(r0, r1):
                    token = int(q_indptr[b]) + i
                    if len(parts) == 1:
                        assert parts[0][2] == -1 and token not in units
                        continue
                    first, chunks = units[token]
                    assert chunks == len(parts)
                    for k, (_, _, dst, stride) in enumerate(parts):
                        assert stride == chunks and dst + (i - r0) * stride == first + k
    assert not ranges
    return s, info


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (3, 3), (8, 2), (64, 8)])
@pytest.mark.parametrize("ctas", [1, 3, 8, 152])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (False, 33), (True, 33), (True, 1)])
def test_plans_cover_every_row_and_token_once(lib, hq, hkv, ctas, causal, window):
    r = np.random.default_rng(hq + ctas)
    for _ in range(6):
        batch = int(r.integers(0, 9))
        lens = [int(x) for x in r.integers(1, 2500, batch)]
        drafts = [int(r.integers(0, min(n, 300) + 1)) for n in lens]
        q_indptr = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        t = table(lens, 16)
        cfg = config(num_qo_heads=hq, num_kv_heads=hkv, num_ctas=ctas, max_batch=max(1, sum(drafts), batch),
                     max_num_pages=int(t[0][-1]), num_pages=2000, min_chunk_tokens=int(r.choice([1, 256])))
        check_plan(cfg, hq, hkv, 16, lens, drafts, causal, window)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 15000)])
def test_plans_that_keep_blocks_together(lib, causal, window):
    """More tokens than L2 holds, shared by several row blocks: in pieces, all cut alike."""
    page = 4096
    for hq, hkv, lens, drafts in ((64, 8, [100_000], [256]), (32, 8, [100_000], [256]), (32, 8, [30_000] * 4, [100] * 4),
                                  (32, 8, [60_000, 50_000, 3], [65, 70, 3]), (8, 1, [400_000, 500], [40, 1])):
        cfg = config(num_qo_heads=hq, num_kv_heads=hkv, num_ctas=152, max_batch=sum(drafts), page_size=page,
                     max_num_pages=200, num_pages=200)
        s, info = check_plan(cfg, hq, hkv, page, lens, drafts, causal, window)
        if not window and lens[0] > 16384:
            cuts = {}
            for req, tb, te, dst, tokens, first, stride in s["items"]:
                if req == 0:
                    cuts.setdefault(first, set()).add(tb)
            assert len({frozenset(c) for c in cuts.values()}) == 1, "blocks of a request cut at different tokens"
        # room for a plan with few tokens, too: no pieces that it cannot hold
    tight = config(num_qo_heads=64, num_kv_heads=8, num_ctas=152, max_batch=256, page_size=page, max_num_pages=30,
                   num_pages=30)
    check_plan(tight, 64, 8, page, [100_000], [256], causal, window)


def test_largest_plans_fit_their_slots(lib):
    """Slots and items of plans that cut as often as they can."""
    for hq, hkv, ctas in ((8, 1, 152), (1, 1, 152), (64, 8, 152)):
        drafts = [128 // (hq // hkv)] * 64
        lens = [700] * 64
        q_indptr = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        cfg = config(num_qo_heads=hq, num_kv_heads=hkv, num_ctas=ctas, max_batch=sum(drafts), max_num_pages=4000,
                     num_pages=4000, min_chunk_tokens=1, alpha=0)
        info = pkd.plan_host_tree(cfg, q_indptr, *table(lens, 16))[1]
        assert info["num_units"] > 0


def test_plans_that_are_refused(lib):
    cfg, t = config(), table([40, 20], 16)
    ok = i32(0, 3, 5)
    plan = lambda *a, **k: pkd.plan_host_tree(cfg, *a, **k)
    plan(ok, *t)
    for bad in (i32(0, 41, 45), i32(0, 3, 2), i32(1, 3, 5), i32(0, 3, 24)):
        with pytest.raises(pkd.PkdError, match="BAD_TABLE"):
            plan(bad, *t)
    with pytest.raises(pkd.PkdError, match="BAD_TABLE"):
        plan(ok, t[0], t[1], i32(8, 17))
    with pytest.raises(pkd.PkdError, match="BAD_TABLE"):
        plan(ok, t[0], i32(0, 1, 2, 3, 600), t[2])
    with pytest.raises(pkd.PkdError, match="BAD_TABLE"):
        plan(ok[:-1], *t)
    with pytest.raises(pkd.PkdError, match="INVALID"):
        plan(ok, *t, window=-1)
    with pytest.raises(pkd.PkdError, match="CAPACITY"):
        plan(i32(0, 60, 65), *table([60, 20], 16))
    with pytest.raises(pkd.PkdError, match="CAPACITY"):
        pkd.plan_host_tree(config(max_num_pages=4), ok, *t)
    with pytest.raises(pkd.PkdError, match="INVALID"):
        pkd.plan_host(cfg, *t)
    with pytest.raises(pkd.PkdError, match="INVALID"):
        pkd.plan_host_tree(config(flags=0), ok, *t)
    page = 1 << 20
    big = lambda n, last: (i32(0, n), np.zeros(n, np.int32), i32(last))
    huge = config(page_size=page, max_num_pages=2048, num_kv_heads=1, num_qo_heads=8)
    with pytest.raises(pkd.PkdError, match="CAPACITY|SHAPE"):
        pkd.plan_host_tree(huge, i32(0, 1), *big(2048, page))


def test_tree_masks():
    mask, depths = pkd.tree_mask(i32(0, 5, 5, 40), i32(-1, 0, 0, 2, -1, *range(-1, 34)))
    assert depths.tolist() == [0, 1, 1, 2, 0] + list(range(35))
    words = mask.view(np.uint32)
    assert words.shape == (40, 2) and words[:5, 0].tolist() == [1, 3, 5, 13, 16] and not words[:5, 1].any()
    for i in range(35):
        assert int(words[5 + i, 0]) | int(words[5 + i, 1]) << 32 == (1 << (i + 1)) - 1
    mask, depths = pkd.tree_mask(i32(0), np.zeros(0, np.int32))
    assert mask.shape == (0, 1) and depths.shape == (0,)
    for q, p in ((i32(0, 2), i32(-1, 1)), (i32(0, 2), i32(-1, -2)), (i32(0, 2), i32(-1)), (i32(1, 2), i32(-1, -1)),
                 (i32(0, 2, 1), i32(-1)), (i32(0, 1, 2), i32(-1, 0))):
        with pytest.raises(ValueError):
            pkd.tree_mask(q, p)


def test_accepted_tables():
    indptr, indices, last = table([40, 20, 16], 16)
    got = pkd.accepted_table(indptr, indices, last, 16, i32(9, 20, 0), i32(1, 4, 0))
    assert got[0].tolist() == [0, 2, 3, 4] and got[2].tolist() == [16, 4, 16]
    assert got[1].tolist() == [indices[0], indices[1], indices[3], indices[5]]
    assert got[3].tolist() == [indices[2], indices[4]]
    same = pkd.accepted_table(indptr, indices, last, 16, i32(9, 20, 0), i32(9, 20, 0))
    assert same[0].tolist() == indptr.tolist() and same[2].tolist() == last.tolist() and not same[3].size
    for drafted, counts in ((i32(9, 20, 0), i32(1, 0, 0)), (i32(9, 21, 0), i32(1, 4, 0)), (i32(9, 20, 0), i32(1, 4, 1)),
                            (i32(-1, 20, 0), i32(-1, 4, 0)), (i32(9, 20), i32(1, 4))):
        with pytest.raises(ValueError):
            pkd.accepted_table(indptr, indices, last, 16, drafted, counts)
    with pytest.raises(pkd.PkdError, match="BAD_TABLE"):
        pkd.accepted_table(indptr, indices, i32(8, 4, 17), 16, i32(9, 20, 0), i32(1, 4, 0))


def rotate_status(lib, **kw):
    a = dict(q=256, qt=1536, qh=128, qo=1 << 20, ot=1024, oh=128, k=2304, kt=1536, kh=128, v=2816, vt=1536, vh=128, qn=None,
             kn=None, f32=0, eps=1e-6, turns=64, axes=64, rotary=128, pairs=0, rs=1.0, rp=64, n_axes=1, bi=64, pos=64, n=2,
             ip=64, ix=64, nnz=4, la=64, batch=1, kv=1 << 21, pages=4, page=16, hq=8, hkv=2, dim=128, ks=1.0, vs=1.0, flags=0,
             err=None)
    a.update(kw)
    return lib.pkd_rotate_append_kv(*a.values(), None)


def test_rotate_append_refusals(lib):
    """(Arguments are refused before any CUDA call; addresses here are never read.)"""
    for kw in (dict(flags=4), dict(n=-1), dict(batch=-1), dict(nnz=-1), dict(pages=0), dict(page=0), dict(hq=-1), dict(hkv=0),
               dict(n_axes=0), dict(n_axes=5), dict(eps=-1.0), dict(eps=float("nan")), dict(rs=float("inf")), dict(rotary=136),
               dict(rotary=24), dict(rotary=-16), dict(rotary=4, pairs=1), dict(pairs=2), dict(f32=2), dict(ks=2.0), dict(vs=0.5),
               dict(flags=8, ks=0.0), dict(flags=8, vs=float("nan")), dict(flags=8, ks=1e-45), dict(q=None), dict(qo=None),
               dict(k=None), dict(v=None), dict(kv=None), dict(turns=None), dict(axes=None), dict(rp=None), dict(bi=None),
               dict(pos=None), dict(ip=None), dict(ix=None), dict(la=None), dict(q=264), dict(qo=8), dict(kv=8), dict(turns=4),
               dict(err=2), dict(qn=1), dict(qn=2, f32=1), dict(qt=1532), dict(qh=132), dict(kt=4), dict(ot=64), dict(oh=64),
               dict(vh=-8), dict(kt=1 << 41)):
        assert rotate_status(lib, **kw) == INVALID, kw
    for dim in (0, 32, 96, 512):
        assert rotate_status(lib, dim=dim, rotary=0) == SHAPE
    assert rotate_status(lib, n=0) == 0


def accept_status(lib, **kw):
    a = dict(layers=2, kv=[256, 512], acc=64, width=4, dr=64, ip=64, ix=64, nnz=4, la=64, batch=1, pages=4, page=16, hkv=2,
             dim=128, flags=0, err=None)
    a.update(kw)
    kv = a.pop("kv")
    layers = a.pop("layers")
    return lib.pkd_accept_kv(layers, (ctypes.c_void_p * len(kv))(*kv) if kv else None, *a.values(), None)


def test_accept_refusals(lib):
    for kw in (dict(layers=0), dict(layers=129), dict(kv=None), dict(kv=[256, 256]), dict(kv=[256, 520]), dict(kv=[256, 0]),
               dict(width=-1), dict(width=1025), dict(batch=-1), dict(nnz=-1), dict(pages=0), dict(page=0), dict(hkv=0),
               dict(dim=0), dict(dim=4), dict(dim=8, flags=8), dict(flags=1), dict(acc=None), dict(dr=None), dict(ip=None),
               dict(ix=None), dict(la=None), dict(acc=2), dict(dr=2), dict(err=1), dict(hkv=1 << 20)):
        assert accept_status(lib, **kw) == INVALID, kw
    assert accept_status(lib, batch=0) == 0 and accept_status(lib, width=0) == 0


def test_tree_calls_without_a_context(lib):
    assert lib.pkd_plan_tree(None, None, None, None, None, 0, 0, 0, None, None) == INVALID
    assert lib.pkd_run_tree(None, None, 0, None, None, None, None, 0, None, None, 1.0, 0.0, 0, None) == INVALID
    assert lib.pkd_run_tree_scaled(None, None, 0, None, None, None, None, 0, None, None, 1.0, 0.0, 1.0, 1.0, 0,
                                   None) == INVALID


@pytest.mark.parametrize("freq", [[500_000.0 ** (-i / 64) for i in range(64)], [10_000.0 ** (-i / 32) / 7 for i in range(32)],
                                  [1.0, -3.7, 0.0, 5e-324, 1e20, -1e30, 2.0 ** -80, 123456.789]])
def test_turns_are_rounded_once(freq):
    """Turns per position times 2^64: the nearest integers, so that position p is off by at most p / 2."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")
    rope = pkd.RotaryPositions(freq, interleaved=True, device="cpu")
    for x, got in zip(freq, rope.turns.numpy().view(np.uint64)):
        off = (Fraction(x) * 2 ** 63 / pi - int(got)) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(1, 2)


def test_accept_refuses_caches_that_overlap(lib):
    """(4 pages of 16 tokens, 2 heads and 128 values: 65,536 bytes for K and V in bf16.)"""
    size = 4 * 2 * 16 * 2 * 128 * 2
    for kv in ([1 << 20, (1 << 20) + 16], [1 << 20, (1 << 20) + size - 16], [(1 << 20) + size // 2, 1 << 20],
               [1 << 20, 1 << 22, (1 << 20) + size // 2, 1 << 23]):
        assert accept_status(lib, layers=len(kv), kv=kv) == INVALID, kv
    assert accept_status(lib, kv=[1 << 20, (1 << 20) + size // 2 - 16], flags=pkd.FLAG_KV_FP8) == INVALID
    assert accept_status(lib, kv=[16, 1 << 40], pages=2 ** 31 - 1, page=2 ** 31 - 1, hkv=1 << 16) == INVALID
