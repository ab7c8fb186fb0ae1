"""Cases of the three operators of a decoding step with drafted tokens, their plain forms and
their calls.

* ``rotate``: new tokens' queries and keys, normed per head where the model does so, rotated by
  their positions (one axis, or several), keys and values written into their page slots;
* ``tree``: attention of every request's drafted tokens (a tree, or a chain) over its cached
  tokens and their own ancestors; scores capped, biased by distance or cut to a window where
  the model does so; a single token per request is the ordinary decode step of such a model;
* ``accept``: the accepted drafts' rows moved to the front of the drafted ones, in every layer.

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits; with
``own`` true it makes the calls a user makes of the package.
"""
import math
import random

import numpy as np
import torch

own = False

HEAD = 128
THETA = 500_000.0
EPS = 1e-6
SCALE = 1.0 / math.sqrt(HEAD)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's new tokens: latency alone counts
        dict(name="rotate step", op="rotate", heads=32, kv_heads=8, batch=64, tokens=1, page=16, kv="bf16",
             layout="NHD", norms=False, axes=1, pairs=False, rotary=128),
        # drafted tokens of a model with norms per head, 8-bit cache
        dict(name="rotate drafts e4m3", op="rotate", heads=64, kv_heads=8, batch=48, tokens=24, page=16, kv="e4m3",
             layout="HND", norms=True, axes=1, pairs=False, rotary=128),
        # prompts of images and text of odd lengths: positions in time, height and width
        dict(name="rotate prompts three axes", op="rotate", heads=32, kv_heads=8, batch=8, tokens=2011, page=64,
             kv="bf16", layout="NHD", norms=False, axes=3, pairs=False, rotary=128),
        # one user's chat with a small tree of drafts: latency alone counts
        dict(name="tree one request", op="tree", heads=32, kv_heads=8, batch=1, longest=517, lens="even", drafts=8,
             shape="tree", page=16, layout="NHD", window=0, cap=0.0, slopes=False),
        # an ordinary serving batch, ragged lengths, trees of 16 drafts
        dict(name="tree batch", op="tree", heads=32, kv_heads=8, batch=64, longest=8192, lens="ragged", drafts=16,
             shape="tree", page=16, layout="NHD", window=0, cap=0.0, slopes=False),
        # wide trees and many heads per KV head: as much arithmetic as bytes
        dict(name="tree wide", op="tree", heads=64, kv_heads=8, batch=16, longest=8192, lens="ragged", drafts=61,
             shape="tree", page=16, layout="NHD", window=0, cap=0.0, slopes=False),
        # a long document beside short chats
        dict(name="tree long document", op="tree", heads=32, kv_heads=8, batch=9, longest=100_003, lens="skewed",
             drafts=12, shape="tree", page=64, layout="HND", window=0, cap=0.0, slopes=False),
        # a plain decode step of a model with capped scores and a sliding window
        dict(name="capped window step", op="tree", heads=32, kv_heads=8, batch=64, longest=8192, lens="ragged",
             drafts=1, shape="chain", page=16, layout="NHD", window=4096, cap=50.0, slopes=False),
        # a model with a bias by distance and no shared heads, small trees
        dict(name="biased trees", op="tree", heads=8, kv_heads=8, batch=24, longest=4001, lens="ragged", drafts=7,
             shape="tree", page=32, layout="NHD", window=0, cap=0.0, slopes=True),
        # pieces of prompts over what is cached of them
        dict(name="causal chunk capped", op="tree", heads=32, kv_heads=8, batch=8, longest=6007, lens="ragged",
             drafts=256, shape="chain", page=16, layout="NHD", window=0, cap=30.0, slopes=False),
        # a step's accepted drafts, all layers
        dict(name="accept step", op="accept", layers=32, kv_heads=8, batch=64, drafts=16, page=16, layout="NHD"),
        # one user's accepted drafts
        dict(name="accept one request", op="accept", layers=32, kv_heads=8, batch=1, drafts=8, page=16, layout="NHD"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "tree", "tree", "tree", "accept"])
    layout = rng.choice(["NHD", "HND"])
    if op == "accept":
        return dict(op=op, layers=rng.choice([1, 2, 8, 32]), kv_heads=rng.choice([1, 2, 4, 8]), batch=_log(rng, 1, 64),
                    drafts=_log(rng, 1, 64), page=rng.choice([1, 5, 16, 64]), layout=layout)
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 8])
    if op == "rotate":
        batch = _log(rng, 1, 256)
        return dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, batch=batch,
                    tokens=_log(rng, 1, max(1, 12_000 // batch)), page=rng.choice([1, 5, 16, 64]),
                    kv=rng.choice(["bf16", "bf16", "e4m3"]), layout=layout, norms=rng.choice([True, False]),
                    axes=rng.choice([1, 1, 2, 3]), pairs=rng.choice([False, True]), rotary=rng.choice([32, 64, 96, 128, 128]))
    batch = _log(rng, 1, 64)
    drafts = _log(rng, 1, max(1, min(256, 1024 // batch)))
    lens = rng.choice(["even", "ragged", "skewed"])
    longest = drafts + _log(rng, 1, min(100_000, 130_000 // batch * (4 if lens == "skewed" else 1)))
    return dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, batch=batch, longest=longest, lens=lens, drafts=drafts,
                shape=rng.choice(["tree", "tree", "chain"]), page=rng.choice([16, 32, 64]), layout=layout,
                window=rng.choice([0, 0, _log(rng, 1, longest)]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                slopes=rng.choice([False, False, True]))


def _lens(case):
    """The cached tokens of a tree case's requests, drafts included: fixed by its sizes."""
    n, longest, least = case["batch"], case["longest"], case["drafts"]
    r = random.Random("%d,%d,%s" % (n, longest, case["lens"]))
    if case["lens"] == "even":
        return [longest] * n
    if case["lens"] == "ragged":
        got = [r.randint(least, longest) for _ in range(n)]
    else:  # one long, the others short
        got = [r.randint(least, max(least, longest // 128)) for _ in range(n)]
    got[r.randrange(n)] = longest
    return got


def _paths(case):
    """The accepted drafts of an accept case's requests, in order: fixed by its sizes."""
    r = random.Random("%d,%d" % (case["batch"], case["drafts"]))
    most = min(-(-case["drafts"] // 2), 8)
    return [sorted(r.sample(range(case["drafts"]), r.randint(-(-most // 2), most))) for _ in range(case["batch"])]


def work(case):
    op, kvh = case["op"], case["kv_heads"]
    if op == "rotate":
        n, h = case["batch"] * case["tokens"], case["heads"]
        size = 1 if case["kv"] == "e4m3" else 2
        return {"bytes": n * ((h + 2 * kvh) * HEAD * 2 + 4 * case["axes"] + 8 + h * HEAD * 2 + 2 * kvh * HEAD * size),
                "flops": n * (h + kvh) * HEAD * (7 if case["norms"] else 3)}
    if op == "accept":
        moved = sum(a != i for path in _paths(case) for i, a in enumerate(path))
        return {"bytes": case["layers"] * moved * 2 * (2 * kvh * HEAD * 2) + 4 * sum(map(len, _paths(case))), "flops": 0}
    h, drafts, window = case["heads"], case["drafts"], case["window"]
    contexts = [n - drafts for n in _lens(case)]
    seen = [min(c, window - 1) if window else c for c in contexts]
    total = sum(seen) + drafts * case["batch"]
    pages = sum(-(-n // case["page"]) for n in seen)
    rows = drafts * case["batch"] * h
    return {"bytes": total * kvh * HEAD * 4 + rows * (HEAD * 4 + 4) + 4 * pages,
            "flops": 4 * HEAD * h * drafts * (sum(seen) + case["batch"])}


# ---------------------------------------------------------------- inputs
class State:
    pass


def _table(case, lens, gen):
    """The page table of the requests, its pages scattered over the pool."""
    s, page = State(), case["page"]
    counts = [-(-n // page) for n in lens]
    s.case, s.pages = case, sum(counts) + 3
    s.indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    s.last = np.array([n - page * (c - 1) for n, c in zip(lens, counts)], np.int32)
    where = torch.randperm(s.pages, generator=gen, device="cuda")[: int(s.indptr[-1])].int()
    s.indices = where.cpu().numpy()
    s.lens = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s.d_indptr = torch.from_numpy(s.indptr).cuda()
    s.d_indices = where.contiguous()
    s.d_last = torch.from_numpy(s.last).cuda()
    return s


def _cache(case, pages, gen, dtype=torch.bfloat16):
    page, h = case["page"], case["kv_heads"]
    shape = (pages, 2, page, h, HEAD) if case["layout"] == "NHD" else (pages, 2, h, page, HEAD)
    return _normal(shape, gen, dtype)


def _normal(shape, gen, dtype=torch.bfloat16):
    """N(0, 1) in `dtype`, made in pieces."""
    x = torch.empty(shape, dtype=dtype, device="cuda")
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        piece = torch.randn(n, generator=gen, device="cuda")
        flat[i:i + n] = (piece * 112.0).clamp_(-448.0, 448.0).to(dtype) if dtype == torch.float8_e4m3fn else piece.to(dtype)
    return x


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return {"rotate": _prepare_rotate, "tree": _prepare_tree, "accept": _prepare_accept}[case["op"]](case, gen, seed)


def _prepare_rotate(case, gen, seed):
    batch, n, h, kvh = case["batch"], case["tokens"], case["heads"], case["kv_heads"]
    r = random.Random("%d,%d" % (batch, n))
    old = [0 if n > 64 else r.randint(0, 200) for _ in range(batch)]  # tokens already there
    s = _table(case, [o + n for o in old], gen)
    e4m3 = case["kv"] == "e4m3"
    s.cache = _cache(case, s.pages, gen, torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    s.k_scale, s.v_scale = (1.0 / 112.0, 1.0 / 90.0) if e4m3 else (1.0, 1.0)
    # one projection's output: queries, keys and values are column ranges of its rows
    both = _normal((batch * n, (h + 2 * kvh) * HEAD), gen)
    s.q = both[:, :h * HEAD].view(-1, h, HEAD)
    s.k = both[:, h * HEAD:(h + kvh) * HEAD].view(-1, kvh, HEAD)
    s.v = both[:, (h + kvh) * HEAD:].view(-1, kvh, HEAD)
    s.q_norm = (1.0 + 0.2 * _normal((HEAD,), gen).float()).bfloat16() if case["norms"] else None
    s.k_norm = (1.0 + 0.2 * _normal((HEAD,), gen).float()).bfloat16() if case["norms"] else None
    s.rows = torch.arange(batch, device="cuda", dtype=torch.int32).repeat_interleave(n)
    s.places = (torch.tensor(old, device="cuda", dtype=torch.int32)[:, None]
                + torch.arange(n, device="cuda", dtype=torch.int32)[None, :]).reshape(-1).contiguous()
    # positions of conversations that are longer than what is still cached of them; behind the first
    # axis those of an image's rows and columns
    far = torch.randint(0, 120_000, (batch,), generator=gen, device="cuda", dtype=torch.int32)
    first = s.places + far.repeat_interleave(n)
    more = torch.randint(0, 256, (batch * n, case["axes"] - 1), generator=gen, device="cuda", dtype=torch.int32)
    s.at = first if case["axes"] == 1 else torch.cat([first[:, None], first[:, None] // 2 + more], 1).contiguous()
    half = case["rotary"] // 2
    s.freq = [THETA ** (-i / half) for i in range(half)]
    # every axis has a run of the frequencies
    s.axis = [i * case["axes"] // half for i in range(half)]
    s.d_freq = torch.tensor(s.freq, dtype=torch.float64, device="cuda")
    s.d_axis = torch.tensor(s.axis, device="cuda")
    if own:
        import paged_kv_decode_host_gb300 as pkd
        s.rope = pkd.RotaryPositions(s.freq, interleaved=case["pairs"], axes=s.axis)
    return s


def _parents(case, seed):
    """Every draft's parent among its request's drafts, -1 for the context's end; a parent comes
    before its children."""
    r, n = random.Random(seed), case["drafts"]
    if case["shape"] == "chain":
        return [[j - 1 for j in range(n)] for _ in range(case["batch"])]
    return [[r.randint(max(-1, j // 3 - 2), j - 1) for j in range(n)] for _ in range(case["batch"])]


def _tree(parents):
    """(bits, depths): words of 32 bits, bit j of row i set where draft j is i or its ancestor."""
    batch, n = len(parents), len(parents[0])
    see = np.zeros((batch, n, n), bool)
    depth = np.zeros((batch, n), np.int32)
    rows = np.arange(batch)
    p = np.array(parents)
    for i in range(n):
        up = p[:, i]
        has = up >= 0
        see[has, i] = see[rows[has], up[has]]
        depth[has, i] = depth[rows[has], up[has]] + 1
        see[:, i, i] = True
    words = -(-n // 32)
    bits = np.zeros((batch, n, words), np.uint32)
    for j in range(n):
        bits[:, :, j // 32] |= see[:, :, j].astype(np.uint32) << np.uint32(j % 32)
    return bits.reshape(batch * n, words).view(np.int32), depth.reshape(-1)


def _prepare_tree(case, gen, seed):
    lens, n = _lens(case), case["drafts"]
    s = _table(case, lens, gen)
    s.kv = _cache(case, s.pages, gen)
    s.q = _normal((case["batch"] * n, case["heads"], HEAD), gen)
    s.causal = case["shape"] == "chain"
    s.mask = s.depths = s.slopes = None
    if not s.causal:
        bits, depths = _tree(_parents(case, seed))
        s.mask, s.depths = torch.from_numpy(bits).cuda(), torch.from_numpy(depths).cuda()
    if case["slopes"]:
        h = case["heads"]
        s.slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], dtype=torch.float32, device="cuda")
    s.q_indptr = (np.arange(case["batch"] + 1) * n).astype(np.int32)
    if own:
        import paged_kv_decode_host_gb300 as pkd
        s.dec = pkd.BatchTreeDecodeWithPagedKVCache(
            case["heads"], case["kv_heads"], HEAD, case["page"], max_tokens=case["batch"] * n,
            max_num_pages=len(s.indices), num_pages=s.pages, kv_layout=case["layout"])
        s.dec.plan(s.q_indptr, s.indptr, s.indices, s.last, causal=s.causal, window=case["window"])
    return s


def _prepare_accept(case, gen, seed):
    n, paths = case["drafts"], _paths(case)
    r = random.Random("%d" % case["batch"])
    # what is cached before the drafts plays no part but for where they start
    s = _table(case, [r.randint(1, 100) + n for _ in paths], gen)
    s.kv = [_cache(case, s.pages, gen) for _ in range(case["layers"])]
    wide = max(len(p) for p in paths)
    s.accepted = torch.tensor([p + [-1] * (wide - len(p)) for p in paths], dtype=torch.int32, device="cuda")
    s.drafted = torch.full((case["batch"],), n, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s.case
    op = case["op"]
    if own:
        import paged_kv_decode_host_gb300 as pkd
        if op == "rotate":
            return pkd.rotate_append_kv(s.q, s.k, s.v, s.rope, s.rows, s.places, s.d_indptr, s.d_indices, s.d_last,
                                        s.cache, rope_positions=s.at, q_norm=s.q_norm, k_norm=s.k_norm, eps=EPS,
                                        k_scale=s.k_scale, v_scale=s.v_scale, kv_layout=case["layout"])
        if op == "tree":
            return s.dec.run(s.q, s.kv, mask=s.mask, depths=s.depths, score_cap=case["cap"], slopes=s.slopes)
        return pkd.accept_kv(s.kv, s.accepted, s.drafted, s.d_indptr, s.d_indices, s.d_last,
                             kv_layout=case["layout"])
    return {"rotate": _plain_rotate, "tree": _plain_tree, "accept": _plain_accept}[op](s)


# ---------------------------------------------------------------- plain forms
def _slots(s, rows, places):
    """(page, place in it) of places of requests."""
    page = s.case["page"]
    return s.d_indices.long()[s.d_indptr.long()[rows] + places // page], places % page


def _norm(x, weight):
    return x if weight is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _rotated(x, cos, sin, pairs):
    """The first 2 * (columns of cos) dims of every head rotated, the others as they are."""
    r = 2 * cos.shape[-1]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., :r // 2], x[..., r // 2:r])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if pairs else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rotate(s):
    case = s.case
    at = s.at[:, None] if s.at.dim() == 1 else s.at
    angle = at.double()[:, s.d_axis] * s.d_freq          # in 64 bits: positions are far
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _rotated(_norm(s.q.float(), s.q_norm), cos, sin, case["pairs"])
    k = _rotated(_norm(s.k.float(), s.k_norm), cos, sin, case["pairs"])
    v = s.v.float()
    if case["kv"] == "e4m3":
        k, v = (x.clamp(-448.0, 448.0) for x in (k / s.k_scale, v / s.v_scale))
    cache = s.cache.view(torch.uint8) if case["kv"] == "e4m3" else s.cache
    k, v = (x.to(s.cache.dtype).view(cache.dtype) for x in (k, v))
    page, place = _slots(s, s.rows.long(), s.places.long())
    if case["layout"] == "NHD":
        cache[page, 0, place], cache[page, 1, place] = k, v
    else:
        cache[page, 0, :, place], cache[page, 1, :, place] = k, v
    return q.bfloat16(), s.cache


def _plain_tree(s):
    case = s.case
    batch, n, kvh, longest = case["batch"], case["drafts"], case["kv_heads"], case["longest"]
    t = torch.arange(longest, device="cuda")
    lens = s.lens.long()[:, None]
    context = lens - n                                                     # [B, 1]
    valid = t[None, :] < lens
    page, place = _slots(s, torch.arange(batch, device="cuda")[:, None], torch.where(valid, t[None, :], 0))
    j = (t[None, :] - context).clamp(0, n - 1)                             # the draft that a token is
    first = torch.arange(n, device="cuda")
    depth = first.expand(batch, n) if s.depths is None else s.depths.long().view(batch, n)
    at_q = context + depth                                                 # [B, n]
    at_k = torch.where(t[None, :] < context, t[None, :], context + depth.gather(1, j))
    if s.causal:
        see = (first[None, :] <= first[:, None]).expand(batch, n, n)
    else:
        see = (s.mask.view(batch, n, -1)[:, :, first // 32] >> (first % 32)) & 1 != 0
    see = see.gather(2, j[:, None, :].expand(batch, n, longest)) | (t[None, :] < context)[:, None, :]
    see = see & valid[:, None, :]
    far = at_q[:, :, None] - at_k[:, None, :]                              # [B, n, L]
    if case["window"]:
        see = see & (far < case["window"])
    k, v = (s.kv[page, c, place] if case["layout"] == "NHD" else s.kv[page, c, :, place] for c in (0, 1))
    k, v = k.float().permute(0, 2, 3, 1), v.float().transpose(1, 2)        # [B, Hkv, D, L], [B, Hkv, L, D]
    q = s.q.float().view(batch, n, kvh, -1, HEAD).permute(0, 2, 3, 1, 4)   # [B, Hkv, g, n, D]
    scores = torch.matmul(q, k[:, :, None]) * SCALE                        # [B, Hkv, g, n, L]
    if case["cap"]:
        scores = case["cap"] * torch.tanh(scores / case["cap"])
    if s.slopes is not None:
        scores = scores - s.slopes.view(1, kvh, -1, 1, 1) * far[:, None, None].float()
    scores = scores.masked_fill(~see[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v[:, :, None]) / torch.where(z == 0, 1.0, z)
    lse = (top + torch.log(z))[..., 0]
    return (out.permute(0, 3, 1, 2, 4).reshape(batch * n, -1, HEAD).bfloat16(),
            lse.permute(0, 3, 1, 2).reshape(batch * n, -1))


def _plain_accept(s):
    case = s.case
    row, i = torch.nonzero(s.accepted >= 0, as_tuple=True)
    context = (s.lens - s.drafted).long()[row]
    from_page, from_place = _slots(s, row, context + s.accepted[row, i].long())
    to_page, to_place = _slots(s, row, context + i)
    for kv in s.kv:
        rows = kv if case["layout"] == "NHD" else kv.transpose(2, 3)      # [pages, 2, P, Hkv, D]
        rows[to_page, :, to_place] = rows[from_page, :, from_place]
    return s.kv


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "tree": _exact_tree, "accept": _exact_accept}[case["op"]](s)


def _exact_rotate(s):
    case = s.case
    page, half = case["page"], case["rotary"] // 2
    at = s.at.reshape(len(s.rows), -1).double()
    turn = torch.stack([at[:, s.axis[i]] * s.freq[i] for i in range(half)], 1)
    z = torch.polar(torch.ones_like(turn), turn)[:, None]                  # [n, 1, half]
    lo = torch.arange(half, device="cuda") * (2 if case["pairs"] else 1)
    hi = lo + (1 if case["pairs"] else half)
    outs = []
    for x, w in ((s.q, s.q_norm), (s.k, s.k_norm)):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / HEAD + EPS) * w.double()
        y = torch.complex(x[..., lo], x[..., hi]) * z
        x = x.clone()
        x[..., lo], x[..., hi] = y.real, y.imag
        outs.append(x)
    top = 448.0 if case["kv"] == "e4m3" else math.inf
    k, v = ((x / c).clamp(-top, top) for x, c in ((outs[1], s.k_scale), (s.v.double(), s.v_scale)))
    cache = s.cache.double()
    slots = [(int(s.indices[int(s.indptr[b]) + t // page]), t % page) for b, t in zip(s.rows.tolist(), s.places.tolist())]
    at = torch.tensor(slots, device="cuda")
    rows = cache if case["layout"] == "NHD" else cache.transpose(2, 3)
    rows[at[:, 0], 0, at[:, 1]] = k
    rows[at[:, 0], 1, at[:, 1]] = v
    return outs[0], cache


def _exact_tree(s):
    case = s.case
    n, kvh, window, cap = case["drafts"], case["kv_heads"], case["window"], case["cap"]
    outs, lses = [], []
    for b, length in enumerate(_lens(case)):
        mine = s.d_indices[int(s.indptr[b]):int(s.indptr[b + 1])].long()
        kv = s.kv[mine].double()
        kv = kv if case["layout"] == "NHD" else kv.transpose(2, 3)
        k, v = (kv[:, c].reshape(-1, kvh, HEAD)[:length] for c in (0, 1))
        q = s.q[b * n:(b + 1) * n].double().view(n, kvh, -1, HEAD)
        x = torch.einsum("nhgd,thd->hgnt", q, k) / math.sqrt(HEAD)
        context = length - n
        depth = torch.arange(n, device="cuda") if s.depths is None else s.depths[b * n:(b + 1) * n].long()
        position = torch.cat([torch.arange(context, device="cuda"), context + depth])
        away = (context + depth)[:, None] - position[None, :]
        see = torch.ones(n, length, dtype=torch.bool, device="cuda")
        words = None if s.causal else s.mask[b * n:(b + 1) * n].cpu().numpy().view(np.uint32)
        for i in range(n):
            row = [j <= i for j in range(n)] if s.causal else [bool(int(words[i, j // 32]) >> (j % 32) & 1) for j in range(n)]
            see[i, context:] = torch.tensor(row, device="cuda")
        if window:
            see &= away < window
        if cap:
            x = cap * torch.tanh(x / cap)
        if s.slopes is not None:
            x = x - s.slopes.double().view(kvh, -1, 1, 1) * away
        x = x.masked_fill(~see, -math.inf)
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[..., None])
        outs.append(torch.einsum("hgnt,thd->nhgd", p, v).reshape(n, -1, HEAD))
        lses.append(lse.permute(2, 0, 1).reshape(n, -1))
    return torch.cat(outs), torch.cat(lses)


def _exact_accept(s):
    case = s.case
    page, lens = case["page"], s.lens.tolist()
    got = []
    for kv in s.kv:
        new = kv.view(torch.int16).cpu().numpy().copy()
        rows = new if case["layout"] == "NHD" else new.swapaxes(2, 3)
        for b, path in enumerate(_paths(case)):
            for i, a in enumerate(path):  # a >= i: what is read was not yet written
                to, src = (lens[b] - case["drafts"] + x for x in (i, a))
                first = int(s.indptr[b])
                rows[s.indices[first + to // page], :, to % page] = rows[s.indices[first + src // page], :, src % page]
        got.append(torch.from_numpy(new).view(torch.bfloat16).cuda().double())
    return got
