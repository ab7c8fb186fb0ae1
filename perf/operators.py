"""Cases of four serving operators over paged caches, their plain forms and their calls.

* ``latent``: decode attention over a paged cache of one shared latent vector per token
  (the absorbed form: every head's query meets the same cached row, whose first columns are
  also the value);
* ``append``: a step's (or a prompt's) new latent rows written into their page slots;
* ``accumulate``: the attention weight that every cached token receives in a step, added to
  the running sum kept beside the cache;
* ``evict``: the cache of a request cut to a budget of tokens by that sum, in place.

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits; with
``own`` true it makes the calls a user makes of the package.
"""
import math
import random

import numpy as np
import torch

own = False

LATENT, ROPE = 512, 64          # cached row: latent columns, then the rotary key's
ROW = LATENT + ROPE
HEAD = 128                      # head dim of the K / V caches
SCALE = 1.0 / math.sqrt(192.0)  # softmax scale of the latent form: heads of 128 + 64 before absorption


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's chat on a slice of the heads: latency alone counts
        dict(name="latent one request", op="latent", heads=16, batch=1, longest=517, lens="even", page=64),
        # an ordinary serving batch, 16 heads per GPU, ragged lengths
        dict(name="latent batch 16 heads", op="latent", heads=16, batch=64, longest=8192, lens="ragged", page=64),
        # every head on one GPU: as much arithmetic as bytes
        dict(name="latent batch 128 heads", op="latent", heads=128, batch=32, longest=8192, lens="ragged", page=16),
        # a long document beside short chats, heads that fill no tile
        dict(name="latent long document", op="latent", heads=40, batch=9, longest=100_003, lens="skewed", page=16),
        # one decode step's new tokens
        dict(name="append step", op="append", batch=64, tokens=1, page=64),
        # prompts of odd lengths written at once
        dict(name="append prompts", op="append", batch=7, tokens=4681, page=16),
        # three short requests
        dict(name="accumulate short", op="accumulate", heads=32, kv_heads=8, batch=3, longest=37, lens="ragged",
             page=16, kv="bf16", layout="NHD"),
        # a decode batch of 64 requests, one layer
        dict(name="accumulate batch", op="accumulate", heads=32, kv_heads=8, batch=64, longest=8192, lens="ragged",
             page=16, kv="bf16", layout="NHD"),
        # 8-bit cache, one long request among short ones
        dict(name="accumulate skewed e4m3", op="accumulate", heads=64, kv_heads=8, batch=17, longest=50_021,
             lens="skewed", page=16, kv="e4m3", layout="HND"),
        # one token over the budget in every request, as in each step of steady decoding
        dict(name="evict step", op="evict", kv_heads=8, batch=32, longest=1025, lens="even", page=16, layers=2,
             budget=1024, per_head=True, layout="NHD"),
        # a block of tokens evicted at once from ragged requests
        dict(name="evict block", op="evict", kv_heads=8, batch=24, longest=4609, lens="ragged", page=16, layers=4,
             budget=2048, per_head=True, layout="NHD"),
        # half of a long document, the same tokens for all heads
        dict(name="evict long shared", op="evict", kv_heads=4, batch=2, longest=65_539, lens="even", page=32,
             layers=2, budget=32_768, per_head=False, layout="HND"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["latent", "latent", "append", "accumulate", "accumulate", "evict", "evict"])
    page = rng.choice([16, 32, 64])
    lens = rng.choice(["even", "ragged", "skewed"])
    if op == "append":
        batch = _log(rng, 1, 256)
        return dict(op=op, batch=batch, tokens=_log(rng, 1, max(1, 32_000 // batch)), page=page)
    if op == "latent":
        batch = _log(rng, 1, 64)
        longest = _log(rng, 1, min(100_000, 130_000 // batch * (4 if lens == "skewed" else 1)))
        return dict(op=op, heads=rng.choice([8, 16, 20, 32, 40, 64, 96, 128]), batch=batch, longest=longest, lens=lens, page=page)
    if op == "accumulate":
        batch = _log(rng, 1, 64)
        longest = _log(rng, 1, min(50_000, 230_000 // batch))
        kv_heads = rng.choice([1, 2, 4, 8])
        return dict(op=op, heads=kv_heads * rng.choice([1, 2, 4, 8]), kv_heads=kv_heads, batch=batch, longest=longest,
                    lens=lens, page=rng.choice([1, 5, 16, 64]), kv=rng.choice(["bf16", "bf16", "e4m3"]),
                    layout=rng.choice(["NHD", "HND"]))
    batch = _log(rng, 1, 32)
    longest = _log(rng, 2, min(60_000, 80_000 // batch))
    return dict(op=op, kv_heads=rng.choice([1, 2, 4, 8]), batch=batch, longest=longest, lens=lens,
                page=rng.choice([1, 16, 64]), layers=rng.choice([1, 2]), budget=max(1, int(longest * rng.uniform(0.3, 1.0))),
                per_head=rng.choice([True, False]), layout=rng.choice(["NHD", "HND"]))


def _lens(case):
    """The lengths of a case's requests: fixed by its sizes."""
    n, longest = case["batch"], case["longest"]
    r = random.Random("%d,%d,%s" % (n, longest, case["lens"]))
    if case["lens"] == "even":
        return [longest] * n
    if case["lens"] == "ragged":
        got = [r.randint(1, longest) for _ in range(n)]
    else:  # one long, the others short
        got = [r.randint(1, max(1, longest // 128)) for _ in range(n)]
    got[r.randrange(n)] = longest
    return got


def _window(case):
    """Sinks and recent tokens that an eviction never takes."""
    return min(4, case["budget"] // 8), case["budget"] // 8


def work(case):
    op = case["op"]
    if op == "append":
        n = case["batch"] * case["tokens"]
        return {"bytes": n * (2 * ROW * 2 + 8), "flops": 0}
    lens = _lens(case)
    total, batch = sum(lens), case["batch"]
    pages = sum(-(-n // case["page"]) for n in lens)
    if op == "latent":
        h = case["heads"]
        return {"bytes": total * ROW * 2 + batch * h * (ROW * 2 + LATENT * 2 + 4) + 4 * pages,
                "flops": 2 * total * h * (ROW + LATENT)}
    if op == "accumulate":
        h, kvh, size = case["heads"], case["kv_heads"], 1 if case["kv"] == "e4m3" else 2
        return {"bytes": total * kvh * (HEAD * size + 8) + batch * h * (HEAD * 2 + 4) + 4 * pages,
                "flops": 2 * total * h * HEAD}
    # evict: the sums and ages of every token of a request over its budget, and each kept
    # token behind the budget moved into a freed slot: read and written once
    over = [n for n in lens if n > case["budget"]]
    moved = sum((n - case["budget"]) * case["budget"] / n for n in over)
    one = case["layers"] * case["kv_heads"]
    return {"bytes": one * (sum(over) * 8 + moved * (2 * 2 * HEAD * 2 + 8)) + 4 * pages + 1, "flops": 0}


# ---------------------------------------------------------------- inputs
class State:
    pass


def _generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _table(case, lens, gen):
    """The page table of the requests, its pages scattered over the pool; and for the plain
    forms every token's pool slot, padded to the longest request."""
    s, page = State(), case["page"]
    counts = [-(-n // page) for n in lens]
    s.pages = sum(counts) + 3
    s.indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    s.last = np.array([n - page * (c - 1) for n, c in zip(lens, counts)], np.int32)
    where = torch.randperm(s.pages, generator=gen, device="cuda")[: int(s.indptr[-1])].int()
    s.indices = where.cpu().numpy()
    s.lens = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s.d_indptr = torch.from_numpy(s.indptr).cuda()
    s.d_indices = where.contiguous()
    s.d_last = torch.from_numpy(s.last).cuda()
    return s


def _slots(case, s):
    """[batch, longest] pool slot (page * page size + place) of every token, 0 behind the
    end, and which of them are tokens."""
    t = torch.arange(case["longest"], device="cuda")
    valid = t[None, :] < s.lens[:, None]
    at = (s.d_indptr[:-1, None].long() + t[None, :] // case["page"]).clamp_(max=len(s.indices) - 1)
    slot = s.d_indices.long()[at] * case["page"] + t[None, :] % case["page"]
    return torch.where(valid, slot, 0), valid


def _kv_shape(case, pages):
    page, h = case["page"], case["kv_heads"]
    return (pages, 2, page, h, HEAD) if case["layout"] == "NHD" else (pages, 2, h, page, HEAD)


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
    gen = _generator(seed)
    op = case["op"]
    if op == "append":
        return _prepare_append(case, gen)
    lens = _lens(case)
    s = _table(case, lens, gen)
    s.case = case
    if op == "latent":
        s.q = _normal((case["batch"], case["heads"], ROW), gen)
        s.cache = _normal((s.pages, case["page"], ROW), gen)
        if own:
            import paged_kv_decode_host_gb300 as pkd
            s.dec = pkd.BatchLatentDecodeWithPagedCache(
                case["heads"], LATENT, ROPE, case["page"], scale=SCALE, max_batch=case["batch"],
                max_num_pages=len(s.indices), num_pages=s.pages)
            s.dec.plan(s.indptr, s.indices, s.last)
    elif op == "accumulate":
        e4m3 = case["kv"] == "e4m3"
        s.k_scale = 1.0 / 112.0 if e4m3 else 1.0
        s.q = _normal((case["batch"], case["heads"], HEAD), gen)
        s.kv = _normal(_kv_shape(case, s.pages), gen, torch.float8_e4m3fn if e4m3 else torch.bfloat16)
        scores, valid = _scores(s)
        s.lse = torch.logsumexp(scores.masked_fill_(~valid[:, None, None, :], -math.inf), -1).reshape(case["batch"], -1)
        del scores
        shape = (s.pages, case["kv_heads"], case["page"])
        s.weights = torch.rand(shape, generator=gen, device="cuda") ** 4
        s.positions = torch.full(shape, -1, dtype=torch.int32, device="cuda")
        s.new = torch.ones(case["batch"], dtype=torch.int32, device="cuda")  # this step's token
        s.seen = s.lens + torch.randint(0, 1000, (case["batch"],), generator=gen, device="cuda", dtype=torch.int32)
        if own:
            import paged_kv_decode_host_gb300 as pkd
            s.dec = pkd.BatchDecodeWithPagedKVCache(
                case["heads"], case["kv_heads"], HEAD, case["page"], max_batch=case["batch"],
                max_num_pages=len(s.indices), num_pages=s.pages, kv_dtype=case["kv"], kv_layout=case["layout"])
            s.dec.plan(s.indptr, s.indices, s.last)
    else:
        layers, shape = case["layers"], (s.pages, case["kv_heads"], case["page"])
        s.kv = [_normal(_kv_shape(case, s.pages), gen) for _ in range(layers)]
        # weights as sums of a few steps' attention: long-tailed, some of them equal
        w = -torch.log(torch.rand((layers,) + shape, generator=gen, device="cuda").clamp_(min=1e-30))
        w = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.3, torch.floor(w * 16) / 16, w)
        # ages of a cache that was cut before: the older half out of order
        slot, valid = _slots(case, s)
        t = torch.arange(case["longest"], device="cuda")[None, :].expand_as(slot)
        half = (s.lens // 2)[:, None]
        order = torch.where(t < half, half - 1 - t, t)[valid].int()
        p = torch.full((layers,) + shape, -1, dtype=torch.int32, device="cuda")
        at = slot[valid]
        odd = torch.randint(0, 2, (layers, at.numel(), case["kv_heads"]), generator=gen, device="cuda", dtype=torch.int32)
        if not case["per_head"]:
            odd = odd[:, :, :1].expand_as(odd)
        p[:, at // case["page"], :, at % case["page"]] = (2 * order[None, :, None] + odd).transpose(0, 1)
        s.seen = 2 * s.lens
        # the sums and ages as a user keeps them, and the step's own (an eviction updates them in
        # place: every pass starts from what the steps before left)
        s.before = torch.stack([w.view(torch.int32), p])
        s.track = s.before.clone()
        s.weights = [s.track[0, l].view(torch.float32) for l in range(layers)]
        s.positions = [s.track[1, l] for l in range(layers)]
    return s


def _prepare_append(case, gen):
    batch, n = case["batch"], case["tokens"]
    r = random.Random("%d,%d" % (batch, n))
    old = [0 if n > 64 else r.randint(0, 4096) for _ in range(batch)]  # tokens already there
    s = _table(dict(case, longest=max(old) + n), [o + n for o in old], gen)
    s.case = case
    s.cache = _normal((s.pages, case["page"], ROW), gen)
    # one projection's output: the latent and the rotary key are column ranges of its rows
    both = _normal((batch * n, ROW + 8), gen)
    s.latent, s.rope = both[:, :LATENT], both[:, LATENT:ROW]
    s.rows = torch.arange(batch, device="cuda", dtype=torch.int32).repeat_interleave(n)
    s.places = (torch.tensor(old, device="cuda", dtype=torch.int32)[:, None]
                + torch.arange(n, device="cuda", dtype=torch.int32)[None, :]).reshape(-1).contiguous()
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    op = s.case["op"]
    if own:
        import paged_kv_decode_host_gb300 as pkd
        if op == "latent":
            return s.dec.run(s.q, s.cache)
        if op == "append":
            return pkd.append_latent(s.latent, s.rope, s.rows, s.places, s.d_indptr, s.d_indices, s.d_last, s.cache)
        if op == "accumulate":
            s.dec.accumulate_weights(s.q, s.kv, s.lse, s.weights, positions=s.positions, new_tokens=s.new,
                                     seen=s.seen, k_scale=s.k_scale)
            return s.weights, s.positions
        s.track.copy_(s.before)
        sinks, recent = _window(s.case)
        pkd.evict_kv(s.kv, s.weights, s.positions, s.d_indptr, s.d_indices, s.d_last, s.seen, s.case["budget"],
                     max_len=s.case["longest"], sinks=sinks, recent=recent, per_head=s.case["per_head"],
                     kv_layout=s.case["layout"])
        return s.kv, s.weights, s.positions
    if op == "latent":
        return _plain_latent(s)
    if op == "append":
        return _plain_append(s)
    if op == "accumulate":
        return _plain_accumulate(s)
    return _plain_evict(s)


# ---------------------------------------------------------------- plain forms
def _plain_latent(s):
    slot, valid = _slots(s.case, s)
    rows = s.cache.view(-1, ROW)[slot].float()                         # [B, L, 576]
    scores = torch.matmul(s.q.float(), rows.transpose(1, 2)) * SCALE   # [B, H, L]
    scores = scores.masked_fill(~valid[:, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows[:, :, :LATENT]) / z
    return out.bfloat16(), (top + torch.log(z))[..., 0]


def _plain_append(s):
    page = s.case["page"]
    slot = s.d_indices.long()[s.d_indptr.long()[s.rows.long()] + s.places.long() // page] * page + s.places.long() % page
    flat = s.cache.view(-1, ROW)
    flat[slot, :LATENT] = s.latent
    flat[slot, LATENT:] = s.rope
    return s.cache


def _scores(s):
    """[B, Hkv, g, L] scaled scores of the step's queries and every cached key."""
    case = s.case
    slot, valid = _slots(case, s)
    page, place = slot // case["page"], slot % case["page"]
    keys = s.kv[:, 0]
    keys = (keys.view(torch.uint8) if case["kv"] == "e4m3" else keys)
    k = keys[page, place] if case["layout"] == "NHD" else keys[page, :, place]          # [B, L, Hkv, D]
    k = (k.view(torch.float8_e4m3fn) if case["kv"] == "e4m3" else k).float().permute(0, 2, 3, 1)
    q = s.q.float().view(case["batch"], case["kv_heads"], -1, HEAD)
    return torch.matmul(q, k) * (s.k_scale / math.sqrt(HEAD)), valid


def _plain_accumulate(s):
    case = s.case
    scores, valid = _scores(s)
    lse = s.lse.view(case["batch"], case["kv_heads"], -1, 1)
    w = torch.exp(scores - lse).sum(2).transpose(1, 2)[valid]           # [tokens, Hkv]
    slot, _ = _slots(case, s)
    page, place = slot[valid] // case["page"], slot[valid] % case["page"]
    t = torch.arange(case["longest"], device="cuda")[None, :].expand_as(valid)
    fresh = (t >= (s.lens - s.new)[:, None])[valid][:, None]
    age = (s.seen[:, None] - s.lens[:, None] + t)[valid][:, None].int()
    s.weights[page, :, place] = torch.where(fresh, 0.0, s.weights[page, :, place]) + w
    s.positions[page, :, place] = torch.where(fresh, age, s.positions[page, :, place])
    return s.weights, s.positions


def _plain_evict(s):
    case = s.case
    layers, heads, keep = case["layers"], case["kv_heads"], case["budget"]
    sinks, recent = _window(case)
    slot, valid = _slots(case, s)
    page, place = slot // case["page"], slot % case["page"]
    s.track.copy_(s.before)
    w = torch.stack(s.weights)[:, page, :, place].permute(2, 0, 3, 1)   # [layers, B, H, L]
    p = torch.stack(s.positions)[:, page, :, place].permute(2, 0, 3, 1)
    if not case["per_head"]:
        total = w[:, :, :1].double()
        for h in range(1, heads):
            total = total + w[:, :, h:h + 1].double()
        w, p = total.float(), p[:, :, :1]
    safe = (p < sinks) | (p >= (s.seen - recent)[None, :, None, None])
    key = w.double().nan_to_num(nan=-math.inf, posinf=1e300, neginf=-1e300).masked_fill(safe, math.inf)
    key = key.masked_fill(~valid[None, :, None, :], -math.inf)
    # behind the end come last: a stable order puts the lower place first among equals
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, torch.arange(case["longest"], device="cuda").expand_as(order).contiguous())
    t = torch.arange(case["longest"], device="cuda")
    n = s.lens[None, :, None, None]
    kept = (rank < keep) & valid[None, :, None, :]
    hole = ~kept & (t < keep) & (n > keep)
    tail = kept & (t >= keep)
    # the i-th hole before the budget takes the i-th kept token behind it
    hl, hb, hh, ht = torch.nonzero(hole, as_tuple=True)
    tl, tb, th, tt = torch.nonzero(tail, as_tuple=True)
    if not case["per_head"]:
        many = torch.arange(heads, device="cuda")
        hl, hb, ht, tl, tb, tt = (x.repeat_interleave(heads) for x in (hl, hb, ht, tl, tb, tt))
        th = many.repeat(len(tt) // heads)
    to_page, to_place, from_page, from_place = page[hb, ht], place[hb, ht], page[tb, tt], place[tb, tt]
    for l in range(layers):
        m = tl == l
        a, b, c, d, h = to_page[m], to_place[m], from_page[m], from_place[m], th[m]
        if case["layout"] == "NHD":
            s.kv[l][a, :, b, h] = s.kv[l][c, :, d, h]
        else:
            s.kv[l][a, :, h, b] = s.kv[l][c, :, h, d]
        s.weights[l][a, h, b] = s.weights[l][c, h, d]
        s.positions[l][a, h, b] = s.positions[l][c, h, d]
    return s.kv, s.weights, s.positions


# ---------------------------------------------------------------- from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case["page"]
    if op == "append":
        out = s.cache.clone()
        slots = [int(s.indices[int(s.indptr[b]) + t // page]) * page + t % page
                 for b, t in zip(s.rows.tolist(), s.places.tolist())]
        out.view(-1, ROW)[torch.tensor(slots, device="cuda")] = torch.cat([s.latent, s.rope], 1)
        return out.double()
    lens = _lens(case)
    if op == "latent":
        outs, lses = [], []
        for i, n in enumerate(lens):
            mine = s.d_indices[int(s.indptr[i]):int(s.indptr[i + 1])].long()
            c = s.cache[mine].reshape(-1, ROW)[:n].double()
            x = torch.einsum("hd,td->ht", s.q[i].double(), c) * SCALE
            lse = torch.logsumexp(x, 1)
            outs.append(torch.exp(x - lse[:, None]) @ c[:, :LATENT])
            lses.append(lse)
        return torch.stack(outs), torch.stack(lses)
    heads = case["kv_heads"]
    if op == "accumulate":
        weights, positions = s.weights.double(), s.positions.clone()
        for i, n in enumerate(lens):
            mine = s.d_indices[int(s.indptr[i]):int(s.indptr[i + 1])].long()
            k = s.kv.view(torch.uint8)[mine, 0].view(s.kv.dtype).double() if case["kv"] == "e4m3" else s.kv[mine, 0].double()
            k = k if case["layout"] == "NHD" else k.transpose(1, 2)
            k = k.reshape(-1, heads, HEAD)[:n]
            q = s.q[i].double().view(heads, -1, HEAD)
            x = torch.einsum("hgd,thd->hgt", q, k) * (s.k_scale / math.sqrt(HEAD))
            got = torch.exp(x - s.lse[i].double().view(heads, -1, 1)).sum(1)
            was = weights[mine].transpose(0, 1).reshape(heads, -1)
            was[:, n - 1] = 0.0
            was[:, :n] += got
            weights[mine] = was.view(heads, -1, page).transpose(0, 1)
            age = positions[mine].transpose(0, 1).reshape(heads, -1)
            age[:, n - 1] = s.seen[i] - 1
            positions[mine] = age.view(heads, -1, page).transpose(0, 1)
        return weights, positions
    if sum(lens) * case["layers"] * heads > 4_000_000:
        return None
    keep = case["budget"]
    sinks, recent = _window(case)
    kvs, ws, ps = [], [], []
    for l in range(case["layers"]):
        kv = s.kv[l].cpu().view(torch.int16).numpy().copy()
        if case["layout"] == "HND":
            kv = kv.swapaxes(2, 3)          # a view: [pages, 2, P, H, D]
        w, p = s.weights[l].cpu().numpy().copy(), s.positions[l].cpu().numpy().copy()
        for i, n in enumerate(lens):
            if n <= keep:
                continue
            at = np.arange(n)
            pg, pl = s.indices[int(s.indptr[i]) + at // page], at % page
            seen = int(s.seen[i])
            for h in range(heads if case["per_head"] else 1):
                x = w[pg, h, pl].astype(np.float64)
                for more in range(1, 1 if case["per_head"] else heads):
                    x = x + w[pg, more, pl].astype(np.float64)
                x = x.astype(np.float32)
                a = p[pg, h, pl]
                safe = (a < sinks) | (a >= seen - recent)
                best = np.lexsort((at, -x.astype(np.float64), ~safe))[:keep]
                kept = np.zeros(n, bool)
                kept[best] = True
                to, src = np.nonzero(~kept[:keep])[0], keep + np.nonzero(kept[keep:])[0]
                for hh in [h] if case["per_head"] else range(heads):
                    kv[pg[to], :, pl[to], hh] = kv[pg[src], :, pl[src], hh]
                for hh in [h] if case["per_head"] else range(heads - 1, -1, -1):
                    w[pg[to], hh, pl[to]] = w[pg[src], hh, pl[src]]
                    p[pg[to], hh, pl[to]] = p[pg[src], hh, pl[src]]
        kv = kv.swapaxes(2, 3) if case["layout"] == "HND" else kv
        kvs.append(torch.from_numpy(np.ascontiguousarray(kv)).view(torch.bfloat16).double())
        ws.append(torch.from_numpy(w).double())
        ps.append(torch.from_numpy(p))
    return kvs, ws, ps
