"""A decoding step with drafted tokens: their queries and keys rotated and
appended, attention of the drafts over cache and ancestors, and the accepted
ones moved into place.

* :class:`RotaryPositions`, :func:`rotate_append_kv` -- norms per head, rotary
  positions of one or more axes and the append in one kernel.
* :class:`BatchTreeDecodeWithPagedKVCache`, :func:`tree_mask` -- plan / run for
  one or more query tokens per request: trees, chains, pieces of prompts.
* :func:`accept_kv`, :func:`accepted_table` -- the accepted drafts to the front
  of the drafted ones, in every layer, and the page table after it.
"""
from __future__ import annotations

import ctypes
import functools
import math

import numpy as np

from . import (_NOT_HANDLED, FLAG_HND, FLAG_KV_FP8, FLAG_TREE, BatchDecodeWithPagedKVCache,
               PkdError, PlanInfo, _check, _empty_on, _err_arg, _fast, _host_i32, _on, _ptr,
               _stream_ptr, _table_args, load, make_config, schedule_layout)

MAX_AXES = 4
STEP_ABI = 1   # PKD_STEP_ABI of pkd.h


@functools.lru_cache(maxsize=8)
def _pi(bits):
    """pi times 2^bits, by Machin's formula."""
    def arctan(n):   # of 1 / n
        total, power, k = 0, (1 << bits) // n, 1
        while power:
            total += power // k if k % 4 == 1 else -(power // k)
            power //= n * n
            k += 2
        return total

    return 16 * arctan(5) - 4 * arctan(239)


def _turns(freq):
    """freq radians per position as turns times 2^64, modulo 2^64, rounded to nearest: in
    integers (a double's 53 bits would be off by up to 2^-56 turns a position)."""
    bits = 160 + max(0, max(math.frexp(x)[1] for x in freq))
    pi, turns = _pi(bits), []
    for x in freq:
        over, under = x.as_integer_ratio()   # x / (2 pi) * 2^64 = x 2^(63 + bits) / pi
        under *= 2 * pi
        turns.append(((over << (64 + bits)) + (under >> 1)) // under % 2 ** 64)
    return np.array(turns, dtype=np.uint64)


_step_module = None   # the calls on tensors (module), False when not built


def _step():
    """The compiled calls on tensors, if built."""
    global _step_module
    if _step_module is None:
        try:
            import torch   # (its libraries come first)
            from . import _pkd_step as m
            lib = load()
            m.init(STEP_ABI, torch.__version__.split("+")[0],
                   *[ctypes.cast(f, ctypes.c_void_p).value for f in (
                       lib.pkd_rotate_append_kv, lib.pkd_run_tree_scaled, lib.pkd_accept_kv)])
            _step_module = m
        except (ImportError, TypeError):   # (TypeError: the init of an older one)
            _step_module = False
    return _step_module or None


class RotaryPositions:
    """The frequencies of a model's rotary positions, kept on the device as turns
    per position, rounded to 64 bits behind the point (the product with a position is
    exact modulo one turn: position p is off by at most p * 2^-65 turns).

    inv_freq: rotary_dim / 2 angles per position (radians), e.g. theta ** (-2 i /
    rotary_dim), with whatever scaling the model applies.  interleaved: pair i is
    dims (2 i, 2 i + 1) instead of (i, i + rotary_dim / 2); rotary_dim a multiple
    of 16 (8 interleaved).  axes: the axis (0 to 3: time, height, width, ...) whose
    position turns each pair, all 0 by default.  scale multiplies the rotated
    dims."""

    def __init__(self, inv_freq, *, interleaved=False, axes=None, scale=1.0, device=None):
        import torch
        freq = [float(x) for x in (inv_freq.tolist() if hasattr(inv_freq, "tolist") else inv_freq)]
        if not freq or not all(math.isfinite(x) for x in freq):
            raise ValueError("inv_freq must be finite numbers, one per pair of dims")
        self.rotary_dim, self.interleaved = 2 * len(freq), bool(interleaved)
        if self.rotary_dim % (8 if interleaved else 16) or self.rotary_dim > 256:
            raise ValueError("rotary_dim must be a multiple of 16 (8 interleaved), at most 256")
        axes = [0] * len(freq) if axes is None else [int(x) for x in axes]
        if len(axes) != len(freq) or min(axes) < 0 or max(axes) >= MAX_AXES:
            raise ValueError(f"axes must name an axis, 0 to {MAX_AXES - 1}, for every pair")
        if not math.isfinite(scale):
            raise ValueError("scale must be finite")
        self.num_axes, self.scale = max(axes) + 1, float(scale)
        turns = _turns(freq)
        device = torch.device("cuda" if device is None else device)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self.axes = torch.tensor(axes, dtype=torch.int32, device=device)
        self._dev = self.turns.get_device()
        self._args = (self.turns.data_ptr(), self.axes.data_ptr(), self.rotary_dim,
                      int(self.interleaved), self.scale)


_NO_ROPE = (0, 0, 0, 0, 1.0)


def _rows(name, t, bf, dev, n, dim=None):
    """(address, token stride, head stride, heads, dim) of rows of heads."""
    if t.dtype is not bf or t.get_device() != dev:
        raise TypeError(f"{name} must be a bfloat16 tensor on cuda:{dev}")
    shape, (token, head, col) = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != n or (dim is not None and shape[2] != dim):
        raise ValueError(f"{name} must be [{n}, heads, {'D' if dim is None else dim}]")
    if n and (col != 1 or (n > 1 and token % 8) or (shape[1] > 1 and head % 8)
              or t.data_ptr() % 16):
        raise ValueError(f"{name}: contiguous heads on 16-byte boundaries are needed")
    return t.data_ptr(), token, head, shape[1], shape[2]


def rotate_append_kv(q, k_new, v_new, rope, batch_indices, positions, indptr, indices,
                     last_page_len, kv_cache, *, rope_positions=None, q_norm=None, k_norm=None,
                     eps=1e-6, q_out=None, k_scale=1.0, v_scale=1.0, err=None, stream=None,
                     kv_layout="NHD"):
    """Norm and rotate new tokens' queries and keys and write keys and values
    into their page slots.  Returns (q_out, kv_cache).

    q [n, Hq, D] (or None), k_new, v_new [n, Hkv, D]: bf16, last dimension
    contiguous, token and head strides multiples of 8 elements (they may be
    column ranges of one projection's output); D 64, 128 or 256.  rope: a
    :class:`RotaryPositions`, or None.  rope_positions: int32 [n], or [n, axes]
    for several axes; by default ``positions``, which together with
    batch_indices names a token's place in its request's cache as for
    :func:`append_kv` (they differ where a cache was cut, in trees, and with
    several axes).  q_norm, k_norm: [D] bf16 or float32 weights of an RMS norm
    over each head before the rotation.  q_out: bf16 [n, Hq, D], by default a
    new tensor; q itself to rotate in place (else not overlapping the inputs).
    An E4M3 cache takes k / k_scale and v / v_scale, rounded to nearest, at most
    448.  No two tokens may have the same slot.  kv_cache, the table, err and
    kv_layout as for :func:`append_kv`; a token outside the table still has its
    query rotated."""
    if stream is None and q_out is None and kv_layout in ("NHD", "HND"):
        m = _step()
        if m is not None:
            got = m.rotate_append(
                q, k_new, v_new, None if rope is None else rope._args,
                1 if rope is None else rope.num_axes, 0 if rope is None else rope._dev,
                batch_indices, positions, indptr, indices, last_page_len, kv_cache, rope_positions,
                q_norm, k_norm, eps, k_scale, v_scale, kv_layout == "HND", err)
            if got is not NotImplemented:
                if got[0]:
                    _check(got[0], "pkd_rotate_append_kv")
                return got[1], kv_cache
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    dev = kv_cache.get_device()
    fp8 = kv_cache.dtype is torch.float8_e4m3fn or kv_cache.dtype is torch.uint8
    if dev < 0 or not kv_cache.is_contiguous() or not (fp8 or kv_cache.dtype is bf):
        raise TypeError("kv_cache must be a contiguous CUDA tensor, bfloat16 or e4m3")
    if kv_layout not in ("NHD", "HND"):
        raise ValueError("kv_layout must be 'NHD' or 'HND'")
    if kv_cache.dim() != 5 or kv_cache.shape[1] != 2:
        raise ValueError("kv_cache must be [pages, 2, P, Hkv, D] or [pages, 2, Hkv, P, D]")
    pages, _, P, hkv, D = kv_cache.shape
    hnd = kv_layout == "HND"
    if hnd:
        P, hkv = hkv, P
    n = batch_indices.numel()
    k = _rows("k_new", k_new, bf, dev, n, D)
    v = _rows("v_new", v_new, bf, dev, n, D)
    if k[3] != hkv or v[3] != hkv:
        raise ValueError(f"k_new and v_new must have the cache's {hkv} heads")
    hq = 0
    qa = qo = (0, 0, 0)
    if q is not None:
        qa = _rows("q", q, bf, dev, n, D)
        hq = qa[3]
        if q_out is None:
            q_out = _empty_on(stream, (n, hq, D), bf, q.device)
            qo = (q_out.data_ptr(), hq * D, D)
        else:
            qo = _rows("q_out", q_out, bf, dev, n, D)
            if qo[3] != hq:
                raise ValueError("q_out must have q's heads")
            if qo[0] == qa[0] and q_out.stride() != q.stride():
                raise ValueError("q_out must be q with its strides, or memory of its own")
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm need q")
    for name, t in (("batch_indices", batch_indices), ("positions", positions)):
        if t.dtype is not i32 or not t.is_contiguous() or t.get_device() != dev:
            raise TypeError(f"{name} must be a contiguous int32 tensor on cuda:{dev}")
    if positions.numel() != n:
        raise ValueError("batch_indices and positions need one entry per new token")
    num_axes, at, rope_args = 1, 0, _NO_ROPE
    if rope is not None:
        if rope._dev != dev:
            raise ValueError(f"rope is on {rope.turns.device}, the cache on {kv_cache.device}")
        t = positions if rope_positions is None else rope_positions
        if t.dtype is not i32 or not t.is_contiguous() or t.get_device() != dev:
            raise TypeError(f"rope_positions must be a contiguous int32 tensor on cuda:{dev}")
        if t.dim() == 2:
            num_axes = t.shape[1]
        if t.numel() != n * num_axes or not rope.num_axes <= num_axes <= MAX_AXES:
            raise ValueError(f"rope_positions must be [{n}, {rope.num_axes}]: one position per "
                             "token and axis")
        if rope.rotary_dim > D:
            raise ValueError(f"rotary_dim {rope.rotary_dim} is more than the heads' {D}")
        at, rope_args = t.data_ptr(), rope._args
    f32, norms = 0, [0, 0]
    if q_norm is not None or k_norm is not None:
        kinds = {t.dtype for t in (q_norm, k_norm) if t is not None}
        for j, (name, t) in enumerate((("q_norm", q_norm), ("k_norm", k_norm))):
            if t is None:
                continue
            if t.dtype not in (bf, torch.float32) or len(kinds) > 1 or t.get_device() != dev:
                raise TypeError("q_norm and k_norm must be bfloat16, or both float32, on "
                                f"cuda:{dev}")
            if t.shape != (D,) or not t.is_contiguous():
                raise ValueError(f"{name} must be [{D}], contiguous")
            norms[j] = t.data_ptr()
        f32 = int(torch.float32 in kinds)
    batch = _table_args(i32, dev, indptr, indices, last_page_len)
    fast = _fast()
    with _on(dev):
        st = (load().pkd_rotate_append_kv if fast is None else fast.rotate_append)(
            qa[0], qa[1], qa[2], qo[0], qo[1], qo[2], k[0], k[1], k[2], v[0], v[1], v[2],
            norms[0], norms[1], f32, eps, *rope_args, at, num_axes, batch_indices.data_ptr(),
            positions.data_ptr(), n, indptr.data_ptr(), indices.data_ptr(), indices.numel(),
            last_page_len.data_ptr(), batch, kv_cache.data_ptr(), pages, P, hq, hkv, D, k_scale,
            v_scale, (FLAG_HND if hnd else 0) | (FLAG_KV_FP8 if fp8 else 0), _err_arg(err, dev),
            _stream_ptr(stream))
    if st:
        _check(st, "pkd_rotate_append_kv")
    return q_out, kv_cache


def tree_mask(q_indptr, parents):
    """(mask, depths) of drafted trees, on the host: int32 [tokens, words] and
    int32 [tokens], for :meth:`BatchTreeDecodeWithPagedKVCache.run`.

    Request b's drafts are tokens q_indptr[b] .. q_indptr[b+1] - 1; parents[j]
    is a draft's parent, numbered among its request's drafts, before it, or -1
    for a draft that follows the context.  A draft sees itself and its
    ancestors (bit j of its row: draft j); a depth is the number of them."""
    q_indptr, parents = _host_i32(q_indptr), _host_i32(parents)
    if q_indptr.ndim != 1 or q_indptr.size < 1 or q_indptr[0] != 0 or \
            (np.diff(q_indptr.astype(np.int64)) < 0).any():
        raise ValueError("q_indptr must start at 0 and not fall")
    if parents.ndim != 1 or parents.size != q_indptr[-1]:
        raise ValueError("parents must have q_indptr[-1] entries")
    first, counts = q_indptr[:-1].astype(np.int64), np.diff(q_indptr.astype(np.int64))
    number = np.arange(parents.size) - np.repeat(first, counts)
    if (parents < -1).any() or (parents >= number).any():
        raise ValueError("a parent must be -1 or a draft of the same request before its child")
    most = int(counts.max()) if counts.size else 0
    mask = np.zeros((parents.size, max(1, -(-most // 32))), np.uint32)
    depths = np.zeros(parents.size, np.int32)
    for j in range(most):
        at = first[counts > j] + j
        up = parents[at]
        row, has = at[up >= 0], (at - j + up)[up >= 0]
        mask[row] = mask[has]
        depths[row] = depths[has] + 1
        mask[at, j // 32] |= np.uint32(1 << (j % 32))
    return mask.view(np.int32), depths


def plan_host_tree(cfg, q_indptr, indptr, indices, last_page_len, causal=False, window=0):
    """The C++ scheduler for a tree step, on the host (see plan_host)."""
    lib = load()
    q_indptr, indptr = _host_i32(q_indptr), _host_i32(indptr)
    indices, last = _host_i32(indices), _host_i32(last_page_len)
    if q_indptr.shape[0] != last.shape[0] + 1 or indptr.shape[0] != last.shape[0] + 1:
        raise PkdError(-2, "q_indptr and indptr must have batch + 1 entries")
    if last.shape[0] and indices.shape[0] < indptr[-1]:
        raise PkdError(-2, "indices shorter than indptr[-1]")
    off = schedule_layout(cfg)
    words = np.zeros(off[5], dtype=np.int32)
    info = PlanInfo()
    _check(lib.pkd_plan_host_tree(ctypes.byref(cfg), _ptr(q_indptr), _ptr(indptr), _ptr(indices),
                                  _ptr(last), int(last.shape[0]), int(bool(causal)), window,
                                  _ptr(words), words.size, ctypes.byref(info)),
           "pkd_plan_host_tree")
    return words, info.as_dict(), off


class BatchTreeDecodeWithPagedKVCache(BatchDecodeWithPagedKVCache):
    """Attention of one or more query tokens per request over its paged cache:
    drafts to verify, as trees or chains, pieces of prompts, and ordinary decode
    steps of models that cap their scores, bias them by distance or see only a
    window.

    A request's query tokens are the last of its cached tokens: append their
    keys and values first (:func:`append_kv`, :func:`rotate_append_kv`), then
    ``plan`` over the table with them, then ``run`` once per layer.  max_tokens:
    the most query tokens of a plan (and requests).  The cache is bf16 or (kv_dtype
    "e4m3") E4M3, layout NHD or HND, head_dim 128, page size a multiple of 16.  Capture a step with
    ``torch.cuda.graph`` around its runs: it replays under later plans of no
    more query tokens than q has rows.  The runs of one context share its
    workspace: order them, captured ones too, by a stream or an event.
    """

    def __init__(self, num_qo_heads, num_kv_heads, head_dim, page_size, *, max_tokens,
                 max_num_pages, num_pages, alpha=-1, min_chunk_tokens=-1, num_ctas=0,
                 kv_layout="NHD", kv_dtype="bf16", device=None):
        import torch
        if kv_dtype not in ("bf16", "e4m3"):
            raise ValueError("kv_dtype must be 'bf16' or 'e4m3'")
        if kv_layout not in ("NHD", "HND"):
            raise ValueError("kv_layout must be 'NHD' [pages, 2, P, Hkv, D] or "
                             "'HND' [pages, 2, Hkv, P, D]")
        self.kv_layout, self.kv_dtype, self._fp8 = kv_layout, kv_dtype, kv_dtype == "e4m3"
        self.device = torch.device("cuda" if device is None else device)
        self.hq, self.hkv, self.d, self.p = num_qo_heads, num_kv_heads, head_dim, page_size
        self.num_pages = num_pages
        self.causal, self._most = False, 0
        self._create(make_config(num_qo_heads, num_kv_heads, head_dim, page_size, max_tokens,
                                 max_num_pages, num_pages, alpha, min_chunk_tokens, num_ctas,
                                 FLAG_TREE | (FLAG_HND if kv_layout == "HND" else 0)
                                 | (FLAG_KV_FP8 if self._fp8 else 0)))
        self._kv_shape = torch.Size((num_pages, 2, page_size, num_kv_heads, head_dim)
                                    if kv_layout == "NHD" else
                                    (num_pages, 2, num_kv_heads, page_size, head_dim))
        self._dev, self._scale = self.workspace.get_device(), head_dim ** -0.5
        self._shape = tuple(self._kv_shape) + (num_qo_heads,)

    def plan(self, q_indptr, indptr, indices, last_page_len, *, causal=False, window=0,
             stream=None):
        """Schedule one step from host int32 arrays: the page table with the
        query tokens appended, and q_indptr [batch + 1], request b's rows of q
        (at most its cached tokens; none for a request that has no part in the
        step).  causal: every request's query tokens are a chain, and run takes
        no mask; window: 0, or the number of positions a query sees back, its
        own included.  Returns the epoch."""
        causal = 1 if causal else 0
        fast, st = _fast(), _NOT_HANDLED
        if fast is not None:
            st, ep = fast.plan_tree(self._hv, q_indptr, indptr, indices, last_page_len, causal,
                                    window, _stream_ptr(stream))
        if st == _NOT_HANDLED:
            qi, indptr = _host_i32(q_indptr), _host_i32(indptr)
            indices, last = _host_i32(indices), _host_i32(last_page_len)
            batch = last.shape[0]
            if qi.shape[0] != batch + 1 or indptr.shape[0] != batch + 1:
                raise PkdError(-2, "q_indptr and indptr must have batch + 1 entries")
            if batch and indices.shape[0] < indptr[batch]:
                raise PkdError(-2, "indices shorter than indptr[-1]")
            if not -2 ** 31 <= window < 2 ** 31:
                raise OverflowError("window must fit 32 bits")
            st = self._lib.pkd_plan_tree(self._h, _ptr(qi), _ptr(indptr), _ptr(indices),
                                         _ptr(last), batch, causal, window, _stream_ptr(stream),
                                         self._ep_ref)
            ep = self._ep.value
        if st:
            _check(st, "pkd_plan_tree")
        self.epoch, self.causal = ep, bool(causal)
        self.batch = int(q_indptr[-1]) if len(last_page_len) else 0
        return ep

    def run(self, q, kv_cache, *, mask=None, depths=None, scale=None, score_cap=0.0, slopes=None,
            out=None, lse=None, return_lse=True, expect_epoch=0, stream=None, k_scale=1.0,
            v_scale=1.0):
        """Attention for one layer.  Returns (out, lse) or out.

        q [rows, Hq, 128], rows at least the planned query tokens (rows behind
        them are not written in out and lse); with l cached tokens, the last n
        of them the request's query tokens, query i sees the first l - n, and
        query token j where bit j % 32 of word j / 32 of its mask row is set
        (causal plans: j <= i).
        mask: int32 [rows, words], words >= ceil(n / 32) for every request
        (:func:`tree_mask`); needed unless the plan is causal.
        depths: int32 [rows], a query token's position behind the request's
        first l - n tokens, by default its number among the request's; for
        windows and slopes only, not in causal plans.
        scale: of q . k, by default 1 / sqrt(128).  score_cap (0: none; 2^-30 to
        2^96): scores become score_cap * tanh(score / score_cap).  slopes:
        float32 [Hq], then -= slope * (position of the query - position of the
        key).
        out: bf16, like q, by default a new tensor; not on q's memory.
        k_scale, v_scale: the attended key is k_scale * K and the value v_scale *
        V (an E4M3 cache needs them).
        A query that sees nothing gets 0 and an lse of -inf."""
        if stream is None and self.batch is not None:
            m = _step()
            if m is not None:
                got = m.run_tree(self._hv, self._dev, self.batch, self.causal, self._shape, q, kv_cache,
                                 mask, depths, slopes, self._scale if scale is None else scale,
                                 score_cap, out, lse, return_lse, expect_epoch, k_scale, v_scale,
                                 self._fp8)
                if got is not NotImplemented:
                    if got[0]:
                        _check(got[0], "pkd_run_tree")
                    return got[1:] if return_lse else got[1]
        import torch
        if self.batch is None:
            raise PkdError(-5, "run before plan")
        bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
        kv_dt = bf if not self._fp8 else \
            torch.uint8 if kv_cache.dtype is torch.uint8 else torch.float8_e4m3fn
        dev, rows = q.get_device(), q.shape[0]
        if dev != self.workspace.get_device():
            raise ValueError(f"q is on {q.device}, the plan on {self.workspace.device}")
        if rows < self.batch:
            raise ValueError(f"q has {rows} rows, the plan {self.batch} query tokens")
        shape = (rows, self.hq, self.d)
        if mask is not None and mask.dim() != 2:
            raise ValueError("mask must be [rows, words]")
        words = mask.shape[1] if mask is not None else 0
        for name, t, dt, want in (("q", q, bf, shape), ("kv_cache", kv_cache, kv_dt, self._kv_shape),
                                  ("out", out, bf, shape), ("lse", lse, f32, shape[:2]),
                                  ("mask", mask, i32, (rows, words)),
                                  ("depths", depths, i32, shape[:1]),
                                  ("slopes", slopes, f32, (self.hq,))):
            if t is not None and (t.dtype is not dt or t.shape != want or not t.is_contiguous()
                                  or t.get_device() != dev):
                raise ValueError(f"{name} must be a contiguous {dt} tensor {list(want)} on "
                                 f"{q.device}, got {t.dtype} {list(t.shape)} on {t.device}")
        if self.causal and (mask is not None or depths is not None):
            raise ValueError("a causal plan takes no mask and no depths")
        if not self.causal and mask is None and self.batch:
            raise ValueError("the plan is not causal: run needs a mask")
        if out is None:
            out = _empty_on(stream, shape, bf, q.device)
        if lse is None and return_lse:
            lse = _empty_on(stream, shape[:2], f32, q.device)
        fast = _fast()
        with _on(dev):
            st = (self._lib.pkd_run_tree_scaled if fast is None else fast.run_tree)(
                self._hv, q.data_ptr(), rows, kv_cache.data_ptr(), out.data_ptr(),
                lse.data_ptr() if lse is not None else 0,
                mask.data_ptr() if mask is not None else 0, words,
                depths.data_ptr() if depths is not None else 0,
                slopes.data_ptr() if slopes is not None else 0,
                self._scale if scale is None else scale, score_cap, k_scale, v_scale, expect_epoch,
                _stream_ptr(stream))
        if st:
            _check(st, "pkd_run_tree")
        return (out, lse) if return_lse else out

    def plan_shared(self, *args, **kwargs):
        raise PkdError(-1, "a tree context plans query tokens of requests (plan)")

    plan_cascade = plan_shared

    def accumulate_weights(self, *args, **kwargs):
        raise PkdError(-1, "weights are accumulated for steps of one token per request")

    def capture(self, *args, **kwargs):
        raise PkdError(-1, "capture a tree step with torch.cuda.graph around its runs")


def accept_kv(kv_caches, accepted, drafted, indptr, indices, last_page_len, *, err=None,
              stream=None, kv_layout="NHD"):
    """Move every request's accepted drafts to the front of its drafted tokens,
    in place; all layers in one launch.

    kv_caches: a list of 1 to 128 caches as for :func:`append_kv`, of one shape, which do
    not overlap.
    drafted [batch] int32: that many tokens at a request's end are drafts.
    accepted [batch, width] int32 (width up to 1024): the drafts that stay, in
    increasing order (0-based; the first negative entry ends a row).  indptr /
    indices / last_page_len: int32 CUDA tensors, the table with the drafts.
    Slots behind the last accepted draft keep what they hold
    (:func:`accepted_table` gives the table).  err: optional int32 CUDA tensor
    of one element, flagged for requests whose rows are wrong (they are left as
    they are)."""
    if stream is None and kv_layout in ("NHD", "HND"):
        m = _step()
        if m is not None:
            st = m.accept_kv(kv_caches, accepted, drafted, indptr, indices, last_page_len,
                             kv_layout == "HND", err)
            if st is not NotImplemented:
                if st:
                    _check(st, "pkd_accept_kv")
                return kv_caches
    import torch
    layers = len(kv_caches)
    if not 1 <= layers <= 128:
        raise ValueError("1 to 128 caches, one per layer")
    if kv_layout not in ("NHD", "HND"):
        raise ValueError("kv_layout must be 'NHD' or 'HND'")
    c0, i32 = kv_caches[0], torch.int32
    dev, dtype, shape = c0.get_device(), c0.dtype, c0.shape
    fp8 = dtype is torch.float8_e4m3fn or dtype is torch.uint8
    if dev < 0 or not (fp8 or dtype is torch.bfloat16):
        raise TypeError("caches must be bfloat16 or e4m3, on the GPU")
    if len(shape) != 5 or shape[1] != 2:
        raise ValueError("caches must be [pages, 2, P, Hkv, D] or [pages, 2, Hkv, P, D]")
    at = []
    for t in kv_caches:
        if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or \
                not t.is_contiguous():
            raise ValueError(f"kv_caches[{len(at)}] must be a contiguous {dtype} tensor "
                             f"{list(shape)} on cuda:{dev}")
        at.append(t.data_ptr())
    pages, _, P, hkv, D = shape
    if kv_layout == "HND":
        P, hkv = hkv, P
    batch = _table_args(i32, dev, indptr, indices, last_page_len)
    for name, t in (("accepted", accepted), ("drafted", drafted)):
        if t.dtype is not i32 or not t.is_contiguous() or t.get_device() != dev:
            raise TypeError(f"{name} must be a contiguous int32 tensor on cuda:{dev}")
    if accepted.dim() != 2 or accepted.shape[0] != batch or drafted.numel() != batch:
        raise ValueError("accepted must be [batch, width], drafted [batch]")
    lib, fast = load(), _fast()
    rest = (accepted.data_ptr(), accepted.shape[1], drafted.data_ptr(), indptr.data_ptr(),
            indices.data_ptr(), indices.numel(), last_page_len.data_ptr(), batch, pages, P, hkv, D,
            (FLAG_HND if kv_layout == "HND" else 0) | (FLAG_KV_FP8 if fp8 else 0),
            _err_arg(err, dev))
    with _on(dev):
        if fast is not None:
            st = fast.accept_kv(at, *rest, _stream_ptr(stream))
        else:
            st = lib.pkd_accept_kv(layers, (ctypes.c_void_p * layers)(*at), *rest,
                                   _stream_ptr(stream))
    if st:
        _check(st, "pkd_accept_kv")
    return kv_caches


def accepted_table(indptr, indices, last_page_len, page_size, drafted, counts):
    """The page table after :func:`accept_kv`, on the host: (indptr, indices,
    last_page_len, freed page ids), int32 arrays.  drafted: the drafts at every
    request's end, counts: those that were accepted.  Every request has to keep a
    token.  Raises PkdError (PKD_E_BAD_TABLE) for a wrong table."""
    indptr, indices, last = _host_i32(indptr), _host_i32(indices), _host_i32(last_page_len)
    drafted, counts = _host_i32(drafted), _host_i32(counts)
    if page_size < 1:
        raise ValueError("page_size must be at least 1")
    batch = last.shape[0]
    if indptr.shape[0] != batch + 1 or (batch and indptr[0] != 0):
        raise PkdError(-2, "indptr must start at 0 and have batch + 1 entries")
    if drafted.shape != (batch,) or counts.shape != (batch,):
        raise ValueError("drafted and counts need one entry per request")
    held = np.diff(indptr.astype(np.int64))
    used = int(indptr[-1]) if batch else 0
    if (held < 1).any() or (last < 1).any() or (last > page_size).any() or used > indices.shape[0]:
        raise PkdError(-2, "wrong page table")
    lens = page_size * (held - 1) + last
    if (drafted < 0).any() or (drafted > lens).any() or (counts < 0).any() or \
            (counts > drafted).any():
        raise ValueError("a request's drafts are some of its tokens, the accepted some of those")
    now = lens - drafted + counts
    if (now < 1).any():
        raise ValueError("a request would keep no token")
    left = -(-now // page_size)
    keep = np.arange(used) - np.repeat(indptr[:-1], held) < np.repeat(left, held)
    ids = indices[:used]
    return (np.concatenate([[0], np.cumsum(left)]).astype(np.int32), np.ascontiguousarray(ids[keep]),
            (now - page_size * (left - 1)).astype(np.int32), np.ascontiguousarray(ids[~keep]))
