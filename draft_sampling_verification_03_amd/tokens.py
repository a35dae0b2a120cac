"""torch-facing wrappers of include/dspark_tokens.h: rotary positions (of a batch,
and on the way into the paged cache) and edits of logits by token histories.

As in serving.py every tensor is checked before anything is launched, outputs and
workspaces are allocated on the launch stream, and no arithmetic of the methods happens
here.  Rows of queries, keys, values and logits may be strided in their first dimension
(slices of one projection's output); everything else is contiguous.
"""
import numpy as np
import torch

from . import _abi as A
from .api import F32, I32, _check, _dt, _empty, _on_stream
from .serving import _PER, _RowArgs, _launch, _ptr, _width, _workspace

I64 = torch.int64
_LAYOUTS = {"half": A.DSPARK_ROTARY_HALF, "interleaved": A.DSPARK_ROTARY_INTERLEAVED}
_SCALINGS = {None: A.DSPARK_ROTARY_PLAIN, "linear": A.DSPARK_ROTARY_LINEAR,
             "base": A.DSPARK_ROTARY_BASE, "by_turns": A.DSPARK_ROTARY_BY_TURNS}


class RotaryPlan:
    """How heads rotate: the frequencies of the rot / 2 pairs, which elements are a pair
    and the factor of the rotated values.  Made once; it needs no table of positions.

    layout     "half" (elements i and i + rot / 2) or "interleaved" (2 i and 2 i + 1)
    scaling    None, "linear" (all frequencies over `factor`), "base" (the base grown so
               that the slowest pair is stretched by `factor`) or "by_turns" (pairs that
               turn less than `slow` times over `context` tokens are stretched by `factor`,
               those with more than `fast` not at all, between them in part)
    frequencies  radians a token instead, rot / 2 of them (any other rule)"""

    def __init__(self, rot, *, base=10000.0, layout="half", scaling=None, factor=1.0, context=0.0,
                 slow=1.0, fast=32.0, magnitude=1.0, frequencies=None, device="cuda"):
        if layout not in _LAYOUTS:
            raise ValueError(f"RotaryPlan: layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
        if scaling not in _SCALINGS:
            raise ValueError(f"RotaryPlan: no scaling {scaling!r}")
        if rot < 2 or rot > 256 or rot % 2:
            raise ValueError(f"RotaryPlan: rot must be even and within [2, 256], got {rot}")
        f, turns = np.empty(rot // 2, np.float64), np.empty(rot // 2, np.uint64)
        if frequencies is None:
            _check(A.dspark_rotary_frequencies(rot, base, _SCALINGS[scaling], factor, context, slow,
                                               fast, f.ctypes.data), "dspark_rotary_frequencies")
        else:
            if scaling is not None:
                raise ValueError("RotaryPlan: frequencies are given or scaled, not both")
            given = (frequencies.detach().cpu().double().numpy() if torch.is_tensor(frequencies)
                     else np.asarray(frequencies, np.float64))
            if given.shape != f.shape:
                raise ValueError(f"RotaryPlan: {rot // 2} frequencies are needed, got {given.shape}")
            f[:] = given
        _check(A.dspark_rotary_turns(rot // 2, f.ctypes.data, turns.ctypes.data), "dspark_rotary_turns")
        self.rot, self.layout, self.magnitude = rot, _LAYOUTS[layout], float(magnitude)
        self.frequencies = f
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)


def _plan(a, plan):
    if not isinstance(plan, RotaryPlan):
        raise TypeError(f"{a.where}: plan must be a RotaryPlan, got {type(plan).__name__}")
    a.req(plan.turns, "plan.turns", I64, (plan.rot // 2,))
    return plan.turns.data_ptr()


def _rotate(where, q, k, plan, positions, row_offset, kv_len, ws, stream, out):
    a = _RowArgs(where)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError(f"{where}: q must be a [rows][heads][D] tensor")
    dt = _dt(q)
    n, Hq, D = q.shape
    q_stride, Hkv, k_stride = a.rows(q, "q", q.dtype, (n, Hq, D)), 0, 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise ValueError(f"{where}: k must be a [rows][heads][D] tensor")
        Hkv = k.shape[1]
        k_stride = a.rows(k, "k", q.dtype, (n, Hkv, D))
    turns = _plan(a, plan)
    R = n
    if row_offset is not None:
        R = _width(a, row_offset, "row_offset") - 1
        a.req(row_offset, "row_offset", I32, (R + 1,))
    if positions is not None:
        a.req(positions, "positions", I32, (n,))
    if kv_len is not None:
        a.req(kv_len, "kv_len", I32, (R,))
    index, dev = a.gpu(), q.device
    with _on_stream(stream):
        if out is None:
            out = {"q": q.new_empty((n, Hq, D)), "k": None if k is None else q.new_empty((n, Hkv, D))}
            qo, ko = Hq * D, Hkv * D
        else:
            qo = a.rows(out.get("q"), "out['q']", q.dtype, (n, Hq, D))
            ko = 0 if k is None else a.rows(out.get("k"), "out['k']", q.dtype, (n, Hkv, D))
            a.gpu()
        buf = _workspace(ws, 256, dev, index, stream)
    _launch("dspark_rotary_backward" if where == "rotary_backward" else "dspark_rotary", index, stream,
            n, Hq, Hkv, D, plan.rot, plan.layout, dt, plan.magnitude, turns, _ptr(positions), R,
            _ptr(row_offset), _ptr(kv_len), q.data_ptr(), q_stride, _ptr(k), k_stride,
            out["q"].data_ptr(), qo, None if k is None else out["k"].data_ptr(), ko, buf.data_ptr(),
            buf.numel())
    return out


def rotary(q, k=None, *, plan, positions=None, row_offset=None, kv_len=None, ws=None, stream=None,
           out=None):
    """q [rows][Hq][D] and k [rows][Hkv][D] with their positions rotated in: positions
    [rows] int32; or of the sequences row_offset [R + 1], each from 0 on or, with kv_len
    [R], the last tokens of so many; or 0, 1, ... (with kv_len [rows] alone: kv_len - 1).
    Returns {"q", "k"}; `out` may name the inputs (in place) or tensors beside them in one
    buffer, not over a part of them."""
    return _rotate("rotary", q, k, plan, positions, row_offset, kv_len, ws, stream, out)


def rotary_backward(g_q, g_k=None, *, plan, positions=None, row_offset=None, kv_len=None, ws=None,
                    stream=None, out=None):
    """From the gradients of rotary()'s outputs to those of its inputs."""
    return _rotate("rotary_backward", g_q, g_k, plan, positions, row_offset, kv_len, ws, stream, out)


def cache_append(q, k_new, v_new, k_pages, v_pages, table, kv_len, *, plan=None, row_offset=None,
                 positions=None, ws=None, stream=None, out=None):
    """What stands before cache_attend() in a layer: the new rows' keys, rotated by their
    place in the cache (or `positions` [rows]), and values go into their pages; returns
    the rotated queries (None without q; `out` may be q itself).  cache_attend() then
    takes no k_new and v_new.  Shapes as there; plan None: no rotation."""
    a = _RowArgs("cache_append")
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 3:
        raise ValueError("cache_append: k_new must be a [rows][Hkv][D] tensor")
    dt, dtype = _dt(k_new), k_new.dtype
    n, Hkv, D = k_new.shape
    kn = a.rows(k_new, "k_new", dtype, (n, Hkv, D))
    vn = a.rows(v_new, "v_new", dtype, (n, Hkv, D))
    if kn != vn:
        raise ValueError("cache_append: k_new and v_new must have the same row stride")
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("cache_append: k_pages must be a [n_pages][Hkv][page][D] tensor")
    n_pages, _, page, _ = k_pages.shape
    k_stride = a.rows(k_pages, "k_pages", dtype, (n_pages, Hkv, page, D))
    v_stride = a.rows(v_pages, "v_pages", dtype, (n_pages, Hkv, D, page))
    R, width = _width(a, kv_len, "kv_len"), _width(a, table, "table")
    a.req(kv_len, "kv_len", I32, (R,))
    a.req(table, "table", I32, (R, width))
    if row_offset is not None:
        a.req(row_offset, "row_offset", I32, (R + 1,))
    elif n != R:
        raise ValueError(f"cache_append: {n} rows for {R} requests need row_offset")
    rot, layout, magnitude, turns = 0, 0, 1.0, None
    if plan is not None:
        turns = _plan(a, plan)
        rot, layout, magnitude = plan.rot, plan.layout, plan.magnitude
    if positions is not None:
        a.req(positions, "positions", I32, (n,))
    Hq, q_stride, qo = 0, 0, 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("cache_append: q must be a [rows][Hq][D] tensor")
        Hq = q.shape[1]
        q_stride = a.rows(q, "q", dtype, (n, Hq, D))
    elif out is not None:
        raise ValueError("cache_append: out is for the queries, and there are none")
    index, dev = a.gpu(), k_new.device
    with _on_stream(stream):
        if q is not None and out is None:
            out, qo = q.new_empty((n, Hq, D)), Hq * D
        elif q is not None:
            qo = a.rows(out, "out", dtype, (n, Hq, D))
            a.gpu()
        buf = _workspace(ws, 256, dev, index, stream)
    _launch("dspark_cache_append", index, stream, R, n, Hq, Hkv, D, page, width, n_pages, dt, rot,
            layout, magnitude, turns, _ptr(positions), _ptr(q), q_stride, _ptr(out), qo,
            k_new.data_ptr(), v_new.data_ptr(), kn, k_pages.data_ptr(), v_pages.data_ptr(), k_stride,
            v_stride, table.data_ptr(), _ptr(row_offset), kv_len.data_ptr(), buf.data_ptr(),
            buf.numel())
    return out


class _Edits:
    """The arguments that both directions of the edits share, checked."""

    def __init__(self, where, X, row_offset, history, hist_len, prompt_len, drafts, repetition, mask,
                 mask_index):
        self.a = a = _RowArgs(where)
        if not isinstance(X, torch.Tensor) or X.dim() != 2:
            raise ValueError(f"{where}: logits must be a [n_rows][V] tensor")
        self.dt = _dt(X)
        self.n, self.V = n, V = X.shape
        self.stride = a.rows(X, "X", X.dtype, (n, V))
        self.R = R = n
        if row_offset is not None:
            self.R = R = _width(a, row_offset, "row_offset") - 1
            a.req(row_offset, "row_offset", I32, (R + 1,))
            if R < 1 or R > n:
                raise ValueError(f"{where}: {n} rows for {R} requests (row_offset is [R + 1], and there "
                                 "are as many rows as requests at least)")
        self.cap = self.gamma = self.words = self.n_masks = 0
        if history is not None:
            self.cap = _width(a, history, "history")
            a.req(history, "history", I32, (R, self.cap))
            a.req(hist_len, "hist_len", I32, (R,))
            a.req(prompt_len, "prompt_len", I32, (R,), optional=True)
        elif hist_len is not None or prompt_len is not None:
            raise ValueError(f"{where}: hist_len and prompt_len belong to a history")
        if drafts is not None:
            self.gamma = _width(a, drafts, "drafts")
            a.req(drafts, "drafts", I32, (R, self.gamma))
        if repetition is not None:
            a.req(repetition, "repetition", F32, (R,))
        if mask is not None:
            self.words = _width(a, mask, "mask")
            if mask.dim() != 2 or self.words < (V + 31) // 32:
                raise ValueError(f"{where}: mask must be [n_masks][{(V + 31) // 32}] int32")
            self.n_masks = mask.shape[0]
            a.req(mask, "mask", I32, (self.n_masks, self.words))
            a.req(mask_index, "mask_index", I32, (n,), optional=True)
            if mask_index is None and self.n_masks < n:
                raise ValueError(f"{where}: {n} rows with {self.n_masks} masks need mask_index")
        elif mask_index is not None:
            raise ValueError(f"{where}: mask_index without a mask")

    def output(self, out, like):
        n, V = self.n, self.V
        if out is None:
            per = _PER[like.dtype]
            out = _empty((n, -(-V // per) * per), like.dtype, like.device)[:, :V]
        return out, self.a.rows(out, "out", like.dtype, (n, V))


def edit_logits(X, *, row_offset=None, history=None, hist_len=None, prompt_len=None, drafts=None,
                repetition=None, frequency=None, presence=None, bias_ids=None, bias=None, mask=None,
                mask_index=None, ws=None, stream=None, out=None):
    """Logits X [n_rows][V] (rows may be strided) of the requests that row_offset [R + 1]
    gives (None: one row each), edited by each request's tokens: history [R][capacity] up
    to hist_len [R], of which the first prompt_len [R] were the prompt (None: none), and
    for its row j the drafts [R][gamma] before it.

    repetition, frequency, presence  [R] fp32: a token seen before is divided (positive)
        or multiplied by `repetition`; one generated n times loses frequency n + presence
    bias_ids, bias  [R][n] int32 (-1: none) and fp32: added
    mask  [n_masks][ceil(V / 32)] int32: bit v % 32 of word v / 32 allows v; mask_index
        [n_rows] int32: the row's mask, -1 for none (None: row i's is mask i)

    Returns out, which may be X itself (not a view over a part of it); rows that no request
    has keep what it held."""
    e = _Edits("edit_logits", X, row_offset, history, hist_len, prompt_len, drafts, repetition, mask,
               mask_index)
    a, R = e.a, e.R
    if frequency is not None:
        a.req(frequency, "frequency", F32, (R,))
    if presence is not None:
        a.req(presence, "presence", F32, (R,))
    n_bias = 0
    if bias_ids is not None or bias is not None:
        n_bias = _width(a, bias_ids, "bias_ids")
        a.req(bias_ids, "bias_ids", I32, (R, n_bias))
        a.req(bias, "bias", F32, (R, n_bias))
    index = a.gpu()
    with _on_stream(stream):
        out, out_stride = e.output(out, X)
        buf = _workspace(ws, 256, X.device, index, stream)
    a.gpu()
    _launch("dspark_edit_logits", index, stream, e.n, e.V, e.stride, e.dt, X.data_ptr(), R,
            _ptr(row_offset), _ptr(history), e.cap, _ptr(hist_len), _ptr(prompt_len), _ptr(drafts),
            e.gamma, _ptr(repetition), _ptr(frequency), _ptr(presence), n_bias, _ptr(bias_ids),
            _ptr(bias), e.n_masks, _ptr(mask), e.words, _ptr(mask_index), out.data_ptr(), out_stride,
            buf.data_ptr(), buf.numel())
    return out


def edit_logits_backward(G, X=None, *, row_offset=None, history=None, hist_len=None, prompt_len=None,
                         drafts=None, repetition=None, mask=None, mask_index=None, ws=None,
                         stream=None, out=None):
    """From the gradient G [n_rows][V] of edit_logits()'s output to that of its input X (the
    raw logits, needed with `repetition` only).  `out` may be G itself."""
    e = _Edits("edit_logits_backward", G, row_offset, history, hist_len, prompt_len, drafts, repetition,
               mask, mask_index)
    a, x_stride = e.a, 0
    if X is not None or repetition is not None:
        x_stride = a.rows(X, "X", G.dtype, (e.n, e.V))
    index = a.gpu()
    with _on_stream(stream):
        out, out_stride = e.output(out, G)
        buf = _workspace(ws, 256, G.device, index, stream)
    a.gpu()
    _launch("dspark_edit_logits_backward", index, stream, e.n, e.V, x_stride, e.dt, _ptr(X),
            G.data_ptr(), e.stride, e.R, _ptr(row_offset), _ptr(history), e.cap, _ptr(hist_len),
            _ptr(prompt_len), _ptr(drafts), e.gamma, _ptr(repetition), e.n_masks, _ptr(mask), e.words,
            _ptr(mask_index), out.data_ptr(), out_stride, buf.data_ptr(), buf.numel())
    return out


def history_append(history, hist_len, tokens, *, n_acc=None, row_offset=None, prompt_len=None, ws=None,
                   stream=None, out=None):
    """Request r's new tokens join history [R][capacity] behind its hist_len [R]: the first
    n_acc[r] + 1 of tokens [R][width] (the y of verify(); all of them without n_acc), or
    with row_offset [R + 1] alone its part of a flat list.  With both, row_offset is
    cache_reserved_rows(): a request with fewer than n_acc + 1 rows stays as it is (a round
    that found no pages changes nothing).  prompt_len [R], if given, becomes the
    new length where a request got tokens (a prompt's).  Returns the lengths (`out`, which
    may be hist_len)."""
    a = _RowArgs("history_append")
    if not isinstance(history, torch.Tensor) or history.dim() != 2:
        raise ValueError("history_append: history must be a [R][capacity] tensor")
    a.add(history, "history")
    R, cap = history.shape
    a.req(history, "history", I32, (R, cap))
    a.req(hist_len, "hist_len", I32, (R,))
    w = _width(a, tokens, "tokens")
    flat = row_offset is not None and n_acc is None
    a.req(tokens, "tokens", I32, (w,) if flat else (R, w))
    a.req(n_acc, "n_acc", I32, (R,), optional=True)
    a.req(row_offset, "row_offset", I32, (R + 1,), optional=True)
    a.req(prompt_len, "prompt_len", I32, (R,), optional=True)
    index, dev = a.gpu(), history.device
    with _on_stream(stream):
        out = _empty((R,), I32, dev) if out is None else a.req(out, "out", I32, (R,))
        buf = _workspace(ws, 256, dev, index, stream)
    a.gpu()
    _launch("dspark_history_append", index, stream, R, w, w, tokens.data_ptr(), _ptr(n_acc),
            _ptr(row_offset), cap, history.data_ptr(), hist_len.data_ptr(), out.data_ptr(),
            _ptr(prompt_len), buf.data_ptr(), buf.numel())
    return out


class TokenHistory:
    """The tokens of up to R requests, on the device: tokens [R][capacity], lens [R], and
    how many of them were prompts, prompt_lens [R].

    start(tokens, row_offset) takes prompts, append(y, n_acc) what a round emitted, and
    edit(X, ...) is edit_logits() with this history.  Nothing waits for the host, and a
    captured round may be replayed.  A request that leaves has its lens and prompt_lens set
    to 0; a fork copies its row of each.  error_code() reads what the device found wrong."""

    def __init__(self, R, capacity, device="cuda"):
        from .api import Workspace
        # a multiple of four tokens: every row is read in whole 16-byte pieces
        width = -(-capacity // 4) * 4
        self.tokens = torch.full((R, width if width < 1 << 20 else capacity), -1, dtype=I32, device=device)
        self.lens = torch.zeros(R, dtype=I32, device=device)
        self.prompt_lens = torch.zeros(R, dtype=I32, device=device)
        self.ws = Workspace(device)
        # made here: a buffer made within a capture would be cleared by every replay
        self.ws.get(256, None, self.lens.device)

    def start(self, tokens, row_offset, stream=None):
        """Request r's prompt is tokens[row_offset[r]:row_offset[r + 1]] (none: it stays)."""
        history_append(self.tokens, self.lens, tokens, row_offset=row_offset,
                       prompt_len=self.prompt_lens, ws=self.ws, stream=stream, out=self.lens)

    def append(self, y, n_acc, row_offset=None, stream=None):
        """The emitted tokens of a round: the first n_acc + 1 of y.  A captured round gives
        the rows of its PagedCache as row_offset: what found no pages changes nothing."""
        history_append(self.tokens, self.lens, y, n_acc=n_acc, row_offset=row_offset, ws=self.ws,
                       stream=stream, out=self.lens)

    def edit(self, X, *, ws=None, stream=None, **edits):
        """edit_logits(X) by this history."""
        return edit_logits(X, history=self.tokens, hist_len=self.lens, prompt_len=self.prompt_lens,
                           ws=self.ws if ws is None else ws, stream=stream, **edits)

    def error_code(self, stream=None):
        return self.ws.error_code(stream)
