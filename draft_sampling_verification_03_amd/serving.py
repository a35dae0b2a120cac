"""torch-facing wrappers of include/dspark_serving.h: log probabilities with
their gradient, attention over a paged key-value cache, and the cache's pages.

As in api.py every tensor is checked before anything is launched, outputs and
workspaces are allocated on the launch stream, and no arithmetic of the methods
happens here.  Logit rows, queries, new keys and values and a layer's pages may
be strided in their first dimension (a slice of a wider buffer); everything
else is contiguous.
"""
import contextlib

import torch

from . import _abi as A
from .api import F32, I32, Workspace, _Args, _check, _dt, _empty, _on_stream, _outputs

_PER = {torch.bfloat16: 8, torch.float32: 4}  # elements of 16 bytes


class _RowArgs(_Args):
    def rows(self, t, name, dtype, shape, optional=False):
        """As req, but the first dimension may have any stride of whole 16-byte
        pieces that keeps its entries apart; returns (tensor, that stride)."""
        if t is None and optional:
            return None, 0
        if not isinstance(t, torch.Tensor) or t.is_contiguous() and t.dim() == len(shape) > 1 \
                and t[:1].numel() % _PER.get(t.dtype, 1) == 0:
            self.req(t, name, dtype, shape)
            return t, t.stride(0) if t.shape[0] > 1 else t[:1].numel()
        if t.dtype != dtype or t.dim() != len(shape) or any(
                s is not None and s != d for s, d in zip(shape, t.shape)):
            self.req(t, name, dtype, shape)
        one = t[0].numel() if t.shape[0] else 0
        if t.shape[0] and not t[0].is_contiguous():
            raise ValueError(f"{self.where}: {name} must be contiguous past its first dimension")
        stride = t.stride(0) if t.shape[0] > 1 else -(-one // _PER[dtype]) * _PER[dtype]
        if stride < one or stride % _PER[dtype]:
            raise ValueError(f"{self.where}: {name} must have rows of whole 16-byte pieces "
                             f"(stride {stride} elements for rows of {one})")
        self.tensors.append((name, t))
        return t, stride


@contextlib.contextmanager
def _guard(dev):
    with torch.cuda.device(dev):
        yield


def _run(dev, stream, call):
    """call(stream) with the tensors' device current."""
    if dev.index == torch.cuda.current_device():
        return call(torch.cuda.current_stream() if stream is None else stream)
    with _guard(dev):
        return call(torch.cuda.current_stream() if stream is None else stream)


def _check_tokens(a, tokens, row_offset, n_rows):
    """(R, token stride) of the ragged layout, (0, 0) without one."""
    if row_offset is None:
        a.req(tokens, "tokens", I32, (n_rows,), optional=True)
        return 0, 0
    a.req(row_offset, "row_offset", I32, (None,))
    R = row_offset.shape[0] - 1
    if R < 1:
        raise ValueError(f"{a.where}: row_offset must have shape [R + 1]")
    if tokens is None:
        return R, 0
    a.req(tokens, "tokens", I32, (R, None))
    return R, tokens.shape[1]


def logprobs(X, tokens=None, *, k=0, row_offset=None, temp=1.0, ws=None, stream=None, out=None):
    """X [n_rows][V] logits (rows may be strided); tokens [n_rows] int32, or with
    row_offset [R + 1] the verified batch's layout [R][w] (y of verify()), -1
    for no token.  Returns logp (None without tokens), entropy and stats
    [n_rows][2] = (m, S), and with k > 0 top_ids and top_logp [n_rows][k].
    Rows from row_offset[R] on keep what `out` held (undefined without `out`)."""
    a = _RowArgs("logprobs")
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError("logprobs: X must be a [n_rows][V] tensor")
    dt = _dt(X)
    n, V = X.shape
    _, stride = a.rows(X, "X", X.dtype, (n, V))
    R, w = _check_tokens(a, tokens, row_offset, n)
    dev = a.device()
    k = int(k)
    with _on_stream(stream):
        out = _outputs(a, out, dict(logp=((n,), F32) if tokens is not None else None,
                                    entropy=((n,), F32), stats=((n, 2), F32),
                                    top_ids=((n, k), I32) if k > 0 else None,
                                    top_logp=((n, k), F32) if k > 0 else None), dev)
        a.device()
        ws = ws or Workspace(dev)
        buf = ws.get(A.dspark_logprobs_workspace(n, V, k, dt), stream, dev)
    st = _run(dev, stream, lambda s: A.dspark_logprobs(
        n, V, stride, dt, float(temp), X, tokens, w, R, row_offset, k, out.get("logp"),
        out["entropy"], out["stats"], out.get("top_ids"), out.get("top_logp"), buf, buf.numel(), s))
    _check(st, "dspark_logprobs")
    return out


def logprobs_backward(X, stats, entropy=None, *, tokens=None, g_logp=None, g_entropy=None,
                      top_ids=None, g_top=None, row_offset=None, temp=1.0, ws=None, stream=None,
                      out=None):
    """Gradient of logprobs() with respect to X from the gradients of its
    outputs: g_logp, g_entropy [n_rows], g_top [n_rows][k] with top_ids (each
    optional).  stats and entropy are logprobs()'s.  `out` may be X itself."""
    a = _RowArgs("logprobs_backward")
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError("logprobs_backward: X must be a [n_rows][V] tensor")
    dt = _dt(X)
    n, V = X.shape
    _, stride = a.rows(X, "X", X.dtype, (n, V))
    R, w = _check_tokens(a, tokens, row_offset, n)
    a.req(stats, "stats", F32, (n, 2))
    a.req(entropy, "entropy", F32, (n,), optional=g_entropy is None)
    a.req(g_logp, "g_logp", F32, (n,), optional=True)
    a.req(g_entropy, "g_entropy", F32, (n,), optional=True)
    k = 0
    if g_top is not None:
        if not isinstance(g_top, torch.Tensor) or g_top.dim() != 2:
            raise ValueError("logprobs_backward: g_top must be a [n_rows][k] tensor")
        k = g_top.shape[1]
        a.req(g_top, "g_top", F32, (n, k))
        a.req(top_ids, "top_ids", I32, (n, k))
    if g_logp is not None and tokens is None:
        raise ValueError("logprobs_backward: g_logp needs tokens")
    dev = a.device()
    with _on_stream(stream):
        if out is None:
            per = _PER[X.dtype]
            out = _empty((n, -(-V // per) * per), X.dtype, dev)[:, :V]
        _, dx_stride = a.rows(out, "out", X.dtype, (n, V))
        a.device()
        ws = ws or Workspace(dev)
        buf = ws.get(256, stream, dev)
    st = _run(dev, stream, lambda s: A.dspark_logprobs_backward(
        n, V, stride, dt, float(temp), X, tokens if g_logp is not None else None, w, R, row_offset,
        stats, entropy, g_logp, g_entropy, k, top_ids if k else None, g_top, out, dx_stride, buf,
        buf.numel(), s))
    _check(st, "dspark_logprobs_backward")
    return out


# -------------------------------------------------------------------- pages
def _state(a, lens, table, refs):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError(f"{a.where}: table must be a [R][max_pages] tensor")
    R, width = table.shape
    a.req(table, "table", I32, (R, width))
    a.req(lens, "lens", I32, (R,))
    a.req(refs, "refs", I32, (None,))
    return R, width, refs.shape[0]


def _pools(a, k_pages, v_pages, n_pages):
    """Bytes of a page in each pool (None both: numbers only)."""
    if k_pages is None and v_pages is None:
        return 0
    size = []
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if not isinstance(t, torch.Tensor) or t.dim() < 2 or t.shape[0] != n_pages:
            raise ValueError(f"{a.where}: {name} must be a [n_pages = {n_pages}][...] tensor")
        a.req(t, name, t.dtype, t.shape)
        size.append(t[0].numel() * t.element_size())
    if size[0] != size[1]:
        raise ValueError(f"{a.where}: k_pages and v_pages must have pages of the same size")
    return size[0]


def _state_out(a, out, lens, table, refs):
    spec = dict(lens=(lens.shape, I32), table=(table.shape, I32), refs=(refs.shape, I32))
    out = dict(_outputs(a, out, spec, lens.device))
    same = [out[n].data_ptr() == t.data_ptr()
            for n, t in (("lens", lens), ("table", table), ("refs", refs))]
    if any(same) and not all(same):
        raise ValueError(f"{a.where}: lens, table and refs change in place all three or none")
    return out


def _cache_call(where, name, page, lens, table, refs, ws, stream, out, extra, args):
    """Checks the state (after the caller's own arguments, given by `extra`),
    makes the outputs and calls dspark_<name>; args(a, s, o, buf) gives the
    arguments behind the sizes."""
    a = _RowArgs(where)
    R, width, n_pages = _state(a, lens, table, refs)
    extra(a, R, n_pages)
    dev = a.device()
    with _on_stream(stream):
        o = _state_out(a, out, lens, table, refs)
        a.device()
        ws = ws or Workspace(dev)
        buf = ws.get(A.dspark_cache_workspace(R, n_pages), stream, dev)
        tail = args(o, dev)
    st = _run(dev, stream, lambda s: getattr(A, name)(R, int(page), width, n_pages, *tail[0], lens,
                                                      table, refs, o["lens"], o["table"], o["refs"],
                                                      *tail[1], buf, buf.numel(), s))
    _check(st, name)
    return o


def _one(o, name, out, dev):
    """A one-element result beside the state: the caller's or a new one."""
    t = None if out is None else out.get(name)
    o[name] = _empty((1,), I32, dev) if t is None else t
    return o[name]


def cache_fork(src, dst, lens, table, refs, *, page, ws=None, stream=None, out=None):
    """Requests dst[i] become copies of src[i] that share their pages.  Returns
    the state (lens, table, refs); `out` may name the inputs (in place)."""
    def extra(a, R, n_pages):
        a.req(src, "src", I32, (None,))
        a.req(dst, "dst", I32, (src.shape[0],))
    return _cache_call("cache_fork", "dspark_cache_fork", page, lens, table, refs, ws, stream, out,
                       extra, lambda o, dev: ((src.shape[0], src, dst), ()))


def cache_reserve(row_offset, lens, table, refs, k_pages, v_pages, *, page, ws=None, stream=None,
                  out=None):
    """Pages for row_offset[r + 1] - row_offset[r] new tokens of every request.
    k_pages, v_pages: the whole pools, [n_pages][...] (None both: the state
    alone).  Returns the state and missing [1] (0: done)."""
    size = [0]

    def extra(a, R, n_pages):
        a.req(row_offset, "row_offset", I32, (R + 1,))
        size[0] = _pools(a, k_pages, v_pages, n_pages)
        if out is not None and out.get("missing") is not None:
            a.req(out["missing"], "out['missing']", I32, (1,))

    return _cache_call("cache_reserve", "dspark_cache_reserve", page, lens, table, refs, ws, stream,
                       out, extra, lambda o, dev: ((row_offset,), (k_pages, v_pages, size[0],
                                                                   _one(o, "missing", out, dev))))


def cache_commit(row_offset, n_acc, lens, table, refs, *, page, ws=None, stream=None, out=None):
    """After verify(): of the rows that cache_reserve made room for, the first
    n_acc + 1 stay.  Returns the state."""
    def extra(a, R, n_pages):
        a.req(row_offset, "row_offset", I32, (R + 1,))
        a.req(n_acc, "n_acc", I32, (R,))
    return _cache_call("cache_commit", "dspark_cache_commit", page, lens, table, refs, ws, stream,
                       out, extra, lambda o, dev: ((row_offset, n_acc), ()))


def cache_release(which, lens, table, refs, *, page, ws=None, stream=None, out=None):
    """Requests `which` leave and give their pages back.  Returns the state."""
    def extra(a, R, n_pages):
        a.req(which, "which", I32, (None,))
    return _cache_call("cache_release", "dspark_cache_release", page, lens, table, refs, ws, stream,
                       out, extra, lambda o, dev: ((which.shape[0], which), ()))


def cache_compact(lens, table, refs, k_pages, v_pages, *, page, ws=None, stream=None, out=None):
    """Moves the pages in use to the front of the pools.  Returns the state and
    n_live [1]."""
    size = [0]

    def extra(a, R, n_pages):
        size[0] = _pools(a, k_pages, v_pages, n_pages)
        if out is not None and out.get("n_live") is not None:
            a.req(out["n_live"], "out['n_live']", I32, (1,))

    return _cache_call("cache_compact", "dspark_cache_compact", page, lens, table, refs, ws, stream,
                       out, extra, lambda o, dev: ((), (k_pages, v_pages, size[0],
                                                        _one(o, "n_live", out, dev))))


# ---------------------------------------------------------------- attention
def cache_attend(q, k_pages, v_pages, table, kv_len, *, row_offset=None, k_new=None, v_new=None,
                 scale=None, window=0, ws=None, stream=None, out=None):
    """Attention of the new rows q [rows][Hq][D] over the pages of their
    requests: k_pages [n_pages][Hkv][page][D] and v_pages [n_pages][Hkv][D][page]
    of one layer (page stride free), table [R][max_pages], kv_len [R] tokens
    with the new rows, row_offset [R + 1] (None: one row per request).  k_new,
    v_new [rows][Hkv][D] are written into their pages first.  scale: 1/sqrt(D)
    by default.  Returns out (as q) and lse [rows][Hq]."""
    a = _RowArgs("cache_attend")
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("cache_attend: q must be a [rows][Hq][D] tensor")
    dt = _dt(q)
    n, Hq, D = q.shape
    _, q_stride = a.rows(q, "q", q.dtype, (n, Hq, D))
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("cache_attend: k_pages must be a [n_pages][Hkv][page][D] tensor")
    n_pages, Hkv, page, _ = k_pages.shape
    _, k_stride = a.rows(k_pages, "k_pages", q.dtype, (n_pages, Hkv, page, D))
    _, v_stride = a.rows(v_pages, "v_pages", q.dtype, (n_pages, Hkv, D, page))
    a.req(kv_len, "kv_len", I32, (None,))
    R = kv_len.shape[0]
    a.req(table, "table", I32, (R, None))
    a.req(row_offset, "row_offset", I32, (R + 1,), optional=True)
    if row_offset is None and n != R:
        raise ValueError(f"cache_attend: {n} rows for {R} requests need row_offset")
    if (k_new is None) != (v_new is None):
        raise ValueError("cache_attend: give both k_new and v_new, or neither")
    _, kn = a.rows(k_new, "k_new", q.dtype, (n, Hkv, D), optional=True)
    _, vn = a.rows(v_new, "v_new", q.dtype, (n, Hkv, D), optional=True)
    if kn != vn:
        raise ValueError("cache_attend: k_new and v_new must have the same row stride")
    dev = a.device()
    with _on_stream(stream):
        out = _outputs(a, out, dict(out=((n, Hq, D), q.dtype), lse=((n, Hq), F32)), dev)
        a.device()
        ws = ws or Workspace(dev)
        buf = ws.get(A.dspark_cache_attend_workspace(R, n, Hq, Hkv, D, dt), stream, dev)
    st = _run(dev, stream, lambda s: A.dspark_cache_attend(
        R, n, Hq, Hkv, D, page, table.shape[1], n_pages, dt, float(D ** -0.5 if scale is None
                                                                   else scale), int(window),
        q, q_stride, k_new, v_new, kn, k_pages, v_pages, k_stride, v_stride, table, row_offset,
        kv_len, out["out"], out["lse"], buf, buf.numel(), s))
    _check(st, "dspark_cache_attend")
    return out


class PagedCache:
    """The keys and values of up to R requests and all layers of a model, in
    n_pages pages that the requests share out among themselves:
    k [n_pages][layers][Hkv][page][D], v [n_pages][layers][Hkv][D][page].

    A round: reserve(row_offset), attend(layer, ...) for every layer, and after
    the verification commit(n_acc).  All state lives on the device and changes
    in place; nothing waits for the host, and a captured round may be replayed.
    error_code() reads what the device found wrong so far."""

    def __init__(self, R, n_pages, *, Hkv, D, layers=1, page=16, max_pages=None,
                 dtype=torch.bfloat16, device="cuda"):
        max_pages = n_pages if max_pages is None else max_pages
        self.page = page
        self.k = torch.zeros((n_pages, layers, Hkv, page, D), dtype=dtype, device=device)
        self.v = torch.zeros((n_pages, layers, Hkv, D, page), dtype=dtype, device=device)
        self.lens = torch.zeros(R, dtype=I32, device=device)
        self.table = torch.full((R, max_pages), -1, dtype=I32, device=device)
        self.refs = torch.zeros(n_pages, dtype=I32, device=device)
        self.missing = torch.zeros(1, dtype=I32, device=device)
        self.n_live = torch.zeros(1, dtype=I32, device=device)
        self.row_offset = None
        self.ws, self.attend_ws = Workspace(device), Workspace(device)

    def _state(self):
        return dict(lens=self.lens, table=self.table, refs=self.refs)

    def reserve(self, row_offset, stream=None):
        """Room for the round's rows; missing[0] says how many pages were short
        (then nothing has changed)."""
        self.row_offset = row_offset
        cache_reserve(row_offset, self.lens, self.table, self.refs, self.k, self.v, page=self.page,
                      ws=self.ws, stream=stream, out=dict(self._state(), missing=self.missing))
        return self.missing

    def attend(self, layer, q, k_new, v_new, *, scale=None, window=0, stream=None, out=None):
        """The reserved rows' keys and values enter layer `layer`, and their
        queries attend over it."""
        if self.row_offset is None:
            raise ValueError("PagedCache.attend: reserve() comes first")
        return cache_attend(q, self.k[:, layer], self.v[:, layer], self.table, self.lens,
                            row_offset=self.row_offset, k_new=k_new, v_new=v_new, scale=scale,
                            window=window, ws=self.attend_ws, stream=stream, out=out)

    def commit(self, n_acc, stream=None):
        """The first n_acc + 1 of every request's reserved rows stay."""
        if self.row_offset is None:
            raise ValueError("PagedCache.commit: reserve() comes first")
        cache_commit(self.row_offset, n_acc, self.lens, self.table, self.refs, page=self.page,
                     ws=self.ws, stream=stream, out=self._state())
        self.row_offset = None

    def fork(self, src, dst, stream=None):
        cache_fork(src, dst, self.lens, self.table, self.refs, page=self.page, ws=self.ws,
                   stream=stream, out=self._state())

    def release(self, which, stream=None):
        cache_release(which, self.lens, self.table, self.refs, page=self.page, ws=self.ws,
                      stream=stream, out=self._state())

    def compact(self, stream=None):
        """Pages in use move to the front; returns n_live [1]."""
        cache_compact(self.lens, self.table, self.refs, self.k, self.v, page=self.page, ws=self.ws,
                      stream=stream, out=dict(self._state(), n_live=self.n_live))
        return self.n_live

    def error_code(self, stream=None):
        """The sticky DSPARK_DEVERR_* bits of the page operations and of attend()."""
        code = 0
        for ws in (self.ws, self.attend_ws):
            if ws.buf is not None:
                code |= ws.error_code(stream)
        return code
