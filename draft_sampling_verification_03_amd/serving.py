"""torch-facing wrappers of include/dspark_serving.h: log probabilities with
their gradient, attention over a paged key-value cache, and the cache's pages.

As in api.py every tensor is checked before anything is launched, outputs and
workspaces are allocated on the launch stream, and no arithmetic of the methods
happens here.  Logit rows, queries, new keys and values and a layer's pages may
be strided in their first dimension (a slice of a wider buffer); everything
else is contiguous.
"""
import functools

import torch

from . import _abi as A
from .api import F32, I32, Workspace, _Args, _check, _dt, _empty, _on_stream

_PER = {torch.bfloat16: 8, torch.float32: 4}  # elements of 16 bytes

# these calls take a few microseconds on the device, so the host's share counts:
# the size queries are pure functions of their arguments and are asked once
_logprobs_ws = functools.lru_cache(1024)(A.dspark_logprobs_workspace)
_cache_ws = functools.lru_cache(1024)(A.dspark_cache_workspace)
_attend_ws = functools.lru_cache(1024)(A.dspark_cache_attend_workspace)


class _RowArgs(_Args):
    """_Args with a short way for arguments that are right (what is not goes
    through _Args.req, which says why), and for row strides."""

    def __init__(self, where):
        super().__init__(where)
        self.index = None  # the GPU of the tensors so far

    def add(self, t, name):
        self.tensors.append((name, t))
        index = t.get_device()
        if index != self.index:
            if self.index is not None:
                self.device()
            self.index = index
        return t

    def right(self, t, dtype, shape):
        """Whether t is such a contiguous tensor on the GPU of the others."""
        return (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape
                and t.is_contiguous() and t.get_device() == self.index)

    def req(self, t, name, dtype, shape, optional=False):
        if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape
                and t.is_contiguous() and t.get_device() == self.index):
            return t
        if super().req(t, name, dtype, shape, optional) is not None:
            self.tensors.pop()
            self.add(t, name)
        return t

    def rows(self, t, name, dtype, shape, optional=False):
        """As req, but the first dimension may have any stride of whole 16-byte
        pieces that keeps its entries apart; returns that stride."""
        if t is None and optional:
            return 0
        if type(t) is not torch.Tensor or t.dtype is not dtype or t.shape != shape:
            self.req(t, name, dtype, shape)
        per, one, strides = _PER[dtype], 1, t.stride()
        for i in range(len(shape) - 1, 0, -1):
            if strides[i] != one and shape[i] != 1:
                raise ValueError(f"{self.where}: {name} must be contiguous past its first dimension")
            one *= shape[i]
        stride = strides[0] if shape[0] > 1 else -(-one // per) * per
        if stride < one or stride % per:
            raise ValueError(f"{self.where}: {name} must have rows of whole 16-byte pieces "
                             f"(stride {stride} elements for rows of {one})")
        if t.get_device() != self.index:
            self.add(t, name)
        return stride

    def gpu(self):
        """Index of the one GPU that every tensor is on."""
        if self.index < 0:
            self.device()
        return self.index


def _ptr(t):
    return None if t is None else t.data_ptr()


def _width(a, t, name):
    """Last dimension of a tensor whose other sizes are checked afterwards."""
    if not isinstance(t, torch.Tensor) or t.dim() == 0:
        a.req(t, name, I32, (None,))
        raise ValueError(f"{a.where}: {name} must have a dimension")
    return t.shape[-1]


def _outs(a, out, spec, dev):
    """Outputs {name: (shape, dtype)}: new, or the caller's checked."""
    if out is None:
        return {n: _empty(s, t, dev) for n, (s, t) in spec.items()}
    for n, (s, t) in spec.items():
        if not a.right(out.get(n), t, s):
            a.req(out.get(n), f"out[{n!r}]", t, s)
    return out


def _workspace(ws, nbytes, dev, index, stream):
    """(keeps alive, address, bytes) of the call's workspace."""
    if ws is None:
        ws = Workspace(dev)
    buf = ws.buf
    if stream is not None or buf is None or buf.get_device() != index or buf.numel() < nbytes:
        buf = ws.get(nbytes, stream, dev)
    return buf


def _launch(name, index, stream, *args):
    """The C function `name` with the tensors' device current; the stream comes last."""
    call = getattr(A.library(), name)
    if index == torch.cuda.current_device():
        st = call(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None
                  else A._s(stream))
    else:
        with torch.cuda.device(index):
            st = call(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None
                      else A._s(stream))
    if st:
        _check(st, name)


def _check_tokens(a, tokens, row_offset, n_rows):
    """(R, token stride) of the ragged layout, (0, 0) without one."""
    if row_offset is None:
        a.req(tokens, "tokens", I32, (n_rows,), optional=True)
        return 0, 0
    R = _width(a, row_offset, "row_offset") - 1
    a.req(row_offset, "row_offset", I32, (R + 1,))
    if R < 1:
        raise ValueError(f"{a.where}: row_offset must have shape [R + 1]")
    if R > n_rows:
        raise ValueError(f"{a.where}: X has {n_rows} rows, {R} requests need as many rows at least "
                         "(those behind row_offset[R] are not read)")
    if tokens is None:
        return R, 0
    w = _width(a, tokens, "tokens")
    a.req(tokens, "tokens", I32, (R, w))
    return R, w


def logprobs(X, tokens=None, *, k=0, row_offset=None, temp=1.0, ws=None, stream=None, out=None):
    """X [n_rows][V] logits (rows may be strided); tokens [n_rows] int32, or with
    row_offset [R + 1] the verified batch's layout [R][w] (y of verify()), -1
    for no token.  Returns logp (None without tokens), entropy and stats
    [n_rows][2] = (m, S), top_ids and top_logp [n_rows][k] (None for k = 0).  Rows from
    row_offset[R] on keep what `out` held (undefined without `out`); X has R rows at
    least, also where the requests' rows are fewer."""
    a = _RowArgs("logprobs")
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        raise ValueError("logprobs: X must be a [n_rows][V] tensor")
    dt = _dt(X)
    n, V = X.shape
    k = int(k)
    stride = a.rows(X, "X", X.dtype, (n, V))
    R, w = _check_tokens(a, tokens, row_offset, n)
    index, dev = a.gpu(), X.device
    spec = {"entropy": ((n,), F32), "stats": ((n, 2), F32)}
    if tokens is not None:
        spec["logp"] = ((n,), F32)
    if k > 0:
        spec["top_ids"], spec["top_logp"] = ((n, k), I32), ((n, k), F32)
    with _on_stream(stream):
        out = _outs(a, out, spec, dev)
        for name in ("logp", "top_ids", "top_logp"):
            if name not in spec:
                out.setdefault(name, None)
        buf = _workspace(ws, _logprobs_ws(n, V, k, dt), dev, index, stream)
    top = (out["top_ids"].data_ptr(), out["top_logp"].data_ptr()) if k > 0 else (None, None)
    _launch("dspark_logprobs", index, stream, n, V, stride, dt, temp, X.data_ptr(), _ptr(tokens), w,
            R, _ptr(row_offset), k, out["logp"].data_ptr() if tokens is not None else None,
            out["entropy"].data_ptr(), out["stats"].data_ptr(), *top, buf.data_ptr(), buf.numel())
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
    stride = a.rows(X, "X", X.dtype, (n, V))
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
    index, dev = a.gpu(), X.device
    with _on_stream(stream):
        if out is None:
            per = _PER[X.dtype]
            out = _empty((n, -(-V // per) * per), X.dtype, dev)[:, :V]
        dx_stride = a.rows(out, "out", X.dtype, (n, V))
        buf = _workspace(ws, 256, dev, index, stream)
    _launch("dspark_logprobs_backward", index, stream, n, V, stride, dt, temp, X.data_ptr(),
            None if g_logp is None else tokens.data_ptr(), w, R, _ptr(row_offset),
            stats.data_ptr(), _ptr(entropy), _ptr(g_logp), _ptr(g_entropy), k,
            top_ids.data_ptr() if k else None, g_top.data_ptr() if k else None, out.data_ptr(),
            dx_stride, buf.data_ptr(), buf.numel())
    return out


# -------------------------------------------------------------------- pages
class _State:
    """The state of a page operation, checked, with its outputs and workspace:
    in place when `out` names the inputs, else new or the caller's arrays."""

    __slots__ = ("a", "R", "width", "n_pages", "lens", "table", "refs")

    def __init__(self, where, lens, table, refs):
        self.a = a = _RowArgs(where)
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError(f"{where}: table must be a [R][max_pages] tensor")
        a.add(table, "table")
        self.R, self.width = R, width = table.shape
        self.n_pages = n = _width(a, refs, "refs")
        self.lens, self.table, self.refs = lens, table, refs
        a.req(table, "table", I32, (R, width))
        a.req(lens, "lens", I32, (R,))
        a.req(refs, "refs", I32, (n,))

    def pools(self, k_pages, v_pages):
        """Bytes of a page in each pool (None both: numbers only)."""
        if k_pages is None and v_pages is None:
            return 0
        size = []
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if not isinstance(t, torch.Tensor) or t.dim() < 2 or t.shape[0] != self.n_pages:
                raise ValueError(f"{self.a.where}: {name} must be a [n_pages = {self.n_pages}][...] "
                                 "tensor")
            self.a.req(t, name, t.dtype, t.shape)
            size.append(t.numel() // self.n_pages * t.element_size())
        if size[0] != size[1]:
            raise ValueError(f"{self.a.where}: k_pages and v_pages must have pages of the same size")
        return size[0]

    def outputs(self, out, dev):
        if out is None:
            return {"lens": _empty((self.R,), I32, dev), "refs": _empty((self.n_pages,), I32, dev),
                    "table": _empty((self.R, self.width), I32, dev)}
        lens, table, refs = out.get("lens"), out.get("table"), out.get("refs")
        if lens is not self.lens or table is not self.table or refs is not self.refs:
            a = self.a
            a.req(lens, "out['lens']", I32, (self.R,))
            a.req(table, "out['table']", I32, (self.R, self.width))
            a.req(refs, "out['refs']", I32, (self.n_pages,))
            if 0 < ((lens.data_ptr() == self.lens.data_ptr()) + (table.data_ptr() == self.table.data_ptr())
                    + (refs.data_ptr() == self.refs.data_ptr())) < 3:
                raise ValueError(f"{a.where}: lens, table and refs change in place all three or none")
        return {"lens": lens, "table": table, "refs": refs}

    def run(self, name, page, ws, stream, out, before, after=(), extra=None):
        """Calls dspark_<name>; `extra` is the one-element output beside the state."""
        a, dev = self.a, self.table.device
        index = a.gpu()
        with _on_stream(stream):
            o = self.outputs(out, dev)
            if extra is not None:
                t = None if out is None else out.get(extra)
                o[extra] = _empty((1,), I32, dev) if t is None else a.req(t, extra, I32, (1,))
                after = (*after, o[extra].data_ptr())
            buf = _workspace(ws, _cache_ws(self.R, self.n_pages), dev, index, stream)
        _launch(name, index, stream, self.R, page, self.width, self.n_pages, *before,
                self.lens.data_ptr(), self.table.data_ptr(), self.refs.data_ptr(),
                o["lens"].data_ptr(), o["table"].data_ptr(), o["refs"].data_ptr(), *after,
                buf.data_ptr(), buf.numel())
        return o


def cache_fork(src, dst, lens, table, refs, *, page, ws=None, stream=None, out=None):
    """Requests dst[i] become copies of src[i] that share their pages.  Returns
    the state (lens, table, refs); `out` may name the inputs (in place)."""
    s = _State("cache_fork", lens, table, refs)
    n = _width(s.a, src, "src")
    s.a.req(src, "src", I32, (n,))
    s.a.req(dst, "dst", I32, (n,))
    return s.run("dspark_cache_fork", page, ws, stream, out, (n, src.data_ptr(), dst.data_ptr()))


def cache_reserved_rows(ws, R):
    """The row offsets [R + 1] that the last cache_reserve() over `ws` left: those it was
    given, or zeros where it found no room.  A view of the workspace: a round that does
    not read `missing` gives it to cache_attend() and cache_commit() as row_offset."""
    if ws.buf is None or ws.buf.numel() < 256 + 4 * (R + 1):
        raise ValueError("cache_reserved_rows: cache_reserve() over this workspace comes first")
    return ws.buf[256:256 + 4 * (R + 1)].view(I32)


def cache_reserve(row_offset, lens, table, refs, k_pages, v_pages, *, page, ws=None, stream=None,
                  out=None):
    """Pages for row_offset[r + 1] - row_offset[r] new tokens of every request.
    k_pages, v_pages: the whole pools, [n_pages][...] (None both: the state
    alone).  Returns the state and missing [1] (0: done; else look at it before
    the round goes on, or go on with cache_reserved_rows())."""
    s = _State("cache_reserve", lens, table, refs)
    s.a.req(row_offset, "row_offset", I32, (s.R + 1,))
    size = s.pools(k_pages, v_pages)
    return s.run("dspark_cache_reserve", page, ws, stream, out, (row_offset.data_ptr(),),
                 (_ptr(k_pages), _ptr(v_pages), size), "missing")


def cache_commit(row_offset, n_acc, lens, table, refs, *, page, ws=None, stream=None, out=None):
    """After verify(): of the rows that cache_reserve made room for, the first
    n_acc + 1 stay.  Returns the state."""
    s = _State("cache_commit", lens, table, refs)
    s.a.req(row_offset, "row_offset", I32, (s.R + 1,))
    s.a.req(n_acc, "n_acc", I32, (s.R,))
    return s.run("dspark_cache_commit", page, ws, stream, out,
                 (row_offset.data_ptr(), n_acc.data_ptr()))


def cache_release(which, lens, table, refs, *, page, ws=None, stream=None, out=None):
    """Requests `which` leave and give their pages back.  Returns the state."""
    s = _State("cache_release", lens, table, refs)
    n = _width(s.a, which, "which")
    s.a.req(which, "which", I32, (n,))
    return s.run("dspark_cache_release", page, ws, stream, out, (n, which.data_ptr()))


def cache_compact(lens, table, refs, k_pages, v_pages, *, page, ws=None, stream=None, out=None):
    """Moves the pages in use to the front of the pools.  Returns the state and
    n_live [1]."""
    s = _State("cache_compact", lens, table, refs)
    size = s.pools(k_pages, v_pages)
    return s.run("dspark_cache_compact", page, ws, stream, out, (),
                 (_ptr(k_pages), _ptr(v_pages), size), "n_live")


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
    q_stride = a.rows(q, "q", q.dtype, (n, Hq, D))
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("cache_attend: k_pages must be a [n_pages][Hkv][page][D] tensor")
    n_pages, Hkv, page, _ = k_pages.shape
    k_stride = a.rows(k_pages, "k_pages", q.dtype, (n_pages, Hkv, page, D))
    v_stride = a.rows(v_pages, "v_pages", q.dtype, (n_pages, Hkv, D, page))
    R, width = _width(a, kv_len, "kv_len"), _width(a, table, "table")
    a.req(kv_len, "kv_len", I32, (R,))
    a.req(table, "table", I32, (R, width))
    if row_offset is not None:
        a.req(row_offset, "row_offset", I32, (R + 1,))
    elif n != R:
        raise ValueError(f"cache_attend: {n} rows for {R} requests need row_offset")
    if (k_new is None) != (v_new is None):
        raise ValueError("cache_attend: give both k_new and v_new, or neither")
    kn = a.rows(k_new, "k_new", q.dtype, (n, Hkv, D), optional=True)
    vn = a.rows(v_new, "v_new", q.dtype, (n, Hkv, D), optional=True)
    if kn != vn:
        raise ValueError("cache_attend: k_new and v_new must have the same row stride")
    index, dev = a.gpu(), q.device
    with _on_stream(stream):
        out = _outs(a, out, {"out": ((n, Hq, D), q.dtype), "lse": ((n, Hq), F32)}, dev)
        buf = _workspace(ws, _attend_ws(R, n, Hq, Hkv, D, dt), dev, index, stream)
    _launch("dspark_cache_attend", index, stream, R, n, Hq, Hkv, D, page, width, n_pages, dt,
            D ** -0.5 if scale is None else scale, window, q.data_ptr(), q_stride, _ptr(k_new),
            _ptr(v_new), kn, k_pages.data_ptr(), v_pages.data_ptr(), k_stride, v_stride,
            table.data_ptr(), _ptr(row_offset), kv_len.data_ptr(), out["out"].data_ptr(),
            out["lse"].data_ptr(), buf.data_ptr(), buf.numel())
    return out


class PagedCache:
    """The keys and values of up to R requests and all layers of a model, in
    n_pages pages that the requests share out among themselves:
    k [n_pages][layers][Hkv][page][D], v [n_pages][layers][Hkv][D][page].

    A round: reserve(row_offset), attend(layer, ...) for every layer (with rotary=, a
    tokens.RotaryPlan, where positions are rotated in), and after the verification
    commit(n_acc).  All state lives on the device and changes
    in place; nothing waits for the host, and a captured round may be replayed.
    A round that finds no room (see reserve()) changes nothing in any of the three.
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
        # made here and never outgrown: a buffer made within a capture would be cleared by
        # every replay, and the errors found so far with it.  Of the attention's, the size
        # for any number of rows and query heads (34 MB for heads of 128).
        self.ws, self.attend_ws = Workspace(device), Workspace(device)
        self.ws.get(_cache_ws(R, n_pages), None, self.lens.device)
        self.attend_ws.get(_attend_ws(R, 1 << 20, Hkv, Hkv, D, A.DSPARK_F32), None, self.lens.device)
        self.rows = cache_reserved_rows(self.ws, R)

    def _state(self):
        return dict(lens=self.lens, table=self.table, refs=self.refs)

    def reserve(self, row_offset, stream=None):
        """Room for the round's rows; missing[0] says how many pages were short (-1: a
        length out of bounds).  Then nothing has changed, and the round's attend() and
        commit() change nothing either: row_offset here is all zeros."""
        self.row_offset = self.rows
        cache_reserve(row_offset, self.lens, self.table, self.refs, self.k, self.v, page=self.page,
                      ws=self.ws, stream=stream, out=dict(self._state(), missing=self.missing))
        return self.missing

    def append(self, layer, q, k_new, v_new, *, rotary=None, positions=None, stream=None, out=None):
        """The reserved rows' keys and values enter layer `layer`, keys and queries rotated
        by the plan `rotary` (None: as they are).  Returns the rotated queries, for attend()
        with k_new = v_new = None; q may be None."""
        if self.row_offset is None:
            raise ValueError("PagedCache.append: reserve() comes first")
        from .tokens import cache_append
        return cache_append(q, k_new, v_new, self.k[:, layer], self.v[:, layer], self.table, self.lens,
                            plan=rotary, row_offset=self.row_offset, positions=positions,
                            ws=self.attend_ws, stream=stream, out=out)

    def attend(self, layer, q, k_new=None, v_new=None, *, rotary=None, positions=None, scale=None,
               window=0, stream=None, out=None):
        """The reserved rows' keys and values enter layer `layer` (None: append() put them
        there), and their queries attend over it.  With `rotary`, a RotaryPlan, queries
        and keys are rotated first, as append() does it."""
        if self.row_offset is None:
            raise ValueError("PagedCache.attend: reserve() comes first")
        if rotary is not None:
            if k_new is None:
                raise ValueError("PagedCache.attend: rotary needs k_new and v_new")
            q = self.append(layer, q, k_new, v_new, rotary=rotary, positions=positions, stream=stream)
            k_new = v_new = None
        elif positions is not None:
            raise ValueError("PagedCache.attend: positions are for rotary")
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
