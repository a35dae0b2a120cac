"""Cases, plain forms and 64-bit values of the serving-side operators: log
probabilities (with their gradient), attention over the paged key-value cache,
and the cache's page operations.

`run` with own = False computes the plain form in elementary torch operations;
with own = True it calls the library.  Sizes are those of the framework's own
workloads (R = 32..512 requests, gamma = 5..16 drafts, V = 151936 and 129280)
or generic ones.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_I32 = torch.int32


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one request, one new token, its five best alternatives: the latency of a chat reply
        dict(name="logprobs one row", op="logprobs", R=1, gamma=0, V=151936, dt="bf16", k=5, temp=1.0,
             masked=False),
        # the verified rows of a 128-request round with drafts of up to 16, 20 alternatives each
        dict(name="logprobs verified batch", op="logprobs", R=128, gamma=16, V=151936, dt="bf16",
             k=20, temp=1.0, masked=False),
        # fp32 logits of an odd vocabulary in padded rows, most of it masked (constrained decoding)
        dict(name="logprobs f32 masked", op="logprobs", R=64, gamma=5, V=129277, dt="f32", k=8,
             temp=0.7, masked=True),
        # a training batch of draft positions: gradients of log probability and entropy
        dict(name="gradient train batch", op="gradient", R=128, gamma=15, V=151936, dt="bf16", k=0,
             temp=1.0, masked=False),
        # a small fp32 distillation batch: gradients through the alternatives too
        dict(name="gradient f32 top", op="gradient", R=13, gamma=4, V=129277, dt="f32", k=10,
             temp=1.3, masked=True),
        # one request, one new token over a short context: latency
        dict(name="attend one token", op="attend", R=1, gamma=0, Hq=32, Hkv=8, D=128, page=16,
             longest=1500, dt="bf16", window=0),
        # the ragged verified rows of a 128-request round over contexts of 1 to 6000 tokens
        dict(name="attend verified batch", op="attend", R=128, gamma=16, Hq=32, Hkv=8, D=128,
             page=16, longest=6000, dt="bf16", window=0),
        # single new tokens of three requests over long contexts, one key-value head, fp32
        dict(name="attend long f32", op="attend", R=3, gamma=0, Hq=8, Hkv=1, D=64, page=64,
             longest=120000, dt="f32", window=0),
        # a round of four requests, one forked
        dict(name="pages round small", op="round", R=4, gamma=7, n_pages=512, page=16,
             max_pages=128, forks=1, page_elems=16384),
        # a round of 512 requests, 96 of them forked from others
        dict(name="pages round stress", op="round", R=512, gamma=15, n_pages=40000, page=16,
             max_pages=320, forks=96, page_elems=8192),
        # a few finished requests leave, the rest of a small pool moves together
        dict(name="pages compact small", op="compact", R=16, n_pages=600, page=16, max_pages=64,
             leave=4, page_elems=8192),
        # a quarter of the requests leave a large pool
        dict(name="pages compact large", op="compact", R=256, n_pages=6000, page=32, max_pages=64,
             leave=64, page_elems=65536),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["logprobs", "gradient", "attend", "attend", "round", "compact"])
    if op in ("logprobs", "gradient"):
        R, gamma = _log(rng, 1, 128), rng.randint(0, 16)
        V, dt = _log(rng, 1000, 151936), rng.choice(["bf16", "f32"])
        rows_most = max(1, int(1.2e8 / V / (_SIZE[dt] // 2)))
        R = max(1, min(R, rows_most // (gamma + 1)))
        return dict(op=op, R=R, gamma=gamma, V=V, dt=dt, k=rng.choice([0, 1, 5, 20, 64]),
                    temp=rng.choice([0.6, 0.7, 1.0, 1.3]), masked=rng.random() < 0.4)
    if op == "attend":
        Hkv = rng.choice([1, 2, 4, 8])
        D, dt = rng.choice([64, 96, 128, 256]), rng.choice(["bf16", "bf16", "f32"])
        longest, gamma = _log(rng, 20, 60000), rng.choice([0, 0, 3, 5, 7, 15])
        Hq = Hkv * rng.choice([1, 3, 4, 7, 8])
        # keep the gathered cache and the plain form's scores near the largest listed case's
        R_most = min(128, int(1.5e9 / (longest * Hkv * D * _SIZE[dt])),
                     int(4e8 / (longest * Hq * (gamma + 1))))
        R = _log(rng, 1, max(1, R_most))
        return dict(op=op, R=R, gamma=gamma, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]),
                    longest=longest, dt=dt, window=rng.choice([0, 0, 0, max(1, longest // 3)]))
    if op == "round":
        R, page = _log(rng, 2, 512), rng.choice([16, 32, 64])
        max_pages = _log(rng, 8, 320)
        return dict(op=op, R=R, gamma=rng.randint(1, 16), n_pages=_log(rng, R * 24, R * 24 + 30000),
                    page=page, max_pages=max_pages, forks=rng.randint(1, max(1, R // 4)),
                    page_elems=8 * _log(rng, 64, 1024))
    R = _log(rng, 2, 256)
    return dict(op=op, R=R, n_pages=_log(rng, 24 * R, 24 * R + 2000), page=rng.choice([16, 32, 64]),
                max_pages=_log(rng, 8, 64), leave=rng.randint(1, max(1, R // 3)),
                page_elems=8 * _log(rng, 64, 4096))


def _spread(n, lo, hi):
    """n whole numbers from hi down to lo, evenly spaced."""
    return np.floor(hi - (hi - lo) * np.arange(n) / max(n - 1, 1) + 0.5).astype(np.int64)


def _rows_of(case):
    """New rows of each request (1 + ell, ell from 0 to gamma), before the seed's permutation."""
    return 1 + _spread(case["R"], 0, case["gamma"])


def _lens_of(case):
    """Context lengths, new rows included: from the request's own rows up to `longest`."""
    return np.maximum(_spread(case["R"], 1, case["longest"]), case["gamma"] + 1)


def _pad(V, dt):
    return -(-V // (16 // _SIZE[dt])) * (16 // _SIZE[dt])


def _held(case):
    """Pages that the requests of a page pool hold at the start, most of the pool."""
    R, per = case["R"], case["n_pages"] / case["R"]
    top = max(1, min(case["max_pages"] - 3, int(1.2 * per)))
    held = _spread(R, 1, top)
    return np.maximum(1, (held * min(1.0, 0.8 * case["n_pages"] / held.sum())).astype(np.int64))


def work(case):
    op = case["op"]
    if op in ("logprobs", "gradient"):
        rows = int(_rows_of(case).sum())
        n, es, k = rows * case["V"], _SIZE[case["dt"]], case["k"]
        small = rows * (4 + 4 + 4 + 8 + 8 * k) + 4 * (case["R"] + 1)
        if op == "logprobs":
            return {"bytes": n * es + small, "flops": 8 * n}
        return {"bytes": 2 * n * es + small, "flops": 8 * n}
    if op == "attend":
        es, D = _SIZE[case["dt"]], case["D"]
        lens, rows = _lens_of(case), _rows_of(case)
        seen = lens if not case["window"] else np.minimum(lens, case["window"] + case["gamma"])
        keys = int(seen.sum())
        n = int(rows.sum())
        mean_rows = n / case["R"]
        return {"bytes": keys * 2 * case["Hkv"] * D * es + n * D * es * (2 * case["Hq"] + 4 * case["Hkv"])
                + 4 * keys // case["page"] + 4 * n * case["Hq"],
                "flops": 4.0 * keys * mean_rows * case["Hq"] * D}
    table = 4 * case["R"] * case["max_pages"]
    meta = 2 * (table + 4 * case["n_pages"] + 4 * case["R"])
    if op == "round":
        return {"bytes": meta + 8 * case["R"] + case["forks"] * 4 * 2 * case["page_elems"], "flops": 0}
    held = _held(case)
    # the leaving requests' pages are spread over the pool, so about that share of what stays moves
    gone = held.sum() * case["leave"] / case["R"]
    stay = held.sum() - gone
    moved = stay * (1 - stay / case["n_pages"])
    return {"bytes": int(meta + moved * 4 * 2 * case["page_elems"]), "flops": 0}


# ----------------------------------------------------------------- prepare
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)


def _offsets(rows):
    return torch.from_numpy(np.concatenate(([0], np.cumsum(rows))).astype(np.int32)).cuda()


def prepare(case, seed):
    return {"logprobs": _prepare_rows, "gradient": _prepare_rows, "attend": _prepare_attend,
            "round": _prepare_pages, "compact": _prepare_pages}[case["op"]](case, seed)


def _prepare_rows(case, seed):
    """Logit rows of the round's verified positions: spread like a language
    model's (a few high values over a broad floor), the emitted tokens of each
    request with -1 behind them, two spare rows behind the last."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    V, dt = case["V"], _DT[case["dt"]]
    rows = rng.permutation(_rows_of(case))
    n = int(rows.sum())
    X = torch.empty((n + 2, _pad(V, case["dt"])), dtype=dt, device="cuda")
    for a in range(0, n + 2, 256):  # in pieces: the 32-bit values of the whole batch are not needed
        b = min(a + 256, n + 2)
        z = torch.randn((b - a, X.shape[1]), generator=g, device="cuda")
        X[a:b] = (2.0 * z + 0.35 * z * z.abs()).to(dt)
    if case["masked"]:
        # a grammar allows about 2% of the vocabulary, and always the first entries
        keep = torch.rand(X.shape[1], generator=g, device="cuda") < 0.02
        keep[:4] = True
        X.masked_fill_(~keep, float("-inf"))
    row_offset = _offsets(rows)
    w = case["gamma"] + 1
    n_acc = (rng.random(case["R"]) * rows).astype(np.int64)
    y = rng.integers(0, V, (case["R"], w))
    if case["masked"]:
        y %= 4
    y[np.arange(w)[None] > n_acc[:, None]] = -1
    st = dict(case=case, X=X[:, :V], tokens=torch.from_numpy(y.astype(np.int32)).cuda(),
              row_offset=row_offset, rows=n, k=case["k"])
    shapes = {"logp": ((n + 2,), torch.float32), "entropy": ((n + 2,), torch.float32),
              "stats": ((n + 2, 2), torch.float32)}
    if case["k"]:
        shapes |= {"top_ids": ((n + 2, case["k"]), _I32), "top_logp": ((n + 2, case["k"]), torch.float32)}
    if case["op"] == "logprobs":
        st["out"] = {k: torch.zeros(s, dtype=t, device="cuda") for k, (s, t) in shapes.items()}
        return st
    # what the forward pass left, and the gradients that come back
    z = {k: torch.zeros(s, dtype=t, device="cuda") for k, (s, t) in shapes.items()}
    for a in range(0, n, 256):
        b = min(a + 256, n)
        x = st["X"][a:b].double() / case["temp"]
        m = x.amax(1, keepdim=True).float()
        e = torch.exp(x - m.double())
        S = e.sum(1)
        t = torch.where(e > 0, e * (x - m.double()), 0.0).sum(1)
        z["stats"][a:b] = torch.stack((m[:, 0], S.float()), 1)
        z["entropy"][a:b] = (torch.log(S) - t / S).float()
        if case["k"]:
            z["top_ids"][a:b] = _top(st["X"][a:b], case["k"])
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    st |= dict(stats=z["stats"], entropy=z["entropy"], g_logp=r(n + 2), g_entropy=0.1 * r(n + 2),
               top_ids=z.get("top_ids"), g_top=r(n + 2, case["k"]) if case["k"] else None,
               out=torch.zeros((n + 2, X.shape[1]), dtype=dt, device="cuda")[:, :V])
    return st


def _prepare_attend(case, seed):
    """Requests whose pages are scattered over a pool, as after many rounds;
    keys and values of the new rows come with the queries."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    dt, D, page = _DT[case["dt"]], case["D"], case["page"]
    Hq, Hkv, R = case["Hq"], case["Hkv"], case["R"]
    rows, lens = rng.permutation(_rows_of(case)), rng.permutation(_lens_of(case))
    n = int(rows.sum())
    pages = -(-lens // page)
    n_pages, width = int(pages.sum()) + 3, int(pages.max()) + 1
    ids = rng.permutation(n_pages)
    table = np.full((R, width), -1, np.int32)
    table[np.arange(width)[None] < pages[:, None]] = ids[: pages.sum()]
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    k = torch.empty((n_pages, Hkv, page, D), dtype=dt, device="cuda")
    v = torch.empty((n_pages, Hkv, D, page), dtype=dt, device="cuda")
    for t in (k, v):
        for a in range(0, n_pages, 4096):
            t[a:a + 4096] = rnd(*t[a:a + 4096].shape).to(dt)
    # queries that lean on some keys: scores of a few units, as trained heads have
    q, kn, vn = 1.5 * rnd(n, Hq, D), rnd(n, Hkv, D), rnd(n, Hkv, D)
    return dict(case=case, q=q.to(dt), k_new=kn.to(dt), v_new=vn.to(dt), k=k, v=v,
                table=torch.from_numpy(table).cuda(),
                kv_len=torch.from_numpy(lens.astype(np.int32)).cuda(), row_offset=_offsets(rows),
                most_rows=int(rows.max()), most_keys=int(lens.max()))


def _prepare_pages(case, seed):
    """A pool after many rounds: every request's pages lie anywhere in it."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    R, page, width, n_pages = case["R"], case["page"], case["max_pages"], case["n_pages"]
    held = rng.permutation(_held(case))
    forks = case.get("forks", 0)
    order = rng.permutation(R)
    dst, src = np.sort(order[:forks]), np.sort(order[forks:])
    held[dst] = 0
    lens = held * page - np.where(held > 0, rng.integers(0, page, R), 0)
    src = rng.choice(src, forks) if forks else src
    # the forked prompts end inside a page
    lens[src] = np.where(lens[src] % page == 0, np.maximum(lens[src] - 1, 1), lens[src])
    table = np.full((R, width), -1, np.int32)
    ids = rng.permutation(n_pages)[: held.sum()]
    table[np.arange(width)[None] < held[:, None]] = ids
    refs = np.zeros(n_pages, np.int32)
    refs[ids] = 1
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.int32))).cuda()  # noqa: E731
    st = dict(case=case, lens=cu(lens), table=cu(table), refs=cu(refs),
              k=torch.randn((n_pages, case["page_elems"]), generator=g, device="cuda",
                            dtype=torch.bfloat16),
              v=torch.randn((n_pages, case["page_elems"]), generator=g, device="cuda",
                            dtype=torch.bfloat16))
    if case["op"] == "compact":
        st["leave"] = cu(rng.permutation(R)[: case["leave"]])
        return st
    rows = rng.permutation(_rows_of(case))
    st |= dict(src=cu(src), dst=cu(dst), row_offset=_offsets(rows),
               n_acc=cu((rng.random(R) * rows).astype(np.int64)))
    return st


# --------------------------------------------------------------------- run
def run(state):
    return {"logprobs": _run_logprobs, "gradient": _run_gradient, "attend": _run_attend,
            "round": _run_round, "compact": _run_compact}[state["case"]["op"]](state)


def _ws(state):
    """The workspace that the program keeps between calls."""
    import draft_sampling_verification_03_amd as ds
    if "ws" not in state:
        state["ws"] = ds.Workspace()
    return ds, state["ws"]


def _top(X, k):
    """Indices of the k largest of each row, ties to the lowest index: the
    value's bits as an ordered integer above the complement of the index."""
    b = (X.float() + 0.0).view(_I32).long()  # + 0: a negative zero equals zero
    b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    key = (b << 20) + (0xFFFFF - torch.arange(X.shape[1], device=X.device))
    return (0xFFFFF - (torch.topk(key, k, dim=1).values & 0xFFFFF)).to(_I32)


def _row_tokens(state):
    """Token of every row (-1: none) and whether the row is in use."""
    row = torch.arange(state["X"].shape[0], device="cuda")
    off = state["row_offset"].long()
    rho = torch.searchsorted(off[1:].contiguous(), row, right=True).clamp(max=off.numel() - 2)
    j = (row - off[rho]).clamp(max=state["tokens"].shape[1] - 1)
    return state["tokens"][rho, j].long(), row < off[-1]


def _run_logprobs(state):
    c = state["case"]
    if own:
        ds, ws = _ws(state)
        return ds.logprobs(state["X"], state["tokens"], k=c["k"], row_offset=state["row_offset"],
                           temp=c["temp"], ws=ws, out=state["out"])
    tok, used = _row_tokens(state)
    x = state["X"].float() / c["temp"]
    m = x.amax(1)
    d = x - m[:, None]
    e = torch.exp(d)
    S = e.sum(1)
    logS = torch.log(S)
    ent = logS - torch.where(e > 0, e * d, 0.0).sum(1) / S
    lp = torch.where(tok >= 0, d.gather(1, tok.clamp(min=0)[:, None])[:, 0] - logS, 0.0)
    out = {"logp": lp, "entropy": ent, "stats": torch.stack((m, S), 1)}
    if c["k"]:
        ids = _top(state["X"], c["k"])
        out |= {"top_ids": ids, "top_logp": d.gather(1, ids.long()) - logS[:, None]}
    return {k: torch.where(used.view(-1, *[1] * (v.dim() - 1)), v, state["out"][k])
            for k, v in out.items()}


def _run_gradient(state):
    c = state["case"]
    if own:
        ds, ws = _ws(state)
        return ds.logprobs_backward(state["X"], state["stats"], state["entropy"],
                                    tokens=state["tokens"], g_logp=state["g_logp"],
                                    g_entropy=state["g_entropy"], top_ids=state["top_ids"],
                                    g_top=state["g_top"], row_offset=state["row_offset"],
                                    temp=c["temp"], ws=ws, out=state["out"])
    tok, used = _row_tokens(state)
    gl = torch.where(tok >= 0, state["g_logp"], 0.0)
    total = gl if not c["k"] else gl + state["g_top"].sum(1)
    d = state["X"].float() / c["temp"] - state["stats"][:, :1]
    p = torch.exp(d) / state["stats"][:, 1:]
    lp = torch.where(p > 0, d - torch.log(state["stats"][:, 1:]), 0.0)
    z = -p * (total[:, None] + state["g_entropy"][:, None] * (lp + state["entropy"][:, None]))
    z.scatter_add_(1, tok.clamp(min=0)[:, None], gl[:, None])
    if c["k"]:
        z.scatter_add_(1, state["top_ids"].long(), state["g_top"])
    return torch.where(used[:, None], (z / c["temp"]).to(state["X"].dtype), state["out"])


def _slots(state):
    """Row, position in its request and request of every new row."""
    off = state["row_offset"].long()
    row = torch.arange(state["q"].shape[0], device="cuda")
    rho = torch.searchsorted(off[1:].contiguous(), row, right=True)
    j = row - off[rho]
    return rho, j, state["kv_len"].long()[rho] - (off[rho + 1] - off[rho]) + j


def _run_attend(state):
    c = state["case"]
    if own:
        ds, ws = _ws(state)
        o = ds.cache_attend(state["q"], state["k"], state["v"], state["table"], state["kv_len"],
                            row_offset=state["row_offset"], k_new=state["k_new"],
                            v_new=state["v_new"], window=c["window"], ws=ws)
        return {"out": o["out"], "lse": o["lse"], "k": state["k"], "v": state["v"]}
    page, Hq, Hkv, D = c["page"], c["Hq"], c["Hkv"], c["D"]
    rho, j, pos = _slots(state)
    table = state["table"].long()
    at = table[rho, pos // page]
    state["k"][at, :, pos % page] = state["k_new"]
    state["v"][at, :, :, pos % page] = state["v_new"]
    # every request's keys and values side by side, as long as the longest
    t = torch.arange(state["most_keys"], device="cuda")
    at = table[:, t // page].clamp(min=0)
    there = (t[None] < state["kv_len"][:, None])[:, None, :, None]
    k = torch.where(there, state["k"][at, :, t % page].float().transpose(1, 2), 0.0)
    v = torch.where(there, state["v"][at, :, :, t % page].float().transpose(1, 2), 0.0)
    R, J = c["R"], state["most_rows"]
    q = torch.zeros((R, J, Hq, D), device="cuda")
    q[rho, j] = state["q"].float()
    last = torch.full((R, J), -1, device="cuda", dtype=torch.long)
    last[rho, j] = pos
    q = q.view(R, J, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, -1, D)
    s = torch.matmul(q, k.transpose(2, 3)).view(R, Hkv, J, Hq // Hkv, -1) / math.sqrt(D)
    sees = t[None, None] <= last[:, :, None]
    if c["window"]:
        sees &= t[None, None] > last[:, :, None] - c["window"]
    s.masked_fill_(~sees[:, None, :, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    s = s.sub_(m).exp_()
    S = s.sum(-1, keepdim=True)
    o = (torch.matmul(s.view(R, Hkv, -1, s.shape[-1]), v).view(R, Hkv, J, Hq // Hkv, D) / S)
    lse = (m + torch.log(S))[..., 0]
    back = lambda a: a.transpose(1, 2).reshape(R, J, Hq, *a.shape[4:])[rho, j]  # noqa: E731
    return {"out": back(o).to(state["q"].dtype), "lse": back(lse), "k": state["k"], "v": state["v"]}


def _pages(lens, page):
    return (lens + page - 1) // page


def _count(refs, table, at, by):
    """refs with `by` added for every table entry that `at` marks."""
    add = torch.zeros(refs.numel() + 1, dtype=_I32, device="cuda")
    add.index_add_(0, torch.where(at, table.long(), refs.numel()).reshape(-1),
                   torch.full((table.numel(),), by, dtype=_I32, device="cuda"))
    return refs + add[:-1]


def _kept(lens, table, refs, new, page):
    """Requests cut to `new` tokens: the pages behind them are given back."""
    i = torch.arange(table.shape[1], device="cuda")[None]
    drop = (i >= _pages(new, page)[:, None]) & (i < _pages(lens, page)[:, None])
    return new, torch.where(drop, -1, table), _count(refs, table, drop, -1)


def _run_round(state):
    c = state["case"]
    page = c["page"]
    if own:
        ds, ws = _ws(state)
        s = ds.cache_fork(state["src"], state["dst"], state["lens"], state["table"], state["refs"],
                          page=page, ws=ws, out=state.get("mid"))
        state["mid"] = {k: s[k] for k in ("lens", "table", "refs")}
        got = ds.cache_reserve(state["row_offset"], s["lens"], s["table"], s["refs"], state["k"],
                               state["v"], page=page, ws=ws, out=state["mid"])
        ds.cache_commit(state["row_offset"], state["n_acc"], s["lens"], s["table"], s["refs"],
                        page=page, ws=ws, out=state["mid"])
        return {**state["mid"], "missing": got["missing"], "k": state["k"], "v": state["v"]}
    R, n_pages = c["R"], c["n_pages"]
    src, dst = state["src"].long(), state["dst"].long()
    i = torch.arange(c["max_pages"], device="cuda")[None]
    # fork: the new request holds the old one's pages
    lens, table = state["lens"].clone(), state["table"].clone()
    lens[dst], table[dst] = lens[src], table[src]
    refs = _count(state["refs"], table[dst], i < _pages(lens[dst], page)[:, None], 1)
    # reserve: a shared last page is copied by all who write it, but the first where nobody else holds it
    off = state["row_offset"]
    n = off[1:] - off[:-1]
    have, want = _pages(lens, page), _pages(lens + n, page)
    r = torch.arange(R, device="cuda")
    tail = torch.where(have > 0, table[r, (have - 1).clamp(min=0)], 0).long()
    writes = (n > 0) & (lens % page != 0)
    to = torch.where(writes, tail, n_pages)
    writers = torch.zeros(n_pages + 1, dtype=_I32, device="cuda").index_add_(
        0, to, torch.ones(R, dtype=_I32, device="cuda"))
    first = torch.full((n_pages + 1,), R, device="cuda").scatter_reduce_(0, to, r, "amin")
    copy = writes & (refs[tail] > 1) & ~((writers[tail] == refs[tail]) & (first[tail] == r))
    need = want - have + copy
    free = refs == 0
    ids = torch.empty(n_pages + 1, dtype=torch.long, device="cuda")
    ids[torch.where(free, torch.cumsum(free, 0) - 1, n_pages)] = torch.arange(n_pages, device="cuda")
    at = torch.cumsum(need, 0) - need
    missing = (need.sum() - free.sum()).clamp(min=0)
    grow = (i >= have[:, None]) & (i < want[:, None])
    table = torch.where(grow, ids[(at + copy - have)[:, None].add(i).clamp(0, n_pages - 1)], table)
    w = copy.nonzero()[:, 0]
    new = ids[at[w]]
    state["k"][new], state["v"][new] = state["k"][tail[w]], state["v"][tail[w]]
    refs = _count(refs, tail[w], torch.ones_like(w, dtype=torch.bool), -1)
    table[w, (have[w] - 1).long()] = new
    refs = _count(refs, table, grow, 1)
    refs[new] = 1
    lens = lens + n
    # commit: the accepted rows stay
    lens, table, refs = _kept(lens, table, refs, lens - n + state["n_acc"] + 1, page)
    return {"lens": lens.to(_I32), "table": table.to(_I32), "refs": refs.to(_I32),
            "missing": missing.to(_I32).view(1), "k": state["k"], "v": state["v"]}


def _run_compact(state):
    c = state["case"]
    page = c["page"]
    if own:
        ds, ws = _ws(state)
        s = ds.cache_release(state["leave"], state["lens"], state["table"], state["refs"], page=page,
                             ws=ws, out=state.get("mid"))
        state["mid"] = {k: s[k] for k in ("lens", "table", "refs")}
        got = ds.cache_compact(s["lens"], s["table"], s["refs"], state["k"], state["v"], page=page,
                               ws=ws, out=state["mid"])
        return {**state["mid"], "n_live": got["n_live"], "k": state["k"], "v": state["v"]}
    stay = state["lens"].clone()
    stay[state["leave"].long()] = 0
    lens, table, refs = _kept(state["lens"], state["table"], state["refs"], stay, page)
    # the i-th page above the live count moves into the i-th hole below it
    live = refs > 0
    n_live = live.sum()
    p = torch.arange(c["n_pages"], device="cuda")
    hole, mover = (~live & (p < n_live)).nonzero()[:, 0], (live & (p >= n_live)).nonzero()[:, 0]
    state["k"][hole], state["v"][hole] = state["k"][mover], state["v"][mover]
    moved = p.clone()
    moved[mover] = hole
    refs = refs.clone()
    refs[hole], refs[mover] = refs[mover], 0
    table = torch.where(table >= 0, moved[table.clamp(min=0).long()], -1)
    return {"lens": lens, "table": table.to(_I32), "refs": refs.to(_I32),
            "n_live": n_live.to(_I32).view(1), "k": state["k"], "v": state["v"]}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, request by request."""
    st = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "gradient": _exact_gradient, "attend": _exact_attend,
            "round": _exact_round, "compact": _exact_compact}[case["op"]](case, st)


def _exact_rows(case, st):
    """(row, token, z) of every row in use, z = x / T in 64 bits."""
    off, y = st["row_offset"].tolist(), st["tokens"].tolist()
    for r in range(case["R"]):
        for row in range(off[r], off[r + 1]):
            yield row, y[r][row - off[r]], st["X"][row].double() / case["temp"]


def _exact_logprobs(case, st):
    out = {k: (v.double() if k != "top_ids" else None) for k, v in st["out"].items()}
    for row, tok, z in _exact_rows(case, st):
        lp = torch.log_softmax(z, 0)
        p = lp.exp()
        out["logp"][row] = lp[tok] if tok >= 0 else 0.0
        out["entropy"][row] = -torch.special.xlogy(p, p).sum()
        m = z.max()
        out["stats"][row, 0], out["stats"][row, 1] = m, torch.exp(z - m).sum()
        if case["k"]:
            out["top_logp"][row] = torch.sort(lp, descending=True).values[: case["k"]]
    return out


def _exact_gradient(case, st):
    out = st["out"].double()
    for row, tok, z in _exact_rows(case, st):
        p = torch.softmax(z, 0)
        g = torch.zeros_like(z)
        if tok >= 0:
            g -= st["g_logp"][row].double() * p
            g[tok] += st["g_logp"][row].double()
        if case["k"]:
            gt = st["g_top"][row].double()
            g -= gt.sum() * p
            g[st["top_ids"][row].long()] += gt
        lp = torch.where(p > 0, p, 1.0).log()
        g -= st["g_entropy"][row].double() * p * (lp - (p * lp).sum())
        out[row] = g / case["temp"]
    return out


def _exact_attend(case, st):
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    grp = case["Hq"] // Hkv
    off, lens = st["row_offset"].tolist(), st["kv_len"].tolist()
    k_all, v_all = st["k"], st["v"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    for r in range(case["R"]):
        n, L = off[r + 1] - off[r], lens[r]
        ids = st["table"][r, : -(-L // page)].long()
        for j in range(n):
            t = L - n + j
            k_all[ids[t // page], :, t % page] = st["k_new"][off[r] + j]
            v_all[ids[t // page], :, :, t % page] = st["v_new"][off[r] + j]
        for h in range(Hkv):
            k = k_all[ids, h].reshape(-1, D)[:L].double()
            v = v_all[ids, h].transpose(1, 2).reshape(-1, D)[:L].double()
            for j in range(n):
                a = 0 if not case["window"] else max(0, L - n + j + 1 - case["window"])
                b = L - n + j + 1
                q = st["q"][off[r] + j, h * grp:(h + 1) * grp].double()
                s = (q @ k[a:b].T) * D ** -0.5
                lse[off[r] + j, h * grp:(h + 1) * grp] = torch.logsumexp(s, 1)
                out[off[r] + j, h * grp:(h + 1) * grp] = torch.softmax(s, 1) @ v[a:b]
    return {"out": out, "lse": lse, "k": k_all.double(), "v": v_all.double()}


def _exact_round(case, st):
    """The round's page operations one request and one page at a time."""
    page = case["page"]
    lens, table, refs = (st[k].tolist() for k in ("lens", "table", "refs"))
    k, v = st["k"], st["v"]
    for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
        lens[d], table[d] = lens[s], list(table[s])
        for p in table[d]:
            if p >= 0:
                refs[p] += 1
    off, n_acc = st["row_offset"].tolist(), st["n_acc"].tolist()
    n = [off[r + 1] - off[r] for r in range(case["R"])]
    tails = [table[r][(lens[r] - 1) // page] if n[r] and lens[r] % page else -1
             for r in range(case["R"])]
    writers = {}
    for r, p in enumerate(tails):
        writers.setdefault(p, []).append(r)
    held = list(refs)
    free = iter([p for p, c in enumerate(refs) if not c])
    for r in range(case["R"]):
        p = tails[r]
        if p >= 0 and held[p] > 1 and not (len(writers[p]) == held[p] and writers[p][0] == r):
            q = next(free)
            k[q], v[q] = k[p], v[p]
            refs[p], refs[q] = refs[p] - 1, 1
            table[r][(lens[r] - 1) // page] = q
        for i in range(-(-lens[r] // page), -(-(lens[r] + n[r]) // page)):
            table[r][i] = next(free)
            refs[table[r][i]] = 1
        lens[r] += n[r]
    for r in range(case["R"]):
        new = lens[r] - n[r] + n_acc[r] + 1
        for i in range(-(-new // page), -(-lens[r] // page)):
            refs[table[r][i]] -= 1
            table[r][i] = -1
        lens[r] = new
    return _whole(lens, table, refs, "missing", 0, k, v)


def _exact_compact(case, st):
    page = case["page"]
    lens, table, refs = (st[k].tolist() for k in ("lens", "table", "refs"))
    for r in st["leave"].tolist():
        for i in range(-(-lens[r] // page)):
            refs[table[r][i]] -= 1
            table[r][i] = -1
        lens[r] = 0
    n_live = sum(1 for c in refs if c)
    holes = iter([p for p in range(n_live) if not refs[p]])
    to = {}
    for p in range(n_live, case["n_pages"]):
        if refs[p]:
            h = to[p] = next(holes)
            refs[h], refs[p] = refs[p], 0
            st["k"][h], st["v"][h] = st["k"][p], st["v"][p]
    table = [[to.get(p, p) for p in row] for row in table]
    return _whole(lens, table, refs, "n_live", n_live, st["k"], st["v"])


def _whole(lens, table, refs, name, count, k, v):
    return {"lens": torch.tensor(lens), "table": torch.tensor(table), "refs": torch.tensor(refs),
            name: torch.tensor([count]), "k": k.double(), "v": v.double()}
