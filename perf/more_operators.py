"""Cases, plain forms and 64-bit values of the operators that the tokens of a
round need: rotary positions (with their gradient), appending rotated keys and
values to the paged cache, edits of logits by the requests' token histories
(penalties, biases, grammar masks, with their gradient), and the histories
themselves.

`run` with own = False computes the plain form in elementary torch operations;
with own = True it calls the library.  Sizes are those of the framework's own
workloads (R = 32..512 requests, gamma = 5..16 drafts, V = 151936 and 129280,
32 query and 8 key-value heads of 128) or generic ones.
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
        # one new token of one request far into a long context: the latency of a step, per layer
        dict(name="rotary one token", op="rotary", rows=1, seqs=0, Hq=32, Hkv=8, D=128, rot=128,
             layout="interleaved", dt="bf16", scaled=True),
        # the backward pass of a packed training batch of seven sequences of unequal length
        dict(name="rotary gradient train batch", op="rotary_gradient", rows=8191, seqs=7, Hq=32, Hkv=8,
             D=128, rot=128, layout="half", dt="bf16", scaled=False),
        # one request, one new token: what stands before its attention in every layer
        dict(name="append one token", op="append", R=1, gamma=0, Hq=32, Hkv=8, D=128, rot=128, page=16,
             longest=1500, whole=0, layout="half", dt="bf16", scaled=False),
        # the verified rows of a 128-request round (1 + ell each), the short pages of a server
        dict(name="append verified batch", op="append", R=128, gamma=16, Hq=32, Hkv=8, D=128, rot=128,
             page=16, longest=2000, whole=0, layout="half", dt="bf16", scaled=True),
        # prompts that enter in chunks while others decode; fp32, half of a head of 96 rotated
        dict(name="append f32 prompts", op="append", R=40, gamma=4, Hq=12, Hkv=4, D=96, rot=48, page=64,
             longest=5001, whole=5, layout="interleaved", dt="f32", scaled=False),
        # one request, one row of logits: the latency of a chat reply with penalties
        dict(name="edit one row", op="edit", R=1, gamma=0, V=151936, dt="bf16", longest=1500, bias=8,
             masks=0),
        # the verified rows of a 128-request round; a quarter of them under a grammar
        dict(name="edit verified batch", op="edit", R=128, gamma=16, V=151936, dt="bf16", longest=6000,
             bias=16, masks=32),
        # few requests with very long histories, fp32 logits of an odd vocabulary
        dict(name="edit f32 long history", op="edit", R=24, gamma=4, V=129277, dt="f32", longest=120000,
             bias=300, masks=3),
        # grammar masks alone, over the target's rows in place (constrained decoding)
        dict(name="edit grammar in place", op="mask", R=128, gamma=7, V=151936, dt="bf16", masks=64),
        # training on sampled replies: the gradient of the edited logits goes back to the raw ones
        dict(name="edit gradient train batch", op="edit_gradient", R=64, gamma=15, V=129280, dt="bf16",
             longest=2000, bias=0, masks=16),
        # the tokens of a small round join four histories
        dict(name="history 4 requests", op="history", R=4, width=6, capacity=2048),
        # the emitted tokens of a 512-request round, gamma = 15
        dict(name="history 512 requests", op="history", R=512, width=16, capacity=8191),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rot(rng, D):
    """All of a head, a half, a quarter, or any even part of it."""
    return rng.choice([D, D, D // 2, D // 4 * 2, 2 * rng.randint(1, D // 2)])


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["rotary", "rotary_gradient", "append", "append", "edit", "edit", "mask",
                     "edit_gradient", "history"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op in ("rotary", "rotary_gradient"):
        D, Hkv = rng.choice([64, 80, 96, 112, 128, 192, 256]), rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 3, 4, 7, 8])
        most = max(1, int(8e7 / ((Hq + Hkv) * D * _SIZE[dt])))
        rows = _log(rng, 1, min(most, 20000))
        return dict(op=op, rows=rows, seqs=rng.choice([0, 1, min(rows, _log(rng, 1, 300))]), Hq=Hq,
                    Hkv=Hkv, D=D, rot=_rot(rng, D), layout=rng.choice(["half", "interleaved"]), dt=dt,
                    scaled=rng.random() < 0.5)
    if op == "append":
        D, Hkv = rng.choice([64, 96, 128, 256]), rng.choice([1, 2, 4, 8])
        longest, gamma = _log(rng, 20, 8000), rng.choice([0, 0, 3, 5, 7, 15])
        R = _log(rng, 1, 256)
        Hq, whole = Hkv * rng.choice([1, 3, 4, 7, 8]), rng.choice([0, 0, 1, R // 4])
        # a pool and new rows no larger than the listed cases'
        R = max(1, min(R, int(3e8 / (longest * Hkv * D * _SIZE[dt]))))
        whole = min(whole, R, int(1.2e8 / (longest * (Hq + 2 * Hkv) * D * _SIZE[dt])))
        return dict(op=op, R=R, gamma=gamma, Hq=Hq, Hkv=Hkv, D=D,
                    rot=_rot(rng, D), page=rng.choice([16, 32, 64, 128]), longest=longest, whole=whole,
                    layout=rng.choice(["half", "interleaved"]), dt=dt, scaled=rng.random() < 0.5)
    if op == "history":
        return dict(op=op, R=_log(rng, 1, 512), width=rng.randint(1, 17), capacity=_log(rng, 100, 8000))
    R, gamma, V = _log(rng, 1, 128), rng.randint(0, 16), _log(rng, 1000, 151936)
    R = max(1, min(R, int(1.6e8 / V / (_SIZE[dt] // 2)) // (gamma + 1)))
    masks = rng.choice([0, 1, _log(rng, 1, 64)])
    if op == "mask":
        return dict(op=op, R=R, gamma=gamma, V=V, dt=dt, masks=max(1, masks))
    # histories of at most two million tokens in all
    longest = _log(rng, 2, max(2, min(120000, 2000000 // R)))
    return dict(op=op, R=R, gamma=gamma, V=V, dt=dt, longest=longest,
                bias=0 if op == "edit_gradient" else rng.choice([0, 1, 16, 300]), masks=masks)


def _spread(n, lo, hi):
    """n whole numbers from hi down to lo, evenly spaced."""
    return np.floor(hi - (hi - lo) * np.arange(n) / max(n - 1, 1) + 0.5).astype(np.int64)


def _rows_of(case):
    """New rows of each request (1 + ell, ell from 0 to gamma), before the seed's permutation."""
    return 1 + _spread(case["R"], 0, case["gamma"])


def _lens_of(case):
    """Context lengths with the new rows, and the new rows: the first `whole` requests
    are new altogether."""
    lens = np.maximum(_spread(case["R"], 1, case["longest"]), case["gamma"] + 1)
    rows = _rows_of(case)[::-1].copy()
    rows[: case["whole"]] = lens[: case["whole"]]
    return lens, rows


def _seqs_of(case):
    """Lengths of the packed sequences of a batch of rows, all different where they can be."""
    n, s = case["rows"], max(1, case["seqs"])
    cuts = np.floor(n * (np.arange(s + 1) / s) ** 1.3 + 0.5).astype(np.int64)
    return np.diff(cuts)


def _pad(V, dt):
    return -(-V // (16 // _SIZE[dt])) * (16 // _SIZE[dt])


# A grammar's state allows few tokens (a keyword, a bracket) or nearly all (inside a text).
_DENSE, _SPARSE = 0.95, 0.02


def _masked(case):
    """Which of the rows in use have a mask, as a share, and the share of a mask that is forbidden."""
    if not case["masks"]:
        return 0.0, 0.0
    dense = (case["masks"] + 1) // 2 / case["masks"]
    return (1.0 if case["op"] == "mask" else 0.25), dense * (1 - _DENSE) + (1 - dense) * (1 - _SPARSE)


def work(case):
    op = case["op"]
    if op in ("rotary", "rotary_gradient"):
        n = case["rows"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 2 * n * case["D"] * _SIZE[case["dt"]] + 4 * case["rows"] + 4 * case["rot"],
                "flops": 3 * n * case["rot"]}
    if op == "append":
        n = int(_lens_of(case)[1].sum())
        return {"bytes": 2 * n * (case["Hq"] + 2 * case["Hkv"]) * case["D"] * _SIZE[case["dt"]]
                + 4 * n + 12 * case["R"],
                "flops": 3 * n * (case["Hq"] + case["Hkv"]) * case["rot"]}
    if op == "history":
        n = case["R"] * (case["width"] + 1) / 2
        return {"bytes": int(8 * n + 12 * case["R"]), "flops": 0}
    rows, V, es = int(_rows_of(case).sum()), case["V"], _SIZE[case["dt"]]
    small = 4 * case["R"] + 4 * rows + case["masks"] * (-(-V // 32)) * 4
    if op == "mask":
        return {"bytes": int(small + rows * V * es * _masked(case)[1]), "flops": 0}
    histories = 4 * int(_spread(case["R"], 1, case["longest"]).sum()) + 24 * case["R"]
    return {"bytes": 2 * rows * V * es + small + histories + 8 * case["R"] * case["bias"],
            "flops": 2 * rows * V}


# ----------------------------------------------------------------- prepare
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)


def _cu(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).cuda()


def _offsets(rows):
    return _cu(np.concatenate(([0], np.cumsum(rows))))


_CONTEXT, _FACTOR, _SLOW, _FAST = 8192, 8.0, 1.0, 32.0


def _frequencies(case):
    """Radians a token of every pair, and the factor of the rotated values: base 10000, or
    a base of 500000 whose slow pairs are stretched eightfold (those that turn less than
    once in 8192 tokens; between one and 32 turns in part)."""
    i = np.arange(case["rot"] // 2, dtype=np.float64)
    f = (500000.0 if case["scaled"] else 10000.0) ** (-2.0 * i / case["rot"])
    if not case["scaled"]:
        return f, 1.0
    keep = np.clip((_CONTEXT * f / (2 * np.pi) - _SLOW) / (_FAST - _SLOW), 0.0, 1.0)
    return f * (keep + (1 - keep) / _FACTOR), 1.0 + 0.1 * math.log(_FACTOR)


def prepare(case, seed):
    return {"rotary": _prepare_rotary, "rotary_gradient": _prepare_rotary, "append": _prepare_append,
            "edit": _prepare_edit, "edit_gradient": _prepare_edit, "mask": _prepare_edit,
            "history": _prepare_history}[case["op"]](case, seed)


def _prepare_rotary(case, seed):
    """Queries and keys of one projection's output (or the gradients that come back for
    them), side by side in each row; far positions, or packed sequences from 0 on."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    n, Hq, Hkv, D = case["rows"], case["Hq"], case["Hkv"], case["D"]
    f, m = _frequencies(case)
    qkv = torch.randn((n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(_DT[case["dt"]])
    st = dict(case=case, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], f=torch.from_numpy(f).cuda(), magnitude=m)
    if case["seqs"]:
        st["row_offset"] = _offsets(rng.permutation(_seqs_of(case)))
    else:
        st["positions"] = _cu(rng.integers(0, 1000000, n))
    return st


def _prepare_append(case, seed):
    """Requests whose pages are scattered over a pool, as after many rounds; queries,
    keys and values of the new rows come from one projection."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    dt, D, page = _DT[case["dt"]], case["D"], case["page"]
    Hq, Hkv, R = case["Hq"], case["Hkv"], case["R"]
    lens, rows = _lens_of(case)
    order = rng.permutation(R)
    lens, rows = lens[order], rows[order]
    n = int(rows.sum())
    pages = -(-lens // page)
    n_pages, width = int(pages.sum()) + 3, int(pages.max()) + 1
    ids = rng.permutation(n_pages)
    table = np.full((R, width), -1, np.int32)
    table[np.arange(width)[None] < pages[:, None]] = ids[: pages.sum()]
    f, m = _frequencies(case)
    qkv = torch.randn((n, Hq + 2 * Hkv, D), generator=g, device="cuda").to(dt)
    k = torch.zeros((n_pages, Hkv, page, D), dtype=dt, device="cuda")
    v = torch.zeros((n_pages, Hkv, D, page), dtype=dt, device="cuda")
    return dict(case=case, q=qkv[:, :Hq], k_new=qkv[:, Hq:Hq + Hkv], v_new=qkv[:, Hq + Hkv:], k=k, v=v,
                table=_cu(table), kv_len=_cu(lens), row_offset=_offsets(rows),
                f=torch.from_numpy(f).cuda(), magnitude=m)


def _tokens(g, shape, V):
    """Tokens as texts have them: a few are frequent, most are rare."""
    return (V ** torch.rand(shape, generator=g, device="cuda", dtype=torch.float64) - 1).to(_I32)


def _prepare_edit(case, seed):
    """Logit rows spread like a language model's; histories of unequal length, about a
    third of each the prompt; the round's drafts, parameters and grammar states.  Two spare
    rows lie behind the last."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    R, V, dt, w = case["R"], case["V"], _DT[case["dt"]], case["gamma"]
    rows = rng.permutation(_rows_of(case))
    n = int(rows.sum())

    def logits():
        X = torch.empty((n + 2, _pad(V, case["dt"])), dtype=dt, device="cuda")
        for a in range(0, n + 2, 256):  # in pieces: 32-bit values of the whole batch are not needed
            b = min(a + 256, n + 2)
            z = torch.randn((b - a, X.shape[1]), generator=g, device="cuda")
            X[a:b] = (2.0 * z + 0.35 * z * z.abs()).to(dt)
        return X[:, :V]

    st = dict(case=case, X=logits(), row_offset=_offsets(rows), rows=n)
    if case["masks"]:
        m, words = case["masks"], -(-V // 32)
        share = torch.where(torch.arange(m, device="cuda") % 2 == 0, _DENSE, _SPARSE)
        bits = torch.rand((m, words * 32), generator=g, device="cuda") < share[:, None]
        bits = bits.view(m, words, 32).long() << torch.arange(32, device="cuda")
        st["mask"] = bits.sum(2).to(_I32)  # bit i of a word: its entry i is allowed
        index = rng.integers(0, m, n + 2)
        if case["op"] != "mask":
            index[rng.random(n + 2) >= 0.25] = -1
        st["mask_index"] = _cu(index)
    if case["op"] == "mask":
        return st
    lens = rng.permutation(_spread(R, 1, case["longest"]))
    u = lambda a, b: (a + (b - a) * torch.rand(R, generator=g, device="cuda"))  # noqa: E731
    st |= dict(history=_tokens(g, (R, case["longest"]), V), hist_len=_cu(lens), prompt_len=_cu(lens // 3),
               drafts=_tokens(g, (R, w), V) if w else None, repetition=u(1.0, 1.3))
    if case["op"] == "edit":
        st |= dict(presence=u(0.0, 1.0), frequency=u(0.0, 0.5), bias_ids=None, bias=None)
        if case["bias"]:
            # distinct within a request: a stretch of the vocabulary in steps of 1 + seed % 3
            at = rng.integers(0, V, (R, 1)) + (1 + seed % 3) * np.arange(case["bias"])[None]
            st["bias_ids"] = _cu(at % V)
            st["bias"] = 2.0 * torch.randn((R, case["bias"]), generator=g, device="cuda")
    else:
        st["G"] = logits()
    st["out"] = torch.zeros((n + 2, _pad(V, case["dt"])), dtype=dt, device="cuda")[:, :V]
    return st


def _prepare_history(case, seed):
    """Histories with room for the round's tokens, of which each request accepted some."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    R, w, cap = case["R"], case["width"], case["capacity"]
    n_acc = rng.permutation(_spread(R, 1, w)) - 1
    y = rng.integers(0, 151936, (R, w))
    y[np.arange(w)[None] > n_acc[:, None]] = -1
    return dict(case=case, history=_tokens(g, (R, cap), 151936), y=_cu(y), n_acc=_cu(n_acc),
                hist_len=_cu(rng.integers(1, cap - w + 1, R)),
                hist_len_out=torch.zeros(R, dtype=_I32, device="cuda"))


# --------------------------------------------------------------------- run
def run(state):
    return {"rotary": _run_rotary, "rotary_gradient": _run_rotary, "append": _run_append,
            "edit": _run_edit, "edit_gradient": _run_gradient, "mask": _run_mask,
            "history": _run_history}[state["case"]["op"]](state)


def _kept(state):
    """The library with the workspace and the plan that a program keeps between calls."""
    import draft_sampling_verification_03_amd as ds
    if "ws" not in state:
        state["ws"] = ds.Workspace()
        c = state["case"]
        if "rot" in c:
            more = dict(base=10000.0)
            if c["scaled"]:
                more = dict(base=500000.0, scaling="by_turns", factor=_FACTOR, context=_CONTEXT,
                            slow=_SLOW, fast=_FAST, magnitude=state["magnitude"])
            state["plan"] = ds.RotaryPlan(c["rot"], layout=c["layout"], **more)
    return ds, state["ws"]


def _rotated(x, positions, state, sign=1.0):
    """x [n][heads][D] with its first `rot` elements rotated: angles in 64 bits, the rest in 32."""
    c = state["case"]
    angle = positions.double()[:, None] * state["f"]
    cos = (state["magnitude"] * torch.cos(angle)).float()[:, None]
    sin = (sign * state["magnitude"] * torch.sin(angle)).float()[:, None]
    x32, rot = x.float(), c["rot"]
    if c["layout"] == "half":
        a, b = x32[..., : rot // 2], x32[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin, x32[..., rot:]), -1)
    else:
        a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        y = torch.cat((y, x32[..., rot:]), -1)
    return y.to(x.dtype)


def _places(row_offset, n):
    """Request and place within the request of every row."""
    off = row_offset.long()
    row = torch.arange(n, device="cuda")
    rho = torch.searchsorted(off[1:].contiguous(), row, right=True).clamp(max=off.numel() - 2)
    return rho, row - off[rho]


def _run_rotary(state):
    c = state["case"]
    back = c["op"] == "rotary_gradient"
    if own:
        ds, ws = _kept(state)
        f = ds.rotary_backward if back else ds.rotary
        return f(state["q"], state["k"], plan=state["plan"], positions=state.get("positions"),
                 row_offset=state.get("row_offset"), ws=ws)
    pos = state["positions"] if not c["seqs"] else _places(state["row_offset"], c["rows"])[1]
    return {k: _rotated(state[k], pos, state, -1.0 if back else 1.0) for k in ("q", "k")}


def _run_append(state):
    if own:
        ds, ws = _kept(state)
        q = ds.cache_append(state["q"], state["k_new"], state["v_new"], state["k"], state["v"],
                            state["table"], state["kv_len"], plan=state["plan"],
                            row_offset=state["row_offset"], ws=ws)
        return {"q": q, "k": state["k"], "v": state["v"]}
    page, off = state["case"]["page"], state["row_offset"].long()
    rho, j = _places(state["row_offset"], state["q"].shape[0])
    pos = state["kv_len"].long()[rho] - (off[rho + 1] - off[rho]) + j
    at = state["table"].long()[rho, pos // page]
    state["k"][at, :, pos % page] = _rotated(state["k_new"], pos, state)
    state["v"][at, :, :, pos % page] = state["v_new"]
    return {"q": _rotated(state["q"], pos, state), "k": state["k"], "v": state["v"]}


def _allowed(state, rho_rows):
    """[rows][V]: what each row's mask allows."""
    V = state["case"]["V"]
    bits = (state["mask"][:, :, None] >> torch.arange(32, device="cuda", dtype=_I32)) & 1
    bits = torch.cat((bits.flatten(1)[:, :V] != 0, torch.ones((1, V), dtype=torch.bool, device="cuda")))
    index = state["mask_index"][:rho_rows].long()
    return bits[torch.where(index >= 0, index, state["mask"].shape[0])]


def _counts(state):
    """How often each row's request has generated each token, and whether it has seen it."""
    c = state["case"]
    R, V = c["R"], c["V"]
    i = torch.arange(state["history"].shape[1], device="cuda")[None]
    tok = state["history"].long()
    made = (i >= state["prompt_len"][:, None]) & (i < state["hist_len"][:, None])
    said = i < state["prompt_len"][:, None]
    one = torch.ones_like(state["history"])
    count = torch.zeros((R, V + 1), dtype=_I32, device="cuda")
    count.scatter_add_(1, torch.where(made, tok, V), one)
    prompt = torch.zeros((R, V + 1), dtype=_I32, device="cuda")
    prompt.scatter_add_(1, torch.where(said, tok, V), one)
    rho, j = _places(state["row_offset"], state["rows"])
    count = count[rho]
    if state["drafts"] is not None:  # a row's drafts before it count as generated
        d = state["drafts"].long()[rho]
        before = torch.arange(d.shape[1], device="cuda")[None] < j[:, None]
        count.scatter_add_(1, torch.where(before, d, V), torch.ones_like(d, dtype=_I32))
    count = count[:, :V]
    return rho, count, (count > 0) | (prompt[rho, :V] > 0)


def _run_edit(state):
    if own:
        ds, ws = _kept(state)
        return ds.edit_logits(state["X"], row_offset=state["row_offset"], history=state["history"],
                              hist_len=state["hist_len"], prompt_len=state["prompt_len"],
                              drafts=state["drafts"], repetition=state["repetition"],
                              presence=state["presence"], frequency=state["frequency"],
                              bias_ids=state["bias_ids"], bias=state["bias"], mask=state.get("mask"),
                              mask_index=state.get("mask_index"), ws=ws, out=state["out"])
    n = state["rows"]
    rho, count, seen = _counts(state)
    x = state["X"][:n].float()
    r = state["repetition"][rho, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - state["frequency"][rho, None] * count
    x = x - torch.where(count > 0, state["presence"][rho, None], 0.0)
    if state["bias"] is not None:
        x.scatter_add_(1, state["bias_ids"].long()[rho], state["bias"][rho])
    if "mask" in state:
        x = torch.where(_allowed(state, n), x, float("-inf"))
    state["out"][:n] = x.to(state["X"].dtype)
    return state["out"]


def _run_gradient(state):
    if own:
        ds, ws = _kept(state)
        return ds.edit_logits_backward(state["G"], state["X"], row_offset=state["row_offset"],
                                       history=state["history"], hist_len=state["hist_len"],
                                       prompt_len=state["prompt_len"], drafts=state["drafts"],
                                       repetition=state["repetition"], mask=state.get("mask"),
                                       mask_index=state.get("mask_index"), ws=ws, out=state["out"])
    n = state["rows"]
    rho, _, seen = _counts(state)
    g = state["G"][:n].float()
    r = state["repetition"][rho, None]
    g = torch.where(seen, torch.where(state["X"][:n].float() > 0, g / r, g * r), g)
    if "mask" in state:
        g = torch.where(_allowed(state, n), g, 0.0)
    state["out"][:n] = g.to(state["G"].dtype)
    return state["out"]


def _run_mask(state):
    if own:
        ds, ws = _kept(state)
        return ds.edit_logits(state["X"], row_offset=state["row_offset"], mask=state["mask"],
                              mask_index=state["mask_index"], ws=ws, out=state["X"])
    n = state["rows"]
    state["X"][:n].masked_fill_(~_allowed(state, n), float("-inf"))
    return state["X"]


def _run_history(state):
    if own:
        ds, ws = _kept(state)
        ds.history_append(state["history"], state["hist_len"], state["y"], n_acc=state["n_acc"], ws=ws,
                          out=state["hist_len_out"])
        return {"history": state["history"], "hist_len": state["hist_len_out"]}
    w = state["y"].shape[1]
    i = torch.arange(w, device="cuda")[None]
    keep = i <= state["n_acc"][:, None]
    at = state["hist_len"].long()[:, None] + i
    r = torch.arange(state["y"].shape[0], device="cuda")[:, None].expand(-1, w)
    state["history"][r, at] = torch.where(keep, state["y"], state["history"][r, at])
    return {"history": state["history"], "hist_len": state["hist_len"] + state["n_acc"] + 1}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    st = prepare(case, seed)
    return {"rotary": _exact_rotary, "rotary_gradient": _exact_rotary, "append": _exact_append,
            "edit": _exact_edit, "edit_gradient": _exact_gradient, "mask": _exact_mask,
            "history": _exact_history}[case["op"]](case, st)


def _turned(x, positions, case, st, conjugate=False):
    """x as complex numbers, times magnitude e^(i position f)."""
    rot, D = case["rot"], case["D"]
    perm = torch.arange(D)  # pairs side by side
    if case["layout"] == "half":
        perm[:rot] = torch.arange(rot).view(2, rot // 2).T.reshape(-1)
    perm = perm.cuda()
    out = x.double()[..., perm]
    z = torch.view_as_complex(out[..., :rot].contiguous().unflatten(-1, (rot // 2, 2)))
    turn = torch.polar(torch.full_like(st["f"], st["magnitude"])[None].expand(len(positions), -1),
                       positions.double()[:, None] * st["f"][None])
    if conjugate:
        turn = turn.conj()
    out[..., :rot] = torch.view_as_real(z * turn[:, None]).flatten(-2)
    back = torch.empty_like(out)
    back[..., perm] = out
    return back


def _exact_rotary(case, st):
    if case["seqs"]:
        off = st["row_offset"].tolist()
        pos = torch.cat([torch.arange(b - a) for a, b in zip(off, off[1:])]).cuda()
    else:
        pos = st["positions"]
    return {k: _turned(st[k], pos, case, st, case["op"] == "rotary_gradient") for k in ("q", "k")}


def _exact_append(case, st):
    """Request by request, page by page."""
    page = case["page"]
    off, lens, table = (st[k].tolist() for k in ("row_offset", "kv_len", "table"))
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    for r in range(case["R"]):
        a, b, L = off[r], off[r + 1], lens[r]
        pos = torch.arange(L - (b - a), L, device="cuda")
        q[a:b] = _turned(st["q"][a:b], pos, case, st)
        kr = _turned(st["k_new"][a:b], pos, case, st)
        t = L - (b - a)
        while t < L:
            e = min(L, (t // page + 1) * page)
            i, s, m = table[r][t // page], t % page, t - (L - (b - a))
            k[i, :, s:s + e - t] = kr[m:m + e - t].transpose(0, 1)
            v[i, :, :, s:s + e - t] = st["v_new"][a + m:a + m + e - t].permute(1, 2, 0).double()
            t = e
    return {"q": q, "k": k, "v": v}


def _rows_with_counts(case, st):
    """(row, request, times generated [V], in the prompt [V]) of every row in use."""
    off, lens, said = (st[k].tolist() for k in ("row_offset", "hist_len", "prompt_len"))
    for r in range(case["R"]):
        tok = st["history"][r].long()
        count = torch.bincount(tok[said[r]:lens[r]], minlength=case["V"])
        prompt = torch.bincount(tok[: said[r]], minlength=case["V"]) > 0
        for row in range(off[r], off[r + 1]):
            if row > off[r]:
                count[st["drafts"][r, row - off[r] - 1].long()] += 1
            yield row, r, count, prompt


def _forbidden(case, st, row):
    """[V]: what the row's mask leaves out, None without a mask."""
    if "mask" not in st or int(st["mask_index"][row]) < 0:
        return None
    words = st["mask"][int(st["mask_index"][row])].long() & 0xFFFFFFFF
    v = torch.arange(case["V"], device="cuda")
    return (words[v // 32] // 2 ** (v % 32)) % 2 == 0


def _exact_edit(case, st):
    out = st["out"].double()
    for row, r, count, prompt in _rows_with_counts(case, st):
        x = st["X"][row].double()
        rep = st["repetition"][r].double()
        again = torch.where(x > 0, x / rep, x * rep)
        x = torch.where(prompt | (count > 0), again, x)
        x = x - st["frequency"][r].double() * count - st["presence"][r].double() * (count > 0)
        if case["bias"]:
            x[st["bias_ids"][r].long()] += st["bias"][r].double()
        no = _forbidden(case, st, row)
        out[row] = x if no is None else x.masked_fill(no, float("-inf"))
    return out


def _exact_gradient(case, st):
    out = st["out"].double()
    for row, r, count, prompt in _rows_with_counts(case, st):
        rep = st["repetition"][r].double()
        slope = torch.where(prompt | (count > 0), torch.where(st["X"][row] > 0, 1 / rep, rep), 1.0)
        no = _forbidden(case, st, row)
        g = st["G"][row].double() * slope
        out[row] = g if no is None else g.masked_fill(no, 0.0)
    return out


def _exact_mask(case, st):
    out = st["X"].double()
    for row in range(st["rows"]):
        out[row].masked_fill_(_forbidden(case, st, row), float("-inf"))
    return out


def _exact_history(case, st):
    history, lens = st["history"].cpu(), st["hist_len"].tolist()
    for r, (n, y) in enumerate(zip(st["n_acc"].tolist(), st["y"].tolist())):
        for tok in y[: n + 1]:
            history[r, lens[r]] = tok
            lens[r] += 1
    return {"history": history, "hist_len": torch.tensor(lens)}
