"""GPU tests of logit edits and token histories against a plain model in 64 bits.

Tolerances (u = 2^-24): the quotient or product rounds once (the quotient's correction is
itself off by less than another u), frequency n, the two differences and the bias's sum
once each, none of them larger than S = |x'| + |frequency n| + |presence| + |bias|: 6 u S
in all; a bf16 result half a step more, 2^-8 of the value.  Untouched logits and masked
ones are exact.
"""
import numpy as np
import pytest
import torch

import draft_sampling_verification_03_amd as ds

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24
TOKEN, LENGTH, NONFINITE = 1, 4, 8
I32 = torch.int32
INF = float("inf")


def i32(a):
    return torch.tensor(a, dtype=I32, device="cuda")


def f32(a):
    return torch.tensor(a, dtype=F, device="cuda")


def pack(allowed):
    """[m][V] bools to [m][ceil(V / 32)] words, on the host."""
    a = np.asarray(allowed, bool)
    a = np.pad(a, ((0, 0), (0, -a.shape[1] % 32)))
    words = (a.reshape(a.shape[0], -1, 32) << np.arange(32, dtype=np.uint64)).sum(2)
    return torch.from_numpy(words.astype(np.uint32).view(np.int32)).cuda()


class Edits:
    """A batch of requests with histories, drafts, parameters, biases and masks."""

    def __init__(self, rows, V, dt, seed=0, longest=50, gamma=None, n_bias=0, masks=0, spare=0, prompt=True,
                 hot=None):
        rng = np.random.default_rng(seed)
        R, n = len(rows), sum(rows)
        self.rows, self.V, self.dt, self.R = rows, V, dt, R
        self.off = np.concatenate(([0], np.cumsum(rows))).astype(int)
        self.n = n
        g = torch.Generator(device="cuda").manual_seed(seed)
        per = 8 if dt == BF else 4
        wide = torch.randn((n + spare, -(-V // per) * per), generator=g, device="cuda")
        self.X = (3 * wide).to(dt)[:, :V]
        self.row_offset = i32(self.off.tolist())
        gamma = max(rows + [1]) - 1 if gamma is None else gamma
        hot = V if hot is None else min(hot, V)
        self.history = rng.integers(0, hot, (R, longest))
        self.hist_len = rng.integers(0, longest + 1, R)
        self.hist_len[0] = longest
        self.prompt_len = (self.hist_len * rng.random(R)).astype(int) if prompt else None
        self.drafts = rng.integers(0, hot, (R, gamma)) if gamma else None
        if gamma and gamma > 1:
            self.drafts[0, 1] = self.drafts[0, 0]  # the same twice in a row
        self.repetition = rng.uniform(0.7, 1.6, R).astype(np.float32)
        self.frequency = rng.uniform(-0.5, 0.5, R).astype(np.float32)
        self.presence = rng.uniform(-0.5, 1.0, R).astype(np.float32)
        self.bias_ids = self.bias = None
        if n_bias:
            self.bias_ids = rng.integers(0, V, (R, n_bias))
            self.bias = rng.standard_normal((R, n_bias)).astype(np.float32)
        self.allowed = self.mask_index = None
        if masks:
            self.allowed = rng.random((masks, V)) < rng.choice([0.02, 0.5, 0.98], (masks, 1))
            self.mask_index = rng.integers(-1, masks, n + spare)

    def args(self, grad=False):
        cu = lambda a: None if a is None else torch.from_numpy(  # noqa: E731
            a.astype(np.int32) if a.dtype.kind == "i" else a).cuda()
        kw = dict(row_offset=self.row_offset, history=cu(self.history), hist_len=cu(self.hist_len),
                  prompt_len=cu(self.prompt_len), drafts=cu(self.drafts), repetition=cu(self.repetition),
                  mask=None if self.allowed is None else pack(self.allowed), mask_index=cu(self.mask_index))
        if not grad:
            kw.update(frequency=cu(self.frequency), presence=cu(self.presence), bias_ids=cu(self.bias_ids),
                      bias=cu(self.bias))
        return kw

    def counts(self, r, j):
        """(times generated [V], in the prompt [V]) of row j of request r."""
        L = self.hist_len[r]
        p = 0 if self.prompt_len is None else self.prompt_len[r]
        made, said = self.history[r, p:L], self.history[r, :p]
        if self.drafts is not None:
            made = np.concatenate([made, self.drafts[r, :j]])
        made, said = made[made >= 0], said[said >= 0]
        prompt = np.zeros(self.V, bool)
        prompt[said] = True
        return np.bincount(made, minlength=self.V), prompt

    def seen(self, r, j):
        c, p = self.counts(r, j)
        return torch.from_numpy((c > 0) | p).cuda()

    def forbidden(self, row):
        if self.allowed is None or self.mask_index[row] < 0:
            return None
        return torch.from_numpy(~self.allowed[self.mask_index[row]]).cuda()

    def each(self):
        for r in range(self.R):
            for j in range(self.rows[r]):
                yield r, j, self.off[r] + j

    def check(self, got, raw):
        for r, j, row in self.each():
            c, p = self.counts(r, j)
            c, p = torch.from_numpy(c).cuda(), torch.from_numpy(p).cuda()
            x, rep = raw[row].double(), float(self.repetition[r])
            again = (c > 0) | p
            x = torch.where(again, torch.where(x > 0, x / rep, x * rep), x)
            f = float(self.frequency[r]) * c
            q = float(self.presence[r]) * (c > 0)
            want, size = x - f - q, x.abs() + f.abs() + q.abs()
            edited = again.clone()
            if self.bias_ids is not None:
                first = {}
                for v, b in zip(self.bias_ids[r], self.bias[r]):
                    if v >= 0:
                        first.setdefault(int(v), float(b))
                at = torch.tensor(list(first), device="cuda")
                if len(first):
                    b = torch.tensor(list(first.values()), dtype=torch.float64, device="cuda")
                    want[at] += b
                    size[at] += b.abs()
                    edited[at] = True
            tol = 6 * U * size
            if self.dt == BF:
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
            tol = torch.where(edited, tol, 0.0)
            no = self.forbidden(row)
            if no is not None:
                want = want.masked_fill(no, -INF)
            have = got[row].double()
            same = have == want
            err = (have - want).abs()
            assert (same | (err <= tol)).all(), (r, j, (err - tol)[~same].max().item())

    def check_gradient(self, got, G, raw):
        for r, j, row in self.each():
            rep = float(self.repetition[r])
            again = self.seen(r, j)
            slope = torch.where(again, torch.where(raw[row] > 0, 1 / rep, rep), 1.0)
            want = G[row].double() * slope
            tol = torch.where(again, 2 * U * want.abs() + (2.0 ** -8 * want.abs() if self.dt == BF else 0), 0.0)
            no = self.forbidden(row)
            if no is not None:
                want, tol = want.masked_fill(no, 0.0), tol.masked_fill(no, 0.0)
            assert ((got[row].double() - want).abs() <= tol).all(), (r, j)


CASES = [
    dict(rows=[1], V=1, longest=1), dict(rows=[1], V=7, longest=3, n_bias=2, masks=1),
    dict(rows=[3], V=16, longest=40, n_bias=5, masks=2), dict(rows=[2, 0, 5], V=1001, n_bias=3, masks=4),
    dict(rows=[1, 17, 2], V=4096, longest=300, n_bias=16), dict(rows=[4, 1], V=4097, longest=301, masks=3),
    dict(rows=[1] * 9, V=8191, longest=77, n_bias=1, masks=5), dict(rows=[5, 9], V=12289, longest=5000, hot=300),
    dict(rows=[2, 1, 6], V=151936, longest=6000, n_bias=1023, masks=2),
    dict(rows=[1, 3], V=129277, longest=30011, n_bias=300, masks=1),
    dict(rows=[0, 0, 3], V=262144, longest=2, masks=1), dict(rows=[40, 1], V=513, longest=9, hot=4),
]


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_values_in_place_and_gradient(case, dt):
    e = Edits(dt=dt, seed=case, spare=2, **CASES[case])
    ws = ds.Workspace()
    raw = e.X.clone()
    wide = torch.full((e.n + 2, -(-e.V // 8) * 8 + 16), 7.0, dtype=dt, device="cuda")
    got = ds.edit_logits(e.X, ws=ws, out=wide[:, :e.V], **e.args())
    assert ws.error_code() == 0
    e.check(got, raw)
    assert (wide[e.n:] == 7).all() and (wide[:, e.V:] == 7).all() and torch.equal(e.X, raw)
    new = ds.edit_logits(e.X, ws=ws, **e.args())
    assert torch.equal(new[:e.n], got[:e.n])
    G = torch.randn(e.X.shape, device="cuda").to(dt)
    G = torch.nn.functional.pad(G, (0, -e.V % 8))[:, :e.V]
    dX = ds.edit_logits_backward(G, raw_rows(raw), ws=ws, **e.args(grad=True))
    e.check_gradient(dX, G, raw)
    # in place: rows behind the last and columns from V on stay
    base = torch.full((e.n + 2, -(-e.V // 8) * 8), 7.0, dtype=dt, device="cuda")
    base[:, :e.V] = raw
    assert ds.edit_logits(base[:, :e.V], ws=ws, out=base[:, :e.V], **e.args()).data_ptr() == base.data_ptr()
    assert torch.equal(base[:e.n, :e.V], got[:e.n]) and torch.equal(base[e.n:, :e.V], raw[e.n:])
    assert (base[:, e.V:] == 7).all()
    ds.edit_logits_backward(G, raw_rows(raw), ws=ws, out=G, **e.args(grad=True))
    assert torch.equal(G[:e.n], dX[:e.n]) and ws.error_code() == 0


def whole_pieces(V, per):
    """Masks [14][V] of whole 16-byte pieces (`per` tokens), lines of eight of them and
    words, of stretches with even and odd ends, and of the row's last piece."""
    v = np.arange(V)
    line, last = 8 * per, v >= V - 1 - (V - 1) % per
    return np.array([(v >= 16) & (v < 24), v < 1000, (v >= 1000) & (v < 2000), v // per % 2 == 0, v // per % 2 == 1,
                     v // line % 2 == 0, v // 32 % 2 == 1, v // per % 8 == 5, v // per % 8 != 2,
                     (v >= 7) & (v < 331), v % 1000 < 500, v != V - 1, ~last, last])


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("V", [1001, 4096, 9000, 151936])
@pytest.mark.parametrize("history", [False, True])
def test_masks_of_whole_pieces_in_place(V, dt, history):
    """In place, where lines of 128 bytes hold pieces wholly forbidden and pieces wholly
    allowed: the values and gradients of another output, bit for bit."""
    e = Edits([14, 1, 70], V, dt, seed=V, longest=6, n_bias=3, masks=14)
    e.allowed = whole_pieces(V, 8 if dt == BF else 4)
    e.mask_index = np.concatenate((np.arange(14), [3], np.random.default_rng(1).integers(-1, 14, 70)))
    kw, grad = e.args(), e.args(grad=True)
    if not history:
        for name in ("history", "hist_len", "prompt_len", "drafts", "repetition", "frequency", "presence",
                     "bias_ids", "bias"):
            kw[name] = None
            if name in grad:
                grad[name] = None
    raw = e.X.clone()
    got = ds.edit_logits(e.X, **kw)
    if history:
        e.check(got, raw)
    else:
        for row, m in enumerate(e.mask_index):
            want = raw[row] if m < 0 else raw[row].masked_fill(torch.from_numpy(~e.allowed[m]).cuda(), -INF)
            assert torch.equal(got[row], want), (row, m)
    X = raw_rows(raw)
    assert torch.equal(ds.edit_logits(X, out=X, **kw), got)
    G = raw_rows(torch.randn(raw.shape, device="cuda").to(dt))
    X = raw_rows(raw)
    dX = ds.edit_logits_backward(G, X, **grad)
    if history:
        e.check_gradient(dX, G, raw)
        # the gradient without penalties has words and no slopes
        H = G.clone()
        want = ds.edit_logits_backward(raw_rows(H), **dict(grad, repetition=None))
        H = raw_rows(H)
        assert torch.equal(ds.edit_logits_backward(H, out=H, **dict(grad, repetition=None)), want)
    ds.edit_logits_backward(G, X, out=G, **grad)
    assert torch.equal(G, dX)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("share", [0.85, 0.95])
def test_random_masks_in_place(share, dt):
    """Nearly all tokens allowed: some lines hold one piece that is wholly forbidden."""
    V = 151936
    g = torch.Generator(device="cuda").manual_seed(5)
    allowed = torch.rand((64, V), generator=g, device="cuda") < share
    X = torch.randn((64, V), generator=g, device="cuda").to(dt)
    want = X.masked_fill(~allowed, -INF)
    G = torch.randn((64, V), generator=g, device="cuda").to(dt)
    mask = pack(allowed.cpu().numpy())
    assert torch.equal(ds.edit_logits(X, mask=mask, out=X), want)
    want = G.masked_fill(~allowed, 0)
    assert torch.equal(ds.edit_logits_backward(G, mask=mask, out=G), want)


def raw_rows(x):
    """x in rows of whole 16-byte pieces."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % 8))[:, :x.shape[1]]


@pytest.mark.parametrize("without", ["history", "prompt_len", "drafts", "repetition", "frequency", "presence",
                                     "bias", "masks", "all but masks", "all"])
def test_each_part_may_be_missing(without):
    e = Edits([3, 1, 4], 3001, F, seed=5, n_bias=4, masks=3)
    kw = e.args()
    if without in ("history", "all but masks", "all"):
        for k in ("history", "hist_len", "prompt_len"):
            kw[k] = None
        e.hist_len[:] = 0
        e.prompt_len = None
    if without == "prompt_len":
        kw["prompt_len"], e.prompt_len = None, None
    if without in ("drafts", "all but masks", "all"):
        kw["drafts"], e.drafts = None, None
    for name, none in (("repetition", 1.0), ("frequency", 0.0), ("presence", 0.0)):
        if without in (name, "all but masks", "all"):
            kw[name] = None
            getattr(e, name)[:] = none
    if without in ("bias", "all but masks", "all"):
        kw["bias_ids"] = kw["bias"] = e.bias_ids = e.bias = None
    if without in ("masks", "all"):
        kw["mask"] = kw["mask_index"] = e.allowed = e.mask_index = None
    e.check(ds.edit_logits(e.X, **kw), e.X)


def test_one_row_each_and_a_mask_for_every_row():
    e = Edits([1] * 6, 777, BF, seed=6, n_bias=3, masks=6)
    e.mask_index[:] = np.arange(6)
    kw = e.args()
    kw["row_offset"] = kw["mask_index"] = None
    e.check(ds.edit_logits(e.X, **kw), e.X)


def test_many_rows_of_one_request():
    """A sequence scored at once: row j stands behind j tokens of it, in parts that each
    count anew; and rows behind the last draft count them all."""
    for rows, gamma in (([700], 699), ([50, 3], 20)):
        e = Edits(rows, 900, F, seed=8, longest=33, gamma=gamma, hot=60)
        e.check(ds.edit_logits(e.X, **e.args()), e.X)


def test_padding_tokens_and_repeated_biases():
    e = Edits([4, 2], 500, F, seed=9, longest=41, n_bias=9, masks=0)
    e.history[0, ::3] = -1
    e.drafts[0, 1] = -1
    e.bias_ids[0, [1, 5]] = e.bias_ids[0, 0]  # counts the first time
    e.bias_ids[1, 3:] = -1
    ws = ds.Workspace()
    e.check(ds.edit_logits(e.X, ws=ws, **e.args()), e.X)
    assert ws.error_code() == 0


@pytest.mark.parametrize("dt", [BF, F])
def test_not_finite_logits_biases_and_empty_masks(dt):
    """Masked entries are -infinity whatever they were, in the gradient 0; a bias of
    -infinity bans, one of +infinity forces; a row may be left with nothing."""
    e = Edits([3], 2000, dt, seed=10, longest=200, n_bias=2, masks=2)
    e.allowed[0], e.allowed[1] = False, np.arange(2000) % 2 == 0
    e.mask_index[:] = [0, 1, -1]
    e.bias_ids[0], e.bias[0] = [40, 42], [-INF, INF]
    X = e.X
    X[:, 1], X[:, 3], X[:, 5] = float("nan"), INF, -INF
    X[2, 7] = float("nan")
    o = ds.edit_logits(X, **e.args())
    assert (o[0] == -INF).all() and (o[1, 1::2] == -INF).all()
    assert o[1, 40] == -INF and o[1, 42] == INF and o[2, 40] == -INF and o[2, 42] == INF
    assert o[2, 1].isnan() and o[2, 7].isnan() and o[2, 3] == INF and o[2, 5] == -INF
    G = torch.full_like(X, float("nan"))
    d = ds.edit_logits_backward(raw_rows(G), raw_rows(X), **e.args(grad=True))
    assert (d[0] == 0).all() and (d[1, 1::2] == 0).all() and d[2].isnan().all()


def test_gradient_against_differences():
    """Between its kinks at 0 the edit is linear in x with slope 1 / r or r: with x and h
    powers of two apart from rounding, the quotient of two fp32 results of size below 16,
    each off by 6 u S, is off by 12 u S / h."""
    e = Edits([4, 3], 600, F, seed=11, longest=500, n_bias=3, masks=2)
    kw = e.args()
    h = 2.0 ** -4
    x = torch.where(e.X.abs() < 2 * h, 1.0, e.X)
    up, down = ds.edit_logits(x + h, **kw), ds.edit_logits(x - h, **kw)
    slope = torch.where(up == -INF, 0.0, (up - down) / (2 * h))
    grad = ds.edit_logits_backward(torch.ones_like(x), x, **e.args(grad=True))
    # n <= 500 draws from 600 tokens: at most 10 times the same, S <= 1.6 * 20 + 5 + 1 + 5
    assert ((slope - grad).abs() <= 12 * U * 45 / (2 * h) * 2 + 2 * U * 2).all()


def test_exact_where_the_arithmetic_is():
    """Powers of two: the edit equals the same float32 operations bit for bit."""
    e = Edits([5, 2], 5000, F, seed=12, longest=900, n_bias=7)
    e.repetition[:], e.frequency[:], e.presence[:] = [2.0, 0.5], [0.25, -0.5], [1.0, 0.125]
    o = ds.edit_logits(e.X, **e.args())
    for r, j, row in e.each():
        c, p = e.counts(r, j)
        c, p = torch.from_numpy(c).cuda(), torch.from_numpy(p).cuda()
        x = e.X[row]
        rep = float(e.repetition[r])
        x = torch.where((c > 0) | p, torch.where(x > 0, x / rep, x * rep), x)
        x = x - float(e.frequency[r]) * c.float()
        x = x - torch.where(c > 0, float(e.presence[r]), 0.0)
        first = {}
        for v, b in zip(e.bias_ids[r], e.bias[r]):
            first.setdefault(int(v), float(b))
        for v, b in first.items():
            x[v] = x[v] + b
        assert torch.equal(o[row], x)


@pytest.mark.parametrize("what,code", [
    ("token", TOKEN), ("draft", TOKEN), ("bias", TOKEN), ("hist_len", LENGTH), ("negative", LENGTH),
    ("prompt_len", LENGTH), ("slice", LENGTH), ("end", LENGTH), ("mask_index", LENGTH),
    ("repetition", NONFINITE), ("repetition nan", NONFINITE), ("frequency", NONFINITE),
    ("presence", NONFINITE),
])
def test_bad_data_is_reported_and_skipped(what, code):
    """What the device finds wrong counts as absent; the rest is edited as if it were."""
    e = Edits([4, 3, 2], 9000, F, seed=13, n_bias=3, masks=2)
    kw = e.args()
    if what == "token":
        kw["history"][1, 0] = 9000
        e.hist_len[1] = kw["hist_len"][1] = 50
        kw["history"][0, 3] = -7
        e.history[1, 0] = e.history[0, 3] = -1
    elif what == "draft":
        kw["drafts"][0, 1] = 1 << 30
        e.drafts[0, 1] = -1
    elif what == "bias":
        kw["bias_ids"][2, 1] = -2
        e.bias_ids[2, 1] = -1
    elif what in ("hist_len", "negative"):
        kw["hist_len"][1] = 51 if what == "hist_len" else -1
        kw["prompt_len"][1] = 0
        e.hist_len[1], e.prompt_len[1] = 0, 0
    elif what == "prompt_len":
        kw["prompt_len"][1] = e.hist_len[1] + 1
        e.prompt_len[1] = 0
    elif what == "mask_index":
        kw["mask_index"][2] = 2
        e.mask_index[2] = -1
    elif what.startswith("repetition"):
        kw["repetition"][1] = 0.0 if what == "repetition" else float("nan")
        e.repetition[1] = 1.0
    elif what in ("frequency", "presence"):
        kw[what][0] = INF if what == "frequency" else float("nan")
        getattr(e, what)[0] = 0.0
    ws = ds.Workspace()
    if what in ("slice", "end"):
        kw["row_offset"] = i32([0, 4, 2, 9] if what == "slice" else [0, 4, 7, 10])
        out = torch.full_like(e.X, 7.0)
        o = ds.edit_logits(e.X, ws=ws, out=out, **kw)
        assert ws.error_code() == LENGTH
        good = ds.edit_logits(e.X, **e.args())
        assert torch.equal(o[:2], good[:2])
        if what == "end":
            assert torch.equal(o[:7], good[:7]) and (o[7:] == 7).all()
        return
    e.check(ds.edit_logits(e.X, ws=ws, **kw), e.X)
    assert ws.error_code() == code


def test_rows_past_32_bit_offsets():
    V, n = 151936, 7200
    X = torch.zeros((n, V), dtype=BF, device="cuda")  # 2.2 GB, 1.1e9 elements
    assert X.numel() * 2 > 1 << 31
    e = Edits([1, 2], V, BF, seed=14, longest=100)
    X[n - 3:] = e.X
    off = i32([n - 3, n - 2, n])
    kw = dict(e.args(), row_offset=off)
    want = ds.edit_logits(e.X, **e.args())
    ds.edit_logits(X, out=X, **kw)
    assert torch.equal(X[n - 3:], want) and not X[: n - 3].any()


@pytest.mark.parametrize("one_each", [True, False])
def test_most_rows(one_each):
    """The largest number of rows, one request each or all of one request."""
    n = 1 << 22
    X = torch.randn((n, 8), device="cuda").to(BF)
    mask = i32([[0b10110101]])
    allowed = torch.tensor([(0b10110101 >> v) & 1 for v in range(8)], device="cuda") != 0
    index = torch.zeros(n, dtype=I32, device="cuda")
    kw, ws = dict(mask=mask, mask_index=index), ds.Workspace()
    rep = f32([2.0] * (n if one_each else 1))
    if one_each:
        kw.update(history=torch.full((n, 1), 4, dtype=I32, device="cuda"), hist_len=index + 1, repetition=rep)
    else:
        kw.update(row_offset=i32([0, n]), history=i32([[4]]), hist_len=i32([1]), repetition=rep)
    want = X.masked_fill(~allowed, -INF)
    x = X[:, 4].float()
    want[:, 4] = torch.where(x > 0, x / 2, x * 2).to(BF)
    assert torch.equal(ds.edit_logits(X, ws=ws, **kw), want) and ws.error_code() == 0


def test_lengths_without_a_history_are_not_read():
    """The C call with hist_len and no history."""
    X = torch.randn((2, 64), device="cuda")
    out, ws = torch.empty_like(X), torch.zeros(256, dtype=torch.uint8, device="cuda")
    drafts = i32([[3, 5], [7, 9]])
    fre = f32([1.0, 2.0])
    st = ds.dspark_edit_logits(2, 64, 64, 0, X, 2, None, None, -7, i32([40, 50]), None, drafts, 2, None, fre,
                               None, 0, None, None, 0, None, 0, None, out, 64, ws, 256,
                               torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(out, X) and not ws.any()  # row 0 stands behind no draft


def test_streams_and_two_graphs_over_one_workspace():
    e = Edits([3, 1, 6], 5003, BF, seed=15, longest=400, n_bias=5, masks=3)
    kw, ws, side = e.args(), ds.Workspace(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = ds.edit_logits(e.X, ws=ws, stream=side, **kw)
    side.synchronize()
    e.check(o, e.X)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    G = raw_rows(torch.randn(e.X.shape, device="cuda").to(BF))
    with torch.cuda.graph(g1):
        a = ds.edit_logits(e.X, ws=ws, **kw)
    grad = e.args(grad=True)
    for name in ("row_offset", "history", "hist_len", "prompt_len", "drafts", "repetition", "mask", "mask_index"):
        grad[name] = kw[name]
    with torch.cuda.graph(g2):
        b = ds.edit_logits_backward(G, e.X, ws=ws, **grad)
    for i in range(4):
        e.X.copy_(torch.randn(e.X.shape, device="cuda").to(BF))
        e.history = np.random.default_rng(i).integers(0, 5003, e.history.shape)
        kw["history"].copy_(torch.from_numpy(e.history.astype(np.int32)))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        e.check(a, e.X)
        e.check_gradient(b, G, e.X)
    assert ws.error_code() == 0


def test_outputs_beside_the_input_and_over_it():
    """Columns and rows of one buffer may hold input and output; an output that lies over
    a part of the input is refused, and nothing is launched."""
    e = Edits([2, 3], 250, BF, seed=16, longest=40, n_bias=2, masks=2)
    kw, grad = e.args(), e.args(grad=True)
    want = ds.edit_logits(e.X, **kw)
    buf = torch.zeros((12, 512), dtype=BF, device="cuda")
    for x, out in ((buf[:5, :250], buf[:5, 256:506]), (buf[:5, 256:506], buf[:5, :250]),
                   (buf[:5, :250], buf[5:10, :250]), (buf[0:10:2, :250], buf[1:11:2, :250]),
                   (buf[1:11:2, :250], buf[0:10:2, :250])):
        buf.zero_()
        x.copy_(e.X)
        ds.edit_logits(x, out=out, **kw)
        assert torch.equal(out, want) and torch.equal(x, e.X)
    wide = torch.arange(12 * 512, device="cuda").view(12, 512).to(BF)
    before = wide.clone()
    flat = wide.view(24, 256)
    for x, out in ((flat[:5, :250], flat[1:6, :250]), (flat[1:6, :250], flat[:5, :250]),
                   (wide[:5, :250], wide[:5, 8:258]), (wide[:5, :250], flat[2:7, :250])):
        with pytest.raises(ds.DSparkError, match="VALUE"):
            ds.edit_logits(x, out=out, **kw)
        with pytest.raises(ds.DSparkError, match="VALUE"):
            ds.edit_logits_backward(x, raw_rows(e.X), out=out, **grad)
        with pytest.raises(ds.DSparkError, match="VALUE"):
            ds.edit_logits_backward(raw_rows(e.X), x, out=out, **grad)
    assert torch.equal(wide, before)
    one = Edits([1], 250, BF, seed=17, longest=40)
    buf[3, :250].copy_(one.X[0])
    ds.edit_logits(buf[3:4, :250], out=buf[4:5, :250], **one.args())
    assert torch.equal(buf[4:5, :250], ds.edit_logits(one.X, **one.args()))
    lens = i32([1, 2, 3, 4])
    with pytest.raises(ds.DSparkError, match="VALUE"):
        ds.history_append(i32([[0] * 8] * 3), lens[:3], i32([[1]] * 3), out=lens[1:])
    assert lens.tolist() == [1, 2, 3, 4]


# ---------------------------------------------------------------- histories
def test_history_append():
    rng = np.random.default_rng(1)
    R, cap, w = 7, 40, 6
    h = rng.integers(0, 100, (R, cap))
    lens = np.array([0, 1, 10, 34, 35, 40, 39])
    y = rng.integers(0, 100, (R, w))
    acc = np.array([5, -1, 0, 5, 5, 0, 0])  # the fifth and sixth do not fit
    ws = ds.Workspace()
    H, L, Y, N = i32(h.tolist()), i32(lens.tolist()), i32(y.tolist()), i32(acc.tolist())
    prompt = i32([3] * R)
    out = ds.history_append(H, L, Y, n_acc=N, prompt_len=prompt, ws=ws)
    assert ws.error_code() == LENGTH
    want_len, want_prompt = lens.copy(), np.full(R, 3)
    for r in range(R):
        n = acc[r] + 1
        if lens[r] + n <= cap and n > 0:
            h[r, lens[r]:lens[r] + n] = y[r, :n]
            want_len[r] += n
            want_prompt[r] = want_len[r]
    assert torch.equal(H.cpu(), torch.from_numpy(h).int()) and out.tolist() == want_len.tolist()
    assert prompt.tolist() == want_prompt.tolist() and L.tolist() == lens.tolist()
    ws.clear_error()
    # all of a width, in place
    L = i32([0] * R)
    assert ds.history_append(H, L, Y, ws=ws, out=L) is L
    assert L.tolist() == [w] * R and torch.equal(H[:, :w], Y)
    # a flat list: prompts, one of them empty
    off = [0, 3, 3, 40, 41, 50, 60, 61]
    flat = rng.integers(0, 100, 61)
    L.zero_()
    ds.history_append(H, L, i32(flat.tolist()), row_offset=i32(off), prompt_len=prompt, ws=ws, out=L)
    assert L.tolist() == np.diff(off).tolist() and ws.error_code() == 0
    for r in range(R):
        assert H[r, :L[r]].tolist() == flat[off[r]:off[r + 1]].tolist()
    assert prompt.tolist() == [off[r + 1] - off[r] if off[r + 1] > off[r] else want_prompt[r] for r in range(R)]


def test_history_append_of_no_tokens():
    """A flat list without a token (no request has a prompt) changes nothing."""
    hist = ds.TokenHistory(3, 10)
    hist.start(i32([7, 8]), i32([0, 0, 2, 2]))
    for _ in range(2):
        hist.start(torch.empty(0, dtype=I32, device="cuda"), i32([0] * 4))
        assert hist.lens.tolist() == [0, 2, 0] and hist.prompt_lens.tolist() == [0, 2, 0]
        assert hist.tokens[1].tolist() == [7, 8] + [-1] * 10 and hist.error_code() == 0
    hist.start(torch.empty(0, dtype=I32, device="cuda"), i32([0, 0, 1, 1]))  # a token that is not there
    assert hist.error_code() == LENGTH and hist.lens.tolist() == [0, 2, 0]


@pytest.mark.parametrize("what", ["n_acc", "length", "offsets", "end", "rows"])
def test_history_append_refuses_bad_data(what):
    """The request that is wrong stays as it is, the others grow."""
    H = torch.full((3, 16), -1, dtype=I32, device="cuda")
    L, Y, N = i32([2, 5, 7]), i32([[1, 2], [3, 4], [5, 6]]), i32([0, 1, 1])
    ws, kw, grown = ds.Workspace(), dict(n_acc=N), [3, 5, 9]
    if what == "n_acc":
        N[1] = 2
    elif what == "length":
        L[1] = 17
        grown[1] = 17
    elif what == "rows":  # the round reserved one row for request 1, two are emitted
        kw["row_offset"] = i32([0, 2, 3, 5])
    else:
        Y = i32([1, 2, 3, 4])
        kw = dict(row_offset=i32([0, 1, 0, 2] if what == "offsets" else [0, 1, 1, 5]))
        grown = [3, 5, 9] if what == "offsets" else [3, 5, 7]
    out = ds.history_append(H, L, Y, ws=ws, **kw)
    assert ws.error_code() == LENGTH and out.tolist() == grown
    assert (H[1] == -1).all()


def test_long_prompts_and_past_32_bit_offsets():
    R, cap = 2200, 1048575  # 9.2 GB
    H = torch.zeros((R, cap), dtype=I32, device="cuda")
    n = 300001
    flat = torch.randint(0, 1000, (n + 5,), dtype=I32, device="cuda")
    off = torch.zeros(R + 1, dtype=I32, device="cuda")
    off[R - 1], off[R] = 5, n + 5
    L = torch.zeros(R, dtype=I32, device="cuda")
    out = ds.history_append(H, L, flat, row_offset=off)
    assert out[-1] == n and out[-2] == 5 and int(out.sum()) == n + 5
    assert torch.equal(H[-1, :n], flat[5:]) and torch.equal(H[-2, :5], flat[:5]) and not H[:-2].any()


def test_token_history_over_replayed_rounds():
    """Prompts, then a captured round of edit and append: each replay edits by what the
    replays before it appended."""
    R, V, w = 3, 1000, 4
    rng = np.random.default_rng(3)
    hist = ds.TokenHistory(R, 64)
    prompts = [rng.integers(0, V, n).tolist() for n in (5, 1, 9)]
    hist.start(i32(sum(prompts, [])), i32([0, 5, 6, 15]))
    X = torch.randn((6, V), device="cuda")
    off = i32([0, 1, 4, 6])
    drafts, y, acc = i32([[0] * 3] * R), i32([[0] * w] * R), i32([0] * R)
    rep, fre = f32([2.0, 1.0, 0.5]), f32([0.5, 0.25, 0.0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hist.edit(X, row_offset=off, drafts=drafts, repetition=rep, frequency=fre)
        hist.append(y, acc)
    e = Edits([1, 3, 2], V, F, longest=64, seed=1)
    e.presence[:] = 0
    e.repetition[:], e.frequency[:] = rep.cpu().numpy(), fre.cpu().numpy()
    e.prompt_len = np.array([5, 1, 9])
    said = [list(p) for p in prompts]
    for i in range(5):
        yy, aa, dd = rng.integers(0, V, (R, w)), rng.integers(0, w, R), rng.integers(0, V, (R, 3))
        y.copy_(i32(yy.tolist())), acc.copy_(i32(aa.tolist())), drafts.copy_(i32(dd.tolist()))
        X.copy_(torch.randn((6, V), device="cuda"))
        e.hist_len = np.array([len(s) for s in said])
        e.history = np.array([s + [0] * (64 - len(s)) for s in said])
        e.drafts = dd
        graph.replay()
        torch.cuda.synchronize()
        e.check(out, X)
        for r in range(R):
            said[r] += yy[r, : aa[r] + 1].tolist()
            assert hist.tokens[r, : hist.lens[r]].tolist() == said[r]
    assert hist.error_code() == 0 and hist.prompt_lens.tolist() == [5, 1, 9]
