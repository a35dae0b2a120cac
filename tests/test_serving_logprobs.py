"""GPU tests of logprobs and logprobs_backward against torch in 64 bits.

Tolerances (u = 2^-24, the half step of fp32).  Forward: a log probability is
(x - max) / T - log S, each step rounded once, so its first part carries 2 u of
itself.  S is a sum of 2^w with w = (x - max) log2(e) / T rounded three times
(the factor, the difference, the product), so a term is off by
3 u |w| ln 2 + 2 u (the exponential's own ulp), and the |w| 2^w of a row with V
entries averages at most log2 V <= 18: 40 u; adding up to 64 terms a lane, 64
lanes, 4 waves and 256 chunks costs less than (64 + 6 + 3 + 9) u.  In all log S
is within 128 u, the entropy (whose sum has one more product a term and is at
most log V <= 13) within 13 * 160 u.  Backward: p inherits 3 u |d| log2(e) from
the exponent d, and the factor's terms as many roundings; the sum of the
incoming gradients of up to 64 alternatives 7 u.  bf16 results add half a step,
2^-8 of the value.
"""
import math

import pytest
import torch

import draft_sampling_verification_03_amd as ds

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32
TOKEN, LENGTH, NONFINITE = 1, 4, 8


def make(n, V, dt, seed, spread=2.0, stride=None, masked=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = 8 if dt == BF else 4
    stride = stride or -(-V // per) * per
    X = (spread * torch.randn((n, stride), generator=g, device="cuda")).to(dt)
    if masked:
        keep = torch.rand((n, stride), generator=g, device="cuda") >= masked
        keep[:, 0] = True
        X.masked_fill_(~keep, float("-inf"))
    return X[:, :V], g


def expect(X, tok, k, T):
    """logp, entropy, m, S, ids, top_logp in 64 bits (tokens -1: 0)."""
    z = X.double() / T
    lp = torch.log_softmax(z, 1)
    p = lp.exp()
    ent = -torch.special.xlogy(p, p).sum(1)
    got = torch.where(tok >= 0, lp.gather(1, tok.clamp(min=0).long()[:, None])[:, 0], 0.0)
    ids = torch.sort(X.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :k]
    return got, ent, z.amax(1), (z - z.amax(1, keepdim=True)).exp().sum(1), ids, lp.gather(1, ids)


def close(a, b, tol):
    a, b = a.double(), b.double()
    same = (a == b) | ((a - b).abs() <= tol)
    assert same.all(), ((a - b).abs() / tol)[~same].max().item()


def check(X, tok, k, T, out):
    logp, ent, m, S, ids, tlp = expect(X, tok, k, T)
    close(out["logp"], logp, U * (128 + 3 * logp.abs()))
    close(out["entropy"], ent, U * 13 * 160)
    close(out["stats"][:, 0], m, 2 * U * m.abs() + 1e-30)
    close(out["stats"][:, 1], S, S * U * (128 + 2 * m.abs()))
    if k:
        assert torch.equal(out["top_ids"].long(), ids)
        # the result is fp32, which ends at 3.4028e38: lowest / 0.9 = -3.78e38 is -infinity there
        tlp = tlp.float().double()
        close(out["top_logp"], tlp, U * (128 + 3 * tlp.abs().clamp(max=3.5e38)))


@pytest.mark.parametrize("n,V,dt,k,T", [
    (1, 1, F, 1, 1.0), (1, 1, BF, 0, 1.0), (3, 2, F, 2, 0.7), (2, 7, BF, 7, 1.0), (5, 63, F, 20, 1.3),
    (4, 255, BF, 64, 1.0), (3, 1025, F, 64, 0.6), (2, 2049, BF, 5, 2.5), (7, 16384, BF, 20, 1.0),
    (1, 151936, BF, 5, 1.0), (1, 151936, F, 64, 1.0), (3, 129277, F, 8, 0.7), (9, 262143, BF, 20, 1.0),
    (200, 50001, BF, 20, 1.0), (1100, 4097, F, 3, 1.0), (3000, 129, BF, 64, 1.0)])
def test_values(n, V, dt, k, T):
    X, g = make(n, V, dt, 7 * n + V)
    tok = torch.randint(-1, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    ws = ds.Workspace()
    out = ds.logprobs(X, tok, k=k, temp=T, ws=ws)
    assert ws.error_code() == 0
    check(X, tok, k, T, out)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("kind", ["equal", "two values", "ascending", "descending", "one wave", "zeros"])
def test_ties_and_uneven_rows(kind, dt):
    """Rows on which a threshold picks far more than k elements, or all of them
    in one chunk or one wave; +0 and -0 are equal."""
    n, V, k = 3, 40007, 20
    X, g = make(n, V, dt, 5)
    i = torch.arange(V, device="cuda").expand(n, V)
    if kind == "equal":
        X.fill_(1.5)
    elif kind == "two values":
        X.copy_((i % 3 == 0).to(dt))
    elif kind == "ascending":
        X.copy_((i / V * 9).to(dt))
    elif kind == "descending":
        X.copy_((9 - i / V * 9).to(dt))
    elif kind == "one wave":
        X.copy_(torch.where((i // 512) % 4 == 2, X.float() + 20, X.float()).to(dt))
    else:
        X.copy_(torch.where(i % 2 == 0, -0.0, 0.0).to(dt))
    tok = torch.tensor([0, V - 1, 77], dtype=torch.int32, device="cuda")
    check(X, tok, k, 1.0, ds.logprobs(X, tok, k=k))


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("V", [257, 400, 1021, 1500, 4097, 9001])
@pytest.mark.parametrize("levels", [1, 2, 3, 9, 70, 0])
def test_small_vocabularies_with_ties(levels, V, dt):
    """Fewer 128-byte lines than alternatives, so all elements reach the first
    threshold; values from few levels, so that many share the one at the end."""
    X, g = make(5, V, dt, 3)
    if levels:
        X.copy_((torch.randint(0, levels, (5, V), generator=g, device="cuda") * 0.25).to(dt))
        X[3, : V // 2] = float("-inf")
        X[4, 200] = 7.0  # one element above all the others
    tok = torch.randint(-1, V, (5,), generator=g, device="cuda", dtype=torch.int32)
    tok[3] = V - 1
    for k in (1, 20, 64):
        check(X, tok, k, 1.0, ds.logprobs(X, tok, k=k))


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("whole,k", [(True, 1), (True, 64), (False, 4), (False, 20)])
def test_many_rows_whose_maxima_tie(whole, k, dt):
    """The first threshold is the maximum already, so no value is counted between the
    reading of a counter and its clearing: whole rows of one value (more lines than are
    read again share it), and every third 128 bytes (fewer lines, but more elements
    than are ranked)."""
    n, V = 1500, 20480 // dt.itemsize * 2
    X, g = make(n, V, dt, 21)
    X.clamp_(max=2.5)
    if whole:
        X.fill_(3.0)
    else:
        X.view(n, -1, 128 // dt.itemsize)[:, ::3] = 3.0
    tok = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    for _ in range(3):
        ws = ds.Workspace()
        out = ds.logprobs(X, tok, k=k, ws=ws)
        assert ws.error_code() == 0
        check(X, tok, k, 1.0, out)


@pytest.mark.parametrize("n,V,dt,k,masked", [(6, 30001, BF, 20, 0.98), (6, 5000, F, 64, 0.999),
                                             (64, 129277, F, 8, 0.5), (3, 70, BF, 64, 0.9)])
def test_masked(n, V, dt, k, masked):
    """Masked logits have probability 0 and follow the others by index; the
    type's lowest value is not a mask."""
    X, g = make(n, V, dt, 11, masked=masked)
    X[0, V // 2:] = torch.finfo(dt).min
    X[1, 1:] = float("-inf")  # one unmasked entry: probability 1
    tok = torch.zeros(n, dtype=torch.int32, device="cuda")
    tok[2] = V - 1
    ws = ds.Workspace()
    out = ds.logprobs(X, tok, k=k, temp=0.9, ws=ws)
    assert ws.error_code() == 0
    check(X, tok, k, 0.9, out)
    assert out["logp"][1] == 0 and out["entropy"][1] == 0


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("end", [1, -1])
def test_rows_at_the_end_of_the_range(dt, end):
    """Rows of the type's lowest (or largest) value alone: every entry alike; and
    with one entry a step of the type apart, far enough to be 0 or 1."""
    V = 5003
    X, _ = make(2, V, dt, 1)
    X.fill_(end * torch.finfo(dt).max)
    X[1, 77] = end * torch.finfo(dt).max * (1 - torch.finfo(dt).eps)
    tok = torch.tensor([5, 77], dtype=torch.int32, device="cuda")
    ws = ds.Workspace()
    out = ds.logprobs(X, tok, k=3, ws=ws)
    assert ws.error_code() == 0
    check(X, tok, 3, 1.0, out)


def test_rows_without_a_distribution_and_bad_tokens():
    X, _ = make(6, 9000, BF, 3)
    X[1] = float("-inf")
    X[2, 8999] = float("nan")
    X[3, 17] = float("inf")
    X[4] = float("-inf")
    X[4, 5000] = float("nan")  # alone in an otherwise masked chunk
    tok = torch.tensor([9000, 0, 0, 0, 0, -2], dtype=torch.int32, device="cuda")
    ws = ds.Workspace()
    out = ds.logprobs(X, tok, k=4, ws=ws)
    assert ws.error_code() == TOKEN | NONFINITE
    assert out["logp"].isnan().all()
    ok = torch.tensor([True, False, False, False, False, True], device="cuda")
    for name in ("entropy", "stats", "top_logp"):
        assert torch.equal(out[name].reshape(6, -1).isnan().any(1), ~ok), name
    assert torch.equal((out["top_ids"] == -1).all(1), ~ok)
    ws.clear_error()
    # gradients: a row without statistics gives zeros, a bad token counts for nothing
    g = torch.ones(6, device="cuda")
    dx = ds.logprobs_backward(X, out["stats"], out["entropy"], tokens=tok, g_logp=g, g_entropy=g, ws=ws)
    assert ws.error_code() == TOKEN | NONFINITE
    assert (dx[1:5] == 0).all()
    want, _ = gradient(X[:1], None, None, g[:1], None, None, 1.0)
    close(dx[0], want[0], 2.0 ** -8 * want[0].abs() + 1e-6)


def ragged(seed, R=9, gamma=4):
    g = torch.Generator().manual_seed(seed)
    rows = 1 + torch.randint(0, gamma + 1, (R,), generator=g)
    off = torch.cat([torch.zeros(1, dtype=torch.long), rows.cumsum(0)]).int()
    return off.cuda(), int(off[-1])


def flat_tokens(y, off, n):
    tok = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    for r in range(off.numel() - 1):
        m = min(int(off[r + 1] - off[r]), y.shape[1])
        tok[off[r]:off[r] + m] = y[r, :m]
    return tok


@pytest.mark.parametrize("dt,V,R", [(BF, 3001, 9), (F, 1000, 9), (F, 40, 150)])
def test_verified_batch_layout(dt, V, R):
    """Tokens by request, -1 behind the last; rows behind the last request are
    neither read (NaN there raises nothing) nor written."""
    off, used = ragged(1, R)
    X, g = make(used + 3, V, dt, 2)
    X[used:] = float("nan")
    y = torch.randint(-1, V, (R, 5), generator=g, device="cuda", dtype=torch.int32)
    out = dict(logp=torch.full((used + 3,), 7.0, device="cuda"),
               entropy=torch.full((used + 3,), 7.0, device="cuda"),
               stats=torch.full((used + 3, 2), 7.0, device="cuda"),
               top_ids=torch.full((used + 3, 6), 7, dtype=torch.int32, device="cuda"),
               top_logp=torch.full((used + 3, 6), 7.0, device="cuda"))
    ws = ds.Workspace()
    ds.logprobs(X, y, k=6, row_offset=off, ws=ws, out=out)
    assert ws.error_code() == 0
    for t in out.values():
        assert (t[used:] == 7).all()
    check(X[:used], flat_tokens(y, off, used), 6, 1.0, {k: v[:used] for k, v in out.items()})
    # narrower tokens than rows: the rest has none; an end past the rows is cut
    off[-1] = used + 4
    out = ds.logprobs(X, y[:, :2].contiguous(), row_offset=off, ws=ws)
    assert ws.error_code() == LENGTH | NONFINITE
    close(out["logp"][:used], expect(X[:used], flat_tokens(y[:, :2], off.clamp(max=used), used), 1, 1.0)[0],
          U * 300)


def gradient(X, tok, gl, gh, ids, gt, T):
    """The formula in 64 bits, and the size of what is added up in it."""
    p = torch.softmax(X.double() / T, 1)
    lp = torch.where(p > 0, p, 1.0).log()
    H = -(p * lp).sum(1, keepdim=True)
    n = X.shape[0]
    G = torch.zeros(n, 1, dtype=torch.float64, device="cuda")
    own, size = torch.zeros_like(p), torch.zeros_like(p)
    if gl is not None:
        g = torch.where(tok >= 0, gl.double(), 0.0)[:, None]
        own.scatter_add_(1, tok.clamp(min=0).long()[:, None], g)
        G = G + g
    if gt is not None:
        own.scatter_add_(1, ids.long(), gt.double())
        G = G + gt.double().sum(1, keepdim=True)
    ge = 0.0 if gh is None else gh.double()[:, None]
    many = (0 if gt is None else gt.double().abs().sum(1, keepdim=True)) + (
        0 if gl is None else gl.double().abs()[:, None])
    size = p * (many + abs(ge) * (lp.abs() + H)) * (3 * 1.45 * lp.abs() + 40) + own.abs() * 8
    return (own - p * (G + ge * (lp + H))) / T, size / T


@pytest.mark.parametrize("n,V,dt,k,T,masked", [
    (1, 1, F, 0, 1.0, 0), (2, 7, BF, 7, 0.7, 0), (5, 300, F, 20, 1.3, 0.5), (33, 129277, F, 10, 1.3, 0.9),
    (3, 151936, BF, 64, 1.0, 0), (130, 16384, BF, 3, 0.6, 0), (2000, 1031, F, 2, 1.0, 0),
    (2, 262141, BF, 0, 1.0, 0)])
def test_gradient(n, V, dt, k, T, masked):
    X, g = make(n, V, dt, n + V, masked=masked)
    tok = torch.randint(-1, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    f = ds.logprobs(X, tok, k=k, temp=T)
    if k:  # the token among the alternatives, and the same alternative twice
        tok[0] = f["top_ids"][0, 0]
        if k > 1:
            f["top_ids"][0, 1] = f["top_ids"][0, 0]
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    gl, gh, gt = r(n), r(n), r(n, k) if k else None
    dx = ds.logprobs_backward(X, f["stats"], f["entropy"], tokens=tok, g_logp=gl, g_entropy=gh,
                              top_ids=f["top_ids"] if k else None, g_top=gt, temp=T)
    want, size = gradient(X, tok, gl, gh, f["top_ids"], gt, T)
    tol = 160 * U * size / 8 + 1e-30 + (2.0 ** -8 * want.abs() if dt == BF else 0)
    # a chunk's statistics carry 128 u, which every probability inherits
    close(dx, want, tol + 160 * U * (want.abs() + size / 40))


def test_gradient_parts_alone_and_in_place():
    n, V = 12, 2051
    X, g = make(n, V, F, 4)
    tok = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    f = ds.logprobs(X, tok, k=3)
    gl = torch.randn(n, generator=g, device="cuda")
    gt = torch.randn((n, 3), generator=g, device="cuda")
    for kw, args in (((dict(tokens=tok, g_logp=gl)), (tok, gl, None, None, None)),
                     (dict(g_entropy=gl), (None, None, gl, None, None)),
                     (dict(top_ids=f["top_ids"], g_top=gt), (None, None, None, f["top_ids"], gt))):
        dx = ds.logprobs_backward(X, f["stats"], f["entropy"], **kw)
        want, size = gradient(X, *args, 1.0)
        close(dx, want, U * (200 * want.abs() + 25 * size) + 1e-30)
    wide = X.as_strided((n, X.stride(0)), (X.stride(0), 1)).clone()
    wide[:, V:] = 5.0
    dx = ds.logprobs_backward(wide[:, :V], f["stats"], f["entropy"], tokens=tok, g_logp=gl,
                              out=wide[:, :V])
    want, size = gradient(X, tok, gl, None, None, None, 1.0)
    close(wide[:, :V], want, U * (200 * want.abs() + 25 * size) + 1e-30)
    assert (wide[:, V:] == 5.0).all() and dx.data_ptr() == wide.data_ptr()


@pytest.mark.parametrize("size", [1e4, -1e6, 3e7])
def test_stats_and_gradient_of_large_logits(size):
    """m = max / T is rounded to a 24th of its bits, which is far from small here; S
    belongs to the rounded m.  A term of S is off by 3 u |d| (d its exponent, |d| e^d
    <= 0.37) and two ulps, the sum by (V / 256 + 16) u, the factor e^off by two:
    within 80 u.  p = e^d / S adds as much for its own term, so 170 u of p / T."""
    V, T = 1000, 0.7
    X, g = make(4, V, F, 12)
    X.mul_(abs(size) * 2.0 ** -22).add_(size)
    tok = torch.tensor([0, 5, V - 1, 77], dtype=torch.int32, device="cuda")
    out = ds.logprobs(X, tok, temp=T)
    z = X.double() / torch.tensor(T, device="cuda").double()
    m, S = out["stats"][:, 0].double(), out["stats"][:, 1].double()
    want = (z - m[:, None]).exp().sum(1)
    close(S, want, 80 * U * want)
    one = torch.ones(4, device="cuda")
    dx = ds.logprobs_backward(X, out["stats"], None, tokens=tok, g_logp=one, temp=T)
    p = z.softmax(1)
    exact = -p
    exact[torch.arange(4), tok.long()] += 1
    close(dx, exact / T, 170 * U * (p + 0.02) / T)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("V", [700, 5003])
@pytest.mark.parametrize("end", [1, -1])
def test_gradient_of_rows_at_the_end_of_the_range(end, V, dt):
    """Rows of the type's lowest (or largest) value, as a finite mask leaves them: every
    entry alike; one entry a step of the type above or below the others; half of them
    masked by -infinity; a large but ordinary floor.  Whole numbers of x - m, so the
    probabilities are 1 / count or 0.  With incoming gradients, without, and in place."""
    X, g = make(6, V, dt, 1)
    top = end * torch.finfo(dt).max
    X[:4] = top
    X[1, 77] = top * (1 - torch.finfo(dt).eps)
    X[2, 1::2] = float("-inf")
    X[3] = -1e31
    tok = torch.tensor([5, 77, 6, 3, -1, 4], dtype=torch.int32, device="cuda")
    ws = ds.Workspace()
    f = ds.logprobs(X, tok, k=3, ws=ws)
    gl, gh, gt = (torch.randn(s, generator=g, device="cuda") for s in ((6,), (6,), (6, 3)))
    kw = dict(tokens=tok, top_ids=f["top_ids"], ws=ws)
    dx = ds.logprobs_backward(X, f["stats"], f["entropy"], g_logp=gl, g_entropy=gh, g_top=gt, **kw)
    want, size = gradient(X, tok, gl, gh, f["top_ids"], gt, 1.0)
    close(dx, want, 20 * U * size + 160 * U * (want.abs() + size / 40) + 1e-30
          + (2.0 ** -8 * want.abs() if dt == BF else 0))
    none = ds.logprobs_backward(X, f["stats"], f["entropy"], g_logp=0 * gl, g_entropy=0 * gh,
                                g_top=0 * gt, **kw)
    assert (none == 0).all()
    # a temperature may take m out of range: such a row counts as one without statistics
    for T in (0.7, 1.3):
        h = ds.logprobs(X, tok, k=3, temp=T, ws=ds.Workspace())
        assert ds.logprobs_backward(X, h["stats"], h["entropy"], tokens=tok, g_logp=gl, g_entropy=gh,
                                    temp=T, ws=ds.Workspace()).isfinite().all()
    wide = X.as_strided((6, X.stride(0)), (X.stride(0), 1)).clone()
    ds.logprobs_backward(wide[:, :V], f["stats"], f["entropy"], g_logp=gl, g_entropy=gh, g_top=gt,
                         out=wide[:, :V], **kw)
    assert torch.equal(wide[:, :V], dx) and ws.error_code() == 0


def test_gradient_against_differences():
    """Central differences of the forward formula in 64 bits, along random directions."""
    n, V, T = 4, 500, 0.8
    X, g = make(n, V, F, 9)
    tok = torch.tensor([3, 499, -1, 0], dtype=torch.int32, device="cuda")
    f = ds.logprobs(X, tok, k=4, temp=T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    gl, gh, gt = r(n), r(n), r(n, 4)
    dx = ds.logprobs_backward(X, f["stats"], f["entropy"], tokens=tok, g_logp=gl, g_entropy=gh,
                              top_ids=f["top_ids"], g_top=gt, temp=T).double()

    def loss(x):
        lp = torch.log_softmax(x / T, 1)
        t = torch.where(tok >= 0, lp.gather(1, tok.clamp(min=0).long()[:, None])[:, 0], 0.0)
        return ((gl * t).sum() - (gh * (lp.exp() * lp).sum(1)).sum()
                + (gt * lp.gather(1, f["top_ids"].long())).sum())

    for _ in range(5):
        d = torch.randn((n, V), generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        num = (loss(X.double() + h * d) - loss(X.double() - h * d)) / (2 * h)
        # the difference's own error is below 1e-8; the gradient's 300 u of |dx| |d|
        assert abs(num - (dx * d).sum()) <= 1e-7 + 300 * U * (dx.abs() * d.abs()).sum()


def test_gradient_of_the_verified_batch_layout():
    off, used = ragged(4)
    X, g = make(used + 2, 777, F, 6)
    X[used:] = float("nan")
    y = torch.randint(-1, 777, (9, 5), generator=g, device="cuda", dtype=torch.int32)
    ws = ds.Workspace()
    f = ds.logprobs(X, y, row_offset=off, ws=ws)
    gl = torch.randn(used + 2, generator=g, device="cuda")
    out = torch.full((used + 2, 780), 3.0, device="cuda")
    ds.logprobs_backward(X, f["stats"], tokens=y, g_logp=gl, row_offset=off, ws=ws, out=out[:, :777])
    assert ws.error_code() == 0
    want, size = gradient(X[:used], flat_tokens(y, off, used), gl[:used], None, None, None, 1.0)
    close(out[:used, :777], want, U * (200 * want.abs() + 25 * size) + 1e-30)
    assert (out[used:] == 3.0).all() and (out[:, 777:] == 3.0).all()


def test_streams_and_captured_replays():
    """A forward and backward on another stream, then captured twice over one
    workspace and replayed with other inputs and eager work in between."""
    n, V, k = 6, 20000, 5
    X, g = make(n, V, BF, 1)
    tok = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    gl = torch.randn(n, generator=g, device="cuda")
    ws = ds.Workspace()

    def both(stream=None):
        f = ds.logprobs(X, tok, k=k, ws=ws, stream=stream)
        return f, ds.logprobs_backward(X, f["stats"], f["entropy"], tokens=tok, g_logp=gl, ws=ws,
                                       stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f, dx = both(side)
    side.synchronize()
    check(X, tok, k, 1.0, f)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        f1, d1 = both()
    with torch.cuda.graph(g2):
        f2, d2 = both()
    for i in range(4):
        X.copy_((2.0 * torch.randn((n, V), generator=g, device="cuda")).to(BF))
        torch.cuda.synchronize()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        f, dx = both()
        for a in (f1, f2):
            for name in f:
                assert torch.equal(a[name], f[name]), (i, name)
        assert torch.equal(d1, dx) and torch.equal(d2, dx)


def test_same_bits_every_time():
    X, g = make(40, 151936, BF, 8)
    tok = torch.randint(0, 151936, (40,), generator=g, device="cuda", dtype=torch.int32)
    a, b = ds.logprobs(X, tok, k=64), ds.logprobs(X, tok, k=64)
    for name in a:
        assert torch.equal(a[name], b[name])
    assert math.isfinite(float(a["logp"].sum()))


@pytest.mark.parametrize("dt", [BF, F])
def test_more_requests_than_rows_in_use(dt):
    """Requests without rows, three of eight with some: the buffer has eight rows."""
    off = torch.tensor([0, 0, 2, 2, 3, 3, 3, 5, 5], dtype=torch.int32, device="cuda")
    X, g = make(8, 501, dt, 2)
    X[5:] = float("nan")
    y = torch.randint(0, 501, (8, 3), generator=g, device="cuda", dtype=torch.int32)
    ws = ds.Workspace()
    f = ds.logprobs(X, y, k=2, row_offset=off, ws=ws)
    tok = flat_tokens(y, off, 5)
    check(X[:5], tok, 2, 1.0, {k: v[:5] for k, v in f.items()})
    gl = torch.randn(8, generator=g, device="cuda")
    dx = ds.logprobs_backward(X, f["stats"], tokens=y, g_logp=gl, row_offset=off, ws=ws)
    want, size = gradient(X[:5], tok, gl[:5], None, None, None, 1.0)
    close(dx[:5], want, U * (200 * want.abs() + 25 * size) + 1e-30
          + (2.0 ** -8 * want.abs() if dt == BF else 0))
    assert ws.error_code() == 0
