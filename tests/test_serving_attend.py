"""GPU tests of cache_attend against attention in 64 bits, request by request.

Tolerances (u = 2^-24): a score is a D-term fp32 sum of exact products (bf16) or
of products rounded once (fp32), scaled and reduced in the exponent: off by at
most (D + 4) u of s = scale sum |q||k|, and a probability by that much of
itself; the exponential's ulp, up to L terms of the running sums and 8 joins add
(L + 16) u; bf16 probabilities enter as two bf16 values, 2^-17 of each left.  So
|out - o| <= e sum p |v| with e = 2 (D + 4) u s + (2 L + 64) u (+ 2^-16 in bf16:
the numerator's, the sum is not rounded), and a bf16 result half a step more,
2^-8 of the value.  lse: (D + 4) u s + (L + 32) u + 2 u |lse|.
"""
import pytest
import torch

import draft_sampling_verification_03_amd as ds

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
U = 2.0 ** -24
LENGTH, PAGE = 4, 32


class Case:
    """Requests over scattered pages; every slot that no request holds is NaN."""

    def __init__(self, rows, lens, Hq, Hkv, D, page, dt, seed=0, layers=1, spare=2, append=True,
                 packed=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
        self.rows, self.lens, self.page, self.dt = rows, lens, page, dt
        R = len(rows)
        pages = [-(-n // page) for n in lens]
        self.n_pages = sum(pages) + spare
        width = max(pages + [1]) + 1
        ids = torch.randperm(self.n_pages, generator=torch.Generator().manual_seed(seed)).int()
        table = torch.full((R, width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(pages):
            table[i, :n] = ids[at:at + n]
            at += n
        self.table = table.cuda()
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        off = [0]
        for n in rows:
            off.append(off[-1] + n)
        self.off, self.n = off, off[-1]
        self.row_offset = torch.tensor(off, dtype=torch.int32, device="cuda")
        nan = float("nan")
        self.k_all = torch.full((self.n_pages, layers, Hkv, page, D), nan, dtype=dt, device="cuda")
        self.v_all = torch.full((self.n_pages, layers, Hkv, D, page), nan, dtype=dt, device="cuda")
        self.k, self.v = self.k_all[:, layers - 1], self.v_all[:, layers - 1]
        if packed:  # one projection's output: queries, keys and values of a row side by side
            qkv = r(self.n, Hq + 2 * Hkv, D)
            self.q, self.kn, self.vn = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            self.q, self.kn, self.vn = r(self.n, Hq, D), r(self.n, Hkv, D), r(self.n, Hkv, D)
        self.K, self.V = [r(n, Hkv, D) for n in lens], [r(n, Hkv, D) for n in lens]
        for i, (n, new) in enumerate(zip(lens, rows)):
            had = max(0, n - new)
            if append:
                if n >= new:
                    self.K[i][had:], self.V[i][had:] = self.kn[off[i]:off[i + 1]], self.vn[off[i]:off[i + 1]]
            else:
                had = n
            self.fill(i, had)
        self.append = append

    def fill(self, i, n):
        """The first n tokens of request i into its pages."""
        for t in range(0, n, self.page):
            m, p = min(self.page, n - t), int(self.table[i, t // self.page])
            self.k[p, :, :m] = self.K[i][t:t + m].transpose(0, 1)
            self.v[p, :, :, :m] = self.V[i][t:t + m].permute(1, 2, 0)

    def run(self, ws=None, **kw):
        if self.append:
            kw = dict(k_new=self.kn, v_new=self.vn, **kw)
        return ds.cache_attend(self.q, self.k, self.v, self.table, self.kv_len,
                               row_offset=self.row_offset, ws=ws, **kw)

    def check(self, o, scale=None, window=0):
        D = self.q.shape[2]
        group = self.q.shape[1] // self.k.shape[1]
        scale = D ** -0.5 if scale is None else scale
        for i, (n, L) in enumerate(zip(self.rows, self.lens)):
            K = self.K[i].double().repeat_interleave(group, 1).transpose(0, 1)
            V = self.V[i].double().repeat_interleave(group, 1).transpose(0, 1)
            for j in range(n):
                row = self.off[i] + j
                b = L - n + 1 + j
                a = max(0, b - window) if window else 0
                if b <= a:
                    assert (o["out"][row] == 0).all() and (o["lse"][row] == float("-inf")).all()
                    continue
                q = self.q[row].double()
                s = scale * (K[:, a:b] @ q[:, :, None])[..., 0]
                size = (scale * (K[:, a:b].abs() @ q.abs()[:, :, None])[..., 0]).amax(1)
                p = torch.softmax(s, 1)
                want = (p[:, None] @ V[:, a:b])[:, 0]
                e = 2 * (D + 4) * U * size + (2 * (b - a) + 64) * U + (2.0 ** -16 if self.dt == BF else 0)
                tol = e[:, None] * (p[:, None] @ V[:, a:b].abs())[:, 0]
                if self.dt == BF:
                    tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
                err = (o["out"][row].double() - want).abs()
                assert (err <= tol).all(), (i, j, (err / tol).max().item())
                lse = torch.logsumexp(s, 1)
                assert ((o["lse"][row].double() - lse).abs()
                        <= (D + 4) * U * size + (b - a + 32) * U + 2 * U * lse.abs()).all(), (i, j)


def pools_equal(c):
    """Every token's key and value lies in its slot."""
    for i, L in enumerate(c.lens):
        for t in range(L):
            p, s = int(c.table[i, t // c.page]), t % c.page
            assert torch.equal(c.k[p, :, s], c.K[i][t]) and torch.equal(c.v[p, :, :, s], c.V[i][t])


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("rows,lens,Hq,Hkv,D,page", [
    ([1], [1], 1, 1, 64, 16),
    ([1], [17], 8, 2, 128, 16),
    ([1, 1, 1], [31, 32, 33], 4, 4, 64, 32),
    ([3, 1, 5], [3, 100, 129], 6, 2, 96, 16),
    ([1, 9, 17, 2], [700, 9, 300, 16], 8, 1, 128, 16),
    ([17, 4], [1000, 2049], 32, 8, 128, 64),
    ([2, 1], [130, 515], 7, 1, 256, 32),
    ([5, 1, 8], [5, 640, 250], 12, 4, 256, 128),
    ([40], [170], 4, 2, 64, 256),
    ([6, 0, 3], [50, 70, 3], 16, 2, 96, 16),
])
def test_values(rows, lens, Hq, Hkv, D, page, dt):
    c = Case(rows, lens, Hq, Hkv, D, page, dt, seed=sum(lens))
    ws = ds.Workspace()
    o = c.run(ws)
    assert ws.error_code() == 0
    c.check(o)
    pools_equal(c)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("rows,lens,Hq,Hkv,page,window", [
    ([17, 4, 70], [300, 37, 70], 8, 2, 16, 0),
    ([17, 4, 70], [300, 37, 1500], 4, 1, 128, 0),
    ([20, 9, 65], [1111, 9, 431], 6, 2, 32, 0),
    ([17, 4, 70], [600, 999, 70], 4, 1, 16, 45),
    ([33, 0, 12], [2500, 5, 47], 16, 4, 256, 700),
])
def test_heads_of_256_in_blocks_of_64_rows(rows, lens, Hq, Hkv, page, window, dt):
    """One step a buffer: odd and even numbers of steps, pages of one and of several
    pieces of 64 bytes, units cut between workgroups, a window that ends inside a step;
    unseen slots are NaN (Case), and so is a new row's key and value afterwards."""
    c = Case(rows, lens, Hq, Hkv, 256, page, dt, seed=sum(rows) + page)
    ws = ds.Workspace()
    good = c.run(ws, window=window)
    assert ws.error_code() == 0
    c.check(good, window=window)
    pools_equal(c)
    c.kn[5], c.vn[5] = float("nan"), float("inf")
    o = c.run(ws, window=window)
    keep = torch.ones(c.n, dtype=torch.bool, device="cuda")
    keep[5:rows[0]] = False
    assert torch.equal(o["out"][keep], good["out"][keep]) and not o["out"][5].isfinite().any()


@pytest.mark.parametrize("dt,window", [(BF, 1), (BF, 40), (F, 7), (F, 200), (BF, 5000), (F, 2 ** 31 - 1)])
def test_window(dt, window):
    c = Case([1, 17, 6], [500, 300, 33], 8, 2, 64, 16, dt, seed=window)
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("dt,rows,L", [(BF, 1, 40000), (F, 3, 20000), (BF, 17, 9000)])
def test_long_context_is_split_and_joined(dt, rows, L):
    c = Case([rows, 1], [L, 5], 4, 2, 64, 64, dt, seed=1)
    c.check(c.run())


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("Hq,Hkv,window,page", [(4, 1, 0, 16), (6, 2, 0, 64), (7, 1, 50, 32), (8, 8, 333, 128)])
def test_prompts(Hq, Hkv, window, page, dt):
    """Many new rows a request: blocks that see the tokens to the end and blocks that
    see a few, in odd and even number, cut and whole."""
    c = Case([300, 1, 131, 70, 9], [300, 40, 400, 1200, 9], Hq, Hkv, 64, page, dt, seed=window)
    ws = ds.Workspace()
    o = c.run(ws, window=window)
    assert ws.error_code() == 0
    c.check(o, window=window)
    pools_equal(c)


@pytest.mark.parametrize("rows", [1, 20])
def test_more_pages_than_a_workgroup_holds_at_once(rows):
    """64 key-value heads leave 8 shares a head, each of more than 1024 pages of 16."""
    c = Case([rows], [141000], 64, 64, 64, 16, BF, seed=8)
    c.check(c.run())


def test_many_short_requests_in_a_share():
    """Stretches of a few tokens one after another, empty ones and whole ones among
    them, more than one block of rows, a bad page in one of them."""
    g = torch.Generator().manual_seed(2)
    rows = torch.randint(0, 40, (300,), generator=g).tolist()
    lens = [max(n, int(x)) if i % 7 else n // 2 for i, (n, x) in
            enumerate(zip(rows, torch.randint(0, 260, (300,), generator=g)))]
    for dt, D in ((BF, 128), (F, 96)):
        c = Case(rows, lens, 8, 2, D, 16, dt, seed=9, append=False)
        c.check(c.run())
        full = [i for i, n in enumerate(lens) if n > 40 and rows[i]]
        before = c.run()
        c.table[full[3], 1] = -5
        ws = ds.Workspace()
        after = c.run(ws)
        assert ws.error_code() == PAGE
        keep = torch.ones(c.n, dtype=torch.bool, device="cuda")
        keep[c.off[full[3]]:c.off[full[3] + 1]] = False
        assert torch.equal(after["out"][keep], before["out"][keep])
        assert torch.isfinite(after["out"].float()).all()


def test_steep_scores_and_scale():
    """Scores of several hundred, rising along the context (the running maximum
    moves in almost every step) or falling."""
    for sign in (1, -1):
        c = Case([2], [900], 4, 4, 64, 16, F, seed=3)
        ramp = torch.linspace(0, 9, 898, device="cuda")[:, None, None] * sign
        c.K[0][:898] = (c.q[0].float()[None] * ramp + c.K[0][:898].float()).to(F)
        c.fill(0, 898)
        c.check(c.run(scale=0.4), scale=0.4)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("L", [128, 9000])
@pytest.mark.parametrize("power,sign", [(40, 1), (40, -1), (113, 1), (113, -1)])
def test_scores_of_any_size(power, sign, L, rows, dt):
    """Scores sign m 2^power, m = t / L rounded down to 127 levels, and token L / 2 the
    largest: all exact in fp32, and so far apart that the row is that token's value."""
    c = Case([rows], [L], 4, 2, 64, 32, dt, append=False)
    level = torch.arange(L, device="cuda") * 126 // L
    level[L // 2] = 127
    if sign < 0:
        level = 128 - level
    half = 2.0 ** (power // 2)
    c.q.zero_()
    c.q[..., 5] = half
    c.K[0].zero_()
    c.K[0][:, :, 5] = (sign * level[:, None] * (2.0 ** power / half)).to(dt)
    c.fill(0, L)
    ws = ds.Workspace()
    o = c.run(ws, scale=1.0)
    out, lse = o["out"], o["lse"]
    assert ws.error_code() == 0
    want = c.V[0][L // 2].repeat_interleave(2, 0)
    assert torch.equal(out, want.expand(rows, 4, 64))
    top = sign * float(level[L // 2]) * 2.0 ** power
    assert torch.equal(lse, torch.full_like(lse, top))


def test_rows_that_see_nothing():
    """kv_len 0, and rows before token 0; nothing is appended before it."""
    c = Case([1, 3, 2], [0, 2, 40], 4, 2, 64, 16, BF, append=False)
    ws = ds.Workspace()
    o = c.run(ws)
    assert ws.error_code() == 0
    c.check(o)
    ds.cache_attend(c.q, c.k, c.v, c.table, c.kv_len, row_offset=c.row_offset, k_new=c.kn,
                    v_new=c.vn, ws=ws)
    assert ws.error_code() == LENGTH


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_a_row_does_not_see_never_reaches_it(dt, bad):
    """A later row's key and value are not finite: the rows before it keep their
    finite results, the row itself does not."""
    c = Case([4, 2], [70, 64], 4, 2, 64, 16, dt, seed=2)
    clean = c.run()
    c.check(clean)
    c.kn[2], c.vn[2] = bad, bad
    o = c.run()
    for row in (0, 1, 4, 5):
        assert torch.equal(o["out"][row], clean["out"][row]), row
        assert torch.equal(o["lse"][row], clean["lse"][row])
    assert not o["out"][2].isfinite().any() and not o["out"][3].isfinite().any()


def test_window_keeps_old_values_out():
    c = Case([3], [200], 2, 1, 64, 16, BF, seed=5)
    want = c.run(window=20)
    c.check(want, window=20)
    for t in range(0, 178):  # row 0 sees tokens 178..197
        p, s = int(c.table[0, t // 16]), t % 16
        c.k[p, :, s] = float("nan")
        c.v[p, :, :, s] = float("inf")
    o = c.run(window=20)
    assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])


@pytest.mark.parametrize("dt", [BF, F])
def test_packed_rows_and_layers_side_by_side(dt):
    """q, k and v as slices of one projection, the pages of three layers side by
    side; the other layers stay as they were."""
    c = Case([5, 1, 2], [90, 33, 2], 8, 2, 64, 16, dt, layers=3, packed=True)
    before = c.k_all[:, :2].clone(), c.v_all[:, :2].clone()
    c.check(c.run())
    assert torch.equal(before[0].view(torch.int16), c.k_all[:, :2].contiguous().view(torch.int16))
    assert torch.equal(before[1].view(torch.int16), c.v_all[:, :2].contiguous().view(torch.int16))


def test_one_row_each_without_row_offset():
    c = Case([1, 1, 1], [50, 1, 129], 8, 8, 64, 16, BF)
    o = ds.cache_attend(c.q, c.k, c.v, c.table, c.kv_len, k_new=c.kn, v_new=c.vn)
    c.check(o)


def test_rows_behind_the_last_stay():
    c = Case([2, 3], [50, 70], 4, 2, 64, 16, BF)
    pad = lambda t: torch.cat([t, torch.full_like(t[:2], 9.0)])  # noqa: E731
    out = dict(out=torch.full((7, 4, 64), 3.0, dtype=BF, device="cuda"),
               lse=torch.full((7, 4), 3.0, device="cuda"))
    ds.cache_attend(pad(c.q), c.k, c.v, c.table, c.kv_len, row_offset=c.row_offset, k_new=pad(c.kn),
                    v_new=pad(c.vn), out=out)
    assert (out["out"][5:] == 3).all() and (out["lse"][5:] == 3).all()
    c.check({k: v[:5] for k, v in out.items()})


def test_bad_pages_and_slices():
    c = Case([2, 1], [100, 60], 4, 2, 64, 16, BF, seed=4)
    good = c.run()
    ws = ds.Workspace()
    c.table[0, 2] = c.n_pages + 5  # tokens 32..47 of request 0 count as masked
    o = c.run(ws)
    assert ws.error_code() == PAGE
    ws.clear_error()
    assert torch.equal(o["out"][2], good["out"][2])
    for t in range(2):
        keep = [i for i in range(99 + t) if not 32 <= i < 48]
        K, V = c.K[0][keep].double(), c.V[0][keep].double()
        for h in range(4):
            p = torch.softmax(K[:, h // 2] @ c.q[t, h].double() / 8, 0)
            # as in check, with p |v| <= 5 for these inputs
            assert ((p @ V[:, h // 2]) - o["out"][t, h].double()).abs().max() <= 5 * 2.0 ** -8
    # the page of the new rows: not written, and masked
    c.table[1, 3] = -3
    c.run(ws)
    assert ws.error_code() == PAGE
    ws.clear_error()
    for off, lens in (([0, 5, 3], [100, 60]), ([0, 2, 2000], [100, 60]), ([-1, 2, 3], [100, 60]),
                      ([0, 2, 3], [-1, 60]), ([0, 2, 3], [1 << 20, 60])):
        c.row_offset = torch.tensor(off, dtype=torch.int32, device="cuda")
        c.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        c.run(ws)
        assert ws.error_code() & LENGTH, (off, lens)
        ws.clear_error()


def test_slices_that_overlap_stay_within_the_workspace():
    """Offsets that jump back and forth name more rows than there are."""
    R = 64
    c = Case([1] * R, [20] * R, 16, 1, 64, 16, F)
    off = [0, R] * (R // 2) + [0]
    c.row_offset = torch.tensor(off, dtype=torch.int32, device="cuda")
    c.append = False
    ws = ds.Workspace()
    c.run(ws)
    assert ws.error_code() & LENGTH


def test_pages_past_32_bit_offsets():
    """A pool of more than 2^32 bytes and 2^31 elements, the request in its last pages."""
    Hkv, D, page = 8, 128, 16
    n_pages = (1 << 31) // (Hkv * D * page) + 40
    c = Case([2], [100], 8, 8, D, page, BF)
    k = torch.empty((n_pages, Hkv, page, D), dtype=BF, device="cuda")
    v = torch.empty((n_pages, Hkv, D, page), dtype=BF, device="cuda")
    k[-c.n_pages:], v[-c.n_pages:] = c.k, c.v
    c.table = torch.where(c.table >= 0, c.table + n_pages - c.n_pages, c.table)
    c.k, c.v = k, v
    c.check(c.run())


def test_streams_and_two_graphs_over_one_workspace():
    c = Case([3, 1, 9], [60, 2000, 30], 8, 2, 64, 16, BF, seed=6)
    ws = ds.Workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = c.run(ws, stream=side)
    side.synchronize()
    c.check(o)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        a = c.run(ws)
    with torch.cuda.graph(g2):
        b = c.run(ws)
    for i in range(4):
        c.q.copy_(torch.randn(c.q.shape, device="cuda").to(BF))
        c.kv_len.copy_(torch.tensor([60, 2000 - 300 * i, 30], dtype=torch.int32))
        torch.cuda.synchronize()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        want = c.run(ws)
        for o in (a, b):
            assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"]), i


def test_prompt_then_rounds():
    """A prompt of many rows, then rounds of reserve, attend and commit on a
    PagedCache with two layers; the rejected rows leave no trace."""
    R, Hq, Hkv, D = 3, 4, 2, 64
    cache = ds.PagedCache(R, 60, Hkv=Hkv, D=D, layers=2, page=16, dtype=F)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    K = [[torch.empty(0, Hkv, D, device="cuda") for _ in range(R)] for _ in range(2)]
    V = [[torch.empty(0, Hkv, D, device="cuda") for _ in range(R)] for _ in range(2)]
    rng = torch.Generator().manual_seed(1)
    for step in range(6):
        rows = [70, 3, 33] if step == 0 else (1 + torch.randint(0, 6, (R,), generator=rng)).tolist()
        off = torch.tensor([0, *torch.tensor(rows).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        acc = [n - 1 for n in rows] if step == 0 else [int(torch.randint(-1, n, (1,), generator=rng))
                                                       for n in rows]
        assert cache.reserve(off).item() == 0
        n = sum(rows)
        for layer in range(2):
            q, kn, vn = r(n, Hq, D), r(n, Hkv, D), r(n, Hkv, D)
            o = cache.attend(layer, q, kn, vn)
            c = Case.__new__(Case)
            c.rows, c.off, c.dt, c.q, c.k = rows, off.tolist(), F, q, cache.k[:, layer]
            c.K = [torch.cat([K[layer][i], kn[off[i]:off[i + 1]]]) for i in range(R)]
            c.V = [torch.cat([V[layer][i], vn[off[i]:off[i + 1]]]) for i in range(R)]
            c.lens = [t.shape[0] for t in c.K]
            assert cache.lens.tolist() == c.lens
            c.check(o)
            for i in range(R):
                left = c.lens[i] - rows[i] + acc[i] + 1
                K[layer][i], V[layer][i] = c.K[i][:left], c.V[i][:left]
        cache.commit(torch.tensor(acc, dtype=torch.int32, device="cuda"))
        if step == 3:
            cache.release(torch.tensor([1], dtype=torch.int32, device="cuda"))
            cache.fork(torch.tensor([0], dtype=torch.int32, device="cuda"),
                       torch.tensor([1], dtype=torch.int32, device="cuda"))
            cache.compact()
            for layer in range(2):
                K[layer][1], V[layer][1] = K[layer][0], V[layer][0]
    assert cache.error_code() == 0


def snapshot(cache):
    return [t.clone() for t in (cache.lens, cache.table, cache.refs, cache.k, cache.v)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("why", ["pages", "length"])
def test_a_round_without_room_changes_nothing(why, captured):
    """Nobody looks at `missing`: the rounds that find no pages (or pass max_pages) leave
    every length, page number, count, key and value as it was, shared pages too, and
    the first round that finds room goes on from there."""
    R, Hq, Hkv, D = 4, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = ds.PagedCache(R, 5, Hkv=Hkv, D=D, page=16, dtype=F, max_pages=3 if why == "pages" else 2)
    cache.reserve(i32([0, 20, 20, 50, 50]))
    cache.attend(0, r(50, Hq, D), r(50, Hkv, D), r(50, Hkv, D))
    cache.commit(i32([19, -1, 29, -1]))
    cache.fork(i32([0]), i32([1]))
    # requests 0 and 1 write a shared page, 2 needs a new one: two pages, one is free (or
    # 33 tokens in two pages of 16)
    off, acc = i32([0, 3, 6, 9, 9]), i32([1, 0, 1, -1])
    q, kn, vn = r(9, Hq, D), r(9, Hkv, D), r(9, Hkv, D)
    out = dict(out=torch.full((9, Hq, D), 3.0, device="cuda"), lse=torch.full((9, Hq), 3.0, device="cuda"))

    def go():
        cache.reserve(off)
        cache.attend(0, q, kn, vn, out=out)
        cache.commit(acc)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
        go = graph.replay
    before = snapshot(cache)
    for _ in range(3):
        go()
        torch.cuda.synchronize()
        assert same(snapshot(cache), before)
        assert cache.missing.item() == (1 if why == "pages" else -1)
        assert (out["out"] == 3).all() and (out["lse"] == 3).all()
        assert cache.error_code() == (LENGTH if why == "length" else LENGTH | 64)
    cache.release(i32([2]))
    go()
    torch.cuda.synchronize()
    assert cache.missing.item() == 0 and cache.lens.tolist() == [22, 21, 2, 0]
    for i, (had, keep) in enumerate(((20, 2), (20, 1), (0, 2))):
        for j in range(had + keep):
            p, s = int(cache.table[i, j // 16]), j % 16
            k = kn[3 * i + j - had] if j >= had else before[3][int(before[1][0, j // 16]), 0, :, s]
            assert torch.equal(cache.k[p, 0, :, s], k)
    assert cache.refs.tolist().count(0) == 1


def test_error_bits_survive_a_larger_call():
    c = Case([1, 1], [40, 9], 8, 1, 64, 16, BF, seed=3)
    big = Case([30, 1], [40, 9], 8, 1, 64, 16, BF, seed=4)
    ws = ds.Workspace()
    c.table[0, 1] = -1
    c.run(ws)
    small = ws.buf.numel()
    big.run(ws)
    assert ws.buf.numel() > small and ws.error_code() == PAGE
    ws.clear_error()
    assert ws.error_code() == 0


def test_a_captured_round_outlives_a_larger_call():
    """Single tokens are captured, a prompt then makes the workspace grow, its old
    memory would be handed out: the replays leave what was allocated since alone."""
    c = Case([1, 1, 1], [700, 30, 1200], 8, 2, 64, 16, BF, seed=6)
    big = Case([90, 1, 3], [700, 30, 1200], 8, 2, 64, 16, BF, seed=7)
    ws = ds.Workspace()
    c.run(ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = c.run(ws)
    size = ws.buf.numel()
    big.check(big.run(ws))
    assert ws.buf.numel() > size
    other = [torch.full((size,), 77, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        c.q.copy_(torch.randn(c.q.shape, device="cuda").to(BF))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        c.check(o)
        assert all((t == 77).all() for t in other)
    c.table[1, 0] = -4  # what a replay finds wrong is reported too
    graph.replay()
    torch.cuda.synchronize()
    assert ws.error_code() == PAGE


def test_a_round_captured_at_once_keeps_its_errors():
    """Nothing ran over the cache's workspaces before the capture: no replay clears what
    an earlier one found."""
    Hq, Hkv, D = 4, 2, 64
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = ds.PagedCache(2, 8, Hkv=Hkv, D=D, page=16, dtype=F)
    off, acc = i32([0, 40, 41]), i32([39, 0])
    q, kn = torch.randn(41, Hq, D, device="cuda"), torch.randn(41, Hkv, D, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.reserve(off)
        cache.attend(0, q, kn, kn)
        cache.commit(acc)
    graph.replay()
    torch.cuda.synchronize()
    assert cache.lens.tolist() == [40, 1] and cache.error_code() == 0
    off.copy_(i32([0, 1, 2])), acc.copy_(i32([0, 0]))
    page = cache.table[0, 0].clone()
    cache.table[0, 0] = -4
    graph.replay()
    cache.table[0, 0] = page
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert cache.error_code() == PAGE
    assert cache.lens.tolist() == [43, 4]
