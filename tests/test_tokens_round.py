"""The operators of a round's tokens together, as a server runs them: positions rotated
into the paged cache, attention, edits of the target's rows, verification, histories."""
import numpy as np
import pytest
import torch

import draft_sampling_verification_03_amd as ds
from draft_sampling_verification_03_amd import decode
from test_serving_decode import D, HKV, HQ, LAYERS, Model, V, head, offsets

pytestmark = pytest.mark.gpu

I32 = torch.int32


def i32(a):
    return torch.tensor(a, dtype=I32, device="cuda")


class RotaryModel(Model):
    """The two-layer model with rotated queries and keys instead of position embeddings."""

    def __init__(self, seed, R, prompts):
        super().__init__(seed, R, prompts)
        self.pos.zero_()
        self.plan = ds.RotaryPlan(D, base=100.0)
        self.f = torch.from_numpy(self.plan.frequencies).cuda()

    def turn(self, x):
        """In 64 bits, position i for row i."""
        a = torch.arange(x.shape[0], device="cuda").double()[:, None] * self.f
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        p, q = x.chunk(2, -1)
        return torch.cat((p * c - q * s, q * c + p * s), -1)

    def whole(self, tokens):
        t = torch.tensor(tokens, device="cuda")
        h = self.emb[t].double()
        mask = torch.ones(len(tokens), len(tokens), device="cuda").triu(1).bool()

        def attend(q, k, v):
            q, k = self.turn(q), self.turn(k)
            k, v = (x.repeat_interleave(HQ // HKV, 1) for x in (k, v))
            s = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
            return torch.einsum("hij,jhd->ihd", torch.softmax(s.masked_fill(mask, -1e300), 2), v)

        for l in range(LAYERS):
            h = self.layer(l, h, attend)
        return h @ self.out.double()

    def logits(self, tokens, cache):
        """Target rows of the tokens that the cache has rows for, all on the device."""
        h = self.emb[tokens]
        for l in range(LAYERS):
            h = self.layer(l, h, lambda q, k, v, l=l: cache.attend(l, q, k, v, rotary=self.plan)["out"])
        return (h @ self.out).contiguous()

    def rows(self, prev, cache):
        off, lens = cache.row_offset.tolist(), cache.lens.tolist()
        prev = torch.as_tensor(np.asarray(prev)).cuda()
        P = self.logits(prev, cache)
        for r in range(len(lens)):
            n = off[r + 1] - off[r]
            self.history[r] = self.history[r][: lens[r] - n] + prev[off[r]:off[r + 1]].tolist()
            if n:
                want = self.whole(self.history[r])[-n:]
                self.worst = max(self.worst, (P[off[r]:off[r + 1]].double() - want).abs().max().item())
        return P


def prefill(model, cache, prompts):
    keep = [p[:-1] for p in prompts]
    cache.reserve(offsets([len(p) for p in keep]))
    model.history = [[] for _ in prompts]
    model.rows(np.concatenate(keep), cache)
    cache.commit(i32([len(p) - 1 for p in keep]))
    return np.array([p[-1] for p in prompts], np.int32)


def plain_edit(P, prev_rows, said, drafts, prompts, repetition, frequency, presence, allowed):
    """The same float32 operations in torch, row by row."""
    out, row = P.clone(), 0
    for r, n in enumerate(prev_rows):
        for j in range(n):
            x = P[row]
            made = said[r][len(prompts[r]):] + drafts[r][:j]
            c = torch.bincount(torch.tensor(made, device="cuda", dtype=torch.long), minlength=V)
            p = torch.zeros(V, dtype=torch.bool, device="cuda")
            p[prompts[r]] = True
            x = torch.where((c > 0) | p, torch.where(x > 0, x / repetition[r], x * repetition[r]), x)
            x = x - frequency[r] * c.float()
            x = x - torch.where(c > 0, presence[r], 0.0)
            out[row] = torch.where(allowed, x, float("-inf"))
            row += 1
    return out


def test_decode_with_rotary_cache_history_and_edits():
    """The loop with edits emits the same tokens as the loop without them whose target
    rows a plain model edits; the histories hold what was said, in both."""
    R, gamma, rounds = 4, 4, 7
    rng = np.random.default_rng(3)
    prompts = [rng.integers(0, V, n).tolist() for n in (2, 17, 33, 5)]
    # powers of two, so that the two sides round alike
    repetition = torch.tensor([2.0, 1.0, 4.0, 0.5], device="cuda")
    frequency = torch.tensor([0.25, 0.5, 0.0, -0.125], device="cuda")
    presence = torch.tensor([0.5, 0.0, 1.0, 0.25], device="cuda")
    allowed = torch.from_numpy(rng.random(V) < 0.8).cuda()
    words = (allowed.cpu().numpy().reshape(1, -1, 32) << np.arange(32, dtype=np.uint64)).sum(2)
    mask = torch.from_numpy(words.astype(np.uint32).view(np.int32)).cuda()
    W1, W2, U = head(2, R, gamma)

    def start():
        cache = ds.PagedCache(R, 60, Hkv=HKV, D=D, layers=LAYERS, page=16, dtype=torch.float32)
        model = RotaryModel(1, R, prompts)
        return cache, model, prefill(model, cache, prompts)

    cache, model, x0 = start()
    hist = ds.TokenHistory(R, 200)
    hist.start(i32(sum(prompts, [])), offsets([len(p) for p in prompts]))

    def edits(prev):
        return dict(repetition=repetition, frequency=frequency, presence=presence, mask=mask,
                    mask_index=torch.zeros(len(prev), dtype=I32, device="cuda"))

    got = decode.decode(rounds, x0, W1, W2, U, model.rows, cache=cache, logprobs=2, token_history=hist,
                        edits=edits)
    assert got["device_errors"] == (0,) * 6 and model.worst < 1e-4
    for r in range(R):
        assert hist.tokens[r, : hist.lens[r]].tolist() == prompts[r] + got["streams"][r]
    assert hist.prompt_lens.tolist() == [len(p) for p in prompts]

    cache, model, x0 = start()
    said = [list(p) for p in prompts]
    log = dict(round=0)

    def target_rows(prev, c):
        P = model.rows(prev, c)
        off = c.row_offset.tolist()
        n = [off[r + 1] - off[r] for r in range(R)]
        drafts = [[int(t) for t in prev[off[r] + 1:off[r + 1]]] for r in range(R)]
        i = log["round"]
        for r in range(R):  # what the edited loop has emitted so far
            said[r] = prompts[r] + sum((got["y"][t][r, : got["n_acc"][t][r] + 1].tolist() for t in range(i)), [])
        log["round"] += 1
        return plain_edit(P, n, said, drafts, prompts, repetition, frequency, presence, allowed)

    want = decode.decode(rounds, x0, W1, W2, U, target_rows, cache=cache, logprobs=2)
    for name in ("x", "ell", "n_acc", "y", "logp", "entropy", "top_ids", "top_logp"):
        assert np.array_equal(got[name], want[name], equal_nan=got[name].dtype.kind == "f"), name
    assert got["streams"] == want["streams"]
    for r in range(R):  # nothing forbidden was emitted
        assert allowed[torch.tensor(got["streams"][r], device="cuda")].all()


def test_decode_with_edits_alone():
    """No history: a grammar's masks, and the drafts before each row."""
    R, gamma = 3, 3
    W1, W2, U = head(5, R, gamma)
    g = torch.Generator(device="cuda").manual_seed(1)
    T = torch.randn((V, V), generator=g, device="cuda")
    allowed = torch.zeros(V, dtype=torch.bool, device="cuda")
    allowed[10:20] = True
    words = (allowed.cpu().numpy().reshape(1, -1, 32) << np.arange(32, dtype=np.uint64)).sum(2)
    mask = torch.from_numpy(words.astype(np.uint32).view(np.int32)).cuda()
    res = decode.decode(6, np.array([1, 2, 3], np.int32), W1, W2, U,
                        lambda prev: T[torch.from_numpy(prev).cuda()],
                        edits=lambda prev: dict(mask=mask, mask_index=i32([0] * len(prev))))
    assert res["device_errors"] == (0,) * 4
    for s in res["streams"]:
        assert all(10 <= t < 20 for t in s)


@pytest.mark.parametrize("room", [True, False])
def test_a_captured_round(room):
    """draft, schedule, reserve, rotated layers, edits, verify, commit and history in one
    graph: every replay equals the same calls made eagerly on copies of the state; where
    the cache has no room, pages and histories stay as they were."""
    R, gamma = 3, 4
    rng = np.random.default_rng(7)
    prompts = [rng.integers(0, V, n).tolist() for n in (9, 16, 20)]
    W1, W2, _ = head(2, R, gamma)
    model = RotaryModel(3, R, prompts)
    sps = torch.ones(R * (gamma + 1) + 1, dtype=torch.float64, device="cuda")
    U = torch.empty((R, gamma, V), device="cuda")
    conf = torch.empty((R, gamma), device="cuda")
    rep, fre = torch.tensor([1.25, 1.0, 2.0], device="cuda"), torch.tensor([0.5, 0.25, 0.0], device="cuda")
    rows = R * (gamma + 1)

    def state():
        cache = ds.PagedCache(R, 40 if room else 4, Hkv=HKV, D=D, layers=LAYERS, page=16, dtype=torch.float32)
        hist = ds.TokenHistory(R, 200)
        hist.start(i32(sum(prompts, [])), offsets([len(p) for p in prompts]))
        anchors = torch.from_numpy(prefill(model, cache, prompts)).cuda()
        return dict(cache=cache, hist=hist, anchors=anchors,
                    ws=[ds.Workspace() for _ in range(3)])

    def once(s):
        cache, hist = s["cache"], s["hist"]
        d = ds.draft(U, W1, W2, s["anchors"], seed=5, round=1, ws=s["ws"][0])
        sch = ds.schedule(conf, sps, ds.DSPARK_SCHED_THRESHOLD, ws=s["ws"][1], threshold=0.5)
        cache.reserve(sch["row_offset"])
        # the previous token of every row of a full batch of rows, without the host
        i = torch.arange(rows, device="cuda")
        off = sch["row_offset"].long()
        rho = torch.searchsorted(off[1:].contiguous(), i, right=True).clamp(max=R - 1)
        j = (i - off[rho]).clamp(0, gamma)
        prev = torch.cat((s["anchors"][:, None], d["x"]), 1)[rho, j].long()
        P = model.logits(prev, cache)
        hist.edit(P, row_offset=sch["row_offset"], drafts=d["x"], repetition=rep, frequency=fre, out=P)
        v = ds.verify(sch["ell"], sch["row_offset"], P, U, W1, W2, s["anchors"], d["x"], d["q_stats"],
                      d["q_x"], seed=5, round=1, ws=s["ws"][2])
        row_offset = cache.row_offset
        cache.commit(v["n_acc"])
        hist.append(v["y"], v["n_acc"], row_offset=row_offset)
        return dict(x=d["x"], ell=sch["ell"], y=v["y"], n_acc=v["n_acc"], P=P, off=sch["row_offset"])

    a, b = state(), state()
    g = torch.Generator(device="cuda").manual_seed(9)

    def inputs():
        U.copy_(torch.randn(U.shape, generator=g, device="cuda"))
        conf.copy_(torch.rand(conf.shape, generator=g, device="cuda"))

    inputs()
    once(b)  # workspaces, libraries
    torch.cuda.synchronize()
    b = dict(state(), ws=b["ws"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = once(b)
    frozen = b["hist"].tokens.clone(), b["hist"].lens.clone(), b["cache"].lens.clone()
    stopped = False
    for step in range(4):
        inputs()
        want = once(a)
        graph.replay()
        torch.cuda.synchronize()
        n = int(want["off"][-1])
        fits = int(a["cache"].missing) == 0
        stopped |= not fits
        for name in ("x", "ell", "n_acc") if fits else ("x", "ell"):
            assert torch.equal(out[name], want[name]), (step, name)
        if fits:
            assert torch.equal(out["P"][:n], want["P"][:n])
            for r in range(R):
                m = int(want["n_acc"][r]) + 1
                assert torch.equal(out["y"][r, :m], want["y"][r, :m])
        for x in ("lens", "table", "refs"):
            assert torch.equal(getattr(a["cache"], x), getattr(b["cache"], x)), (step, x)
        assert torch.equal(a["hist"].tokens, b["hist"].tokens) and torch.equal(a["hist"].lens, b["hist"].lens)
        if fits:
            last = torch.stack([want["y"][r, int(want["n_acc"][r])] for r in range(R)]).clone()
            a["anchors"].copy_(last), b["anchors"].copy_(last)
            for r in range(R):
                assert int(a["hist"].lens[r]) == int(a["cache"].lens[r]) + 1
            frozen = b["hist"].tokens.clone(), b["hist"].lens.clone(), b["cache"].lens.clone()
        else:  # nothing has changed
            now = b["hist"].tokens, b["hist"].lens, b["cache"].lens
            assert all(torch.equal(x, y) for x, y in zip(frozen, now))
    assert stopped != room
    if room:
        assert a["cache"].error_code() == 0 and a["hist"].error_code() == 0
        assert b["cache"].error_code() == 0 and b["hist"].error_code() == 0


def test_decode_stops_where_a_history_is_full():
    """The round whose tokens do not fit raises and changes neither the cache nor any
    history; a history that they just fill takes them."""
    R, gamma, rounds = 3, 3, 8
    rng = np.random.default_rng(11)
    prompts = [rng.integers(0, V, n).tolist() for n in (2, 17, 5)]
    W1, W2, U = head(4, R, gamma)
    repetition = torch.tensor([2.0, 1.0, 0.5], device="cuda")

    def run(capacity, rounds):
        cache = ds.PagedCache(R, 60, Hkv=HKV, D=D, layers=LAYERS, page=16, dtype=torch.float32)
        model = RotaryModel(1, R, prompts)
        x0 = prefill(model, cache, prompts)
        hist = ds.TokenHistory(R, capacity)
        hist.tokens = torch.full((R, capacity), -1, dtype=I32, device="cuda")
        hist.start(i32(sum(prompts, [])), offsets([len(p) for p in prompts]))
        try:
            return decode.decode(rounds, x0, W1, W2, U, model.rows, cache=cache, token_history=hist,
                                 edits=dict(repetition=repetition)), cache, hist
        except RuntimeError as e:
            return e, cache, hist

    want, cache, hist = run(200, rounds)
    said = [prompts[r] + want["streams"][r] for r in range(R)]
    lens = np.array([len(p) for p in prompts]) + np.cumsum(np.array(want["n_acc"]) + 1, 0)  # after each round
    assert hist.lens.tolist() == lens[-1].tolist()
    longest = int(lens[-1].max())
    got, cache, hist = run(longest, rounds)
    assert got["streams"] == want["streams"] and hist.lens.tolist() == lens[-1].tolist()
    for capacity in (longest - 1, 19):  # 17 and at least 8 tokens do not fit
        whole = int((lens.max(1) <= capacity).sum())  # rounds that fit
        assert whole < rounds
        got, cache, hist = run(capacity, rounds)
        assert isinstance(got, RuntimeError) and f"round {whole}" in str(got) and "history" in str(got)
        kept = lens[whole - 1].tolist() if whole else [len(p) for p in prompts]
        assert hist.lens.tolist() == kept and cache.lens.tolist() == [n - 1 for n in kept]
        for r in range(R):
            assert hist.tokens[r, : kept[r]].tolist() == said[r][: kept[r]]
            assert (hist.tokens[r, kept[r]:] == -1).all()
        assert hist.error_code() == 0 and cache.error_code() == 0
