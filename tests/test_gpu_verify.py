"""mq_verify against a plain 64-bit reference: every token and count has to be equal, but where the reference says that
a decision fell within 2^-22 of its border (weights are right to 5 x 2^-26)."""
import numpy as np
import pytest

import synth
from oracle import decode as ref

pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -22


@pytest.fixture(scope="module")
def mq():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quant_quantized_gemv_gb300 import build
    build.build()
    import quant_quantized_gemv_gb300 as m
    m.lib()
    yield m
    m.mq_set_pdl(False)


def dev(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Sequences of drafts[i] drafted tokens; a draft model near the target."""

    def __init__(self, v, drafts, probs=True, noise=0.4, flat=False, key="", lead=0, behind=0):
        g = synth.rng("verify", v, len(drafts), sum(drafts), probs, flat, key)
        rng = np.random.default_rng(int(g.integers(1 << 30)))
        self.v, self.rows = v, lead + sum(d + 1 for d in drafts) + behind
        self.starts = (lead + np.concatenate([[0], np.cumsum([d + 1 for d in drafts])])).astype(np.int32)
        self.n = len(drafts)
        self.logits = rng.standard_normal((self.rows, v), np.float32) * np.float32(0.3 if flat else 2.5)
        draft = self.logits + rng.standard_normal((self.rows, v), np.float32) * np.float32(noise)
        q = np.exp(draft - draft.max(1, keepdims=True))
        self.q = (q / q.sum(1, keepdims=True)).astype(np.float32)
        c = np.cumsum(self.q.astype(np.float64), 1)
        self.drafts = np.array([min(v - 1, int(np.searchsorted(r, x * r[-1]))) for r, x in zip(c, rng.random(self.rows))], np.int32)
        if not probs:
            self.q = None
        self.u, self.u_draw = rng.random(self.rows).astype(np.float32), rng.random(self.n).astype(np.float32)
        self.f = {}

    def filters(self, **f):
        """One value, or one a sequence."""
        kinds = dict(temperature=np.float32, top_k=np.int32, top_p=np.float32, min_p=np.float32)
        self.f = {n: np.broadcast_to(np.asarray(x, kinds[n]), (self.n,)).copy() for n, x in f.items()}
        return self

    def args(self):
        return dict(logits=dev(self.logits), drafts=dev(self.drafts), starts=dev(self.starts), u=dev(self.u),
                    u_draw=dev(self.u_draw), draft_probs=dev(self.q), **{n: dev(x) for n, x in self.f.items()})

    def run(self, mq, **more):
        import torch
        a = dict(tokens=torch.full((self.rows,), -9, dtype=torch.int32, device="cuda"),
                 counts=torch.full((self.n,), -9, dtype=torch.int32, device="cuda"),
                 ws=mq.mq_verify_workspace(self.n, self.rows))
        a.update(self.args())
        a.update(more)
        r = mq.mq_verify(**a)
        torch.cuda.synchronize()
        room = mq.mq_verify_workspace_bytes(1, 1)
        assert not a["ws"].view(-1, room).view(torch.int32)[:, :3].any()   # the counts are zero again
        return r

    def want(self, i):
        a, b = self.starts[i], self.starts[i + 1]
        names = dict(temperature="t", top_k="k", top_p="p", min_p="m")
        f = {names[k]: x[i].item() for k, x in self.f.items()}
        return ref.verify(self.logits[a:b], self.drafts[a:b], self.u[a:b].astype(float), float(self.u_draw[i]),
                          None if self.q is None else self.q[a:b], **f)

    def check(self, tokens, counts):
        t, c = tokens.cpu().numpy(), counts.cpu().numpy()
        inside = np.zeros(self.rows, bool)
        refused = near = 0
        for i in range(self.n):
            a, b = self.starts[i], self.starts[i + 1]
            inside[a:b] = True
            if a == b:
                assert c[i] == 0
                continue
            want, n, gap = self.want(i)
            if gap > NEAR:
                assert c[i] == n and np.array_equal(t[a:b], want), (i, gap)
            near += gap <= NEAR
            refused += n < b - a
        # (a draw is near with a probability of 2^-21 over the token's share: one in twenty where that is 10^-5)
        assert np.all(t[~inside] == -9) and near <= 2 + self.n // 4
        return refused


FILTERS = [dict(), dict(temperature=0.7), dict(top_p=0.9), dict(top_k=40), dict(top_k=1000, top_p=0.8), dict(min_p=0.05),
           dict(temperature=1.3, top_k=50, top_p=0.95, min_p=0.02)]


@pytest.mark.parametrize("v", [1, 7, 1000, 4099, 50257])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("f", range(len(FILTERS)))
def test_against_reference(mq, v, probs, f):
    c = Case(v, [0, 4, 1, 7, 2, 3] if v < 50000 else [0, 2, 3], probs, key=f).filters(**FILTERS[f])
    c.check(*c.run(mq))


@pytest.mark.parametrize("f", [0, 2, 3, 6])
def test_a_large_vocabulary(mq, f):
    c = Case(152064, [4, 2], key=f).filters(**FILTERS[f])
    c.check(*c.run(mq))


@pytest.mark.parametrize("f", [0, 1, 2, 4])
def test_flat_logits(mq, f):
    """Nothing stands out: long kept sets, rests spread over the whole vocabulary."""
    c = Case(30000, [5] * 5, flat=True, noise=0.05, key=f).filters(**FILTERS[f])
    c.check(*c.run(mq))


def test_sequences_of_all_kinds(mq):
    """Empty ones, rows of nobody before and behind, long drafts, a filter a sequence, greedy ones."""
    drafts = [0, 3, 0, 30, 1, 1, 5, 8, 2, 0]
    c = Case(2000, drafts, key="kinds", lead=2, behind=3)
    c.starts[3] = c.starts[2]          # sequence 2 has no row; sequence 3 takes it
    c.filters(temperature=[0.0, 1.0, 0.5, 0.0, 2.0, 1.0, 1.0, 0.3, -1.0, 1.0], top_k=[0, 5, 0, 0, 1, 3, 0, 100, 0, 0],
              top_p=[1, 1, 1, 1, 1, 0.5, 0.0, 0.9, 1, 1], min_p=[0, 0, 0.1, 0, 0, 0, 0, 0, 0, 0.7])
    c.check(*c.run(mq))


def test_many_sequences(mq):
    """More than a CTA's threads."""
    c = Case(300, [i % 4 for i in range(1500)], key="many").filters(top_p=0.9)
    assert 200 < c.check(*c.run(mq)) < 1300


def test_many_rows_of_one_sequence(mq):
    c = Case(500, [300], noise=0.0, key="long")
    c.u[:] = 0.3
    c.u[211] = 0.999
    c.q[211, c.drafts[211]] = 1.0      # a probability far above the target's
    t, n = c.run(mq)
    c.check(t, n)
    assert int(n) == 212


def test_drafts_that_equal_the_target_stand(mq):
    """q = p: everything stands, whatever u is below 1 (but for p's own rounding: u ends at 0.999)."""
    c = Case(5000, [6, 6, 6], noise=0.0, key="equal")
    c.u[:] = np.float32(0.999)
    t, n = c.run(mq)
    assert n.tolist() == [7, 7, 7]
    c.check(t, n)


def test_borders_of_the_random_numbers(mq):
    """Outside [0, 1) a number counts as the nearest end; at the ends of a sum the token may be one of no weight to speak
    of, so there the counts, and that it is a token, are looked at."""
    c = Case(3000, [3] * 8, key="borders")
    c.u[:] = np.tile(np.float32([0, -1, 2, 0.5]), 8)
    c.u_draw[:] = np.float32([0, 1 - 2.0 ** -24, 1, 2, -1, 0.5, 1e-30, -0.0])
    t, n = c.run(mq)
    c.u = np.clip(c.u, 0, 1 - 2.0 ** -24).astype(np.float32)
    c.u_draw = np.clip(c.u_draw, 0, 1 - 2.0 ** -24).astype(np.float32)
    got, cnt = t.cpu().numpy(), n.cpu().numpy()
    for i in range(8):
        a, b = c.starts[i], c.starts[i + 1]
        want, m, _ = c.want(i)
        assert cnt[i] == m and np.array_equal(got[a:a + m - 1], want[:m - 1]) and 0 <= got[a + m - 1] < 3000
        assert np.all(got[a + m:b] == -1)


def test_probabilities_that_are_none(mq):
    """NaN, negative ones, ones above 1, all of them 1 (nothing is left of p: the draw is from p itself), all 0."""
    c = Case(4000, [2] * 6, key="no probabilities")
    for i, x in enumerate([np.nan, -1.0, 7.0, 1.0, 0.0]):
        c.q[c.starts[i]:c.starts[i + 1]] = x
    c.u[:] = np.float32(0.9)
    for f in (dict(), dict(top_p=0.7), dict(top_k=20)):
        c.filters(**f).check(*c.run(mq))


def test_drafts_outside_the_vocabulary_never_stand(mq):
    c = Case(1000, [3, 3, 3], key="outside")
    c.drafts[c.starts[:-1]] = [-1, 1000, 2 ** 31 - 1]
    c.u[:] = 0
    t, n = c.run(mq)
    assert n.tolist() == [1, 1, 1]
    c.check(t, n)


def test_infinite_and_nan_logits(mq):
    c = Case(3000, [2, 2, 2, 2], key="special")
    s = c.starts
    c.logits[s[0]] = -np.inf                             # nothing to draw from
    c.logits[s[1], [7, 2000]] = np.inf                   # two tokens share it all
    c.drafts[s[1]], c.u[s[1]] = 2000, 0.0
    c.logits[s[2]] = np.nan
    c.logits[s[2], 55] = 1.0
    c.drafts[s[2]] = 54
    c.logits[s[3], ::2] = np.nan
    t, n = c.run(mq)
    got = t.cpu().numpy()
    assert n[0] == 1 and got[s[0]] == -1
    assert got[s[1]] == 2000 and got[s[2]] == 55 and n[2] == 1
    want, m, gap = c.want(3)
    assert gap <= NEAR or (np.array_equal(got[s[3]:s[4]], want) and n[3] == m)
    c.drafts[s[1]], c.u[s[1]] = 8, 0.0                   # stands for nothing beside them; what is left is theirs
    t, n = c.run(mq)
    assert n[1] == 1 and int(t[s[1]]) in (7, 2000)


@pytest.mark.parametrize("starts", [[0, 5, 3, 9], [-1, 2, 4, 9], [0, 2, 4, 10], [9, 6, 3, 0], [5, 5, 5, 2 ** 31 - 1]])
def test_starts_that_do_not_ascend(mq, starts):
    """Nothing is written but the status, and the workspace serves the next call."""
    import torch
    c = Case(1000, [2, 2, 2], key="starts")
    good = c.run(mq)
    ws = mq.mq_verify_workspace(3, 9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, n = c.run(mq, starts=dev(np.int32(starts)), status=status, ws=ws)
    assert int(status) == 1 and (t == -9).all() and (n == -9).all()
    again = c.run(mq, ws=ws)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


def test_one_workspace_for_calls_of_all_sizes(mq):
    import torch
    ws = mq.mq_verify_workspace(100, 400)
    for drafts in ([3] * 100, [1], [20, 0, 3], [0] * 50, [7] * 9):
        c = Case(700, drafts, key="workspace")
        a, b = c.run(mq, ws=ws), c.run(mq)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_strides_odd_addresses_and_tokens_over_the_drafts(mq):
    import torch
    c = Case(1003, [3, 1, 4], key="strides").filters(top_p=0.9)
    want = c.run(mq)
    wide = torch.full((c.rows, 1003 * 2 + 7), 50.0, device="cuda")
    wide[:, 5:1008] = dev(c.logits)
    wide[:, 5:1008] = dev(c.logits)
    wide[:, 1008:2011] = dev(c.q)
    drafts = dev(c.drafts)
    t, n = c.run(mq, logits=wide[:, 5:1008], draft_probs=wide[:, 1008:2011], drafts=drafts, tokens=drafts)
    assert torch.equal(t, want[0]) and torch.equal(n, want[1]) and t is drafts


def test_made_outputs_streams_and_a_captured_chain(mq):
    import torch
    c = Case(20000, [4, 0, 2], key="graph").filters(temperature=0.8, top_p=0.95)
    want = c.run(mq)
    a, st, gr = c.args(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    got = mq.mq_verify(**a)
    torch.cuda.synchronize()
    other = mq.mq_verify(**a, stream=st)
    torch.cuda.synchronize()
    ws = mq.mq_verify_workspace(c.n, c.rows)
    tokens, counts = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    logits = torch.zeros_like(a["logits"])
    torch.cuda.synchronize()
    mq.mq_set_pdl(True)
    try:
        with torch.cuda.graph(gr, stream=st):
            for _ in range(3):
                mq.mq_copy(logits, a["logits"])
                mq.mq_verify(**{**a, "logits": logits}, tokens=tokens, counts=counts, ws=ws)
    finally:
        mq.mq_set_pdl(False)
    gr.replay()
    torch.cuda.synchronize()
    for t, n in (got, other, (tokens, counts)):
        assert torch.equal(t, want[0]) and torch.equal(n, want[1])


def test_rows_without_drafts_are_draws(mq):
    """A sequence of one row is mq_sample with the same numbers."""
    import torch
    c = Case(50257, [0] * 20, key="draws").filters(temperature=0.9, top_k=60, top_p=0.9, min_p=0.01)
    t, n = c.run(mq)
    f = {k: dev(x) for k, x in c.f.items()}
    assert torch.equal(t, mq.mq_sample(dev(c.logits), dev(c.u_draw), **f)) and (n == 1).all()


def test_refusals(mq):
    import torch
    c = Case(100, [2, 1], key="refusals")
    a = dict(c.args(), tokens=torch.full((5,), -9, dtype=torch.int32, device="cuda"),
             counts=torch.zeros(2, dtype=torch.int32, device="cuda"), ws=mq.mq_verify_workspace(2, 5))
    for change, error in [(dict(drafts=a["drafts"][:4]), ValueError), (dict(drafts=a["drafts"].long()), TypeError),
                          (dict(u=a["u"][:4]), ValueError), (dict(u_draw=a["u"]), ValueError),
                          (dict(draft_probs=a["draft_probs"][:, :99]), ValueError), (dict(ws=a["ws"][:39]), mq.MQError),
                          (dict(starts=a["starts"][:1], u_draw=a["u_draw"][:0], counts=a["counts"][:0]), mq.MQError),
                          (dict(top_k=a["u_draw"]), TypeError), (dict(temperature=a["u"]), ValueError),
                          (dict(logits=a["logits"].t().contiguous().t()), ValueError), (dict(counts=a["tokens"]), ValueError),
                          (dict(logits=a["logits"].cpu()), TypeError), (dict(starts=a["starts"].cpu()), TypeError)]:
        with pytest.raises(error):
            mq.mq_verify(**{**a, **change})
    torch.cuda.synchronize()
    assert (a["tokens"] == -9).all()


# ------------------------------------------------------------------ many rows: those without a filter go by chunks
LEAST = 8 << 20


def many(v, key, probs=True, **more):
    drafts, rows = [], 0
    while rows * v < LEAST:
        drafts.append((len(drafts) * 5 + 2) % 7)
        rows += drafts[-1] + 1
    return Case(v, drafts, probs, key=key, **more)


@pytest.mark.parametrize("v", [30011, 152064])
@pytest.mark.parametrize("probs", [True, False])
def test_many_rows_without_filters(mq, v, probs):
    import torch
    c = many(v, "chunks", probs, lead=3, behind=2).filters(temperature=0.8)
    t, n = c.run(mq)
    assert c.check(t, n) > 3
    a = c.args()
    del a["temperature"]
    c.f = {}
    t, n = mq.mq_verify(**a)                                  # nothing but chunks is launched
    u, m = c.run(mq, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    inside = slice(int(c.starts[0]), int(c.starts[-1]))
    assert torch.equal(t[inside], u[inside]) and torch.equal(n, m)
    c.check(u, m)


def test_many_rows_some_with_filters(mq):
    """Greedy ones, filters of all kinds and none, in one call."""
    c = many(30011, "mixed")
    i = np.arange(c.n)
    c.filters(temperature=np.where(i % 5 == 1, 0.0, 0.5 + 0.1 * (i % 7)), top_k=np.where(i % 4 == 2, 30, 0),
              top_p=np.where(i % 6 == 3, 0.9, 1.0), min_p=np.where(i % 9 == 4, 0.05, 0.0))
    c.check(*c.run(mq))


def test_many_rows_of_flat_logits(mq):
    c = many(30011, "flat", flat=True, noise=0.05)
    c.check(*c.run(mq))


def test_many_rows_special_values(mq):
    """Rows of nothing, infinite logits, NaN, probabilities that are none, drafts outside the vocabulary, the ends of the
    random numbers; empty sequences."""
    c = many(30011, "special many", lead=1)
    s = c.starts
    c.starts = s = np.concatenate([s[:4], s[3:]]).astype(np.int32)       # sequence 3 has no row
    c.n += 1
    c.u_draw = np.concatenate([c.u_draw[:4], c.u_draw[3:]])
    first = s[:-1]
    c.logits[first[5]] = -np.inf
    c.logits[first[6], [7, 20000]] = np.inf
    c.logits[first[8]] = np.nan
    c.logits[first[8], 55] = 1.0
    c.drafts[first[8]] = 54
    c.logits[first[9], ::2] = np.nan
    for i, x in zip(range(10, 15), [np.nan, -1.0, 7.0, 1.0, 0.0]):
        c.q[s[i]:s[i + 1]] = x
    c.drafts[first[15:18]] = [-1, 30011, 2 ** 31 - 1]
    c.u[s[10]:s[18]] = np.float32(0.9)
    t, n = c.run(mq)
    got, cnt = t.cpu().numpy(), n.cpu().numpy()
    assert cnt[3] == 0 and cnt[5] == 1 and got[first[5]] == -1
    assert got[first[6]] in (7, 20000) and got[first[8]] == 55 and cnt[8] == 1
    for i in range(c.n):
        if i in (3, 5, 6, 8):
            continue
        want, m, gap = c.want(i)
        assert gap <= NEAR or (cnt[i] == m and np.array_equal(got[s[i]:s[i + 1]], want)), (i, gap)


def test_many_rows_strides_in_place_and_captured(mq):
    import torch
    c = many(30011, "strides many").filters(top_p=np.float32(1.0))
    want = c.run(mq)
    wide = torch.full((c.rows, 2 * 30011 + 5), 60.0, device="cuda")
    wide[:, 2:30013] = dev(c.logits)
    wide[:, 30013:60024] = dev(c.q)
    drafts = dev(c.drafts)
    a = dict(c.args(), logits=wide[:, 2:30013], draft_probs=wide[:, 30013:60024], drafts=drafts)
    t, n = c.run(mq, **dict(a, tokens=drafts))
    assert torch.equal(t, want[0]) and torch.equal(n, want[1])
    a["drafts"] = dev(c.drafts)
    ws = mq.mq_verify_workspace(c.n, c.rows)
    tokens, counts, st, gr = torch.zeros_like(want[0]), torch.zeros_like(want[1]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    logits = torch.zeros_like(dev(c.logits))
    torch.cuda.synchronize()
    mq.mq_set_pdl(True)
    try:
        with torch.cuda.graph(gr, stream=st):
            for _ in range(3):
                logits.copy_(a["logits"])
                mq.mq_verify(**{**a, "logits": logits}, tokens=tokens, counts=counts, ws=ws)
    finally:
        mq.mq_set_pdl(False)
    for _ in range(2):
        gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(tokens, want[0]) and torch.equal(counts, want[1])


def test_many_rows_starts_that_do_not_ascend(mq):
    import torch
    c = many(30011, "starts many").filters(top_k=0)
    good, ws = c.run(mq), mq.mq_verify_workspace(c.n, c.rows)
    bad = c.starts.copy()
    bad[7] = bad[9] + 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, n = c.run(mq, starts=dev(bad), status=status, ws=ws)
    assert int(status) == 1 and (t == -9).all() and (n == -9).all()
    again = c.run(mq, ws=ws)
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


@pytest.mark.parametrize("v", [30011, 152064])
def test_many_rows_without_a_temperature(mq, v):
    """The most likely tokens: equal largest logits, infinite ones, NaN, rows of nothing; the draft is the first of them,
    or another."""
    c = many(v, "greedy many", lead=1).filters(temperature=0.0)
    c.f["temperature"][4] = np.nan
    s = c.starts
    best = c.logits.argmax(1)
    c.drafts[::2] = best[::2]                                    # many stand
    g = np.random.default_rng(9)
    for r in range(1, c.rows, 3):                                # equal ones; the draft is one of them, mostly the first
        at = np.sort(g.choice(v, 5, replace=False))
        c.logits[r, at] = [30.0, np.inf][r % 2]
        c.drafts[r] = at[0 if r % 4 else 3]
    for r in range(2, c.rows, 7):
        c.logits[r, g.choice(v, v // 2, replace=False)] = np.nan
    c.logits[s[6]] = -np.inf
    c.logits[s[7]] = np.nan
    for probs in (c.q, None):
        c.q = probs
        t, n = c.run(mq)
        assert c.check(t, n) > 3
    u, m = c.run(mq, top_k=dev(np.ones(c.n, np.int32)), temperature=None)   # the clusters' way to one token
    t, u = t.cpu().numpy(), u.cpu().numpy()
    for i in range(c.n):
        if not np.isposinf(c.logits[s[i]:s[i + 1]]).any():
            assert np.array_equal(t[s[i]:s[i + 1]], u[s[i]:s[i + 1]]), i


def test_more_sequences_than_rows(mq):
    c = many(152064, "empty many", lead=2)
    s = c.starts
    for n_seqs in (c.rows + 9, c.rows - 1):
        starts = np.sort(np.concatenate([s, g_starts(s, n_seqs + 1 - len(s))])).astype(np.int32)
        of = np.flatnonzero(np.diff(starts))
        c2 = many(152064, "empty many", lead=2)
        c2.starts, c2.n = starts, n_seqs
        c2.u_draw = np.full(n_seqs, 0.25, np.float32)
        c2.u_draw[of] = c.u_draw
        t, n = c2.run(mq)
        c2.check(t, n)


def g_starts(s, more):
    """Starts of empty sequences: some of those that are there, again."""
    return np.random.default_rng(more).choice(s, more)


def test_many_short_rows(mq):
    """Rows of one chunk, by chunks."""
    c = Case(129, [i % 6 for i in range(3000)], key="short", lead=3, behind=5).filters(
        temperature=np.where(np.arange(3000) % 7 == 3, 0.0, 0.7))
    assert c.rows * c.v >= 1 << 20
    assert c.check(*c.run(mq)) > 100


def test_many_rows_on_two_streams_at_once(mq):
    import torch
    c = many(30011, "two streams").filters(top_k=np.where(np.arange(many(30011, "two streams").n) % 5 == 2, 30, 0))
    want = c.run(mq)
    a = c.args()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.full_like(want[0], -9), torch.full_like(want[1], -9), mq.mq_verify_workspace(c.n, c.rows)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, (tokens, counts, ws) in zip(streams, outs):
            mq.mq_verify(**a, tokens=tokens, counts=counts, ws=ws, stream=st)
    torch.cuda.synchronize()
    for tokens, counts, _ in outs:
        assert torch.equal(tokens, want[0]) and torch.equal(counts, want[1])


@pytest.mark.parametrize("f", [dict(), dict(temperature=0.0), dict(top_p=0.9), dict(top_k=30)])
def test_the_largest_vocabulary(mq, f):
    c = Case(mq.MQ_SAMPLE_MAX_VOCAB, [2, 0, 1], key=("largest", str(f)), lead=1).filters(**f)
    c.check(*c.run(mq))


# ------------------------------------------------------------------ faint ends, addresses
def borders(c, tokens, counts, i, near=2.0 ** -21):
    """Sequence i's tokens where a random number may lie on a border: what stands is the reference's, and the drawn token is
    one of a finite logit whose interval reaches to within `near` of the draw."""
    names = dict(temperature="t", top_k="k", top_p="p", min_p="m")
    a, b = int(c.starts[i]), int(c.starts[i + 1])
    want, n, _ = c.want(i)
    got = tokens[a:b]
    assert counts[i] == n and np.array_equal(got[:n - 1], want[:n - 1]) and np.all(got[n:] == -1)
    r, at = a + n - 1, int(got[n - 1])
    assert 0 <= at < c.v and np.isfinite(c.logits[r, at])
    w = p = ref.distribution(c.logits[r], **{names[k]: x[i].item() for k, x in c.f.items()})
    if r + 1 < b:
        q = np.zeros(c.v)
        if c.q is not None:
            q = np.clip(np.nan_to_num(c.q[r].astype(np.float64), nan=0.0), 0, 1)
        else:
            q[c.drafts[r]] = 1.0
        w = np.maximum(p - q, 0)
        w = w if w.sum() > 0 else p
    sums = np.cumsum(w) / w.sum()
    u = float(c.u_draw[i])
    assert sums[at] - w[at] / w.sum() - near <= u <= sums[at] + near, (i, at)


def faint(v, probs, temperature, key, other=1.0):
    """Rows of one or a few likely tokens amid ones that have 2^-43 of the row or less: as many as chunks hold, the first and
    the last among them.  Drafts that stand, drafts that do not, none."""
    drafts = [0, 1, 2] * 8
    c = Case(v, drafts, probs, key=key).filters(temperature=np.float32(temperature))
    g = np.random.default_rng(v)
    c.logits = (g.standard_normal(c.logits.shape).astype(np.float32) * np.float32(0.1) - np.float32(30.5)) * np.float32(temperature)
    c.u[:] = np.float32(0.25)
    for r in range(c.rows):
        likely = v // 2 + 3 * np.arange(1 + r % 3)
        c.logits[r, likely] = np.float32([0.0, -1.0, -2.0])[:len(likely)] * np.float32(temperature)
        c.drafts[r] = likely[0] if r % 2 else 5             # one that stands, one that does not
        if probs:
            c.q[r] = 0.0
            c.q[r, c.drafts[r]] = np.float32(other)
    ends = np.float32([0.0, 1e-30, 2.0 ** -24, 0.5, 1 - 2.0 ** -24, 1.0, 2.0, -1.0])
    c.u_draw = ends[np.arange(c.n) // 3 % 8]
    return c


@pytest.mark.parametrize("v", [152064, 50257])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("temperature", [1.0, 0.2])
def test_many_rows_the_ends_of_the_draw(mq, v, probs, temperature):
    c = faint(v, probs, temperature, "ends")
    assert c.rows * v >= 2 << 20
    t, n = (x.cpu().numpy() for x in c.run(mq))
    c.u_draw = np.clip(c.u_draw, 0, 1 - 2.0 ** -24).astype(np.float32)
    for i in range(c.n):
        borders(c, t, n, i)


@pytest.mark.parametrize("v", [152064, 50257])
def test_many_rows_the_ends_of_a_draw_from_p_itself(mq, v):
    """Probabilities of 1 everywhere: nothing is left of p."""
    c = faint(v, True, 1.0, "ends of p")
    c.q[:] = 1.0
    c.u[:] = np.float32(1 - 2.0 ** -24)
    c.drafts[:] = 5
    t, n = (x.cpu().numpy() for x in c.run(mq))
    c.u_draw = np.clip(c.u_draw, 0, 1 - 2.0 ** -24).astype(np.float32)
    for i in range(c.n):
        borders(c, t, n, i)


def test_many_rows_a_padded_vocabulary(mq):
    """Nothing in the last two chunks: a draw of 1 ends in front of them."""
    c = faint(50257, False, 0.5, "padded")
    c.logits[:, 40000:] = -np.inf
    t, n = (x.cpu().numpy() for x in c.run(mq))
    c.u_draw = np.clip(c.u_draw, 0, 1 - 2.0 ** -24).astype(np.float32)
    for i in range(c.n):
        borders(c, t, n, i)


def test_many_rows_the_borders_of_the_random_numbers(mq):
    """Rows as any, by chunks; u at its ends as well."""
    c = many(30011, "borders many")
    c.u[::3] = np.resize(np.float32([0, -1, 2, 1 - 2.0 ** -24]), len(c.u[::3]))
    c.u_draw = np.resize(np.float32([0, 1 - 2.0 ** -24, 1, 2, -1, 0.5, 1e-30, -0.0]), c.n)
    t, n = (x.cpu().numpy() for x in c.run(mq))
    c.u = np.clip(c.u, 0, 1 - 2.0 ** -24).astype(np.float32)
    c.u_draw = np.clip(c.u_draw, 0, 1 - 2.0 ** -24).astype(np.float32)
    for i in range(c.n):
        near = False                                        # (u = 1 - 2^-24 over equal probabilities decides by 2^-24 of them)
        for r in range(c.starts[i], c.starts[i + 1] - 1):
            least, x = float(c.u[r]) * float(c.q[r, c.drafts[r]]), ref.distribution(c.logits[r])[c.drafts[r]]
            near = near or abs(least - x) <= NEAR * max(least, x)
        if not near:
            borders(c, t, n, i)


def test_many_rows_wherever_they_begin(mq):
    """A row among 16 bytes: its sums, and so its token, do not change.  Draws of many numbers over many tokens of nearly
    equal weight, so that some fall near a border."""
    import torch
    v, n = 152063, 64                                       # an odd stride: four rows begin in four ways
    g = torch.Generator(device="cuda").manual_seed(5)
    ws = mq.mq_verify_workspace(n, n)
    starts = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    zeros, u = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda")
    tokens, counts = torch.zeros_like(zeros), torch.zeros_like(zeros)
    other = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(4):
        logits = (torch.randn(n // 4, 1, v, device="cuda", generator=g) * 0.5).expand(-1, 4, -1).contiguous().view(n, v)
        for _ in range(3000):
            draws = torch.rand(n // 4, 1, device="cuda", generator=g).expand(-1, 4).reshape(n)
            mq.mq_verify(logits, zeros, starts, u, draws, tokens=tokens, counts=counts, ws=ws)
            t = tokens.view(-1, 4)
            other += (t != t[:, :1]).sum()
    assert int(other) == 0


@pytest.mark.parametrize("v", [20000, 152064])
@pytest.mark.parametrize("f", [dict(), dict(top_k=700), dict(top_p=0.95)])
def test_what_is_left_of_nearly_equal_probabilities(mq, v, f):
    """q within a thousandth of p: the differences are exact, so what is left is off by what the weights are (5 x 2^-26 of p) as a
    share of all that is left."""
    c = Case(v, [1] * (8 if v < 50000 else 40), noise=0.0, key=("nearly", str(f))).filters(**f)
    g = np.random.default_rng(v)
    names = dict(top_k="k", top_p="p")
    for i in range(c.n):
        r = c.starts[i]
        p = ref.distribution(c.logits[r], **{names[k]: x[i].item() for k, x in c.f.items()})
        c.q[r] = np.clip(p * (1 + 1e-3 * g.uniform(-1, 1, v)), 0, 1)
        c.q[r, c.drafts[r]] = 1.0                             # refused
    c.u[:] = np.float32(0.9999)
    t, n = (x.cpu().numpy() for x in c.run(mq))
    for i in range(c.n):
        borders(c, t, n, i, 2.0 ** -23 / 2.0 ** -13)          # what is left adds up to 1 / 4 x 10^-3 > 2^-13


@pytest.mark.parametrize("v", [1000, 152064])
@pytest.mark.parametrize("starts", [[0, 3, 1, 9], [0, 9, 0, 9], [0, 4, 3, 9]])
def test_starts_that_overlap(mq, v, starts):
    """A row of two sequences, of one of them the last, whose draft is no token: refused as a whole, nothing read for it."""
    import torch
    c = Case(v, [2, 2, 2], key="overlap")
    c.drafts[:] = [-1, -2 ** 31, v, 2 ** 31 - 1, -1, 5, -1, v, -1]
    for f in (dict(), dict(top_p=0.9)):
        c.filters(**f)
        for _ in range(20):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            t, n = c.run(mq, starts=dev(np.int32(starts)), status=status)
            assert int(status) == 1 and (t == -9).all() and (n == -9).all()


@pytest.mark.parametrize("v", [50257, 131071, 152064])
@pytest.mark.parametrize("probs", [True, False, "ones"])
def test_many_rows_tokens_at_the_ends_of_chunks(mq, v, probs):
    """All of a row in one to three tokens beside the borders of 8192: rows that begin anywhere among 16 bytes; what is left of p,
    p, and p itself where nothing is left."""
    g = np.random.default_rng(v)
    c = Case(v, [1, 0, 2, 1] * 5, probs is not False, key=("chunk ends", str(probs)))
    c.logits[:] = -60.0
    for r in range(c.rows):
        at = 8192 * int(g.integers(1, v // 8192 + 1)) + np.arange(-2, 2)[r % 4] + np.array([0, 1, 5])[:1 + r // 4 % 3]
        c.logits[r, at] = g.uniform(-2, 0, len(at))
        c.drafts[r] = at[0] if r % 2 else 7
    c.u[:] = np.float32(1 - 2.0 ** -24 if probs == "ones" else 0.5)
    if probs:
        c.q[:] = 1.0 if probs == "ones" else 0.0
        c.q[np.arange(c.rows), c.drafts] = 1.0
    c.u_draw = np.resize(np.float32([0.5, 0.0, 1 - 2.0 ** -24, 0.25, 0.9]), c.n)
    t, n = (x.cpu().numpy() for x in c.run(mq))
    for i in range(c.n):
        borders(c, t, n, i)
