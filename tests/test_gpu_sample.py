"""mq_sample against a plain 64-bit reference.

Tokens have to be equal unless the draw falls within 2^-22 of a border of the
reference's token.  A weight, in units of 2^-26 and relative to 2^f >= 0.707:
its exponent's fraction 0.7, the series' last sum 1, the product with the
fraction 1, the terms before 0.5: 4.5, under 5.  Sums of weights are no worse, so
a share of the kept sum is off by at most 10 units, 2^-22.6.
Probabilities: the same 10 units and the result's rounding 2^-24: 14 units,
under 2^-22; and 2^-42 of the largest weight absolutely."""
import numpy as np
import pytest

import synth
from oracle import decode as ref

pytestmark = pytest.mark.gpu


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
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(mq, logits, u, t=None, k=None, p=None, m=None, **more):
    import torch
    n = len(logits)
    f = lambda x, ty: None if x is None else dev(np.broadcast_to(np.asarray(x, ty), (n,)).copy())  # noqa: E731
    prob = torch.full((n,), -1.0, device="cuda")
    lg = logits if isinstance(logits, torch.Tensor) else dev(logits)
    tok = mq.mq_sample(lg, f(u, np.float32), temperature=f(t, np.float32), top_k=f(k, np.int32),
                       top_p=f(p, np.float32), min_p=f(m, np.float32), prob=prob, **more)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), prob.cpu().numpy()


def check(logits, u, got, t=1.0, k=0, p=1.0, m=0.0):
    n = len(logits)
    b = lambda x: np.broadcast_to(np.asarray(x), (n,))  # noqa: E731
    f32 = lambda x: float(np.float32(x))  # noqa: E731
    close = 0
    for i in range(n):
        tok, pr, kept, gap = ref.sample(logits[i], f32(b(u)[i]), f32(b(t)[i]), int(b(k)[i]), f32(b(p)[i]), f32(b(m)[i]))
        if got[0][i] != tok:
            assert gap < 2.0 ** -22 and kept[got[0][i]], (i, got[0][i], tok, gap)
            close += 1
            continue
        assert abs(got[1][i] - pr) <= pr * 2.0 ** -22 + 2.0 ** -42, (i, got[1][i], pr)
    assert close <= 1 + n // 50


def rows(key, n, v, std=2.0, peaks=0):
    g = synth.rng("sample", key, n, v)
    x = (synth.normal(g, n * v) * np.float32(std)).reshape(n, v)
    for i in range(n if peaks else 0):
        x[i, g.integers(0, v, peaks)] = 6 + 4 * synth.normal(g, peaks)
    return x.astype(np.float32), g.uniform(0, 1, n).astype(np.float32)


FILTERS = [dict(), dict(t=0.7), dict(k=1), dict(k=40), dict(k=5000), dict(p=0.9), dict(p=0.1), dict(m=0.05),
           dict(t=0.8, k=40, p=0.95, m=0.05), dict(k=3000, p=0.9), dict(t=1.7, p=0.99, m=1e-4), dict(t=0.0),
           dict(k=20, m=0.3), dict(p=0.0), dict(m=1.0), dict(m=2.0), dict(t=5.0, k=100, p=0.5)]


@pytest.mark.parametrize("f", FILTERS, ids=lambda f: "-".join(f"{k}{v}" for k, v in f.items()) or "plain")
@pytest.mark.parametrize("v,peaks", [(1, 0), (5, 0), (1000, 8), (4099, 0), (50257, 16)])
def test_filters(mq, f, v, peaks):
    x, u = rows("filters", 9, v, 2.5, peaks)
    check(x, u, run(mq, x, u, **f), **f)


@pytest.mark.parametrize("n,f", [(1, dict(t=0.8, k=40, p=0.95, m=0.05)), (3, dict(p=0.9)), (17, dict(k=1000, p=0.8)),
                                 (64, dict(p=0.9, t=1.5)), (200, dict(m=0.02))])
def test_the_152064_token_head(mq, n, f):
    x, u = rows("head", n, 152064, 2.5, 0 if n > 3 else 64)
    sub = slice(None) if n <= 17 else slice(0, n, 13)
    tok, pr = run(mq, x, u, **f)
    check(x[sub], u[sub], (tok[sub], pr[sub]), **f)


def test_the_largest_vocabulary(mq):
    x, u = rows("largest", 2, mq.MQ_SAMPLE_MAX_VOCAB, 2.0)
    for f in (dict(p=0.95), dict(k=77)):
        check(x, u, run(mq, x, u, **f), **f)


def test_parameters_of_each_row(mq):
    x, u = rows("each", 12, 3001, 2.0, 8)
    t = np.array([0, 0.5, 1, 2, 0.9, 1, 1, 1, 3, 1e-3, 1e3, 1], np.float32)
    k = np.array([0, 5, 0, 50, 3001, 4000, -1, 1, 2, 0, 7, 0], np.int32)
    p = np.array([1, 0.9, 0.5, 1, 0.99, 0.3, 1.5, 1, 0.9, 0.9, 0.9, -1], np.float32)
    m = np.array([0, 0, 0.1, 0, 0, 0, 0.01, 0, 0, 0, 0.9, 0], np.float32)
    check(x, u, run(mq, x, u, t=t, k=k, p=p, m=m), t=t, k=k, p=p, m=m)


@pytest.mark.parametrize("f", [dict(), dict(k=4), dict(k=1500), dict(p=0.5), dict(k=3000, p=0.25), dict(m=0.5), dict(t=0.0)])
@pytest.mark.parametrize("kind", ["equal", "two levels", "ties at the border", "near", "minus zero"])
def test_ties_go_to_the_lowest_index(mq, f, kind):
    """Equal logits by the thousand: bins of more tokens than one list are
    narrowed down to one place in the order."""
    v = 20011
    x = np.zeros((4, v), np.float32)
    g = synth.rng("ties", kind)
    if kind == "two levels":
        x[:, g.integers(0, v, 9000)] = 1.0
    elif kind == "ties at the border":
        x[:] = np.round(synth.normal(g, 4 * v).reshape(4, v) * 2) / 2
    elif kind == "near":
        x[:] = 1.0 + g.integers(0, 3, (4, v)) * np.float32(2.0 ** -23)
    elif kind == "minus zero":
        x[:, ::2] = -0.0
    u = np.array([0.0, 0.2500001, 0.7123, 0.9999999], np.float32)
    check(x, u, run(mq, x, u, **f), **f)


def test_equal_logits_have_exact_borders(mq):
    """Weights of 1 are exact: 8 equal tokens, top-p of one half keeps four of
    them, and u * 4 falls on borders exactly."""
    x = np.zeros((5, 8), np.float32)
    u = np.array([0.0, 0.25, 0.5, 0.75, 0.999], np.float32)
    tok, pr = run(mq, x, u, p=0.5)
    assert tok.tolist() == [0, 1, 2, 3, 3] and np.all(pr == 0.25)
    tok, pr = run(mq, x, u)
    assert tok.tolist() == [0, 2, 4, 6, 7] and np.all(pr == 0.125)


def test_infinities_and_nan(mq):
    inf, nan = np.inf, np.nan
    x = np.full((9, 600), -inf, np.float32)
    x[1, 77] = -5.0
    x[2] = nan
    x[3, :] = nan
    x[3, 5], x[3, 9] = 1.0, 1.0
    x[4, 3:6] = 0.0
    x[5, [10, 20]] = inf
    x[6] = 3.0e38 * np.where(np.arange(600) % 2, 1, -1)
    x[7, 599] = -3.4e38
    x[8, :] = 0.0
    x[8, 44] = nan
    u = np.array([.5, .5, .5, .75, .5, .6, .3, .5, .999], np.float32)
    for f in (dict(), dict(k=2), dict(p=0.9), dict(k=100, p=0.9, m=0.1), dict(t=0.0), dict(t=1e-30, p=0.9), dict(t=1e30, k=3)):
        got = run(mq, x, u, **f)
        assert got[0][0] == -1 and got[1][0] == 0.0 and got[0][2] == -1
        check(x, u, got, **f)


@pytest.mark.parametrize("t", [np.inf, 1e-38, 1e-45, -1.0, np.nan])
def test_temperatures_at_the_ends(mq, t):
    """Infinite: every finite logit weighs the same.  Vanishing, negative and
    NaN: the largest (equal ones share the draw where the temperature is positive)."""
    x, u = rows("ends", 6, 900, 2.0)
    x[2, 40:] = -np.inf
    x[4, [7, 300]] = 20.0
    for f in (dict(), dict(k=30), dict(p=0.5), dict(m=0.5)):
        got = run(mq, x, u, t=t, **f)
        if np.isinf(t):
            kept = np.isfinite(x)
            if "k" in f or "p" in f:
                order = np.argsort(-x, kind="stable", axis=1)
                n = np.full(6, f["k"]) if "k" in f else np.ceil(kept.sum(1) * 0.5).astype(int)
                kept = np.zeros_like(kept)
                for i in range(6):
                    kept[i, order[i, :n[i]]] = True
            for i in range(6):
                at = np.flatnonzero(kept[i])
                assert got[0][i] == at[int(np.float64(np.float32(u[i])) * len(at))]
                assert abs(got[1][i] * len(at) - 1) < 2.0 ** -22
        else:
            check(x, u, got, t=t if t > 0 else 0.0, **f)


def test_u_outside_its_range(mq):
    x, _ = rows("u", 4, 700)
    u = np.array([-1.0, 1.0, 2.0, np.nan], np.float32)
    tok, pr = run(mq, x, u, k=3)
    kept = [np.sort(np.argsort(-r, kind="stable")[:3]) for r in x]
    assert tok.tolist() == [kept[0][0], kept[1][-1], kept[2][-1], kept[3][0]]


def test_draws_follow_the_kept_distribution(mq):
    """One row, u on a grid of 4096: every token comes as often as its share says."""
    x, _ = rows("grid", 1, 500, 2.0)
    n = 4096
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    tok, pr = run(mq, np.repeat(x, n, 0), u, k=50, p=0.9)
    _, _, kept, _ = ref.sample(x[0], 0.0, 1.0, 50, float(np.float32(0.9)))
    assert np.all(np.diff(tok) >= 0) and set(tok) <= set(np.flatnonzero(kept))
    w = np.where(kept, np.exp(x[0].astype(np.float64) - x[0].max()), 0)
    share = w / w.sum()
    assert np.all(np.abs(np.bincount(tok, minlength=500) - share * n) <= 1.001)
    assert np.all(np.abs(pr - share[tok]) <= share[tok] * 2.0 ** -22)


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_strides_and_unaligned_rows(mq, offset):
    import torch
    v = 3001
    x, u = rows("stride", 5, v, 2.0, 8)
    want = run(mq, x, u, t=0.9, k=30, p=0.9)
    wide = torch.full((5, v + 9), 50.0, device="cuda")
    wide[:, offset:offset + v] = dev(x)
    got = run(mq, wide[:, offset:offset + v], u, t=0.9, k=30, p=0.9)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_the_split_over_ctas_does_not_matter(mq):
    """The same row alone (many CTAs) and in a batch (few): the same bits."""
    x, u = rows("split", 300, 30011, 2.5)
    f = dict(t=1.2, k=2500, p=0.95, m=1e-3)
    tok, pr = run(mq, x, u, **f)
    for i in range(0, 300, 37):
        t1, p1 = run(mq, x[i:i + 1], u[i:i + 1], **f)
        assert t1[0] == tok[i] and p1[0] == pr[i]


def test_captured_replayed_and_on_another_stream(mq):
    import torch
    x, u = rows("graph", 3, 20000, 2.0, 16)
    want, wp = run(mq, x, u, t=0.9, k=50, p=0.9)
    lg, ud = torch.zeros(3, 20000, device="cuda"), torch.zeros(3, device="cuda")
    t, p = torch.full((3,), 0.9, device="cuda"), torch.full((3,), 0.9, device="cuda")
    k = torch.full((3,), 50, dtype=torch.int32, device="cuda")
    tok, pr = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, device="cuda")
    args = dict(temperature=t, top_k=k, top_p=p, token=tok, prob=pr)
    st = torch.cuda.Stream()
    for pdl in (False, True):
        mq.mq_set_pdl(pdl)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            for _ in range(3):
                mq.mq_sample(lg, ud, **args)
        mq.mq_set_pdl(False)
        lg.copy_(dev(x)), ud.copy_(dev(u)), tok.zero_(), pr.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert np.array_equal(tok.cpu().numpy(), want) and np.array_equal(pr.cpu().numpy(), wp)
        tok.zero_()
        torch.cuda.synchronize()
        mq.mq_sample(lg, ud, stream=st, **args)
        st.synchronize()
        assert np.array_equal(tok.cpu().numpy(), want)


def test_refusals(mq):
    import torch
    x, u = torch.zeros(2, 100, device="cuda"), torch.zeros(2, device="cuda")
    mq.mq_sample(x, u)
    for bad in (dict(logits=x.half()), dict(logits=x.t()), dict(u=u[:1]), dict(u=u.double()), dict(u=u.cpu()),
                dict(top_k=u), dict(temperature=u[:1]), dict(token=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(prob=torch.zeros(3, device="cuda"))):
        a = dict(logits=x, u=u)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            mq.mq_sample(a.pop("logits"), a.pop("u"), **a)
    for shape in ((0, 100), (2, 0)):
        with pytest.raises(mq.MQError) as e:
            mq.mq_sample(torch.zeros(shape, device="cuda"), torch.zeros(shape[0], device="cuda"))
        assert e.value.status == mq.MQ_ERR_SHAPE
    wide = torch.zeros(1, mq.MQ_SAMPLE_MAX_VOCAB + 1, device="cuda")
    with pytest.raises(mq.MQError) as e:
        mq.mq_sample(wide, u[:1])
    assert e.value.status == mq.MQ_ERR_SHAPE


def test_a_token_made_for_another_stream_is_of_its_memory(mq):
    """Not of what the current stream has just given back, which its kernels may still use."""
    import torch
    x, u = torch.zeros(2, 100, device="cuda"), torch.zeros(2, device="cuda")
    given_back = torch.empty(2, dtype=torch.int32, device="cuda").data_ptr()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    token = mq.mq_sample(x, u, stream=st)
    st.synchronize()
    assert token.data_ptr() != given_back and token.tolist() == [0, 0]


@pytest.mark.parametrize("kind", ["spread", "ties", "many ties", "near", "one place", "few finite", "infinite"])
@pytest.mark.parametrize("v", [700, 4100, 9001, 20011, 152064])
def test_short_top_k(mq, v, kind):
    """Top-k small enough to be chosen from what each part of a row sends, up to and past its limits:
    parts with nothing, ties within and across parts, fewer tokens than k."""
    ks = [2, 3, 40, 55, 56, 57, 111, 112, 113, 223, 224, 225, 255, 256, 257, 300, 600, v - 1]
    x, u = rows("short " + kind, len(ks), v)
    g = synth.rng("short", kind, v)
    if kind == "ties":                       # some 55 equal ones in every sixteenth, places differ alone
        x[:, :: max(v // 880, 1)] = 20.0
    elif kind == "many ties":                # more than any part may send
        x[:, ::5] = 20.0
    elif kind == "near":                     # the order lies in the last bits
        at = g.choice(v, min(v, 800), replace=False)
        x[:, at] = 20.0 + g.integers(0, 3, (len(ks), len(at))) * np.float32(2.0 ** -19)
    elif kind == "one place":                # all of them in one part
        x[:, v // 2:v // 2 + 300] += 30.0
    elif kind == "few finite":
        keep = g.choice(v, 37, replace=False)
        y = np.full_like(x, -np.inf)
        y[:, keep] = x[:, keep]
        x = y
    elif kind == "infinite":
        x[:, g.choice(v, 3, replace=False)] = np.inf
    for more in (dict(), dict(p=0.9, m=0.05, t=0.7)):
        for a in range(0, len(ks), 6):       # 6 rows: the widest split of each
            s = slice(a, a + 6)
            check(x[s], u[s], run(mq, x[s], u[s], k=ks[s], **more), k=ks[s], **more)
    check(x[:1], u[:1], run(mq, x[:1], u[:1], k=40, p=0.95), k=40, p=0.95)


@pytest.mark.parametrize("kind", ["spread", "flat", "ties", "ties at the end", "near", "one place", "half infinite"])
@pytest.mark.parametrize("v", [2100, 9001, 50257, 152064])
def test_longer_top_k(mq, v, kind):
    """Top-k whose tokens one CTA takes from all of them, up to and past what it has room for; top-p among
    them ends anywhere; ties by the hundred, within and across parts."""
    ks = [300, 511, 513, 1000, 1500, 1990, 2040, 2046, 2047, 2048, 2060, 4000]
    x, u = rows("longer " + kind, len(ks), v, 0.5 if kind == "flat" else 2.5, 40 if kind == "one place" else 0)
    g = synth.rng("longer", kind, v)
    if kind == "ties":                       # 700 equal ones above the rest
        x[:, g.choice(v, 700, replace=False)] = 20.0
    elif kind == "ties at the end":          # top-k ends among 1900 equal ones
        x[:, g.choice(v, 1900, replace=False)] = 20.0
        x[:, g.choice(v, 100, replace=False)] = 20.5
    elif kind == "near":                     # one bin, the order in the last bits
        x[:, g.choice(v, 1800, replace=False)] = 20.0 + g.integers(0, 5, 1800) * np.float32(2.0 ** -19)
    elif kind == "one place":                # nearly all of them in one part
        x[:, v // 3:v // 3 + 1700] += 15.0
    elif kind == "half infinite":
        x[:, g.choice(v, v // 2, replace=False)] = -np.inf
    for more in (dict(), dict(p=0.9), dict(p=0.3, t=0.5), dict(m=0.2, t=2.0), dict(p=0.97, m=0.01, t=1.3)):
        for a in range(0, len(ks), 6):
            s = slice(a, a + 6)
            check(x[s], u[s], run(mq, x[s], u[s], k=ks[s], **more), k=ks[s], **more)


@pytest.mark.parametrize("v", [900, 9001, 50257, 152064])
@pytest.mark.parametrize("kind", ["peaks", "few", "ties", "room", "infinite"])
def test_small_nucleus(mq, v, kind):
    """Top-p alone, of one token to some thousands: peaks, ties by the hundred, a plateau, infinities."""
    x, u = rows("nucleus " + kind, 12, v, 1.0, 30 if kind == "peaks" else 0)
    g = synth.rng("nucleus", kind, v)
    for i in range(len(x)):
        if kind == "few":
            x[i, g.choice(v, 5, replace=False)] = 25.0 + i
        elif kind == "ties":
            x[i, g.choice(v, min(v // 2, 100 + 170 * i), replace=False)] = 20.0
        elif kind == "room":                 # 1500 to 2600 tokens within an octave, above all others
            n = min(v - 10, 1500 + 100 * i)
            x[i, g.choice(v, n, replace=False)] = 30.0 - g.uniform(0, 0.7, n)
        elif kind == "infinite":
            x[i, g.choice(v, 1 + i % 3, replace=False)] = np.inf
    for more in (dict(p=0.5), dict(p=0.9), dict(p=0.999, t=0.6), dict(p=0.95, m=0.1, t=1.4), dict(p=1e-6), dict(p=0.9999999)):
        for a in (0, 6):
            s = slice(a, a + 6)
            check(x[s], u[s], run(mq, x[s], u[s], **more), **more)


@pytest.mark.parametrize("n", [1, 2, 40])
def test_an_estimate_that_stops_short(mq, n):
    """The sum by bins of 1/64 octave takes the first token for the whole nucleus; by the weights, the next ones,
    five octaves below, are needed too: equal, at the heavy end of their bin, n of the 64 by their index."""
    v, w = 5000, 2.0 ** -(5 - 0.45 / 64)
    x = np.full((1, v), -60.0, np.float32)
    x[0, 7] = 0.0
    tail = np.sort(synth.rng("short", n).choice(np.arange(10, v), 64, replace=False))
    x[0, tail] = np.float32(-(5 - 0.45 / 64) * np.log(2))
    p = (1 + (n - 0.5) * w) / (1 + 64 * w) if n > 1 else (1 + 0.02 * w) / (1 + 64 * w)
    for u in (0.0, 0.5, 0.9, 0.99, 0.9999):
        got = run(mq, x, np.array([u], np.float32), p=p)
        tok, pr, kept, _ = ref.sample(x[0], float(np.float32(u)), p=float(np.float32(p)))
        assert kept.sum() == n + 1
        check(x, np.array([u], np.float32), got, p=p)


@pytest.mark.parametrize("t", [1e-28, 1e-31, 1e-33, 1e-36])
def test_logits_as_small_as_their_temperature(mq, t):
    """What counts is the quotient: logits and temperature of vanishing size draw as their multiples do."""
    x, u = rows("vanishing", 6, 3001, 2.0, 8)
    x = (x.astype(np.float64) * t).astype(np.float32)
    for f in (dict(), dict(k=40), dict(p=0.9), dict(k=1500, p=0.95), dict(m=0.05)):
        check(x, u, run(mq, x, u, t=t, **f), t=t, **f)
