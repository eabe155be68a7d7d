"""mq_attn_decode on inputs whose results are known to a few roundings: every
cached token counts once wherever tiles, rounds, shares and windows end, and no
part of a query or of a weight is missing.  The bounds are of oracle.decode
(exact_mean_bound, TwoTokens.bound); that a lost token or part breaks them is
tested on the CPU in test_attention_checks.py.  And forms of a call that the
other tests leave out: sequences named by many rows, strided q8 pages, groups of
more than 8 heads in every type."""
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
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def stored(x, kv, shifts=None):
    """Pages [n, heads, ps, d] of float32 values that the type holds exactly (NaN: a place that nobody may use)
    as the cache's tensor; shifts: q8's scales are 2^-shift."""
    import torch
    if kv != "q8":
        return dev(x).to(torch.float16 if kv == "f16" else torch.bfloat16)
    n, h, ps, d = x.shape
    b = x.reshape(n, h, ps, d // 32, 32)
    scale = np.where(np.isnan(b[..., 0]), np.nan, 1.0 if shifts is None else 2.0 ** -shifts).astype(np.float16)
    with np.errstate(invalid="ignore"):
        codes = np.nan_to_num(b / scale[..., None].astype(np.float32), nan=77).astype(np.int8)
    return dev(np.concatenate([codes.reshape(n, h, -1).view(np.uint8), scale.reshape(n, h, -1).view(np.uint8)], -1))


class Rows:
    """Sequences of given lengths in a cache of shuffled pages; all places behind them are NaN."""

    def __init__(self, g, kv, d, hkv, ps, lens, fill):
        """fill(length) -> keys and values [hkv, length, d] of a sequence"""
        self.kv, self.d, self.hkv, self.ps = kv, d, hkv, ps
        need = [max(0, -(-int(n) // ps)) for n in lens]
        self.n_pages, self.width = sum(need) + 2, max(1, max(need))
        order = g.permutation(self.n_pages - 1)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        k, v = (np.full((self.n_pages, hkv, ps, d), np.nan, np.float32) for _ in range(2))
        self.keys, self.values, at = [], [], 0
        for i, n in enumerate(lens):
            kk, vv = fill(max(0, int(n)))
            self.keys.append(kk), self.values.append(vv)
            self.table[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
            for j in range(need[i]):
                m = min(ps, int(n) - j * ps)
                k[self.table[i, j], :, :m] = kk[:, j * ps:j * ps + m]
                v[self.table[i, j], :, :m] = vv[:, j * ps:j * ps + m]
        self.k, self.v = k, v

    def cache(self, mq, shifts=None):
        return mq.MQKVCache(self.kv, self.n_pages, self.ps, self.hkv, self.d, k=stored(self.k, self.kv, shifts),
                            v=stored(self.v, self.kv, shifts))


def whole_numbers(g, hkv, d):
    def fill(n):
        return (g.integers(lo, 128, (hkv, n, d)).astype(np.float32) for lo in (-3, -127))
    return fill


BORDERS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 0, -1, 255, 256, 257, 383, 385, 4095,
           4096, 4097, 2047, 2049, 6144, 6145]


def check_means(rows, out, hq, lens, window=0, seq=None, untouched=7.0):
    got = out.cpu().numpy().reshape(len(lens), rows.hkv, hq // rows.hkv, rows.d).astype(np.float64)
    for i, n in enumerate(lens):
        if n < 0:
            assert np.all(got[i] == untouched), i
            continue
        v = rows.values[i if seq is None else seq[i]][:, max(0, n - window) if window else 0:n].astype(np.float64)
        want = v.sum(1) / v.shape[1] if n else np.zeros((rows.hkv, rows.d))
        assert np.all(np.abs(got[i] - want[:, None]) <= ref.exact_mean_bound(want)[:, None]), (i, n)


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("lens,ps,window", [(BORDERS, 16, 0), (BORDERS, 48, 0), (BORDERS, 16, 200), ([20001], 64, 0),
                                            ([70001], 16, 0), ([9001, 3, 8193, 6145], 32, 4095),
                                            ([1000, 1500] * 20, 16, 0)])
def test_every_token_counts_once(mq, kv, d, lens, ps, window):
    """Queries of zero over whole numbers: each result is a mean that one token more, less or twice would change."""
    import torch
    g, hq, hkv = synth.rng("every token", kv, d, len(lens), ps, window), 6, 2
    rows = Rows(g, kv, d, hkv, ps, lens, whole_numbers(g, hkv, d))
    out = torch.full((len(lens), hq * d), 7.0, device="cuda")
    mq.mq_attn_decode(rows.cache(mq), torch.zeros_like(out), dev(np.int32(lens)), dev(rows.table), 0.1, out=out,
                      window=window)
    torch.cuda.synchronize()
    check_means(rows, out, hq, lens, window)


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("nt", [40, 1000, 1024, 1100])
def test_sequences_named_by_many_rows(mq, kv, nt):
    """seq in the launches of more than 32 rows, and of more than are shared out: rows in any order, several of one
    sequence with lengths of their own, empty and padding ones, and their q8 planes."""
    import torch
    g, hq, hkv, d, n_seq = synth.rng("many rows", kv, nt), 4, 2, 64, 37
    full = [int(x) for x in g.integers(1, 600, n_seq)]
    full[5] = 5000
    rows = Rows(g, kv, d, hkv, 16, full, whole_numbers(g, hkv, d))
    seq = g.integers(0, n_seq, nt).astype(np.int32)
    lens = np.array([g.integers(0, full[s] + 1) for s in seq], np.int32)
    lens[::17] = -1
    lens[3::29] = 0
    nb = mq.mq_q8_bytes(hq * d)
    plane = torch.full((nt * nb,), 0x55, dtype=torch.uint8, device="cuda")
    out = torch.full((nt, hq * d), 7.0, device="cuda")
    mq.mq_attn_decode(rows.cache(mq), torch.zeros_like(out), dev(lens), dev(rows.table), 0.1, out=out, seq=dev(seq),
                      q8=plane)
    torch.cuda.synchronize()
    check_means(rows, out, hq, lens, seq=seq)
    got = plane.view(nt, nb).cpu()
    for i in range(0, nt, 7):
        if lens[i] < 0:
            assert (got[i] == 0x55).all()
            continue
        want = mq.mq_quantize_q8(out[i].clone()).cpu().numpy()
        for a, b in zip(mq.mq_q8_unpack_host(got[i].numpy(), hq * d), mq.mq_q8_unpack_host(want, hq * d)):
            assert np.array_equal(a, b), i


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("of", ["queries", "weights"])
def test_no_part_is_missing(mq, kv, d, of):
    """Two tokens alone matter, so that every bit of a query or of a weight shows, at every place of a head and in
    every row of a tile."""
    import torch
    g, hq, hkv, nt = synth.rng("parts", kv, d, of), 10, 2, 64
    lens = g.integers(17, 200, nt)
    rng = np.random.default_rng(int(g.integers(1 << 30)))
    cases = [ref.TwoTokens(rng, hq, hkv, d, int(n), of) for n in lens]
    it = iter(cases)

    def fill(n):
        t = next(it)
        return t.k.astype(np.float32), t.v.astype(np.float32)
    rows = Rows(g, kv, d, hkv, 16, lens, fill)
    shifts = g.integers(0, 6, (rows.n_pages, hkv, 16, d // 32)).astype(np.float64)
    q = np.stack([t.q.reshape(-1) for t in cases])
    out = torch.empty((nt, hq * d), device="cuda")
    mq.mq_attn_decode(rows.cache(mq, shifts), dev(q), dev(lens.astype(np.int32)), dev(rows.table), 1.0, out=out)
    torch.cuda.synchronize()
    got = out.cpu().numpy().reshape(nt, hq, d).astype(np.float64)
    for i, t in enumerate(cases):
        want = ref.attention(t.q, t.k, t.v, 1.0)
        ratio = np.abs(got[i] - want) / t.bound(want, kv != "bf16")
        assert ratio.max() <= 1, (i, ratio.max())


@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("hq,hkv", [(9, 1), (16, 1), (20, 2), (33, 3)])
def test_groups_of_more_than_eight_heads(mq, kv, hq, hkv):
    from test_gpu_attn_decode import Case
    c = Case(mq, kv, 128, hq, hkv, 32, [1, 70, 1500, 5000])
    c.check(c.run())


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
def test_strided_pages(mq, kv):
    """Keys and values of a page side by side in one array, with room between pages."""
    import torch
    from test_gpu_attn_decode import Case
    c = Case(mq, kv, 96, 8, 2, 48, [500, 33, 0, 2100])
    want = c.run()
    flat = [t.reshape(c.n_pages, -1).view(torch.uint8) for t in (c.k, c.v)]
    page = flat[0].shape[1]
    both = torch.full((c.n_pages, 2 * page + 64), 0xff, dtype=torch.uint8, device="cuda")
    both[:, :page], both[:, page:2 * page] = flat
    views = []
    for at in (0, page):
        t = both[:, at:at + page]
        t = t.view(c.k.dtype) if kv != "q8" else t
        views.append(t.unflatten(1, c.k.shape[1:]))
    c.cache = mq.MQKVCache(kv, c.n_pages, 48, 2, 96, k=views[0], v=views[1])
    assert torch.equal(c.run(), want)


def test_a_few_rows_of_one_sequence_in_any_type(mq):
    """The tokens of a speculative step over each type, with the query heads of two groups."""
    from test_gpu_attn_decode import Case
    for kv in ("f16", "bf16", "q8"):
        c = Case(mq, kv, 128, 20, 2, 16, [0, 3003, 0, 0])
        seq = np.array([1, 1, 1, 1], np.int32)
        c.lens = np.array([3000, 3001, 3002, 3003], np.int32)
        c.check(c.run(seq=dev(seq)), seq=seq)
