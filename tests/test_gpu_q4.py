"""The 4-bit cache on the GPU: the append's codes and scales, byte for byte where its input is exact, and the
attention over it against a plain 64-bit reference over the same bytes.

Tolerance of the attention: oracle.decode.attention_bound, as for the other types: the codes less 8 are exact in the
products."""
import math

import numpy as np
import pytest

import synth
from oracle import decode as ref
from test_gpu_attn_decode import Case, RAGGED
from test_gpu_rope_append import UNIT
from test_gpu_rope_append import Case as AppendCase

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


# ------------------------------------------------------------------ append
class Append(AppendCase):
    def run(self, mq, kv=None, **more):
        import torch
        kv = kv or mq.MQKVCache("q4", self.n_pages, self.ps, self.hkv, self.d)
        kv.k.fill_(0x99), kv.v.fill_(0x99)
        q_out = torch.full((self.rows, self.hq * self.d), 5.0, device="cuda")
        args = dict(q_out=q_out, rope=mq.mq_rope_table(self.freqs) if self.r else None, style=self.style,
                    q_bias=dev(self.qb), k_bias=dev(self.kb), v_bias=dev(self.vb), q_gain=dev(self.qg),
                    k_gain=dev(self.kg), eps=1e-6)
        args.update(more)
        out = mq.mq_rope_append(kv, dev(self.q), dev(self.k), dev(self.v), dev(self.pos), dev(self.table), **args)
        torch.cuda.synchronize()
        return out, kv

    def check(self, out, kv, seq=None):
        """A value is off by what f32 loses before it, half a step (a whole one where the range ends at 7), and the
        scale's rounding to fp16, 2^-11 of up to 8 steps."""
        seq = self.seq if seq is None else seq
        (q, qm), (k, km), (v, vm) = self.want()
        got = out.cpu().numpy().reshape(self.rows, self.hq, self.d)
        live = self.pos >= 0
        assert np.all(np.abs(got - q)[live] <= UNIT * qm[live]) and np.all(got[~live] == 5.0)
        for t, want, mag, keys in ((kv.k, k, km, True), (kv.v, v, vm, False)):
            codes, scales = ref.unpack_q4(t.cpu().numpy(), self.ps, self.d, keys)
            vals, _ = ref.q4_values(codes, scales)
            written = np.zeros(vals.shape, bool)
            for i in np.flatnonzero(live):
                page, slot = self.table[seq[i], self.pos[i] // self.ps], self.pos[i] % self.ps
                blocks = want[i].reshape(self.hkv, -1, 32)
                step = np.repeat(np.abs(blocks).max(-1) / 8, 32, -1)
                far = np.where(np.abs(want[i]) > 7.4 * step, 1.0, 0.5)
                tol = UNIT * mag[i] + step * (far + 8 * 2.0 ** -11 + 1e-4)
                assert np.all(np.abs(vals[page, :, slot] - want[i]) <= tol), i
                # the scale itself, but for which of two nearly equal values leads
                d = np.abs(scales[page, :, slot].astype(np.float64))
                assert np.all(np.abs(d - np.abs(blocks).max(-1) / 8) <= d * 2.0 ** -11 + UNIT * mag[i].max() + 2.0 ** -25)
                written[page, :, slot] = True
            assert np.all(codes[~written] == 9)
            assert np.all(scales.view(np.uint16)[~written[..., ::32]] == 0x9999)


@pytest.mark.parametrize("d,r,style", [(128, 128, "half"), (128, 128, "pairs"), (64, 32, "half"), (64, 64, "half"),
                                       (64, 64, "pairs"), (96, 96, "half"), (96, 48, "pairs"), (256, 128, "half"),
                                       (256, 256, "pairs"), (256, 256, "half"), (128, 0, "half"), (128, 8, "half")])
@pytest.mark.parametrize("bias,norm", [(False, False), (True, True)])
def test_append(mq, d, r, style, bias, norm):
    c = Append(5, 10, 2, d, r, style, "q4", 16, bias, norm, [0, 1, 15, 16, 4097], pad=2)
    c.check(*c.run(mq))


@pytest.mark.parametrize("d,r,style", [(128, 128, "half"), (128, 24, "half"), (96, 64, "pairs"), (64, 64, "half"),
                                       (64, 64, "pairs"), (256, 256, "half")])
def test_append_of_many_rows(mq, d, r, style):
    nt = (1250 if d > 64 or style == "half" else 19600) // 15 + 9
    c = Append(nt, 9, 3, d, r, style, "q4", 48, True, True, [(i * 37) % 500 for i in range(nt)], pad=3)
    c.check(*c.run(mq))


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("nt", [3, 700])
def test_append_is_the_quantization_byte_for_byte(mq, d, nt):
    """Values without a rotation reach the quantizer as they are: zeros, equal magnitudes, vanishing, huge, infinite and
    NaN blocks among them."""
    c = Append(nt, 8, 4, d, 0, "half", "q4", 16, False, False, [(i * 7) % 90 for i in range(nt)])
    for x in (c.k, c.v):
        b = x.reshape(nt, -1, 32)
        b[0, 0] = 0
        b[0, 1] = np.where(np.arange(32) % 2, 1.5, -1.5)
        b[1, 0] *= np.float32(1e-7)
        b[1, 1] *= np.float32(1e5)
        b[2, 0, 7] = np.inf
        b[2, 1, 31] = np.nan
        b[2, 2] = np.float32(3e-8)
        b[2, 3, 4] = -6e5
    out, kv = c.run(mq)
    for t, x, keys in ((kv.k, c.k, True), (kv.v, c.v, False)):
        codes, scales = ref.unpack_q4(t.cpu().numpy(), 16, d, keys)
        u, s = ref.quantize_q4(x.reshape(nt, 4, d))
        for i in range(nt):
            page, slot = c.table[i, c.pos[i] // 16], c.pos[i] % 16
            assert np.array_equal(codes[page, :, slot], u[i]), (i, keys)
            got, want = scales[page, :, slot], s[i]
            assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


# ------------------------------------------------------------------ attention
class Q4(Case):
    """Rows of given lengths over a cache whose unused places are codes of all kinds with NaN scales."""

    def __init__(self, mq, d, hq, hkv, ps, lens, key="", q_std=2.0, v_scale=1.0, k_shift=True):
        g = synth.rng("attn q4", d, hq, hkv, ps, len(lens), key)
        self.__dict__.update(kv="q4", d=d, hq=hq, hkv=hkv, ps=ps, lens=np.asarray(lens, np.int32), mq=mq)
        need = [max(0, -(-int(n) // ps)) for n in lens]
        self.n_pages, self.width = sum(need) + 2, max(1, max(need))
        order = g.permutation(self.n_pages - 1)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        used = np.zeros((self.n_pages, ps), bool)
        for i, c in enumerate(need):
            self.table[i, :c] = order[at:at + c]
            at += c
            for j in range(c):
                used[self.table[i, j], : min(ps, int(lens[i]) - j * ps)] = True
        shape = (self.n_pages, hkv, ps, d)
        rng = np.random.default_rng(int(g.integers(1 << 30)))
        k, v = (rng.standard_normal(shape, np.float32) for _ in range(2))
        if k_shift:
            k += rng.standard_normal((hkv, 1, d), np.float32)
        self.codes, self.scales = [], []
        for x in (k, v * np.float32(v_scale)):
            u, s = ref.quantize_q4(x)
            s[np.broadcast_to(~used[:, None, :, None], s.shape)] = np.nan
            self.codes.append(u), self.scales.append(s)
        self.q = (synth.normal(g, len(lens) * hq * d) * np.float32(q_std)).reshape(len(lens), hq * d)
        self.scale = 1 / math.sqrt(d)
        self.store()

    def store(self):
        self.k, self.v = (dev(ref.pack_q4(u, s, keys)) for u, s, keys in zip(self.codes, self.scales, (True, False)))
        self.cache = self.mq.MQKVCache("q4", self.n_pages, self.ps, self.hkv, self.d, k=self.k, v=self.v)

    def want(self, i, n, softcap=0.0, window=0, seq=None):
        row = self.table[i if seq is None else seq[i]]
        (k, km), (v, vm) = (tuple(ref.gather(x, row, n) for x in ref.q4_values(u, s))
                            for u, s in zip(self.codes, self.scales))
        scale = np.float32(self.scale).astype(float)
        first = max(0, n - window) if window else 0
        k, km, v, vm = (x[:, first:] for x in (k, km, v, vm))
        q = self.q[i].reshape(self.hq, self.d)
        want, parts = ref.attention(q, k, v, scale, softcap, parts=True)
        if parts is None:
            return want, np.zeros_like(want)
        qg = np.abs(q.astype(np.float64)).reshape(self.hkv, -1, self.d)
        mag = np.matmul(qg, km.transpose(0, 2, 1)) * abs(scale)
        return want, ref.attention_bound(want, (parts[0], mag, parts[2], vm), softcap)

    def check(self, out, softcap=0.0, window=0, rows=None, seq=None, lens=None):
        got = out.cpu().numpy().reshape(len(self.q), self.hq, self.d)
        lens = self.lens if lens is None else lens
        for i in range(len(self.q)) if rows is None else rows:
            n = int(lens[i])
            if n < 0:
                assert np.all(got[i] == 7.0)
                continue
            want, tol = self.want(i, n, softcap, window, seq)
            err = np.abs(got[i] - want)
            assert np.all(err <= tol), (i, n, err.max(), (err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("hq,hkv,ps", [(10, 2, 16), (4, 4, 48)])
def test_ragged_rows(mq, d, hq, hkv, ps):
    c = Q4(mq, d, hq, hkv, ps, RAGGED)
    c.check(c.run())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (8, 1), (9, 1), (16, 1), (20, 2), (33, 3)])
def test_head_groups(mq, hq, hkv):
    c = Q4(mq, 128, hq, hkv, 32, [1, 70, 1500])
    c.check(c.run())


@pytest.mark.parametrize("d,lens,ps", [(128, [4097], 16), (128, [20001], 64), (64, [70000], 4096),
                                       (128, [3000, 1, 2999, 64, 65], 16), (256, [9000, 777], 32), (96, [12345], 48)])
def test_long_rows_are_split_and_joined(mq, d, lens, ps):
    import torch
    c = Q4(mq, d, 10, 2, ps, lens)
    ws = mq.mq_attn_workspace(c.cache, 10, len(lens), max(lens))
    assert ws is not None
    out = c.run(ws=ws, max_len=max(lens))
    c.check(out)
    assert torch.equal(out, c.run(ws=ws, max_len=max(lens)))           # the order of sums is fixed
    assert not ws[: mq.mq_device_sms() * 4].any()                      # the counters in front are zero again


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 1024, 5000])
def test_windows(mq, window):
    """Tokens that left the window have NaN scales and are not used."""
    import torch
    lens = [1, 16, 99, 101, 1500, 4000, 0, -1]
    c = Q4(mq, 64, 6, 2, 16, lens)
    clean = [s.copy() for s in c.scales]
    for i, n in enumerate(lens):
        for j in range(max(0, n - window)):
            for s in c.scales:
                s[c.table[i, j // 16], :, j % 16] = np.nan
    c.store()
    out = c.run(window=window)
    assert torch.isfinite(out).all()
    c.scales = clean
    c.check(out, window=window)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("window,ps", [(1, 16), (17, 16), (100, 16), (100, 48), (1024, 16), (1000, 64)])
def test_pages_that_left_the_window_may_be_gone(mq, d, window, ps):
    """Only what a row sees needs a page: the entries before it name none, or one that does not exist."""
    import torch
    lens = [1, 16, 99, 101, 1500, 4000, 0, -1]
    c = Q4(mq, d, 6, 2, ps, lens)
    full = c.table.copy()
    for i, n in enumerate(lens):
        gone = max(0, n - window) // ps
        c.table[i, :gone] = np.where(np.arange(gone) % 2, -1, 2 ** 31 - 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.run(window=window, status=status)
    assert int(status) == 0 and torch.isfinite(out).all()
    c.table = full
    c.check(out, window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cap,window", [(30.0, 0), (50.0, 700), (0.5, 0)])
def test_capped_scores(mq, d, cap, window):
    c = Q4(mq, d, 8, 4, 16, [1, 40, 777, 2500], q_std=6.0)
    c.check(c.run(softcap=cap, window=window), softcap=cap, window=window)


@pytest.mark.parametrize("q_std,v_scale", [(1e-30, 1.0), (1e4, 1.0), (2.0, 1e-3), (2.0, 2e3), (0.0, 1.0)])
def test_magnitudes(mq, q_std, v_scale):
    c = Q4(mq, 128, 8, 2, 16, [1, 50, 600], q_std=q_std, v_scale=v_scale)
    c.check(c.run())


def test_huge_queries_over_vanishing_keys(mq):
    """Queries of 2^120 against scales of 2^-24: scores of a few hundred thousand at most after the scale."""
    c = Q4(mq, 64, 4, 2, 16, [40, 90])
    c.q = (np.sign(c.q) * np.float32(2.0 ** 120)).astype(np.float32)
    c.scales[0] = np.where(np.isnan(c.scales[0]), np.nan, 2.0 ** -24).astype(np.float16)
    c.store()
    c.scale = 2.0 ** -97
    c.check(c.run())


def test_a_nan_or_infinite_scale_that_is_seen(mq):
    """It makes the heads that see it NaN, and no others."""
    c = Q4(mq, 128, 4, 2, 16, [40, 90])
    c.scales[1][c.table[0, 1], 0, 3, 2] = np.nan      # a value's block of row 0, kv head 0
    c.scales[0][c.table[1, 2], 1, 5, 0] = np.nan      # a key's block of row 1, kv head 1
    c.store()
    got = c.run().cpu().numpy().reshape(2, 2, 2, 128)
    assert np.isnan(got[0, 0, :, 64:96]).all() and np.isfinite(got[0, 1]).all()
    assert np.isnan(got[1, 1]).all() and np.isfinite(got[1, 0]).all()


def whole(g, kind):
    """Codes of whole numbers under scales of powers of two."""
    return g.integers(0, 16, kind).astype(np.uint8)


BORDERS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 0, -1, 255, 256, 257, 383, 385, 4095,
           4096, 4097, 2047, 2049, 6144, 6145]


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("lens,ps,window", [(BORDERS, 16, 0), (BORDERS, 48, 0), (BORDERS, 16, 200), ([20001], 64, 0),
                                            ([9001, 3, 8193, 6145], 32, 4095), ([1000, 1500] * 20, 16, 0)])
def test_every_token_and_code_counts_once(mq, d, lens, ps, window):
    """Queries of zero over whole numbers: each result is a mean that one token, or one code, more or less would change."""
    c = Q4(mq, d, 6, 2, ps, lens, key="means")
    hole = np.isnan(c.scales[1])
    c.codes[1] = whole(synth.rng("means", d, len(lens)), c.codes[1].shape)
    c.scales[1] = np.where(hole, np.nan, 1.0).astype(np.float16)
    c.q[:] = 0
    c.store()
    got = c.run(window=window).cpu().numpy().reshape(len(lens), 2, 3, d).astype(np.float64)
    v, _ = ref.q4_values(c.codes[1], c.scales[1])
    for i, n in enumerate(lens):
        if n < 0:
            assert np.all(got[i] == 7.0)
            continue
        x = ref.gather(v, c.table[i], n)[:, max(0, n - window) if window else 0:]
        mean = x.sum(1) / x.shape[1] if n else np.zeros((2, d))
        assert np.all(np.abs(got[i] - mean[:, None]) <= ref.exact_mean_bound(mean)[:, None]), (i, n)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("of", ["queries", "weights"])
def test_no_part_is_missing(mq, d, of):
    """Two tokens alone matter (oracle.decode.TwoTokens), so every bit of a query or of a weight shows.  The bound is of
    sums without a bias; the codes' 8s add, for the scores, a sum of up to 16 |q| a block that loses 2^-23 of itself
    twice (32 values, of which the two parts and the bias), and for the results the same of 16 w."""
    g, hq, hkv, nt = synth.rng("q4 parts", d, of), 10, 2, 48
    lens = g.integers(17, 200, nt)
    c = Q4(mq, d, hq, hkv, 16, lens)
    rng = np.random.default_rng(int(g.integers(1 << 30)))
    cases = [ref.TwoTokens(rng, hq, hkv, d, int(n), of) for n in lens]
    shifts = 2.0 ** -g.integers(0, 3, c.scales[0].shape).astype(np.float64)
    for x, name in ((0, "k"), (1, "v")):
        vals = np.zeros(c.codes[x].shape)
        for i, t in enumerate(cases):
            y = getattr(t, name)
            for j in range(-(-int(lens[i]) // 16)):
                m = min(16, int(lens[i]) - j * 16)
                vals[c.table[i, j], :, :m] = y[:, j * 16:j * 16 + m]
        c.codes[x] = (vals / np.repeat(shifts, 32, -1) + 8).astype(np.uint8)
        c.scales[x] = np.where(np.isnan(c.scales[x]), np.nan, shifts).astype(np.float16)
    c.store()
    c.q = np.stack([t.q.reshape(-1) for t in cases])
    c.scale = 1.0
    got = c.run().cpu().numpy().reshape(nt, hq, d).astype(np.float64)
    for i, t in enumerate(cases):
        want = ref.attention(t.q, t.k, t.v, 1.0)
        w = np.abs(want)
        sums = np.abs(t.q).astype(np.float64).sum(-1, keepdims=True) * 16 * 2 * 2 if of == "queries" else \
            np.abs(t.q).astype(np.float64).sum(-1, keepdims=True) * 16 * 2
        more = 2.0 ** -23 * (w * (1 - w) * sums + 2 * 16 * 2)
        ratio = np.abs(got[i] - want) / (t.bound(want, True) + more)
        assert ratio.max() <= 1, (i, ratio.max())


def test_strided_pages(mq):
    import torch
    c = Q4(mq, 96, 8, 2, 48, [500, 33, 0, 2100])
    want = c.run()
    flat = [t.reshape(c.n_pages, -1) for t in (c.k, c.v)]
    page = flat[0].shape[1]
    both = torch.full((c.n_pages, 2 * page + 64), 0xff, dtype=torch.uint8, device="cuda")
    both[:, :page], both[:, page:2 * page] = flat
    views = [both[:, at:at + page].unflatten(1, c.k.shape[1:]) for at in (0, page)]
    c.cache = mq.MQKVCache("q4", c.n_pages, 48, 2, 96, k=views[0], v=views[1])
    assert torch.equal(c.run(), want)


@pytest.mark.parametrize("nt", [40, 1024, 1100])
def test_many_rows_of_few_sequences(mq, nt):
    import torch
    g = synth.rng("q4 many rows", nt)
    c = Q4(mq, 64, 4, 2, 16, [int(x) for x in g.integers(1, 400, 21)] + [3000])
    seq = g.integers(0, 22, nt).astype(np.int32)
    full = c.lens
    c.lens = np.array([g.integers(0, full[s] + 1) for s in seq], np.int32)
    c.lens[::17] = -1
    c.q = (synth.normal(g, nt * 4 * 64)).reshape(nt, 256)
    out = c.run(seq=dev(seq))
    c.check(out, rows=range(0, nt, 13), seq=seq)
    nb = mq.mq_q8_bytes(256)
    plane = torch.full((nt * nb,), 0x55, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.run(seq=dev(seq), q8=plane), out)
    for i in (1, nt - 2):
        want = mq.mq_quantize_q8(out[i].clone()).cpu().numpy()
        got = plane.view(nt, nb)[i].cpu().numpy()
        for a, b in zip(mq.mq_q8_unpack_host(got, 256), mq.mq_q8_unpack_host(want, 256)):
            assert np.array_equal(a, b), i


def test_bad_pages_and_lengths(mq):
    import torch
    c = Q4(mq, 128, 4, 2, 16, [40, 90, 33, 50])
    good = c.run()
    c.table[1, 2] = c.n_pages
    c.lens[2] = 16 * c.width + 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.run(status=status)
    assert int(status) == 1 and torch.isnan(out[1:3]).all()
    assert torch.equal(out[[0, 3]], good[[0, 3]])


def test_what_is_appended_is_attended(mq):
    """The two together, a prompt and then single tokens, and the same steps in a captured graph."""
    import torch
    g, hq, hkv, d, ps, n = synth.rng("q4 together"), 8, 2, 128, 16, 77
    x = [dev((synth.normal(g, (n + 4) * w * d)).reshape(n + 4, -1)) for w in (hq, hkv, hkv)]
    table = dev(np.random.default_rng(5).permutation(8)[None].astype(np.int32))
    rope = mq.mq_rope_table(1e4 ** (-np.arange(0, d, 2) / d))

    def steps(kv, outs):
        mq.mq_rope_append(kv, *(t[:n] for t in x), torch.arange(n, dtype=torch.int32, device="cuda"), table, rope=rope,
                          seq=torch.zeros(n, dtype=torch.int32, device="cuda"))
        pos = torch.full((1,), n, dtype=torch.int32, device="cuda")
        length = pos + 1
        for i in range(4):
            q = mq.mq_rope_append(kv, *(t[n + i:n + i + 1] for t in x), pos, table, rope=rope)
            mq.mq_attn_decode(kv, q, length, table, 1 / math.sqrt(d), out=outs[i])
            pos.add_(1), length.add_(1)
        return q
    a, b = (mq.MQKVCache("q4", 8, ps, hkv, d) for _ in range(2))
    out_a, out_b = (torch.zeros(4, 1, hq * d, device="cuda") for _ in range(2))
    q = steps(a, out_a)
    torch.cuda.synchronize()
    k, v = (ref.q4_values(*ref.unpack_q4(t.cpu().numpy(), ps, d, keys)) for t, keys in ((a.k, True), (a.v, False)))
    row = table[0].cpu().numpy()
    qn = q[0].cpu().numpy().reshape(hq, d)
    want, parts = ref.attention(qn, ref.gather(k[0], row, n + 4), ref.gather(v[0], row, n + 4),
                                1 / math.sqrt(d), parts=True)
    mag = np.matmul(np.abs(qn.astype(np.float64)).reshape(hkv, -1, d), ref.gather(k[1], row, n + 4).transpose(0, 2, 1)) / math.sqrt(d)
    tol = ref.attention_bound(want, (parts[0], mag, parts[2], ref.gather(v[1], row, n + 4)))
    assert np.all(np.abs(out_a[3, 0].cpu().numpy().reshape(hq, d) - want) <= tol)
    st, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=st):
        steps(b, out_b)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out_a, out_b) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)


def test_a_cache_past_32_bits(mq):
    """Pages behind the first 4 GiB: appended to and attended as those in front."""
    import torch
    hq, hkv, d, ps, n = 8, 2, 128, 64, 300
    page = mq.mq_kv_page_bytes("q4", hkv, ps, d)
    n_pages = (1 << 32) // page + 64
    g = synth.rng("q4 far")
    x = [dev(synth.normal(g, n * w * d).reshape(n, -1)) for w in (hq, hkv, hkv)]
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    outs = []
    for first in (0, n_pages - 5):
        kv = mq.MQKVCache("q4", n_pages, ps, hkv, d)
        table = dev(np.arange(first, first + 5, dtype=np.int32)[None])
        q = mq.mq_rope_append(kv, *x, pos, table, seq=torch.zeros_like(pos))
        outs.append((mq.mq_attn_decode(kv, q, pos + 1, table, 1 / math.sqrt(d), seq=torch.zeros_like(pos)),
                     kv.k[first:first + 5].clone(), kv.v[first:first + 5].clone()))
        del kv
        torch.cuda.empty_cache()
    assert outs[0][1].any() and all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("hq,hkv", [(8, 2), (20, 2), (8, 8)])
def test_in_place_and_strided_rows(mq, hq, hkv):
    import torch
    c = Q4(mq, 128, hq, hkv, 16, [9000, 3, 0, 700, 4000])
    want = c.run()
    q = dev(c.q)
    c.run(q=q, out=q)
    assert torch.equal(q, want)
    wide = torch.full((5, hq * 128 + 8), 3.0, device="cuda")
    wide[:, 4:-4] = dev(c.q)
    out = torch.full((5, 2 * hq * 128), 7.0, device="cuda")
    c.run(q=wide[:, 4:-4], out=out[:, hq * 128:])
    assert torch.equal(out[:, hq * 128:], want) and (out[:, :hq * 128] == 7.0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_std", [1e-30, 1e20, 1e36])
def test_queries_of_all_magnitudes(mq, d, q_std):
    c = Q4(mq, d, 8, 2, 16, [1, 50, 600], q_std=q_std)
    assert np.isfinite(c.q).all()
    c.scale = 2 / (math.sqrt(d) * q_std)
    c.check(c.run())


@pytest.mark.parametrize("cap", [1e-30, 1e-39, 1e-44])
def test_caps_whose_inverse_overflows(mq, cap):
    """A cap that leaves nothing of any score: the mean of the values."""
    c = Q4(mq, 64, 4, 2, 16, [90, 1, 300])
    c.q.reshape(3, 4, 64)[:, ::2] = 0.0
    c.check(c.run(softcap=cap), softcap=cap)


# ------------------------------------------------------------------ small values
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("v_scale", [1e-2, 1e-4, 1e-5, 2e-6])
def test_small_values(mq, d, v_scale):
    """Scales down to fp16's least: the bound is a share of the values."""
    c = Q4(mq, d, 8, 2, 16, [1, 50, 600, 5000], v_scale=v_scale, key="small")
    c.check(c.run())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("order", ["up", "down", "zeros first", "by block"])
def test_scales_that_change_along_a_sequence(mq, d, order):
    """From 2^-20 to 2^11 and back: the sums' units follow the largest that has been met."""
    c = Q4(mq, d, 8, 2, 16, [700, 4100, 33], key=order)
    u, s = c.codes[1], c.scales[1]
    factor = np.ones(s.shape)
    for i, n in enumerate(c.lens):
        e = np.linspace(-18, 12, int(n))
        e = {"up": e, "down": e[::-1], "zeros first": np.where(np.arange(n) < n // 2, -np.inf, -16), "by block": e * 0 - 10}[order]
        for t in range(int(n)):
            at = c.table[i, t // 16], slice(None), t % 16
            factor[at] = 2.0 ** e[t] * (2.0 ** (4 * np.arange(d // 32)) if order == "by block" else 1.0)
    with np.errstate(invalid="ignore"):
        c.scales[1] = np.clip(s.astype(np.float64) * factor, -60000, 60000).astype(np.float16)
    c.store()
    c.check(c.run())


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("of,shift", [("queries", 0), ("weights", 0), ("weights", -10), ("weights", -12), ("weights", -20)])
def test_every_bit_shows_at_every_scale(mq, d, of, shift):
    """Two tokens alone matter (oracle.decode.TwoTokens) and nothing is allowed for but what its bound counts, under value
    scales of 1 to 2^-20."""
    g, hq, hkv, nt = synth.rng("q4 bits", d, of, shift), 10, 2, 24
    lens = g.integers(17, 200, nt)
    c = Q4(mq, d, hq, hkv, 16, lens)
    rng = np.random.default_rng(int(g.integers(1 << 30)))
    cases = [ref.TwoTokens(rng, hq, hkv, d, int(n), of) for n in lens]
    for x, name in ((0, "k"), (1, "v")):
        vals = np.zeros(c.codes[x].shape)
        for i, t in enumerate(cases):
            y = getattr(t, name)
            for j in range(-(-int(lens[i]) // 16)):
                m = min(16, int(lens[i]) - j * 16)
                vals[c.table[i, j], :, :m] = y[:, j * 16:j * 16 + m]
        c.codes[x] = (vals + 8).astype(np.uint8)
        c.scales[x] = np.where(np.isnan(c.scales[x]), np.nan, 2.0 ** shift if x else 1.0).astype(np.float16)
    c.store()
    c.q = np.stack([t.q.reshape(-1) for t in cases])
    c.scale = 1.0
    got = c.run().cpu().numpy().reshape(nt, hq, d).astype(np.float64) * 2.0 ** -shift
    for i, t in enumerate(cases):
        want = ref.attention(t.q, t.k, t.v, 1.0)
        ratio = np.abs(got[i] - want) / t.bound(want, True)
        assert ratio.max() <= 1, (i, ratio.max())
