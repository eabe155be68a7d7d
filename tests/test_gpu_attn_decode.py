"""mq_attn_decode against a plain 64-bit reference over the same cache bytes.

The tolerance of every value is oracle.decode.attention_bound, the error of an
f32 evaluation term by term (its docstring derives it)."""
import math

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


class Case:
    """Rows of given lengths over a cache whose unused places are all NaN."""

    def __init__(self, mq, kv, d, hq, hkv, ps, lens, key="", q_std=2.0, v_scale=1.0, k_shift=True):
        import torch
        g = synth.rng("attn", kv, d, hq, hkv, ps, len(lens), key)
        self.__dict__.update(kv=kv, d=d, hq=hq, hkv=hkv, ps=ps, lens=np.asarray(lens, np.int32))
        need = [max(0, -(-int(n) // ps)) for n in lens]
        self.n_pages = sum(need) + 2
        self.width = max(1, max(need))
        order = g.permutation(self.n_pages - 1)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for i, c in enumerate(need):
            self.table[i, :c] = order[at:at + c]
            at += c
        shape = (self.n_pages, hkv, ps, d)
        gt = torch.Generator(device="cuda")
        gt.manual_seed(int(g.integers(1 << 30)))
        k = torch.randn(shape, generator=gt, device="cuda")
        if k_shift:
            k += torch.randn((hkv, 1, d), generator=gt, device="cuda")
        v = torch.randn(shape, generator=gt, device="cuda") * v_scale
        used = torch.zeros((self.n_pages, ps), dtype=torch.bool, device="cuda")
        for i, n in enumerate(lens):
            for j in range(need[i]):
                used[self.table[i, j], : min(ps, int(n) - j * ps)] = True
        hole = (~used)[:, None, :, None]
        if kv == "q8":
            self.k, self.v = self.pack(k, hole), self.pack(v, hole)
        else:
            dtype = torch.float16 if kv == "f16" else torch.bfloat16
            self.k, self.v = (x.masked_fill(hole, math.nan).to(dtype) for x in (k, v))
        self.cache = mq.MQKVCache(kv, self.n_pages, ps, hkv, d, k=self.k, v=self.v)
        self.q = (synth.normal(g, len(lens) * hq * d) * np.float32(q_std)).reshape(len(lens), hq * d)
        self.scale = 1 / math.sqrt(d)
        self.mq = mq

    def pack(self, x, hole):
        import torch
        n, h, ps, d = x.shape
        b = x.reshape(n, h, ps, d // 32, 32)
        step = b.abs().amax(-1, keepdim=True) / 127
        codes = torch.round(b / step).clamp(-128, 127).to(torch.int8)
        step = step[..., 0].masked_fill(hole, math.nan).half()
        return torch.cat([codes.reshape(n, h, -1).view(torch.uint8), step.reshape(n, h, -1).view(torch.uint8)], -1)

    def values(self, t):
        import torch
        raw = (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy()
        return ref.unpack_pages(raw.view(np.uint16) if t.dtype == torch.bfloat16 else raw, self.kv, self.ps, self.d)

    def run(self, q=None, out=None, **more):
        import torch
        out = torch.full(self.q.shape, 7.0, device="cuda") if out is None else out
        r = self.mq.mq_attn_decode(self.cache, dev(self.q) if q is None else q, dev(self.lens), dev(self.table),
                                   self.scale, out=out, **more)
        torch.cuda.synchronize()
        return r

    def check(self, out, softcap=0.0, window=0, rows=None, seq=None, lens=None):
        got = out.cpu().numpy().reshape(len(self.q), self.hq, self.d)
        kp, vp = self.values(self.k), self.values(self.v)
        lens = self.lens if lens is None else lens
        for i in range(len(self.q)) if rows is None else rows:
            n = int(lens[i])
            if n < 0:
                assert np.all(got[i] == 7.0)
                continue
            row = self.table[i if seq is None else seq[i]]
            k, v = ref.gather(kp, row, n), ref.gather(vp, row, n)
            want, parts = ref.attention(self.q[i].reshape(self.hq, self.d), k, v, np.float32(self.scale).astype(float),
                                        softcap, window, parts=True)
            tol = ref.attention_bound(want, parts, softcap)
            err = np.abs(got[i] - want)
            assert np.all(err <= tol), (i, n, err.max(), (err / np.maximum(tol, 1e-300)).max())


RAGGED = [1, 2, 15, 16, 17, 0, 63, 64, 65, 130, 333, -1, 1000, -1]


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("hq,hkv,ps", [(10, 2, 16), (4, 4, 48)])
def test_ragged_rows(mq, kv, d, hq, hkv, ps):
    c = Case(mq, kv, d, hq, hkv, ps, RAGGED)
    c.check(c.run())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (8, 1), (9, 1), (16, 1), (20, 2), (33, 3)])
def test_head_groups(mq, hq, hkv):
    c = Case(mq, "f16", 128, hq, hkv, 32, [1, 70, 1500])
    c.check(c.run())


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("lens,ps", [([4097], 16), ([20001], 64), ([70000], 4096), ([3000, 1, 2999, 64, 65], 16)])
def test_long_rows_are_split_and_joined(mq, kv, lens, ps):
    c = Case(mq, kv, 128, 10, 2, ps, lens)
    ws = mq.mq_attn_workspace(c.cache, 10, len(lens), max(lens))
    assert ws is not None
    out = c.run(ws=ws, max_len=max(lens))
    c.check(out)
    again = c.run(ws=ws, max_len=max(lens))
    import torch
    assert torch.equal(out, again)                                     # the order of sums is fixed
    assert not ws[: mq.mq_device_sms() * 4].any()                      # the counters in front are zero again


def test_many_rows(mq):
    """More units than a wave of CTAs: pieces of 1024 tokens and more."""
    lens = [1 + (i * 2741) % 9000 for i in range(70)]
    c = Case(mq, "f16", 128, 16, 8, 64, lens)
    c.check(c.run(), rows=list(range(0, 70, 9)))


@pytest.mark.parametrize("window", [0, 100])
def test_more_rows_than_are_shared_out(mq, window):
    """Past 1024 rows every unit has a CTA of its own (no workspace, no cut)."""
    lens = [(i * 37) % 700 - (1 if i % 11 == 0 else 0) for i in range(1100)]
    c = Case(mq, "f16", 64, 4, 2, 16, lens)
    out = c.run(window=window)
    rows = [i for i in range(0, 1100, 97) if lens[i] > window] + [0, 1099]
    c.check(out, rows=rows, window=window)
    for i in np.flatnonzero(c.lens < 0):
        assert (out[i] == 7.0).all()


def test_exactly_the_rows_that_are_shared_out(mq):
    """1024 rows, the most of one shared launch: empty, padded, short and long ones."""
    lens = [0 if i % 5 == 0 else -1 if i % 7 == 0 else 1 + (i * 131) % 300 for i in range(1023)] + [5000]
    c = Case(mq, "q8", 64, 2, 1, 16, lens)
    out = c.run()
    c.check(out, rows=list(range(0, 1024, 61)) + [1023])
    assert (out[c.lens == 0] == 0).all() and (out[c.lens < 0] == 7.0).all() and torch_finite(out[c.lens > 0])


def torch_finite(t):
    import torch
    return bool(torch.isfinite(t).all())


@pytest.mark.parametrize("kv", ["f16", "q8"])
@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 1024, 5000])
def test_windows(mq, kv, window):
    """Tokens that left the window are NaN and not used."""
    lens = [1, 16, 99, 101, 1500, 4000, 0, -1]
    c = Case(mq, kv, 64, 6, 2, 16, lens)
    for i, n in enumerate(lens):
        for j in range(max(0, n - window)):
            page, slot = c.table[i, j // 16], j % 16
            if kv == "q8":
                sc = 16 * 64 + slot * 4
                for t in (c.k, c.v):
                    t[page, :, sc:sc + 4] = 0xff                         # fp16 NaN scales
            else:
                c.k[page, :, slot] = math.nan
                c.v[page, :, slot] = math.inf
    out = c.run(window=window)
    import torch
    assert torch.isfinite(out).all()
    # the reference over the window alone
    kp, vp = c.values(c.k), c.values(c.v)
    got = out.cpu().numpy().reshape(len(lens), 6, 64)
    for i, n in enumerate(lens):
        if n <= 0:
            assert np.all(got[i] == (0.0 if n == 0 else 7.0))
            continue
        a = max(0, n - window)
        k, v = ref.gather(kp, c.table[i], n)[:, a:], ref.gather(vp, c.table[i], n)[:, a:]
        want, parts = ref.attention(c.q[i].reshape(6, 64), k, v, np.float32(c.scale).astype(float), parts=True)
        assert np.all(np.abs(got[i] - want) <= ref.attention_bound(want, parts))


@pytest.mark.parametrize("kv,d", [("f16", 128), ("bf16", 256), ("q8", 96)])
@pytest.mark.parametrize("cap,window", [(30.0, 0), (50.0, 700), (0.5, 0)])
def test_capped_scores(mq, kv, d, cap, window):
    c = Case(mq, kv, d, 8, 4, 16, [1, 40, 777, 2500], q_std=6.0)
    c.check(c.run(softcap=cap, window=window), softcap=cap, window=window)


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("q_std,v_scale", [(1e-30, 1.0), (1e4, 1.0), (2.0, 1e-3), (2.0, 2e3), (0.0, 1.0)])
def test_magnitudes(mq, kv, q_std, v_scale):
    """Vanishing and huge queries and values: the parts keep their 22 bits."""
    c = Case(mq, kv, 128, 8, 2, 16, [1, 50, 600], q_std=q_std, v_scale=v_scale)
    c.check(c.run())


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
def test_one_token_dominates_and_equal_scores(mq, kv):
    """A score 200 above the rest gives that token's value; equal keys the mean."""
    import torch
    c = Case(mq, kv, 64, 4, 2, 16, [90, 90], k_shift=False)
    if kv == "q8":
        c.k[:, :, : 16 * 64] = 0
        c.k[:, :, 16 * 64:] = 0
    else:
        c.k.zero_()
    out = c.run()
    c.check(out)
    mean = ref.gather(c.values(c.v), c.table[0], 90).mean(1)
    got = out[0].cpu().numpy().reshape(2, 2, 64)
    assert np.abs(got - mean[:, None]).max() < 1e-5
    assert torch.equal(out[0].view(2, 2, 64)[:, 0], out[0].view(2, 2, 64)[:, 1])


@pytest.mark.parametrize("lens", [[300, 0, 17, -1], [9000, 0, 2, -1]])
def test_q8_plane_is_the_quantized_row(mq, lens):
    """out's planes equal mq_quantize_q8 of each row, byte for byte (one piece
    and joined pieces); a padding row's plane is left as it was."""
    import torch
    c = Case(mq, "f16", 128, 10, 2, 16, lens)
    nb = mq.mq_q8_bytes(1280)
    plane = torch.full((4 * nb,), 0x55, dtype=torch.uint8, device="cuda")
    out = c.run(q8=plane)
    c.check(out)
    for i in range(3):
        d, qs, s = mq.mq_q8_unpack_host(mq.mq_quantize_q8(out[i].clone()).cpu().numpy(), 1280)
        d2, qs2, s2 = mq.mq_q8_unpack_host(plane[i * nb:(i + 1) * nb].cpu().numpy(), 1280)
        assert np.array_equal(d, d2) and np.array_equal(qs, qs2) and np.array_equal(s, s2)
    assert (plane[3 * nb:] == 0x55).all()


def test_rows_of_one_sequence(mq):
    """The tokens of a speculative step: four rows, one sequence, growing lengths."""
    c = Case(mq, "f16", 128, 8, 2, 16, [0, 2050, 0, 0])
    seq = np.array([1, 1, 1, 1], np.int32)
    c.lens = np.array([2047, 2048, 2049, 2050], np.int32)
    c.check(c.run(seq=dev(seq)), seq=seq)


def test_one_workspace_for_calls_of_other_sizes(mq):
    """A workspace sized for the larger call serves the smaller ones, in any order."""
    import torch
    big = Case(mq, "f16", 128, 16, 8, 16, [2500] * 9)
    one = Case(mq, "q8", 64, 4, 1, 32, [6000])
    ws = torch.zeros(max(mq.mq_attn_workspace_bytes(big.cache, 16, 64, 9000),
                         mq.mq_attn_workspace_bytes(one.cache, 4, 1, 9000)), dtype=torch.uint8, device="cuda")
    first = big.run(ws=ws, max_len=2500)
    for _ in range(2):
        one.check(one.run(ws=ws, max_len=6000))
        assert torch.equal(big.run(ws=ws, max_len=2500), first)
        big.run(ws=ws, max_len=9000)
    big.check(first, rows=[0, 8])


def test_strided_rows_and_pages(mq):
    import torch
    c = Case(mq, "f16", 128, 8, 2, 16, [500, 33, 0])
    want = c.run()
    both = torch.empty((c.n_pages, 2, 2, 16, 128), dtype=torch.float16, device="cuda")
    both[:, 0], both[:, 1] = c.k, c.v
    c.cache = mq.MQKVCache("f16", c.n_pages, 16, 2, 128, k=both[:, 0], v=both[:, 1])
    wide = torch.zeros(3, 1024 + 8, device="cuda")
    q = wide[:, 4:1028]
    q.copy_(dev(c.q))
    out = torch.full((3, 2048), 7.0, device="cuda")
    c.run(q=q, out=out[:, 1024:])
    assert torch.equal(out[:, 1024:], want) and (out[:, :1024] == 7.0).all()


@pytest.mark.parametrize("kv,hq,hkv", [("f16", 8, 2), ("bf16", 20, 2), ("q8", 8, 8)])
def test_in_place(mq, kv, hq, hkv):
    """out is q: rows that are cut over many CTAs, and head groups of one kv head."""
    import torch
    c = Case(mq, kv, 128, hq, hkv, 16, [9000, 3, 0, 700, 4000])
    want = c.run()
    q = dev(c.q)
    c.run(q=q, out=q)
    assert torch.equal(q, want)


def test_cache_beyond_32_bits(mq):
    """Pages past 4 GB: their offsets need 64 bits."""
    import torch
    c = Case(mq, "f16", 128, 8, 8, 16, [40, 200])
    want = c.run()
    page = 8 * 16 * 128 * 2
    n = (1 << 32) // page + 64
    k, v = (torch.empty((n, 8, 16, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    k[n - c.n_pages:], v[n - c.n_pages:] = c.k, c.v
    c.cache = mq.MQKVCache("f16", n, 16, 8, 128, k=k, v=v)
    c.table = np.where(c.table >= 0, c.table + n - c.n_pages, -1).astype(np.int32)
    assert torch.equal(c.run(), want)


def test_rows_out_of_range_are_nan(mq):
    """A missing page, a length behind max_len or the table, a sequence that is
    not there: NaN and status 1; the other rows are served."""
    import torch
    lens = [100, 5000, 100, 5000, 100, 100]
    c = Case(mq, "f16", 64, 4, 2, 16, lens)
    good = c.run()
    c.table[1, 200] = -1
    c.table[2, 0] = c.n_pages
    c.lens = np.array([100, 5000, 100, 5001, 16 * c.width + 1, 100], np.int32)
    seq = np.array([0, 1, 2, 3, 4, 6], np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.run(seq=dev(seq), status=status, max_len=5000)
    assert status.item() == 1
    assert torch.equal(out[0], good[0]) and torch.isnan(out[1:]).all()
    status.zero_()
    c2 = Case(mq, "f16", 64, 4, 2, 16, lens)
    assert torch.equal(c2.run(status=status), good) and status.item() == 0


def test_captured_replayed_and_on_another_stream(mq):
    """A captured call replays with new lengths and queries in the same
    buffers, with and without programmatic dependent launch."""
    import torch
    c = Case(mq, "bf16", 128, 8, 2, 16, [3000, 17, 500])
    want = c.run(max_len=4000)
    # without a workspace: one is made, zeroed and used in the stream's order; out is of its memory too, not
    # of what the current stream has just given back
    side = torch.cuda.Stream()
    given_back = torch.empty_like(want).data_ptr()
    torch.cuda.synchronize()
    free = mq.mq_attn_decode(c.cache, dev(c.q), dev(c.lens), dev(c.table), c.scale, max_len=4000, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(free, want) and free.data_ptr() != given_back
    ws = mq.mq_attn_workspace(c.cache, 8, 3, 4000)
    q, lens, table = torch.zeros_like(dev(c.q)), torch.zeros(3, dtype=torch.int32, device="cuda"), dev(c.table)
    out = torch.zeros_like(q)
    st = torch.cuda.Stream()
    for pdl in (False, True):
        mq.mq_set_pdl(pdl)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            for _ in range(3):  # back to back: the workspace passes from one to the next
                mq.mq_attn_decode(c.cache, q, lens, table, c.scale, out=out, ws=ws, max_len=4000)
        mq.mq_set_pdl(False)
        q.copy_(dev(c.q)), lens.copy_(dev(c.lens))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_(), q.mul_(0.5), lens.copy_(torch.tensor([1, 2, 3]))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(out).all() and not torch.equal(out, want)
        q.copy_(dev(c.q)), lens.copy_(dev(c.lens)), out.zero_()
        torch.cuda.synchronize()
        mq.mq_attn_decode(c.cache, q, lens, table, c.scale, out=out, ws=ws, max_len=4000, stream=st)
        st.synchronize()
        assert torch.equal(out, want)


def test_refusals(mq):
    import torch
    c = Case(mq, "f16", 128, 8, 2, 16, [3000])
    q, lens, table = dev(c.q), dev(c.lens), dev(c.table)
    ok = mq.mq_attn_workspace(c.cache, 8, 1, 3008)

    def call(q=q, lens=lens, table=table, scale=c.scale, **more):
        return mq.mq_attn_decode(c.cache, q, lens, table, scale, **{"ws": ok, **more})

    call()
    for bad in (dict(q=q.cpu()), dict(q=q.half()), dict(lens=lens.long()), dict(table=table.long()),
                dict(q=torch.zeros(1, 1000, device="cuda")), dict(table=table[0]), dict(lens=lens[:0]),
                dict(out=torch.zeros(1, 512, device="cuda")), dict(q8=torch.zeros(16, dtype=torch.uint8, device="cuda")),
                dict(q=torch.zeros(2, 1024, device="cuda"), lens=lens.expand(2).contiguous())):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    for bad, status in ((dict(q=torch.zeros(1, 3 * 128, device="cuda")), mq.MQ_ERR_SHAPE),
                        (dict(window=-1), mq.MQ_ERR_SHAPE), (dict(max_len=0), mq.MQ_ERR_SHAPE),
                        (dict(max_len=2 ** 30 + 1), mq.MQ_ERR_SHAPE), (dict(max_len=2 ** 32 + 3000), mq.MQ_ERR_SHAPE),
                        (dict(max_len=2 ** 32 + 3000, ws=None), mq.MQ_ERR_SHAPE),
                        (dict(window=2 ** 32), mq.MQ_ERR_SHAPE), (dict(window=2 ** 31), mq.MQ_ERR_SHAPE),
                        (dict(scale=math.nan), mq.MQ_ERR_SHAPE), (dict(softcap=-1.0), mq.MQ_ERR_SHAPE),
                        (dict(softcap=math.inf), mq.MQ_ERR_SHAPE),
                        (dict(ws=ok[:64]), mq.MQ_ERR_WORKSPACE), (dict(ws=ok[8:]), mq.MQ_ERR_ALIGN)):
        with pytest.raises(mq.MQError) as e:
            call(**bad)
        assert e.value.status == status, bad


@pytest.mark.parametrize("kv,q_std", [("f16", 5e30), ("f16", 1e33), ("f16", 5e37), ("q8", 1e33), ("q8", 5e37),
                                      ("bf16", 1e33)])
def test_the_largest_queries(mq, kv, q_std):
    """Queries of every finite magnitude, under a scale that brings their scores back: the factor of a head's
    parts follows its largest value to the end of f32.  (bf16 sums q k itself, so less room.)"""
    c = Case(mq, kv, 128, 8, 2, 16, [1, 50, 600], q_std=q_std)
    assert np.isfinite(c.q).all()
    c.scale = 2 / (math.sqrt(128) * q_std)
    c.check(c.run())


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("cap", [1e-30, 1e-39, 1e-44])
def test_caps_whose_inverse_overflows(mq, kv, cap):
    """A cap that leaves nothing of any score, over scores of 0 and others: the mean of the values."""
    c = Case(mq, kv, 64, 4, 2, 16, [90, 1, 300])
    c.q.reshape(3, 4, 64)[:, ::2] = 0.0
    c.check(c.run(softcap=cap), softcap=cap)
