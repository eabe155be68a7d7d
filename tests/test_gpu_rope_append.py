"""mq_rope_append against a plain 64-bit reference: every cache type, head
size, rotation style and partial rotation, norms and biases on and off, padding
rows, shared sequences, strides, pages that are missing, and far positions.

Tolerance of an f32 result, in units of 2^-24 of |a| + |b| (the values a
rotation mixes, with |x| + |bias| for x): the bias add 1; the norm's sum of
squares (at most 8 fused adds in a lane and 5 across lanes, halved by the root),
division, root, reciprocal and two products 11; sine and cosine 2 ulp = 4 and
the angle's one rounding, pi; two products 2: 21.2, taken as 24.  A cache entry
adds half a step of its type."""
import numpy as np
import pytest

import synth
from oracle import decode as ref

pytestmark = pytest.mark.gpu
UNIT = 24 * 2.0 ** -24


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


def raw(t):
    """A cache tensor as numpy (bf16 as its bits)."""
    import torch
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy().view(
        np.uint16 if t.dtype == torch.bfloat16 else None or t.cpu().numpy().dtype)


class Case:
    def __init__(self, nt, hq, hkv, d, r, style, kv, ps, bias, norm, pos, pad=0, key=""):
        g = synth.rng("append", nt, hq, hkv, d, r, style, kv, ps, bias, norm, key)
        self.__dict__.update(nt=nt, hq=hq, hkv=hkv, d=d, r=r, style=style, kv=kv, ps=ps, rows=nt + pad)
        n = self.rows
        self.q, self.k, self.v = synth.normal(g, n * hq * d), synth.normal(g, n * hkv * d), synth.normal(g, n * hkv * d)
        self.q, self.k, self.v = (x.reshape(n, -1) * np.float32(2) for x in (self.q, self.k, self.v))
        self.qb, self.kb, self.vb = ((synth.normal(g, w * d) for w in (hq, hkv, hkv)) if bias else (None,) * 3)
        self.qg, self.kg = ((synth.normal(g, d, 1.0, 0.1) for _ in range(2)) if norm else (None, None))
        self.pos = np.concatenate([np.asarray(pos, np.int32), np.full(pad, -1, np.int32)])
        self.freqs = 1e6 ** (-np.arange(0, r, 2) / max(r, 1)) if r else np.zeros(0)
        self.seq = np.arange(n, dtype=np.int32)
        self.width = int(max(pos)) // ps + 1
        self.n_pages = n + 3
        self.table = np.full((n, self.width), -1, np.int32)
        for i in range(nt):
            self.table[i, pos[i] // ps] = (i * 7 + 2) % self.n_pages if self.n_pages % 7 else i

    def run(self, mq, kv=None, **more):
        import torch
        kv = kv or mq.MQKVCache(self.kv, self.n_pages, self.ps, self.hkv, self.d)
        if self.kv == "q8":
            kv.k.fill_(9), kv.v.fill_(9)
        else:
            kv.k.fill_(9.0), kv.v.fill_(9.0)
        q_out = torch.full((self.rows, self.hq * self.d), 5.0, device="cuda")
        rope = mq.mq_rope_table(self.freqs) if self.r else None
        args = dict(q_out=q_out, rope=rope, style=self.style, q_bias=dev(self.qb), k_bias=dev(self.kb),
                    v_bias=dev(self.vb), q_gain=dev(self.qg), k_gain=dev(self.kg), eps=1e-6)
        args.update(more)
        out = mq.mq_rope_append(kv, dev(self.q), dev(self.k), dev(self.v), dev(self.pos), dev(self.table), **args)
        torch.cuda.synchronize()
        return out, kv

    def want(self):
        q, mq_ = ref.rotate(*ref.heads_of(self.q, self.qb, self.qg, 1e-6, self.d), self.pos, self.freqs, self.style)
        k, mk = ref.rotate(*ref.heads_of(self.k, self.kb, self.kg, 1e-6, self.d), self.pos, self.freqs, self.style)
        v, mv = ref.heads_of(self.v, self.vb, None, 1e-6, self.d)
        return (q, mq_), (k, mk), (v, mv)

    def check(self, out, kv, seq=None):
        seq = self.seq if seq is None else seq
        (q, qm), (k, km), (v, vm) = self.want()
        got = out.cpu().numpy().reshape(self.rows, self.hq, self.d)
        live = self.pos >= 0
        assert np.all(np.abs(got - q)[live] <= UNIT * qm[live])
        assert np.all(got[~live] == 5.0)                      # padding rows stay as they were
        for t, want, mag in ((kv.k, k, km), (kv.v, v, vm)):
            bits = raw(t)
            vals = ref.unpack_pages(bits, self.kv, self.ps, self.d)
            written = np.zeros(vals.shape, bool)
            for i in np.flatnonzero(live):
                page, slot = self.table[seq[i], self.pos[i] // self.ps], self.pos[i] % self.ps
                w, tol = want[i], UNIT * mag[i]
                if self.kv == "q8":  # half a code, the scale's rounding to fp16, and f32
                    blk = np.abs(w).reshape(self.hkv, -1, 32).max(-1)
                    step = np.repeat(blk / 127, 32, -1)
                    tol = tol + step * (0.5 + 127 * 2.0 ** -11 + 1e-4)
                else:
                    tol = tol + np.abs(w) * (2.0 ** -11 if self.kv == "f16" else 2.0 ** -8) + 2.0 ** -25
                assert np.all(np.abs(vals[page, :, slot] - w) <= tol), (i, np.abs(vals[page, :, slot] - w).max())
                written[page, :, slot] = True
            if self.kv == "q8":
                codes = bits[..., : self.ps * self.d].reshape(written.shape)
                assert np.all(codes[~written] == 9)
            else:
                assert np.all(vals[~written] == 9.0)           # nothing else of the cache is touched


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("d,r,style", [(128, 128, "half"), (128, 128, "pairs"), (64, 32, "half"), (64, 64, "pairs"),
                                       (96, 96, "half"), (96, 48, "pairs"), (256, 128, "half"), (256, 256, "pairs"),
                                       (128, 0, "half"), (128, 8, "half")])
@pytest.mark.parametrize("bias,norm", [(False, False), (True, True)])
def test_against_reference(mq, kv, d, r, style, bias, norm):
    c = Case(5, 10, 2, d, r, style, kv, 16, bias, norm, [0, 1, 15, 16, 4097], pad=2)
    c.check(*c.run(mq))


@pytest.mark.parametrize("nt,hq,hkv", [(1, 1, 1), (1, 40, 8), (3, 7, 1), (700, 12, 4)])
def test_row_counts_and_groups(mq, nt, hq, hkv):
    """700 rows of 20 heads: several heads a warp share the angles."""
    c = Case(nt, hq, hkv, 128, 128, "half", "f16", 48, True, nt == 3, [3 + 11 * i for i in range(nt)])
    c.check(*c.run(mq))


@pytest.mark.parametrize("kv", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("hq,hkv", [(7, 1), (9, 3), (40, 8)])
@pytest.mark.parametrize("d,r,style", [(128, 128, "half"), (128, 16, "half"), (128, 24, "half"), (128, 80, "pairs"),
                                       (96, 96, "half"), (96, 64, "pairs"), (96, 0, "half"), (64, 64, "half"),
                                       (64, 32, "half"), (64, 64, "pairs")])
def test_many_rows_several_heads_a_warp(mq, kv, hq, hkv, d, r, style):
    """Heads go two (65 to 128 values) or four a warp when rows are many: odd counts, heads of 96 in 12 of 16
    lanes, and rotations whose pairs do not lie whole lanes apart (24), which stay as they are for few rows."""
    nt = (1250 if d > 64 or (r == 64 and style == "half") else 19600) // (hq + 2 * hkv) + 9
    c = Case(nt, hq, hkv, d, r, style, kv, 16, hkv != 8, True, [(i * 37) % 500 for i in range(nt)], pad=3)
    c.check(*c.run(mq))


def test_rows_of_many_heads(mq):
    """More heads than a CTA's share of a row, in CTAs of equal shares."""
    for nt, d in ((3, 128), (300, 128), (600, 64), (300, 256)):
        c = Case(nt, 90, 15, d, d, "half", "q8", 16, True, False, [7 + i for i in range(nt)])
        c.check(*c.run(mq))


def test_many_rows_of_small_heads(mq):
    c = Case(2000, 14, 2, 64, 64, "half", "bf16", 32, False, True, [5 * i for i in range(2000)], pad=1)
    c.check(*c.run(mq))


@pytest.mark.parametrize("pos", [131071, 1 << 24, (1 << 24) + 1, 2 ** 31 - 64])
def test_far_positions_lose_nothing(mq, pos):
    """At 2^31 an f32 angle would be off by a hundred radians; the fixed-point
    angle keeps the same tolerance (the reference's own f64 angle is off by
    2^31 * 2^-53)."""
    c = Case(1, 4, 2, 128, 128, "half", "bf16", 1 << 20, False, False, [0])
    c.pos = np.array([pos], np.int32)
    c.width = pos // c.ps + 1
    c.table = np.full((1, c.width), 1, np.int32)
    c.n_pages = 2
    c.check(*c.run(mq))


def test_rows_of_one_sequence(mq):
    """A prompt chunk: every row names the same sequence."""
    n = 37
    c = Case(n, 4, 2, 128, 128, "half", "f16", 16, False, False, list(range(90, 90 + n)))
    seq = np.full(n, 1, np.int32)
    c.table = np.full((2, 8), -1, np.int32)
    c.table[1] = np.arange(8)[::-1]
    c.n_pages = 9
    out, kv = c.run(mq, seq=dev(seq))
    c.check(out, kv, seq)


def test_q8_entries_are_the_producers_blocks(mq):
    """Values without rotation: codes and scales equal mq_quantize_q8's, byte for byte."""
    import torch
    c = Case(3, 4, 2, 128, 128, "half", "q8", 16, False, False, [0, 17, 40])
    _, kv = c.run(mq)
    for i in range(3):
        plane = mq.mq_quantize_q8(dev(c.v[i].copy()))
        d, qs, _ = mq.mq_q8_unpack_host(plane.cpu().numpy(), 256)
        page, slot = c.table[i, c.pos[i] // 16], c.pos[i] % 16
        b = kv.v[page].cpu().numpy()
        codes = b[:, : 16 * 128].reshape(2, 16, 128)[:, slot].view(np.int8).reshape(-1)
        scale = np.ascontiguousarray(b[:, 16 * 128:]).view(np.uint16).reshape(2, 16, 4)[:, slot].reshape(-1)
        assert np.array_equal(codes, qs) and np.array_equal(scale, d)


def test_strided_rows_in_place_and_strided_pages(mq):
    """q, k, v as column ranges of one array, queries rotated in place, and k
    and v pages interleaved in one array: the bits of the plain call."""
    import torch
    c = Case(9, 8, 2, 128, 64, "half", "f16", 32, True, True, [7 * i for i in range(9)], pad=1)
    out, kv = c.run(mq)
    both = torch.full((c.n_pages, 2, c.hkv, c.ps, c.d), 9.0, dtype=torch.float16, device="cuda")
    kv2 = mq.MQKVCache("f16", c.n_pages, c.ps, c.hkv, c.d, k=both[:, 0], v=both[:, 1])
    qkv = torch.cat([dev(c.q), dev(c.k), dev(c.v), torch.zeros(c.rows, 4, device="cuda")], 1)
    nq, nk = c.hq * c.d, c.hkv * c.d
    q = qkv[:, :nq]
    pad = q[-1].clone()
    mq.mq_rope_append(kv2, q, qkv[:, nq:nq + nk], qkv[:, nq + nk:nq + 2 * nk], dev(c.pos), dev(c.table),
                      q_out=q, rope=mq.mq_rope_table(c.freqs), q_bias=dev(c.qb), k_bias=dev(c.kb),
                      v_bias=dev(c.vb), q_gain=dev(c.qg), k_gain=dev(c.kg))
    torch.cuda.synchronize()
    assert torch.equal(q[:-1], out[:-1]) and torch.equal(q[-1], pad)
    assert torch.equal(both[:, 0], kv.k) and torch.equal(both[:, 1], kv.v)
    assert torch.equal(qkv[:, nq:nq + nk], dev(c.k))


def test_rows_without_a_page_are_refused_on_the_device(mq):
    """A page that is missing or out of range, a position behind the table, a
    sequence that is not there: NaN queries, no write, status 1; the rows beside
    them are served."""
    import torch
    c = Case(6, 4, 2, 128, 128, "half", "f16", 16, False, False, [0, 20, 40, 60, 63, 5])
    good_out, good_kv = c.run(mq)
    c.table[1, 1] = -1
    c.table[2, 2] = c.n_pages
    pos = c.pos.copy()
    pos[3] = 16 * c.width
    seq = c.seq.copy()
    seq[4] = 99
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.pos = pos
    out, kv = c.run(mq, seq=dev(seq), status=status)
    assert status.item() == 1
    assert torch.isnan(out[1:5]).all()
    assert torch.equal(out[[0, 5]], good_out[[0, 5]])
    for i in (0, 5):
        page, slot = c.table[i, pos[i] // 16], pos[i] % 16
        assert torch.equal(kv.k[page, :, slot], good_kv.k[page, :, slot])
        kv.k[page, :, slot] = 9.0
    assert (kv.k == 9.0).all()
    ok = torch.zeros(1, dtype=torch.int32, device="cuda")
    c2 = Case(2, 4, 2, 128, 128, "half", "f16", 16, False, False, [0, 20])
    c2.run(mq, status=ok)
    assert ok.item() == 0


def test_captured_replayed_and_on_another_stream(mq):
    """A captured call replays with new positions and rows in the same buffers,
    with and without programmatic dependent launch; a side stream gives the same."""
    import torch
    c = Case(4, 8, 2, 128, 128, "half", "q8", 16, True, True, [1, 30, 47, 5])
    want, kv_want = c.run(mq)
    kv = mq.MQKVCache(c.kv, c.n_pages, c.ps, c.hkv, c.d)
    q, k, v, pos, table = (torch.zeros_like(dev(x)) for x in (c.q, c.k, c.v, c.pos, c.table))
    out = torch.full((c.rows, c.hq * c.d), 5.0, device="cuda")
    more = dict(q_out=out, rope=mq.mq_rope_table(c.freqs), q_bias=dev(c.qb), k_bias=dev(c.kb), v_bias=dev(c.vb),
                q_gain=dev(c.qg), k_gain=dev(c.kg))
    st = torch.cuda.Stream()
    for pdl in (False, True):
        mq.mq_set_pdl(pdl)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            mq.mq_rope_append(kv, q, k, v, pos, table, **more)
        mq.mq_set_pdl(False)
        for t, x in ((q, c.q), (k, c.k), (v, c.v), (pos, c.pos), (table, c.table)):
            t.copy_(dev(x))
        kv.k.fill_(9), kv.v.fill_(9)
        out.fill_(0)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kv.k, kv_want.k) and torch.equal(kv.v, kv_want.v)
        out.fill_(0)
        torch.cuda.synchronize()
        mq.mq_rope_append(kv, q, k, v, pos, table, stream=st, **more)
        st.synchronize()
        assert torch.equal(out, want)


def test_refusals(mq):
    import torch
    kv = mq.MQKVCache("f16", 4, 16, 2, 128)
    q, k, v = (torch.zeros(1, w * 128, device="cuda") for w in (4, 2, 2))
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    rope = mq.mq_rope_table(np.ones(64))
    mq.mq_rope_append(kv, q, k, v, pos, table, rope=rope)
    for bad in (dict(q=q.cpu()), dict(q=q.double()), dict(k=q), dict(pos=pos.long()), dict(q=q.t()),
                dict(pos=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(rope=rope.int()),
                dict(q=torch.zeros(1, 300, device="cuda"))):
        a = dict(q=q, k=k, v=v, pos=pos, rope=rope)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            mq.mq_rope_append(kv, a["q"], a["k"], a["v"], a["pos"], table, rope=a["rope"])
    for bad, status in ((dict(q=torch.zeros(1, 3 * 128, device="cuda")), mq.MQ_ERR_SHAPE),   # 3 heads over 2
                        (dict(rope=mq.mq_rope_table(np.ones(2))), mq.MQ_ERR_SHAPE),           # rope_dims 4
                        (dict(rope=mq.mq_rope_table(np.ones(68))), mq.MQ_ERR_SHAPE),
                        (dict(q=torch.zeros(513, device="cuda")[1:].view(1, 512)), mq.MQ_ERR_ALIGN)):
        a = dict(q=q, rope=rope)
        a.update(bad)
        with pytest.raises(mq.MQError) as e:
            mq.mq_rope_append(kv, a["q"], k, v, pos, table, rope=a["rope"])
        assert e.value.status == status
    with pytest.raises(ValueError):
        mq.mq_rope_append(kv, q.expand(3, -1).contiguous(), k.expand(3, -1).contiguous(),
                          v.expand(3, -1).contiguous(), pos.expand(3).contiguous(), table, rope=rope)
    with pytest.raises(mq.MQError):
        mq.MQKVCache("f16", 4, 24, 2, 128)
    with pytest.raises(mq.MQError):
        mq.MQKVCache("f16", 4, 16, 2, 80)


def test_pages_that_overlap_are_refused(mq):
    """A stride of 0 between pages would read as pages back to back."""
    import torch
    for kv, dtype, page in (("f16", torch.float16, (2, 16, 64)), ("q8", torch.uint8, (2, 16 * 68))):
        one, four = (torch.zeros(n, *page, dtype=dtype, device="cuda") for n in (1, 4))
        pages = one.expand(4, *page)
        with pytest.raises(ValueError):
            mq.MQKVCache(kv, 4, 16, 2, 64, k=pages, v=pages)
        with pytest.raises(ValueError):
            mq.MQKVCache(kv, 4, 16, 2, 64, k=four, v=pages)
        halves = torch.as_strided(four, (4, *page), (four.stride(0) // 2, *four.stride()[1:]))
        with pytest.raises(ValueError):
            mq.MQKVCache(kv, 4, 16, 2, 64, k=halves, v=halves)
        assert mq.MQKVCache(kv, 1, 16, 2, 64, k=pages[:1], v=four[:1])._struct.page_stride == 0


def test_queries_made_for_another_stream_are_of_its_memory(mq):
    """Not of what the current stream has just given back, which its kernels may still use."""
    import torch
    kv = mq.MQKVCache("f16", 4, 16, 2, 128)
    q, k, v = (torch.ones(1, w * 128, device="cuda") for w in (4, 2, 2))
    pos, table = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    given_back = torch.empty_like(q).data_ptr()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = mq.mq_rope_append(kv, q, k, v, pos, table, stream=st)
    st.synchronize()
    assert out.data_ptr() != given_back and torch.equal(out, q)


@pytest.mark.parametrize("d,style,norm", [(128, "half", True), (64, "pairs", False)])
def test_inputs_written_just_before_under_pdl(mq, d, style, norm):
    """The kernel right before writes the rotation's table, a bias, a gain, the positions or the page table
    of a captured step with programmatic dependent launch: nothing is read before it has finished."""
    import torch
    c = Case(24, 8, 2, d, d, style, "f16", 16, True, norm, [3 + 17 * i for i in range(24)], key="pdl")
    want_q, want = c.run(mq)
    torch.cuda.synchronize()
    args = dict(rope=mq.mq_rope_table(c.freqs), q_bias=dev(c.qb), k_bias=dev(c.kb), v_bias=dev(c.vb),
                q_gain=dev(c.qg), k_gain=dev(c.kg))
    fixed = dict(positions=dev(c.pos), pages=dev(c.table))
    big = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    sink = torch.empty_like(big)
    for name, new in [*args.items(), *fixed.items()]:
        if new is None:
            continue
        live = torch.zeros_like(new)
        call = {**args, **fixed, name: live}
        positions, pages = call.pop("positions"), call.pop("pages")
        kv = mq.MQKVCache(c.kv, c.n_pages, c.ps, c.hkv, c.d)
        q, k, v, q_out = dev(c.q), dev(c.k), dev(c.v), torch.full((c.rows, c.hq * d), 5.0, device="cuda")
        whole = new.numel() * new.element_size() // 16 * 16       # what mq_copy takes; the rest is there already
        live.view(torch.uint8).view(-1)[whole:] = new.view(torch.uint8).view(-1)[whole:]
        old = live.clone()
        mq.mq_set_pdl(True)
        try:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=torch.cuda.Stream()):
                mq.mq_copy(sink, big)                              # what the copy behind it waits for
                mq.mq_copy(live, new, whole)
                mq.mq_rope_append(kv, q, k, v, positions, pages, q_out=q_out, style=style, eps=1e-6, **call)
        finally:
            mq.mq_set_pdl(False)
        for _ in range(3):
            live.copy_(old), kv.k.fill_(9.0), kv.v.fill_(9.0), q_out.fill_(5.0)
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(q_out, want_q), name
            assert torch.equal(kv.k, want.k) and torch.equal(kv.v, want.v), name
