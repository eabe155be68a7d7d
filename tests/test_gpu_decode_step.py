"""A whole decode step on the device: rms_norm -> q8 -> q/k/v GEMVs -> rotation
and append -> attention with its q8 plane -> o GEMV -> FFN -> head GEMV -> draw
-> the next token's row, with positions and lengths advanced in the step.  One
captured step, replayed with programmatic dependent launch, draws the tokens
and leaves the bits of the same steps run one call at a time; the operators of
the eager run are checked against the 64-bit references on the way."""
import math

import numpy as np
import pytest

import synth
from oracle import decode as ref

pytestmark = pytest.mark.gpu
H, HQ, HKV, D, INTER, VOCAB, LAYERS, PS, CTX = 1024, 16, 4, 64, 1280, 2048, 2, 16, 400


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


class Model:
    def __init__(self, mq, kv_type):
        import torch
        self.mq, g = mq, synth.rng("decode-step")
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        pack = lambda fmt, r, c: (fmt, dev(mq.mq_repack(fmt, synth.blocks(fmt, g, r, c), r, c)), r)  # noqa: E731
        self.layers = []
        for _ in range(LAYERS):
            self.layers.append(dict(
                qkv=[pack("q4k", HQ * D, H), pack("q4k", HKV * D, H), pack("q6k", HKV * D, H)], o=pack("q4k", H, HQ * D),
                gate=pack("q4k", INTER, H), up=pack("q4k", INTER, H), down=pack("q6k", H, INTER),
                g1=dev(synth.normal(g, H, 1.0, 0.1)), g2=dev(synth.normal(g, H, 1.0, 0.1)),
                qg=dev(synth.normal(g, D, 1.0, 0.1)), kg=dev(synth.normal(g, D, 1.0, 0.1)),
                bias=[dev(synth.normal(g, n * D) * np.float32(0.1)) for n in (HQ, HKV, HKV)]))
        self.head, self.gf = pack("q6k", VOCAB, H), dev(synth.normal(g, H, 1.0, 0.1))
        self.embed = dev(synth.normal(g, VOCAB * H).reshape(VOCAB, H))
        self.rope = mq.mq_rope_table(1e6 ** (-np.arange(0, D, 2) / D))
        self.kv_type, self.pages_per_layer = kv_type, CTX // PS + 1
        self.table = dev(np.random.default_rng(3).permutation(self.pages_per_layer).astype(np.int32)[None, : CTX // PS])
        self.u = dev(g.uniform(0, 1, 64).astype(np.float32))
        self.params = dict(temperature=dev(np.float32([0.9])), top_k=dev(np.int32([50])), top_p=dev(np.float32([0.95])),
                           min_p=dev(np.float32([0.01])))

    def state(self, length):
        """Caches filled with `length` tokens, the buffers of a step."""
        import torch
        mq = self.mq
        gen = torch.Generator(device="cuda")
        gen.manual_seed(7)
        s = type("S", (), {})()
        s.kv = [mq.MQKVCache(self.kv_type, self.pages_per_layer, PS, HKV, D) for _ in range(LAYERS)]
        n = length
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        seq = torch.zeros(n, dtype=torch.int32, device="cuda")
        for c in s.kv:
            r = [torch.randn(n, w * D, generator=gen, device="cuda") for w in (HQ, HKV, HKV)]
            mq.mq_rope_append(c, *r, pos, self.table, rope=self.rope, seq=seq)
        e = lambda *k, dtype=torch.float32: torch.zeros(*k, dtype=dtype, device="cuda")  # noqa: E731
        s.x, s.xn, s.q, s.k, s.v = e(H), e(H), e(1, HQ * D), e(1, HKV * D), e(1, HKV * D)
        s.q8h, s.att, s.o, s.act, s.down = e(mq.mq_q8_bytes(H), dtype=torch.uint8), e(1, HQ * D), e(H), e(INTER), e(H)
        s.q8a, s.q8i = e(mq.mq_q8_bytes(HQ * D), dtype=torch.uint8), e(mq.mq_q8_bytes(INTER), dtype=torch.uint8)
        s.logits, s.token, s.prob = e(1, VOCAB), e(1, dtype=torch.int32), e(1)
        s.pos, s.len = torch.full((1,), n, dtype=torch.int32, device="cuda"), torch.full((1,), n + 1, dtype=torch.int32, device="cuda")
        s.step = torch.zeros(1, dtype=torch.int64, device="cuda")
        s.tokens = torch.full((64,), -9, dtype=torch.int32, device="cuda")
        s.ws = mq.mq_attn_workspace(s.kv[0], HQ, 1, CTX)
        s.ws_qkv = mq.mq_gemv_group_workspace(self.layers[0]["qkv"], H)
        s.ws_o, s.ws_d, s.ws_h = (mq.mq_gemv_workspace(*x) for x in ((H, HQ * D), (H, INTER), (VOCAB, H)))
        s.x.copy_(self.embed[11])
        return s

    def step(self, s, check=None):
        import torch
        mq = self.mq
        for i, L in enumerate(self.layers):
            mq.mq_rmsnorm_quant_q8(s.x, L["g1"], 1e-6, y=s.xn, q8=s.q8h)
            mq.mq_gemv_group_q8(L["qkv"], s.q8h, H, ys=[s.q[0], s.k[0], s.v[0]], ws=s.ws_qkv)
            mq.mq_rope_append(s.kv[i], s.q, s.k, s.v, s.pos, self.table, q_out=s.q, rope=self.rope,
                              q_bias=L["bias"][0], k_bias=L["bias"][1], v_bias=L["bias"][2], q_gain=L["qg"], k_gain=L["kg"])
            mq.mq_attn_decode(s.kv[i], s.q, s.len, self.table, 1 / math.sqrt(D), out=s.att, q8=s.q8a, ws=s.ws, max_len=CTX)
            if check:
                check(s, i)
            mq.mq_gemv(L["o"][0], L["o"][1], s.q8a, H, HQ * D, y=s.o, ws=s.ws_o)
            s.x.add_(s.o)
            mq.mq_rmsnorm_quant_q8(s.x, L["g2"], 1e-6, y=s.xn, q8=s.q8h)
            mq.mq_gemv_gateup_swiglu_q8("q4k", L["gate"][1], L["up"][1], s.q8h, INTER, H, act=s.act, q8_out=s.q8i)
            mq.mq_gemv("q6k", L["down"][1], s.q8i, H, INTER, y=s.down, ws=s.ws_d)
            s.x.add_(s.down)
        mq.mq_rmsnorm_quant_q8(s.x, self.gf, 1e-6, y=s.xn, q8=s.q8h)
        mq.mq_gemv("q6k", self.head[1], s.q8h, VOCAB, H, y=s.logits[0], ws=s.ws_h)
        mq.mq_sample(s.logits, self.u[s.step], token=s.token, prob=s.prob, **self.params)
        s.tokens.scatter_(0, s.step, s.token)
        torch.index_select(self.embed, 0, s.token, out=s.x.view(1, H))
        s.pos.add_(1), s.len.add_(1), s.step.add_(1)


def values(c):
    import torch
    raw = (c.k.view(torch.int16), c.v.view(torch.int16)) if c.kv_type == "bf16" else (c.k, c.v)
    return [ref.unpack_pages(t.cpu().numpy().view(np.uint16) if c.kv_type == "bf16" else t.cpu().numpy(), c.kv_type, PS, D)
            for t in raw]


@pytest.mark.parametrize("kv_type,length", [("f16", 12), ("q8", 300), ("bf16", 190)])
def test_a_captured_step_draws_the_tokens_of_the_eager_steps(mq, kv_type, length):
    import torch
    m = Model(mq, kv_type)
    steps = 10
    eager = m.state(length)
    worst = []

    def check(s, i):
        torch.cuda.synchronize()
        n = int(s.len.item())
        kp, vp = values(s.kv[i])
        table = m.table[0].cpu().numpy()
        want, parts = ref.attention(s.q[0].cpu().numpy().reshape(HQ, D), ref.gather(kp, table, n), ref.gather(vp, table, n),
                                    1 / math.sqrt(D), parts=True)
        err = np.abs(s.att[0].cpu().numpy().reshape(HQ, D) - want)
        worst.append((err / ref.attention_bound(want, parts)).max())
        d, qs, sm = mq.mq_q8_unpack_host(mq.mq_quantize_q8(s.att[0].clone()).cpu().numpy(), HQ * D)
        d2, qs2, sm2 = mq.mq_q8_unpack_host(s.q8a.cpu().numpy(), HQ * D)
        assert np.array_equal(d, d2) and np.array_equal(qs, qs2) and np.array_equal(sm, sm2)

    for k in range(steps):
        m.step(eager, check if k in (0, steps - 1) else None)
        torch.cuda.synchronize()
        tok, pr, kept, gap = ref.sample(eager.logits[0].cpu().numpy(), float(m.u[k]), float(np.float32(0.9)), 50,
                                        float(np.float32(0.95)), float(np.float32(0.01)))
        assert int(eager.token) == tok or gap < 2.0 ** -22
    assert max(worst) <= 1.0

    graph = m.state(length)
    st = torch.cuda.Stream()
    mq.mq_set_pdl(True)
    try:
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            m.step(graph)
        for _ in range(steps):
            gr.replay()
        torch.cuda.synchronize()
    finally:
        mq.mq_set_pdl(False)
    assert graph.tokens[:steps].tolist() == eager.tokens[:steps].tolist()
    assert len(set(eager.tokens[:steps].tolist())) > 1
    assert torch.equal(graph.logits, eager.logits) and torch.equal(graph.x, eager.x)
    for a, b in zip(graph.kv, eager.kv):
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
