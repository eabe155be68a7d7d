"""Under programmatic dependent launch every input of the decode step's
operators may change between two calls of one captured chain, written by the
kernel right before: nothing may be read early, and nothing may be kept from the
call before (not in L1 either, where the first call has left the old values)."""
import math

import numpy as np
import pytest

import synth

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


def changes_in_a_chain(mq, inputs, others, fresh, call):
    """fresh() -> outputs, call(inputs, outputs) launches.  For each input: first with its value, then, in the same
    chain, with the other one copied over it by the kernel right before; against the same calls one at a time."""
    import torch
    for name, second in others.items():
        first = inputs[name]
        want = []
        for value in (first, second):
            want.append(fresh())
            call({**inputs, name: value}, want[-1])
            torch.cuda.synchronize()
        assert not all(torch.equal(a, b) for a, b in zip(*want)), name   # the change shows
        live, a, b = first.clone(), fresh(), fresh()
        st = torch.cuda.Stream()
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        mq.mq_set_pdl(True)
        try:
            with torch.cuda.graph(gr, stream=st):
                mq.mq_copy(live, first)
                call({**inputs, name: live}, a)
                mq.mq_copy(live, second)
                call({**inputs, name: live}, b)
        finally:
            mq.mq_set_pdl(False)
        for _ in range(5):
            gr.replay()
        torch.cuda.synchronize()
        for got, ref in zip((a, b), want):
            assert all(torch.equal(x, y) for x, y in zip(got, ref)), name


def normal(g, *shape):
    import torch
    return torch.from_numpy((synth.normal(g, int(np.prod(shape))) * np.float32(2)).reshape(shape)).cuda()


@pytest.mark.parametrize("kv,d,style", [("f16", 128, "half"), ("q8", 128, "half"), ("bf16", 64, "pairs")])
def test_append(mq, kv, d, style):
    import torch
    g, nt, hq, hkv, ps = synth.rng("chain append", kv, d), 160, 16, 4, 16
    i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()  # noqa: E731
    inputs = dict(q=normal(g, nt, hq * d), k=normal(g, nt, hkv * d), v=normal(g, nt, hkv * d),
                  positions=i32(np.arange(nt)), pages=i32(np.arange(2 * 64).reshape(2, 64)), seq=i32(np.arange(nt) % 2),
                  rope=mq.mq_rope_table(1e4 ** (-np.arange(0, d, 2) / d)), q_bias=normal(g, hq * d),
                  k_bias=normal(g, hkv * d), v_bias=normal(g, hkv * d), q_gain=normal(g, d), k_gain=normal(g, d))
    others = {n: normal(g, *t.shape) for n, t in inputs.items() if t.dtype == torch.float32}
    others.update(positions=i32(np.arange(nt) + 700), pages=i32(np.arange(2 * 64).reshape(2, 64)[::-1]),
                  seq=i32((np.arange(nt) + 1) % 2), rope=mq.mq_rope_table(5e5 ** (-np.arange(0, d, 2) / d)))

    def fresh():
        c = mq.MQKVCache(kv, 128, ps, hkv, d)
        return torch.zeros(nt, hq * d, device="cuda"), c.k, c.v

    def call(a, out):
        a = dict(a)
        c = mq.MQKVCache(kv, 128, ps, hkv, d, k=out[1], v=out[2])
        mq.mq_rope_append(c, a.pop("q"), a.pop("k"), a.pop("v"), a.pop("positions"), a.pop("pages"), q_out=out[0],
                          style=style, **a)
    changes_in_a_chain(mq, inputs, others, fresh, call)


@pytest.mark.parametrize("kv,lens", [("f16", [3000, 17, 500, 64]), ("q8", [3000, 17, 500, 64]), ("bf16", [40, 1, 0, -1] * 10)])
def test_attention(mq, kv, lens):
    import torch
    g, hq, hkv, d, ps = synth.rng("chain attention", kv), 8, 2, 128, 16
    nt, width = len(lens), 192
    i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()  # noqa: E731
    cache = mq.MQKVCache(kv, 256, ps, hkv, d)
    pos = i32(np.arange(256 * ps))
    mq.mq_rope_append(cache, normal(g, 256 * ps, hq * d), normal(g, 256 * ps, hkv * d), normal(g, 256 * ps, hkv * d), pos,
                      i32(np.arange(256).reshape(1, 256)), seq=torch.zeros_like(pos))
    table = np.stack([g.permutation(256)[:width] for _ in range(nt)])
    inputs = dict(q=normal(g, nt, hq * d), lens=i32(lens), pages=i32(table), seq=i32(np.arange(nt)))
    others = dict(q=normal(g, nt, hq * d), lens=i32(np.roll(lens, 1)), pages=i32(table[:, ::-1]),
                  seq=i32(np.arange(nt)[::-1]))
    ws = mq.mq_attn_workspace(cache, hq, nt, width * ps)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda") if ws is None else ws

    def call(a, out):
        mq.mq_attn_decode(cache, a["q"], a["lens"], a["pages"], 1 / math.sqrt(d), out=out[0], ws=ws, seq=a["seq"])
    changes_in_a_chain(mq, inputs, others, lambda: [torch.zeros(nt, hq * d, device="cuda")], call)


@pytest.mark.parametrize("v,nt", [(3000, 8), (152064, 4)])
def test_draw(mq, v, nt):
    import torch
    g = synth.rng("chain draw", v)
    f32 = lambda x: torch.full((nt,), x, device="cuda")  # noqa: E731
    k = torch.full((nt,), 300, dtype=torch.int32, device="cuda")
    inputs = dict(logits=normal(g, nt, v), u=f32(0.4), temperature=f32(0.9), top_k=k, top_p=f32(0.8), min_p=f32(1e-3))
    others = dict(logits=normal(g, nt, v), u=f32(0.9), temperature=f32(2.5), top_k=k // 100, top_p=f32(0.1),
                  min_p=f32(0.5))

    def fresh():
        return torch.zeros(nt, dtype=torch.int32, device="cuda"), torch.zeros(nt, device="cuda")

    def call(a, out):
        mq.mq_sample(a["logits"], a["u"], temperature=a["temperature"], top_k=a["top_k"], top_p=a["top_p"],
                     min_p=a["min_p"], token=out[0], prob=out[1])
    changes_in_a_chain(mq, inputs, others, fresh, call)
