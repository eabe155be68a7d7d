"""The operators of a decode step around its GEMVs, as measurable cases: the
position rotation with the paged cache's append, the attention over that
cache, and the draw of a token.  `run` computes each in a plain form
(elementary torch operations), or calls the library's own where `own` is set.
"""
import math

import torch

own = False

GROUPS = [(40, 8), (28, 4), (32, 8), (16, 8), (16, 2), (14, 2), (8, 8), (12, 1)]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of the 14B shape (40 query and 8 key heads of 128, q/k/v biases): latency
        dict(name="append 1", op="append", nt=1, hq=40, hkv=8, d=128, rope=128, style="half", bias=True,
             norm=False, kv="f16", ps=16, pos=8191, chunk=False, pad=0),
        # a batched step with per-head norms, positions spread over the context
        dict(name="append 64 norm", op="append", nt=64, hq=32, hkv=8, d=128, rope=128, style="half",
             bias=False, norm=True, kv="bf16", ps=64, pos=32000, chunk=False, pad=0),
        # a padded batch, interleaved pairs, half of the head rotated, an odd page size
        dict(name="append 37 padded", op="append", nt=37, hq=14, hkv=2, d=64, rope=32, style="pairs",
             bias=True, norm=True, kv="f16", ps=48, pos=1000000, chunk=False, pad=5),
        # a prompt chunk of one sequence: bandwidth
        dict(name="append chunk 4096", op="append", nt=4096, hq=40, hkv=8, d=128, rope=128, style="half",
             bias=True, norm=False, kv="f16", ps=16, pos=20000, chunk=True, pad=0),
        # the first tokens of a chat: latency
        dict(name="attn 1 x 117", op="attn", nt=1, hq=40, hkv=8, d=128, kv="f16", ps=16, lo=117, hi=117,
             cap=0.0, window=0, pad=0),
        # one user, a full context
        dict(name="attn 1 x 32768", op="attn", nt=1, hq=40, hkv=8, d=128, kv="f16", ps=16, lo=32768,
             hi=32768, cap=0.0, window=0, pad=0),
        # a ragged batch over a q8 cache (28 query and 4 key heads), an empty row and padding behind it
        dict(name="attn 63 ragged q8", op="attn", nt=63, hq=28, hkv=4, d=128, kv="q8", ps=32, lo=0,
             hi=8191, cap=0.0, window=0, pad=2),
        # wide heads, capped scores, a sliding window
        dict(name="attn 8 cap window", op="attn", nt=8, hq=16, hkv=8, d=256, kv="bf16", ps=64, lo=700,
             hi=9001, cap=50.0, window=4096, pad=0),
        # the largest: a full batch of long contexts
        dict(name="attn 16 x 16384", op="attn", nt=16, hq=40, hkv=8, d=128, kv="f16", ps=64, lo=16001,
             hi=16384, cap=0.0, window=0, pad=0),
        # one user's draw from the 152064-token head with the usual chain of filters
        dict(name="sample 1", op="sample", b=1, v=152064, t=0.8, k=40, p=0.95, m=0.05, peaks=64),
        # a batch, nucleus only, near-flat logits (a nucleus of thousands)
        dict(name="sample 64 flat top-p", op="sample", b=64, v=152064, t=1.0, k=0, p=0.9, m=0.0, peaks=0),
        # an odd vocabulary, rows that start off 16-byte borders, one of them greedy
        dict(name="sample 7 odd min-p", op="sample", b=7, v=50257, t=1.3, k=0, p=1.0, m=0.02, peaks=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "sample"])
    if op == "sample":
        return dict(op=op, b=_log(rng, 1, 64), v=_log(rng, 1000, 152064), t=rng.choice([0.5, 0.7, 1.0, 1.5]),
                    k=rng.choice([0, 1, 20, 50, 1000]), p=rng.choice([1.0, 0.5, 0.9, 0.95]),
                    m=rng.choice([0.0, 0.01, 0.1]), peaks=rng.choice([0, 8, 64]))
    hq, hkv = rng.choice(GROUPS)
    d = rng.choice([64, 96, 128, 256])
    ps = rng.choice([16, 32, 48, 64, 256])
    if op == "append":
        chunk = rng.random() < 0.5
        nt = _log(rng, 1, 4096 if chunk else 256)
        nt = max(1, min(nt, 4096 * 56 * 128 // ((hq + 2 * hkv) * d)))
        return dict(op=op, nt=nt, hq=hq, hkv=hkv, d=d, rope=rng.choice([d, d, d // 2]),
                    style=rng.choice(["half", "pairs"]), bias=rng.random() < 0.5, norm=rng.random() < 0.5,
                    kv=rng.choice(["f16", "bf16"]), ps=ps, pos=_log(rng, 8192, 1000000), chunk=chunk,
                    pad=rng.choice([0, 0, 3]))
    nt = _log(rng, 1, 64)
    most = int(5e8 // (nt * hkv * d * 4))
    hi = max(1, min(_log(rng, 1, 32768), most))
    return dict(op=op, nt=nt, hq=hq, hkv=hkv, d=d, kv=rng.choice(["f16", "bf16", "q8"]), ps=ps,
                lo=_log(rng, 1, hi), hi=hi, cap=rng.choice([0.0, 0.0, 30.0]),
                window=rng.choice([0, 0, 1024]), pad=rng.choice([0, 0, 3]))


def lens_of(c):
    """Cached tokens of each row: spread over [lo, hi] by ratio; -1 for the padding rows behind them."""
    n = c["nt"]
    lo, hi = max(1, c["lo"]), c["hi"]
    lens = [int(round(hi * (lo / hi) ** (i / max(1, n - 1)))) for i in range(n)]
    if c["lo"] == 0:
        lens[-1] = 0
    return lens + [-1] * c["pad"]


def kv_bytes(kv):
    return 17 / 16 if kv == "q8" else 2


def work(case):
    c = case
    if c["op"] == "sample":
        return {"bytes": c["b"] * (4 * c["v"] + 28), "flops": 4 * c["b"] * c["v"]}
    if c["op"] == "append":
        n = c["nt"] * c["d"]
        values = c["hq"] * 8 + c["hkv"] * (8 + 2 * kv_bytes(c["kv"]))
        return {"bytes": n * values, "flops": n * (6 * c["hq"] + 7 * c["hkv"])}
    lens = [min(n, c["window"]) if c["window"] else n for n in lens_of(c) if n >= 0]
    return {"bytes": sum(lens) * 2 * c["hkv"] * c["d"] * kv_bytes(c["kv"]) + len(lens) * c["hq"] * c["d"] * 8,
            "flops": 4 * c["hq"] * c["d"] * sum(lens)}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return g


def _pack_q8(x):
    """[..., ps, D] values -> one byte row per (page, head): the int8 codes, then the fp16 scales."""
    n, h, ps, d = x.shape
    blocks = x.float().reshape(n, h, ps, d // 32, 32)
    scale = blocks.abs().amax(-1, keepdim=True) / 127
    codes = torch.round(blocks / scale.clamp_min(1e-30)).clamp(-128, 127).to(torch.int8)
    return torch.cat([codes.reshape(n, h, ps * d).view(torch.uint8),
                      scale.half().reshape(n, h, ps * d // 32).view(torch.uint8)], -1).contiguous()


def _tables(g, need, n_pages):
    """A page table: rows of distinct random pages, -1 behind each row's last."""
    width = max(1, max(need))
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    need_t = torch.tensor(need, device="cuda")
    start = torch.cumsum(need_t, 0) - need_t
    j = torch.arange(width, device="cuda")
    at = (start[:, None] + j).clamp_max(n_pages - 1)
    return torch.where(j < need_t[:, None], order[at], -1).int().contiguous()


def prepare(case, seed):
    c, g = case, _gen(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    if c["op"] == "sample":
        b, v = c["b"], c["v"]
        logits = normal(b, v, std=2.0 if c["peaks"] else 2.5)
        if c["peaks"]:  # the few tokens that a context allows
            at = torch.randint(v, (b, c["peaks"]), generator=g, device="cuda")
            logits.scatter_(1, at, 6 + 4 * normal(b, c["peaks"]))
        t = torch.full((b,), c["t"], device="cuda")
        if b > 4:
            t[3] = 0.0  # one row asks for the most likely token
        return dict(c=c, logits=logits, t=t, k=torch.full((b,), c["k"], dtype=torch.int32, device="cuda"),
                    p=torch.full((b,), c["p"], device="cuda"), m=torch.full((b,), c["m"], device="cuda"),
                    u=torch.rand(b, generator=g, device="cuda"),
                    token=torch.zeros(b, dtype=torch.int32, device="cuda"),
                    prob=torch.zeros(b, device="cuda"))

    hq, hkv, d, ps = c["hq"], c["hkv"], c["d"], c["ps"]
    dtype = torch.bfloat16 if c["kv"] == "bf16" else torch.float16
    if c["op"] == "append":
        nt, rows = c["nt"], c["nt"] + c["pad"]
        if c["chunk"]:
            pos = torch.arange(c["pos"], c["pos"] + nt, device="cuda")
            seq = torch.zeros(rows, dtype=torch.int32, device="cuda")
            width = -(-(c["pos"] + nt) // ps)
            used = -(-nt // ps) + 2  # only the chunk's pages are backed; the table names them from its place on
            table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
            order = torch.randperm(used, generator=g, device="cuda").int()
            first = c["pos"] // ps
            table[0, first:] = order[: width - first]
            n_pages = used + 1
        else:
            pos = torch.randint(max(1, c["pos"] // 2), c["pos"] + 1, (nt,), generator=g, device="cuda")
            seq = torch.arange(rows, dtype=torch.int32, device="cuda")
            width = c["pos"] // ps + 1
            n_pages = nt + 1
            table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
            table[torch.arange(nt, device="cuda"), pos // ps] = torch.randperm(nt, generator=g, device="cuda").int()
        pos = torch.cat([pos, torch.full((c["pad"],), -1, device="cuda")]).int()
        s = dict(c=c, pos=pos, seq=seq, table=table, n_pages=n_pages,
                 q=normal(rows, hq * d, std=2.0), x=normal(rows, hkv * d, std=2.0), v=normal(rows, hkv * d),
                 k_pages=normal(n_pages, hkv, ps, d, dtype=dtype), v_pages=normal(n_pages, hkv, ps, d, dtype=dtype),
                 q_out=normal(rows, hq * d), bq=None, bk=None, bv=None, gq=None, gk=None, eps=1e-6)
        if c["bias"]:
            s.update(bq=normal(hq * d), bk=normal(hkv * d, std=4.0), bv=normal(hkv * d, std=0.2))
        if c["norm"]:
            s.update(gq=1 + normal(d, std=0.1), gk=1 + normal(d, std=0.1))
        freqs = 1e6 ** (-torch.arange(0, c["rope"], 2, dtype=torch.float64) / c["rope"])
        s["freqs"] = freqs.cuda()
        if own:
            import quant_quantized_gemv_gb300 as mq
            s["rope"] = mq.mq_rope_table(freqs.numpy())
            s["kv"] = mq.MQKVCache(c["kv"], n_pages, ps, hkv, d, k=s["k_pages"], v=s["v_pages"])
        return s

    lens = lens_of(c)
    need = [-(-max(0, n) // ps) for n in lens]
    n_pages = sum(need) + 1
    shift = normal(hkv, 1, d)  # keys have channels with a mean of their own
    k_pages = normal(n_pages, hkv, ps, d, dtype=torch.float16 if c["kv"] == "q8" else dtype) + shift.to(dtype)
    v_pages = normal(n_pages, hkv, ps, d, dtype=torch.float16 if c["kv"] == "q8" else dtype)
    if c["kv"] == "q8":
        k_pages, v_pages = _pack_q8(k_pages), _pack_q8(v_pages)
    s = dict(c=c, k_pages=k_pages, v_pages=v_pages, table=_tables(g, need, n_pages),
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q=normal(len(lens), hq * d, std=2.0),
             out=normal(len(lens), hq * d), scale=1 / math.sqrt(d))
    if own:
        import quant_quantized_gemv_gb300 as mq
        s["kv"] = mq.MQKVCache(c["kv"], n_pages, ps, hkv, d, k=k_pages, v=v_pages)
        s["ws"] = mq.mq_attn_workspace(s["kv"], hq, len(lens), max(1, max(lens)))
        s["max_len"] = max(1, max(lens))
    return s


# ------------------------------------------------------------------ the library's calls
def _own_append(s):
    import quant_quantized_gemv_gb300 as mq
    mq.mq_rope_append(s["kv"], s["q"], s["x"], s["v"], s["pos"], s["table"], q_out=s["q_out"], rope=s["rope"],
                      style=s["c"]["style"], q_bias=s["bq"], k_bias=s["bk"], v_bias=s["bv"], q_gain=s["gq"],
                      k_gain=s["gk"], eps=s["eps"], seq=s["seq"])
    return s["q_out"], s["k_pages"], s["v_pages"]


def _own_attn(s):
    import quant_quantized_gemv_gb300 as mq
    return mq.mq_attn_decode(s["kv"], s["q"], s["lens"], s["table"], s["scale"], out=s["out"], ws=s["ws"],
                             softcap=s["c"]["cap"], window=s["c"]["window"], max_len=s["max_len"])


def _own_sample(s):
    import quant_quantized_gemv_gb300 as mq
    mq.mq_sample(s["logits"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"],
                 token=s["token"], prob=s["prob"])
    return s["token"], s["prob"]


# ------------------------------------------------------------------ the plain forms
def _plain_append(s):
    c, pos, d, r = s["c"], s["pos"], s["c"]["d"], s["c"]["rope"]
    angle = pos.double()[:, None, None] * s["freqs"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

    def heads(x, bias, gain):
        x = (x if bias is None else x + bias).reshape(len(pos), -1, d)
        if gain is None:
            return x
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * gain

    def rotate(x):
        a, b = (x[..., : r // 2], x[..., r // 2: r]) if c["style"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat([a, b], -1) if c["style"] == "half" else torch.stack([a, b], -1).flatten(-2)
        return torch.cat([turned, x[..., r:]], -1)

    live = (pos >= 0)[:, None]
    q = rotate(heads(s["q"], s["bq"], s["gq"])).reshape(len(pos), -1)
    s["q_out"].copy_(torch.where(live, q, s["q_out"]))
    # rows without a position write the last page, which is nobody's, with what it holds
    at = pos.clamp_min(0).long()
    page = torch.where(pos >= 0, s["table"][s["seq"].long(), at // c["ps"]], s["n_pages"] - 1).long()
    slot = at % c["ps"]
    for pages, x in ((s["k_pages"], rotate(heads(s["x"], s["bk"], s["gk"]))), (s["v_pages"], heads(s["v"], s["bv"], None))):
        old = pages[page, :, slot]
        pages[page, :, slot] = torch.where(live[:, :, None], x.to(pages.dtype), old)
    return s["q_out"], s["k_pages"], s["v_pages"]


def _values(pages, c):
    """Cache pages as [n_pages, heads, page_size, D] in 32 bits."""
    if c["kv"] != "q8":
        return pages.float()
    n, d, ps = pages.shape[0], c["d"], c["ps"]
    codes = pages[..., : ps * d].view(torch.int8).float().reshape(n, c["hkv"], ps, d // 32, 32)
    scale = pages[..., ps * d:].contiguous().view(torch.float16).float().reshape(n, c["hkv"], ps, d // 32, 1)
    return (codes * scale).reshape(n, c["hkv"], ps, d)


def _plain_attn(s):
    c, lens, d = s["c"], s["lens"], s["c"]["d"]
    n, width = s["table"].shape
    rows = s["table"].clamp_min(0).long()

    def dense(pages):  # [n, heads, tokens, D]
        x = _values(pages[rows.reshape(-1)], c).reshape(n, width, c["hkv"], c["ps"], d)
        return x.transpose(1, 2).reshape(n, c["hkv"], width * c["ps"], d)

    q = s["q"].reshape(n, c["hkv"], -1, d)
    x = torch.matmul(q, dense(s["k_pages"]).transpose(2, 3)) * s["scale"]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    j = torch.arange(width * c["ps"], device="cuda")
    seen = j < lens[:, None]
    if c["window"]:
        seen &= j >= lens[:, None] - c["window"]
    seen = seen[:, None, None, :]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.where(seen, torch.exp(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
    total = e.sum(-1, keepdim=True)
    v = dense(s["v_pages"])
    v = torch.where(seen.transpose(2, 3), v, 0.0)
    out = torch.matmul(e, v) / torch.where(total == 0, 1.0, total)
    return torch.where((lens >= 0)[:, None], out.reshape(n, -1), s["out"])


def _plain_sample(s):
    # 64 bits: the draw compares sums over the whole vocabulary with borders
    v = s["logits"].shape[1]
    x, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    t = s["t"].double()[:, None]
    greedy = t == 0
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, 1.0, t))
    rank = torch.arange(v, device="cuda")
    k = torch.where(greedy, 1, torch.where(s["k"][:, None] > 0, s["k"][:, None], v))
    w = torch.where(rank < k, w, 0.0)
    before = torch.cumsum(w, 1) - w
    p = s["p"].double()[:, None]
    keep = (rank < k) & ((p >= 1) | (before < p * w.sum(1, keepdim=True)) | (rank == 0))
    keep &= (w >= s["m"].double()[:, None]) | (rank == 0)
    # back to the order of the vocabulary
    kept = torch.zeros_like(w).scatter(1, order, torch.where(keep, w, 0.0))
    run_sum = torch.cumsum(kept, 1)
    total = run_sum[:, -1:]
    hit = (run_sum > s["u"].double()[:, None] * total) & (kept > 0)
    token = torch.argmax(hit.to(torch.uint8), 1, keepdim=True)
    prob = kept.gather(1, token) / total
    return token[:, 0].int(), prob[:, 0].float()


def run(state):
    op = state["c"]["op"]
    if own:
        return {"append": _own_append, "attn": _own_attn, "sample": _own_sample}[op](state)
    return {"append": _plain_append, "attn": _plain_attn, "sample": _plain_sample}[op](state)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _exact_append(s):
    c, d, r = s["c"], s["c"]["d"], s["c"]["rope"]
    half, n = r // 2, len(s["pos"])
    phase = torch.outer(s["pos"].double(), s["freqs"])
    turn = torch.polar(torch.ones_like(phase), phase)[:, None, :]  # a rotation is a complex product

    def place(x, bias, gain, rotated):
        x = x.double()
        if bias is not None:
            x = x + bias.double()
        x = x.view(n, -1, d)
        if gain is not None:
            x = x * (gain.double() * torch.rsqrt(x.square().sum(-1, keepdim=True) / d + s["eps"]))
        if not rotated:
            return x
        x = x.clone()
        if c["style"] == "half":
            z = torch.complex(x[..., :half], x[..., half:r]) * turn
            x[..., :half], x[..., half:r] = z.real, z.imag
        else:
            z = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * turn
            x[..., 0:r:2], x[..., 1:r:2] = z.real, z.imag
        return x

    q_out = s["q_out"].double()
    q_out[: c["nt"]] = place(s["q"], s["bq"], s["gq"], True).reshape(n, -1)[: c["nt"]]
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    k, v = place(s["x"], s["bk"], s["gk"], True), place(s["v"], s["bv"], None, False)
    pos = s["pos"][: c["nt"]].long()
    page = s["table"][s["seq"][: c["nt"]].long(), torch.div(pos, c["ps"], rounding_mode="floor")].long()
    for dst, src in ((k_pages, k), (v_pages, v)):
        flat = dst.transpose(1, 2).reshape(-1, c["hkv"], d)  # (page, slot) rows
        flat[page * c["ps"] + pos % c["ps"]] = src[: c["nt"]]
        dst.copy_(flat.view(s["n_pages"], c["ps"], c["hkv"], d).transpose(1, 2))
    return q_out, k_pages, v_pages


def _exact_attn(s):
    c, d, ps = s["c"], s["c"]["d"], s["c"]["ps"]
    g = c["hq"] // c["hkv"]
    out = s["out"].double()
    for i, n in enumerate(lens_of(c)):
        if n < 0:
            continue
        out[i] = 0
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        pages = s["table"][i, : -(-n // ps)].long()
        k, v = (_values(x[pages], c).transpose(0, 1).reshape(c["hkv"], -1, d)[:, first:n].double()
                for x in (s["k_pages"], s["v_pages"]))
        q = s["q"][i].double().view(c["hkv"], g, d)
        x = torch.einsum("hgd,htd->hgt", q, k) / math.sqrt(d)
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        out[i] = torch.einsum("hgt,htd->hgd", torch.softmax(x, -1), v).reshape(-1)
    return out


def _exact_sample(s):
    import numpy
    logits = s["logits"].double().cpu().numpy()
    t, k, p, m, u = (s[x].cpu().numpy() for x in "tkpmu")
    tokens, probs = [], []
    for i, x in enumerate(logits):
        if t[i] == 0:
            tokens.append(int(x.argmax()))
            probs.append(1.0)
            continue
        order = numpy.argsort(-x, kind="stable")
        w = numpy.exp((x[order] - x[order[0]]) / float(t[i]))
        n = len(w) if k[i] <= 0 else min(int(k[i]), len(w))
        if p[i] < 1:
            n = min(n, 1 + int(numpy.searchsorted(numpy.cumsum(w[:n]), float(p[i]) * w[:n].sum(), "left")))
        n = max(1, min(n, int((w >= float(m[i])).sum())))
        chosen = numpy.sort(order[:n])
        weight = numpy.exp((x[chosen] - x[order[0]]) / float(t[i]))
        at = int(numpy.searchsorted(numpy.cumsum(weight), float(u[i]) * weight.sum(), "right"))
        at = min(at, n - 1)
        tokens.append(int(chosen[at]))
        probs.append(weight[at] / weight.sum())
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "sample": _exact_sample}[case["op"]](s)
