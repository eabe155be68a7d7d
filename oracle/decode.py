"""Plain 64-bit numpy references of the operators around the GEMVs of a decode
step: rotation and paged append, attention over a paged cache, the draw of a
token.  TEST INFRASTRUCTURE ONLY, like the rest of this package; it imports
nothing from the library and works on dense per-sequence arrays and on cache
pages in the layouts that include/mq.h states.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ cache pages
def unpack_pages(raw: np.ndarray, kv: str, ps: int, d: int) -> np.ndarray:
    """Pages as stored -> [n_pages, heads, ps, d] float64.  raw: float16 values
    (f16), uint16 bits (bf16) or uint8 bytes (q8: codes, then fp16 scales)."""
    if kv == "f16":
        return raw.astype(np.float64)
    if kv == "bf16":
        return (raw.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    n, h = raw.shape[:2]
    codes = np.ascontiguousarray(raw[..., : ps * d]).view(np.int8).reshape(n, h, ps, d // 32, 32)
    scale = np.ascontiguousarray(raw[..., ps * d:]).view(np.float16).reshape(n, h, ps, d // 32, 1)
    return (codes.astype(np.float64) * scale.astype(np.float64)).reshape(n, h, ps, d)


def gather(pages: np.ndarray, table_row, n: int) -> np.ndarray:
    """The first n cached tokens of a sequence: [heads, n, d]."""
    _, h, ps, d = pages.shape
    used = np.asarray(table_row[: -(-n // ps)], np.int64)
    return pages[used].transpose(1, 0, 2, 3).reshape(h, -1, d)[:, :n]


# ------------------------------------------------------------------ rotation and append
def heads_of(x, bias, gain, eps, d):
    """[nt, heads * d] -> [nt, heads, d] after bias and norm, and the same of
    the magnitudes (|x| + |bias| in x's place), which bound the roundings."""
    x = x.astype(np.float64)
    mag = np.abs(x)
    if bias is not None:
        x, mag = x + bias.astype(np.float64), mag + np.abs(bias.astype(np.float64))
    x, mag = x.reshape(len(x), -1, d), mag.reshape(len(x), -1, d)
    if gain is not None:
        s = gain.astype(np.float64) / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        x, mag = x * s, mag * np.abs(s)
    return x, mag


def rotate(x, mag, pos, freqs, style):
    """Rotated heads, and |a| + |b| of each value's pair (its own magnitude
    where it is not rotated)."""
    r = 2 * len(freqs)
    phi = np.outer(np.asarray(pos, np.float64), np.asarray(freqs, np.float64))[:, None, :]
    i = np.arange(r // 2)
    ia, ib = (i, i + r // 2) if style == "half" else (2 * i, 2 * i + 1)
    out, m = x.copy(), mag.copy()
    out[..., ia] = x[..., ia] * np.cos(phi) - x[..., ib] * np.sin(phi)
    out[..., ib] = x[..., ib] * np.cos(phi) + x[..., ia] * np.sin(phi)
    m[..., ia] = m[..., ib] = mag[..., ia] + mag[..., ib]
    return out, m


# ------------------------------------------------------------------ attention
def attention(q, k, v, scale, softcap=0.0, window=0, parts=False):
    """One query row [heads, d] over k, v [kv heads, n, d] (float64).  parts:
    also the probabilities, |score| sums and v that an error bound needs."""
    hq, d = q.shape
    hkv, n, _ = k.shape
    first = max(0, n - window) if window else 0
    if n - first == 0:
        return (np.zeros((hq, d)), None) if parts else np.zeros((hq, d))
    qg = q.astype(np.float64).reshape(hkv, hq // hkv, d)
    s = np.matmul(qg, k[:, first:].transpose(0, 2, 1)) * scale
    if softcap:
        s = softcap * np.tanh(s / softcap)
    e = np.exp(s - s.max(-1, keepdims=True))
    e /= e.sum(-1, keepdims=True)
    out = np.matmul(e, v[:, first:]).reshape(hq, d)
    if not parts:
        return out
    mag = np.matmul(np.abs(qg), np.abs(k[:, first:]).transpose(0, 2, 1)) * abs(scale)
    return out, (e, mag, s.max(-1, keepdims=True) - s, v[:, first:])


def attention_bound(out, parts, softcap=0.0):
    """How far an f32 evaluation of `attention` with exact products may be off,
    value by value, in units of 2^-24:
    a score: q's parts (2^-22) 4, 16 sums of the products (truncating, 2^-23) 32,
      the factor 3, all of sum |q k| scale; the difference to the maximum 2 of it;
      a capped score: tanh 4 and two products of the cap;
    a probability: its score's error, exp2 4, its split 4, one rescaling product
      a tile is common to the sum and cancels but for its rounding: taken as 16;
    the sums over tokens: 2 a tile of 16 of a warp's quarter, of sum p |v|; the
    division and the join 16;
    and, not relative to p: its fp16 parts end at fp16's last step, 2^-25 under
    a factor of 2^14 (and of up to 2 of the largest value in a q8 tile), so a
    term is off by up to 2^-38 max |v| however small p is (f32 itself ends at
    2^-126)."""
    if parts is None:
        return np.zeros_like(out)
    e, mag, gap, v = parts
    n = e.shape[-1]
    r = 39 * mag + 2 * gap + 24 + 6 * softcap
    hkv, grp, _ = e.shape
    pv = np.matmul(e * (r + n / 32 + 16), np.abs(v))       # each term's own error
    common = (e * r).sum(-1, keepdims=True)                              # the sum that divides
    floor = 2.0 ** -38 * n * np.abs(v).max(axis=(1, 2), keepdims=True)
    return (2.0 ** -24 * (pv + common * np.matmul(e, np.abs(v))) + floor).reshape(out.shape)


# ------------------------------------------------------------------ sampling
def sample(logits, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, probability among the kept, kept mask, distance of the draw
    from the nearest border of the token's interval).  NaN counts as -inf."""
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    if x.max() == -np.inf:
        return -1, 0.0, np.zeros(len(x), bool), np.inf
    order = np.argsort(-x, kind="stable")
    top = x[order[0]]
    if t <= 0:
        n, w = 1, np.ones(1)
    else:
        with np.errstate(invalid="ignore"):
            z = np.where(x[order] == top, 0.0, (x[order] - top) / t)
        w = np.exp(z)
        n = len(x) if k <= 0 else min(k, len(x))
        if p < 1:
            c = np.cumsum(w[:n])
            n = min(n, 1 + int(np.searchsorted(c, p * c[-1], "left")))
        n = max(1, min(n, int((w >= m).sum())))
        while n > 1 and w[n - 1] == 0.0:
            n -= 1
    kept = np.zeros(len(x), bool)
    kept[order[:n]] = True
    weight = np.zeros(len(x))
    weight[order[:n]] = w[:n]
    c = np.cumsum(weight)
    at = int(np.searchsorted(c, u * c[-1], "right"))
    at = min(at, int(np.flatnonzero(kept)[-1]))
    lo = c[at] - weight[at]
    return at, weight[at] / c[-1], kept, min(u * c[-1] - lo, c[at] - u * c[-1]) / c[-1]


# ------------------------------------------------------------------ sharp checks of an attention
U = 2.0 ** -24  # half a step of f32


def parts_of(x, kind, n):
    """x as the sum of n successive roundings to fp16 or bf16 (float64)."""
    rest, out = np.asarray(x, np.float64), 0.0
    for _ in range(n):
        if kind == "bf16":
            b = rest.astype(np.float32).view(np.uint32).astype(np.uint64)
            p = ((b + 0x7fff + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32).astype(np.float64)
        else:
            p = rest.astype(np.float16).astype(np.float64)
        out, rest = out + p, rest - p
    return out


def attention_in_parts(q, k, v, scale, kind, n_q, n_p):
    """`attention` with q in n_q parts and the weights of the values in n_p parts,
    and nothing else rounded: what an evaluation through 16-bit products loses.
    fp16 parts are of q under a power of two that brings a head's largest value
    to [2^13, 2^14), and of 2^14 p."""
    hq, d = q.shape
    hkv = len(k)
    q = q.astype(np.float64)
    f, g = np.ones((hq, 1)), 1.0
    if kind == "fp16":
        f, g = 2.0 ** (13 - np.floor(np.log2(np.abs(q).max(-1, keepdims=True)))), 2.0 ** 14
    qg = (parts_of(q * f, kind, n_q) / f).reshape(hkv, hq // hkv, d)
    s = np.matmul(qg, k.transpose(0, 2, 1)) * scale
    e = np.exp(s - s.max(-1, keepdims=True))
    return (np.matmul(parts_of(e * g, kind, n_p) / g, v) / e.sum(-1, keepdims=True)).reshape(hq, d)


class TwoTokens:
    """A row in which two tokens alone matter, and every rounding on the way to
    the result can be counted: key A is one value of 1, key B another, and all
    other keys are -1 at a third place, where the queries are large.  Value B is
    +1 or -1, all others are 0, so a result is +-w or 0 with w = 1 / (1 + e^(s_A - s_B)).

    of="queries": s_A and s_B are 8 to 16, of 24 bits, so what a query's parts
    lose shows.  of="weights": s_A = 0 and s_B = -0.7 to 0, so that the weight of
    B is 0.5 to 1, of 24 bits, beside the largest in the same tile of 16."""

    def __init__(self, rng, hq, hkv, d, n, of):
        self.of, grp = of, hq // hkv
        self.q = rng.uniform(-15, 15, (hkv, grp, d)).astype(np.float32)
        self.k, self.v = np.zeros((hkv, n, d)), np.zeros((hkv, n, d))
        for h in range(hkv):
            a, b, c = rng.choice(d, 3, replace=False)
            tile = 16 * rng.integers(0, n // 16) if of == "weights" else 0
            ta, tb = tile + rng.choice(min(16, n) if of == "weights" else n, 2, replace=False)
            self.k[h, :, c] = -1.0
            self.k[h, [ta, tb]] = 0.0
            self.k[h, ta, a] = self.k[h, tb, b] = 1.0
            self.v[h, tb] = rng.choice([-1.0, 1.0], d)
            if of == "queries":
                self.q[h, :, a] = rng.uniform(8, 16, grp)
                self.q[h, :, b] = self.q[h, :, a] + rng.uniform(-2, 2, grp)
                self.q[h, :, c] = 15.9
            else:
                self.q[h, :, a], self.q[h, :, b], self.q[h, :, c] = 0.0, -rng.uniform(0, 0.69, grp), 25.0
        self.q = self.q.reshape(hq, d)

    def bound(self, want, fp16):
        """How far an f32 evaluation with every part may be off, value by value.
        s: fp16 parts end 2^-23 below a head's largest query, bf16's three hold
        all of it; their sum rounds 2, the factor 1 (its own 3 roundings are
        common, so relative to s_A - s_B), the difference to the maximum 1;
        exp2: 2 ulp = 4.
        w: the parts of p 1; the sums 4 of the value's side and 6 of the
        divisor's, two rescalings and the warps' exchange 2 each side, the
        division and its product 2: 17, of |w|."""
        w = np.abs(want)
        top = np.abs(self.q).max(-1, keepdims=True)
        s = 16.0 + 2 if self.of == "queries" else 0.69
        gap = 2.0 if self.of == "queries" else 0.69
        raw = (2 * 2.0 ** np.floor(np.log2(top)) if fp16 else 0.0) + 2 * s
        return U * (w * (1 - w) * (2 * raw + 2 * s + 4 * gap + 4) + 17 * w + 1)


def exact_mean_bound(want):
    """The mean of whole numbers under equal scores: weights of 1 and sums under
    2^24 are exact in f32, so the division and its product round once each."""
    return 2.0 ** -23 * (1 + 2.0 ** -20) * np.abs(want)
