"""The sharp checks of test_gpu_attn_exact.py, with mistakes planted in the
reference: a token lost, repeated or taken for its neighbour, a part of the
queries or of the weights left out."""
import numpy as np
import pytest

from oracle import decode as ref


def test_parts_hold_the_bits_of_their_number():
    x = np.random.default_rng(0).uniform(0.5, 1, 1000).astype(np.float32)
    for kind, bits in (("fp16", (11, 22)), ("bf16", (8, 16, 24))):
        for n, b in enumerate(bits, 1):
            err = np.abs(ref.parts_of(x, kind, n) - x).max()
            assert err <= 2.0 ** -(b + 1) and (b == 24 or err > 2.0 ** -(b + 3)), (kind, n)
    assert np.all(ref.parts_of(x, "bf16", 3) == x)


@pytest.mark.parametrize("of", ["queries", "weights"])
@pytest.mark.parametrize("kind,parts", [("fp16", 2), ("bf16", 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_missing_part_breaks_the_two_token_bound(kind, parts, d, of):
    rng = np.random.default_rng(d)
    over = {"all": [], "one query part less": [], "one weight part less": []}
    for _ in range(40):
        t = ref.TwoTokens(rng, 10, 2, d, int(rng.integers(17, 200)), of)
        want = ref.attention(t.q, t.k, t.v, 1.0)
        bound = t.bound(want, kind == "fp16")
        for name, n_q, n_p in (("all", parts, parts), ("one query part less", parts - 1, parts),
                               ("one weight part less", parts, parts - 1)):
            got = ref.attention_in_parts(t.q, t.k, t.v, 1.0, kind, n_q, n_p)
            over[name].append((np.abs(got - want) / bound).max(-1))
    assert np.max(over["all"]) < 0.2
    assert np.mean(np.array(over["one query part less" if of == "queries" else "one weight part less"]) > 1) > 0.3


@pytest.mark.parametrize("n", [17, 4097, 20001, 70001])
def test_a_lost_token_breaks_the_mean_bound(n):
    g = np.random.default_rng(n)
    v = g.integers(-127, 128, (n, 64)).astype(np.float64)
    total = v.sum(0)
    want = total / n
    bound = ref.exact_mean_bound(want)
    assert np.abs(total).max() < 2 ** 24
    for j in g.integers(0, n - 1, 200):
        for got in ((total - v[j]) / (n - 1), (total + v[j]) / (n + 1), (total + v[j + 1] - v[j]) / n,
                    (total - v[j]) / n):
            assert np.any(np.abs(got - want) > 4 * bound)
