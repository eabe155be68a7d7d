"""mq_add_rmsnorm_quant_q8 against a plain 64-bit reference (oracle.decode.add_rmsnorm derives the tolerance), its q8
planes against mq_quantize_q8 of what it wrote, byte for byte."""
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
    def __init__(self, nt, n, post=False, gate="", scale=1.0, std=1.0):
        g = synth.rng("residual", nt, n, post, gate, scale)
        normal = lambda *k: synth.normal(g, int(np.prod(k))).reshape(k)  # noqa: E731
        self.nt, self.n, self.scale = nt, n, scale
        self.x, self.y = normal(nt, n) * np.float32(3 * std), normal(nt, n) * np.float32(std)
        self.gain = 1 + normal(n) * np.float32(0.1)
        self.post = 1 + normal(n) * np.float32(0.1) if post else None
        self.gate = None if not gate else normal(1 if gate == "channel" else nt, n)

    def args(self, mq):
        import torch
        return dict(x=dev(self.x), y=dev(self.y), gain=dev(self.gain), eps=1e-6, post_gain=dev(self.post),
                    gate=dev(self.gate), scale=self.scale, x_out=torch.full((self.nt, self.n), 7.0, device="cuda"),
                    z=torch.full((self.nt, self.n), 7.0, device="cuda"),
                    q8=torch.full((self.nt * mq.mq_q8_bytes(self.n) + 16,), 0x55, dtype=torch.uint8, device="cuda"))

    def check(self, mq, out, z, q8):
        import torch
        torch.cuda.synchronize()
        # a lane's groups of four (a whole warp's row, at the most, below 4096 values), a butterfly, up to 32 warps
        depth = 4 * -(-self.n // 4 // 32) if self.n < 4096 else 4 * max(8, -(-self.n // 4096))
        want_x, want_z, tol_x, tol_z = ref.add_rmsnorm(self.x, self.y, self.gain.astype(np.float64), float(np.float32(1e-6)),
                                                       self.post, self.gate, float(np.float32(self.scale)), depth + 37)
        assert np.all(np.abs(out.cpu().numpy() - want_x) <= tol_x)
        assert np.all(np.abs(z.cpu().numpy() - want_z) <= tol_z)
        nb = mq.mq_q8_bytes(self.n)
        planes = q8[:self.nt * nb].reshape(self.nt, nb).cpu().numpy()
        for i in range(0, self.nt, max(1, self.nt // 9)):
            row = mq.mq_quantize_q8(z[i].clone()).cpu().numpy()
            for a, b in zip(mq.mq_q8_unpack_host(planes[i], self.n), mq.mq_q8_unpack_host(row, self.n)):
                assert np.array_equal(a, b), i
        if q8.numel() > self.nt * nb:
            assert (q8[self.nt * nb:] == 0x55).all()


@pytest.mark.parametrize("n", [32, 64, 96, 160, 1024, 2080, 3584, 4096, 4128, 5120, 8192, 8224, 13824, 16384, 16416, 32768,
                               32800, 70016])
@pytest.mark.parametrize("nt,post,gate,scale", [(1, False, "", 1.0), (3, True, "channel", 0.22), (2, True, "row", -1.5)])
def test_against_reference(mq, n, nt, post, gate, scale):
    c = Case(nt, n, post, gate, scale)
    c.check(mq, *mq.mq_add_rmsnorm_quant_q8(**c.args(mq)))


@pytest.mark.parametrize("nt,n", [(64, 5120), (700, 3584), (2000, 96), (333, 8192), (150, 16416), (160, 33024)])
@pytest.mark.parametrize("post", [False, True])
def test_many_rows(mq, nt, n, post):
    c = Case(nt, n, post, "row" if nt % 2 else "channel", 0.7)
    c.check(mq, *mq.mq_add_rmsnorm_quant_q8(**c.args(mq)))


@pytest.mark.parametrize("std", [1e-6, 1e4])
def test_magnitudes(mq, std):
    c = Case(4, 5120, True, "", 1.0, std)
    c.check(mq, *mq.mq_add_rmsnorm_quant_q8(**c.args(mq)))


def test_zero_rows(mq):
    """x + y = 0: z is 0, its plane too."""
    import torch
    c = Case(2, 160)
    c.y = -c.x
    out, z, q8 = mq.mq_add_rmsnorm_quant_q8(**c.args(mq))
    torch.cuda.synchronize()
    assert not out.any() and not z.any()
    for plane in q8[:2 * mq.mq_q8_bytes(160)].reshape(2, -1).cpu().numpy():
        assert not any(x.any() for x in mq.mq_q8_unpack_host(plane, 160))


@pytest.mark.parametrize("n", [5120, 33024])
def test_in_place_and_made_outputs(mq, n):
    """x_out = x, z = y, planes made by the call, a strided gate, one row of one dimension: the same bits."""
    import torch
    c = Case(5, n, True, "row", 0.5)
    a = c.args(mq)
    want = mq.mq_add_rmsnorm_quant_q8(**a)
    b = c.args(mq)
    wide = torch.zeros(5, n + 64, device="cuda")
    wide[:, :n] = b["gate"]
    b.update(x_out=b["x"], z=b["y"], q8=None, gate=wide[:, :n])
    got = mq.mq_add_rmsnorm_quant_q8(**b)
    torch.cuda.synchronize()
    assert got[0] is b["x"] and got[1] is b["y"]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[2], want[2][:got[2].numel()])
    one = mq.mq_add_rmsnorm_quant_q8(dev(c.x[2]), dev(c.y[2]), a["gain"], 1e-6, post_gain=a["post_gain"],
                                     gate=a["gate"][2], scale=0.5)
    torch.cuda.synchronize()
    assert one[0].shape == (n,) and torch.equal(one[0], want[0][2]) and torch.equal(one[1], want[1][2])


def test_a_nan_stays_in_its_row(mq):
    import torch
    c = Case(3, 4096, True)
    c.y[1, 77] = np.nan
    out, z, _ = mq.mq_add_rmsnorm_quant_q8(**c.args(mq))
    torch.cuda.synchronize()
    assert torch.isnan(z[1]).all() and torch.isfinite(z[[0, 2]]).all() and torch.isfinite(out[[0, 2]]).all()


def test_equals_the_two_calls_it_replaces(mq):
    """Without a norm behind the block: x + y, bit for bit, then what mq_rmsnorm_quant_q8 gives: two f32 evaluations of
    one factor, each within the reference's bound of it (depth 8 + 37 and 12 + 21 roundings, halved, and 5.5 each)."""
    import torch
    c = Case(1, 5120)
    out, z, _ = mq.mq_add_rmsnorm_quant_q8(**c.args(mq))
    x = dev(c.x) + dev(c.y)
    torch.cuda.synchronize()
    assert torch.equal(out, x)
    z2, _ = mq.mq_rmsnorm_quant_q8(x[0].contiguous(), dev(c.gain), 1e-6)
    assert ((z2 - z[0]).abs() <= 2.0 ** -24 * (22.5 + 16.5 + 11) * z[0].abs()).all()


def test_another_stream_and_a_captured_chain(mq):
    """Each call's x is the last one's x_out, under programmatic dependent launch."""
    import torch
    c = Case(2, 5120, True, "channel", 0.3)
    a = c.args(mq)
    want = a["x"].clone()
    for _ in range(4):
        want = mq.mq_add_rmsnorm_quant_q8(want, a["y"], a["gain"], 1e-6, post_gain=a["post_gain"], gate=a["gate"],
                                          scale=0.3)[0]
    x, st, gr = a["x"].clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    mq.mq_set_pdl(True)
    try:
        with torch.cuda.graph(gr, stream=st):
            for _ in range(4):
                mq.mq_add_rmsnorm_quant_q8(x, a["y"], a["gain"], 1e-6, post_gain=a["post_gain"], gate=a["gate"], scale=0.3,
                                           x_out=x, z=a["z"], q8=a["q8"])
    finally:
        mq.mq_set_pdl(False)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want)
    b, d = c.args(mq), c.args(mq)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        other = mq.mq_add_rmsnorm_quant_q8(**b)
    third = mq.mq_add_rmsnorm_quant_q8(**{**d, "x_out": None, "z": None, "q8": None}, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(other[0], third[0]) and torch.equal(other[1], third[1])


def test_refusals(mq):
    import torch
    c = Case(2, 96)
    a = c.args(mq)
    for change, error in [(dict(y=a["y"][:1]), ValueError), (dict(gain=a["gain"][:64]), ValueError),
                          (dict(gate=a["x"][:, :64]), ValueError), (dict(gate=torch.zeros(3, 96, device="cuda")), ValueError),
                          (dict(x=a["x"].double()), TypeError), (dict(y=a["y"].cpu()), TypeError),
                          (dict(q8=a["q8"][:16]), ValueError), (dict(x_out=a["x"].t().contiguous().t()), ValueError),
                          (dict(x=a["x"][:0], y=a["y"][:0], x_out=a["x"][:0], z=a["z"][:0]), mq.MQError),
                          (dict(scale=float("nan")), mq.MQError), (dict(eps=float("inf")), mq.MQError)]:
        with pytest.raises(error):
            mq.mq_add_rmsnorm_quant_q8(**{**a, **change})
    x = torch.zeros(2, 48, device="cuda")
    with pytest.raises(mq.MQError):
        mq.mq_add_rmsnorm_quant_q8(x, x, x[0], 1e-6, x_out=x, z=x, q8=a["q8"])
    torch.cuda.synchronize()
    assert (a["x_out"] == 7.0).all()


@pytest.mark.parametrize("n", [1 << 15 | 32, 1 << 21, (1 << 26) - 32])
@pytest.mark.parametrize("post", [False, True])
def test_long_rows_of_equal_magnitudes(mq, n, post):
    """Squares that all round to one side, in a bound that does not grow with the row: 16 groups of four of a thread, a
    butterfly and 32 warps are 101 roundings; what is kept beside the sums 2 more."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(n)
    x, y = ((torch.randint(0, 2, (1, n), device="cuda", generator=g) * 2 - 1) * v for v in (1.1, 0.77))
    x, y = x.float(), y.float()
    gain, more = torch.full((n,), 1.25, device="cuda"), torch.full((n,), 0.75, device="cuda") if post else None
    out, z, _ = mq.mq_add_rmsnorm_quant_q8(x, y, gain, 1e-6, post_gain=more, scale=0.5, q8=False)
    host = [None if t is None else t.cpu().numpy() for t in (x, y, gain, more)]
    want_x, want_z, tol_x, tol_z = ref.add_rmsnorm(host[0], host[1], host[2].astype(np.float64), float(np.float32(1e-6)),
                                                   host[3], None, 0.5, 103)
    assert np.all(np.abs(out.cpu().numpy() - want_x) <= tol_x)
    assert np.all(np.abs(z.cpu().numpy() - want_z) <= tol_z)


def test_a_long_row_whose_squares_overflow(mq):
    """The mean is infinite, its root's inverse 0, as in shorter rows."""
    import torch
    for n in (1024, 40000):
        x, gain = torch.full((1, n), 1e19, device="cuda"), torch.ones(n, device="cuda")
        x[0, 5] = 3e19
        out, z, _ = mq.mq_add_rmsnorm_quant_q8(x, x, gain, 1e-6)
        assert torch.equal(out, x + x) and not z.any()


@pytest.mark.parametrize("n", [1024, 33024])
def test_outputs_that_are_not_wanted(mq, n):
    import torch
    c = Case(3, n, True, "row", 0.5)
    a = c.args(mq)
    want = mq.mq_add_rmsnorm_quant_q8(**a)
    out, z, q8 = mq.mq_add_rmsnorm_quant_q8(**{**c.args(mq), "z": False})
    assert z is None and torch.equal(out, want[0]) and torch.equal(q8, want[2])
    out, z, q8 = mq.mq_add_rmsnorm_quant_q8(**{**c.args(mq), "q8": False})
    assert q8 is None and torch.equal(out, want[0]) and torch.equal(z, want[1])
    with pytest.raises(mq.MQError):
        mq.mq_add_rmsnorm_quant_q8(**{**c.args(mq), "z": False, "q8": False})
    with pytest.raises(ValueError):
        mq.mq_add_rmsnorm_quant_q8(**{**c.args(mq), "q8": want[2][:0]})
