"""Host side of the operators around the GEMVs of a decode step, without a GPU:
sizes, the rotation's table, and every refusal before a launch."""
import ctypes
import math

import numpy as np
import pytest

NO_GPU = pytest.mark.skipif(__import__("torch").cuda.is_available(),
                            reason="fake device pointers are only passed where no GPU exists")


class RopeAppend(ctypes.Structure):
    """mq_rope_append_args of include/mq.h"""
    _fields_ = ([(n, ctypes.c_int) for n in ("nt", "n_heads", "rope_dims", "rope_style")]
                + [("eps", ctypes.c_float)]
                + [(n, ctypes.c_void_p) for n in ("q", "k", "v")]
                + [(n, ctypes.c_longlong) for n in ("q_stride", "k_stride", "v_stride")]
                + [("q_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_longlong)]
                + [(n, ctypes.c_void_p) for n in ("q_bias", "k_bias", "v_bias", "q_gain", "k_gain",
                                                  "rope_table", "positions", "seq", "pages")]
                + [("n_seqs", ctypes.c_int), ("pages_stride", ctypes.c_int), ("status", ctypes.c_void_p)])


class Attn(ctypes.Structure):
    """mq_attn_args of include/mq.h"""
    _fields_ = ([(n, ctypes.c_int) for n in ("nt", "n_heads", "max_len", "window")]
                + [(n, ctypes.c_float) for n in ("scale", "softcap")]
                + [("q", ctypes.c_void_p), ("out", ctypes.c_void_p)]
                + [("q_stride", ctypes.c_longlong), ("out_stride", ctypes.c_longlong)]
                + [(n, ctypes.c_void_p) for n in ("q8", "lens", "seq", "pages")]
                + [("n_seqs", ctypes.c_int), ("pages_stride", ctypes.c_int)]
                + [("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p)])


class Sample(ctypes.Structure):
    """mq_sample_args of include/mq.h"""
    _fields_ = ([("nt", ctypes.c_int), ("vocab", ctypes.c_int), ("logits", ctypes.c_void_p),
                 ("stride", ctypes.c_longlong)]
                + [(n, ctypes.c_void_p) for n in ("u", "temperature", "top_p", "min_p", "top_k", "token", "prob")])


@pytest.fixture(scope="module")
def mq():
    from quant_quantized_gemv_gb300 import build
    build.build()
    import quant_quantized_gemv_gb300 as m
    m.lib()
    return m


def test_page_bytes(mq):
    assert mq.mq_kv_page_bytes("f16", 8, 16, 128) == 8 * 16 * 128 * 2
    assert mq.mq_kv_page_bytes("bf16", 1, 48, 96) == 48 * 96 * 2
    assert mq.mq_kv_page_bytes("q8", 4, 32, 64) == 4 * 32 * (64 + 4)
    for bad in (("f16", 0, 16, 128), ("f16", 8, 0, 128), ("f16", 8, 24, 128), ("f16", 8, 16, 80),
                ("f16", -1, 16, 128), ("q8", 8, -16, 128)):
        assert mq.mq_kv_page_bytes(*bad) == 0, bad
    assert mq.lib().mq_kv_page_bytes(4, 8, 16, 128) == 0


def table_of(mq, freqs):
    f = np.asarray(freqs, np.float64)
    out = np.zeros(f.size, np.uint64)
    st = mq.lib().mq_rope_table(f.ctypes.data_as(ctypes.c_void_p), f.size, out.ctypes.data_as(ctypes.c_void_p))
    assert st == mq.MQ_OK
    return out


def test_rope_table_is_the_fraction_of_a_turn(mq):
    freqs = [1.0, 0.5, 1e-6, 0.0, 2 * math.pi, 7.0, -1.0, 1e6 ** (-126 / 128)]
    for f, got in zip(freqs, table_of(mq, freqs)):
        want = f / (2 * math.pi)
        diff = (int(got) / 2 ** 64 - want) % 1.0
        # one division and one subtraction in 53 bits; 2^-64 of the truncation
        assert min(diff, 1 - diff) <= 2.0 ** -52 * max(1.0, abs(want)), f


def test_rope_table_angle_at_far_positions(mq):
    """position * F mod 2^64 is the angle: checked in exact integers against
    the fraction of position * freq / 2 pi in 80 digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563")
    freqs = [1e6 ** (-2 * i / 128) for i in range(64)]
    for f, F in zip(freqs, table_of(mq, freqs)):
        for pos in (1, 4097, 1 << 20, 2 ** 31 - 1):
            turns = Decimal(pos) * Decimal(f) / two_pi
            want = turns - int(turns)
            got = Decimal((pos * int(F)) % 2 ** 64) / Decimal(2 ** 64)
            diff = abs(got - want)
            # the step's division rounds twice at 2^-53 of f / 2 pi < f, and its last
            # bit is 2^-64 of a turn (truncated); the product is exact
            tol = Decimal(pos) * (Decimal(2) ** -52 * Decimal(f) + Decimal(2) ** -64)
            assert min(diff, 1 - diff) <= tol, (f, pos)


def test_rope_table_refusals(mq):
    L, one = mq.lib(), np.ones(1)
    p = one.ctypes.data_as(ctypes.c_void_p)
    assert L.mq_rope_table(None, 1, p) == mq.MQ_ERR_NULL
    assert L.mq_rope_table(p, 1, None) == mq.MQ_ERR_NULL
    assert L.mq_rope_table(p, 0, p) == mq.MQ_ERR_SHAPE
    for bad in (math.inf, math.nan):
        b = np.array([bad])
        assert L.mq_rope_table(b.ctypes.data_as(ctypes.c_void_p), 1, p) == mq.MQ_ERR_SHAPE


def cache(mq, **kw):
    a = dict(type=1, n_pages=4, page_size=16, n_kv_heads=2, head_dim=128, k=0x10000, v=0x20000, page_stride=0)
    a.update(kw)
    return mq._KVStruct(**a)


BAD_CACHES = [(dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(type=0), "SHAPE"), (dict(type=4), "SHAPE"),
              (dict(n_pages=0), "SHAPE"), (dict(page_size=24), "SHAPE"), (dict(head_dim=80), "SHAPE"),
              (dict(n_kv_heads=0), "SHAPE"), (dict(page_stride=-16), "SHAPE"), (dict(page_stride=16), "SHAPE"),
              (dict(page_stride=2 * 16 * 128 * 2 + 8), "ALIGN"), (dict(k=0x10008), "ALIGN"), (dict(v=0x20002), "ALIGN")]


def append_args(mq, **kw):
    a = dict(nt=1, n_heads=4, rope_dims=128, rope_style=0, eps=1e-6, q=0x30000, k=0x40000, v=0x50000,
             q_stride=512, k_stride=256, v_stride=256, q_out=0x60000, q_out_stride=512, rope_table=0x70000,
             positions=0x80000, pages=0x90000, n_seqs=1, pages_stride=4)
    a.update(kw)
    return RopeAppend(**a)


@NO_GPU
@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_append_refuses_a_bad_cache(mq, bad, status):
    st = mq.lib().mq_rope_append(ctypes.byref(cache(mq, **bad)), ctypes.byref(append_args(mq)), None)
    assert st == getattr(mq, "MQ_ERR_" + status)


@NO_GPU
@pytest.mark.parametrize("bad,status", [
    (dict(nt=0), "SHAPE"), (dict(nt=-1), "SHAPE"), (dict(n_heads=0), "SHAPE"), (dict(n_heads=3), "SHAPE"),
    (dict(nt=2 ** 31 - 1), "SHAPE"), (dict(rope_dims=-8), "SHAPE"), (dict(rope_dims=136), "SHAPE"),
    (dict(rope_dims=4), "SHAPE"), (dict(rope_style=2), "SHAPE"), (dict(rope_style=-1), "SHAPE"),
    (dict(n_seqs=0), "SHAPE"), (dict(pages_stride=0), "SHAPE"), (dict(q_stride=508), "SHAPE"),
    (dict(q_out_stride=0), "SHAPE"), (dict(k_stride=252), "SHAPE"), (dict(v_stride=-256), "SHAPE"),
    (dict(q=None), "NULL"), (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(q_out=None), "NULL"),
    (dict(positions=None), "NULL"), (dict(pages=None), "NULL"), (dict(rope_table=None), "NULL"),
    (dict(q=0x30004), "ALIGN"), (dict(q_out=0x60008), "ALIGN"), (dict(k_bias=0x10004), "ALIGN"),
    (dict(q_gain=0x10008), "ALIGN"), (dict(q_stride=514), "ALIGN"), (dict(v_stride=257), "ALIGN"),
    (dict(rope_table=0x70004), "ALIGN"), (dict(positions=0x80002), "ALIGN"), (dict(status=0x80001), "ALIGN")])
def test_append_refuses_bad_arguments(mq, bad, status):
    st = mq.lib().mq_rope_append(ctypes.byref(cache(mq)), ctypes.byref(append_args(mq, **bad)), None)
    assert st == getattr(mq, "MQ_ERR_" + status)


@NO_GPU
def test_append_refuses_null_structs_and_odd_wide_rotations(mq):
    L = mq.lib()
    assert L.mq_rope_append(None, ctypes.byref(append_args(mq)), None) == mq.MQ_ERR_NULL
    assert L.mq_rope_append(ctypes.byref(cache(mq)), None, None) == mq.MQ_ERR_NULL
    wide = append_args(mq, rope_dims=24, q_stride=1024, q_out_stride=1024, k_stride=512, v_stride=512)
    assert L.mq_rope_append(ctypes.byref(cache(mq, head_dim=256)), ctypes.byref(wide), None) == mq.MQ_ERR_SHAPE


def attn_args(mq, **kw):
    a = dict(nt=1, n_heads=4, max_len=1000, window=0, scale=0.1, softcap=0.0, q=0x30000, out=0x40000,
             q_stride=512, out_stride=512, lens=0x50000, pages=0x60000, n_seqs=1, pages_stride=64, ws=0x70000,
             ws_bytes=1 << 30)
    a.update(kw)
    return Attn(**a)


@NO_GPU
@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_attention_refuses_a_bad_cache(mq, bad, status):
    st = mq.lib().mq_attn_decode(ctypes.byref(cache(mq, **bad)), ctypes.byref(attn_args(mq)), None)
    assert st == getattr(mq, "MQ_ERR_" + status)


@NO_GPU
@pytest.mark.parametrize("bad,status", [
    (dict(nt=0), "SHAPE"), (dict(n_heads=0), "SHAPE"), (dict(n_heads=5), "SHAPE"), (dict(nt=1 << 24), "SHAPE"),
    (dict(max_len=0), "SHAPE"), (dict(max_len=-1), "SHAPE"), (dict(max_len=2 ** 31 - 1), "SHAPE"),
    (dict(max_len=2 ** 30 + 1), "SHAPE"), (dict(max_len=2 ** 30, n_heads=256, q_stride=1 << 15, out_stride=1 << 15), "SHAPE"),
    (dict(window=-1), "SHAPE"), (dict(scale=math.inf), "SHAPE"), (dict(scale=math.nan), "SHAPE"),
    (dict(softcap=-2.0), "SHAPE"), (dict(softcap=math.nan), "SHAPE"), (dict(q_stride=508), "SHAPE"),
    (dict(out_stride=-512), "SHAPE"), (dict(n_seqs=0), "SHAPE"), (dict(pages_stride=0), "SHAPE"),
    (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(lens=None), "NULL"), (dict(pages=None), "NULL"),
    (dict(q=0x30004), "ALIGN"), (dict(out=0x40008), "ALIGN"), (dict(q8=0x10004), "ALIGN"),
    (dict(ws=0x70008), "ALIGN"), (dict(q_stride=513), "ALIGN"), (dict(lens=0x50002), "ALIGN"),
    (dict(seq=0x50001), "ALIGN"), (dict(pages=0x60002), "ALIGN"), (dict(status=0x10002), "ALIGN")])
def test_attention_refuses_bad_arguments(mq, bad, status):
    st = mq.lib().mq_attn_decode(ctypes.byref(cache(mq)), ctypes.byref(attn_args(mq, **bad)), None)
    assert st == getattr(mq, "MQ_ERR_" + status)


@NO_GPU
def test_attention_refuses_null_structs(mq):
    L = mq.lib()
    assert L.mq_attn_decode(None, ctypes.byref(attn_args(mq)), None) == mq.MQ_ERR_NULL
    assert L.mq_attn_decode(ctypes.byref(cache(mq)), None, None) == mq.MQ_ERR_NULL
    assert L.mq_attn_workspace_bytes(None, 4, 1, 100) == 0
    assert L.mq_attn_workspace_bytes(ctypes.byref(cache(mq)), 5, 1, 100) == 0
    assert L.mq_attn_workspace_bytes(ctypes.byref(cache(mq)), 4, 0, 100) == 0


@NO_GPU
@pytest.mark.parametrize("bad,status", [
    (dict(nt=0), "SHAPE"), (dict(nt=-3), "SHAPE"), (dict(nt=(1 << 24) + 1), "SHAPE"), (dict(vocab=0), "SHAPE"),
    (dict(vocab=655361, stride=655361), "SHAPE"), (dict(stride=99), "SHAPE"), (dict(stride=-100), "SHAPE"),
    (dict(logits=None), "NULL"), (dict(u=None), "NULL"), (dict(token=None), "NULL"),
    (dict(logits=0x10002), "ALIGN"), (dict(top_k=0x10001), "ALIGN"), (dict(prob=0x10003), "ALIGN")])
def test_sample_refuses_bad_arguments(mq, bad, status):
    a = dict(nt=1, vocab=100, logits=0x10000, stride=100, u=0x20000, token=0x30000)
    a.update(bad)
    st = mq.lib().mq_sample(ctypes.byref(Sample(**a)), None)
    assert st == getattr(mq, "MQ_ERR_" + status)


@NO_GPU
def test_sample_refuses_null_arguments(mq):
    assert mq.lib().mq_sample(None, None) == mq.MQ_ERR_NULL


class Described:
    """What the calls read of a cache, without one on a GPU."""

    def __init__(self, mq):
        self._struct = cache(mq)
        self._address, self.device_index, self.page_size, self.head_dim = ctypes.addressof(self._struct), 0, 16, 128


def test_calls_refuse_what_is_no_cuda_tensor(mq):
    """Without a launch: the checks of the compiled calls, up to the first that fails."""
    import torch
    x = torch.zeros(2, 100)
    for bad in (x, x[0], 3, None, "x", x.to_sparse(), x.double()):
        with pytest.raises(TypeError):
            mq.mq_sample(bad, x[:, 0], token=x)
    b = mq._calls
    for f in (b.rope_append, b.attn_decode, b.sample, b.setup):
        with pytest.raises(TypeError):
            f(1, 2)
        with pytest.raises(TypeError):
            f()


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="there is a current device")
def test_calls_without_a_device_raise(mq):
    """The device's own error, as an exception."""
    import torch
    kv, x, i = Described(mq), torch.zeros(1, 512), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises((RuntimeError, ValueError, TypeError)):
        mq.mq_rope_append(kv, x, x, x, i[0], i)
    with pytest.raises((RuntimeError, ValueError, TypeError)):
        mq.mq_attn_decode(kv, x, i[0], i, 0.1, ws=x)


# the references against what they can be checked with on paper
def test_reference_sample_by_hand():
    from oracle import decode as ref
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert ref.sample(x, 0.0)[0] == 0 and ref.sample(x, 0.3)[0] == 1 and ref.sample(x, 0.95)[0] == 3
    tok, p, kept, _ = ref.sample(x, 0.5, k=2)          # keeps 0.4 and 0.3
    assert kept.tolist() == [False, True, False, True] and tok == 1 and abs(p - 4 / 7) < 1e-12
    assert ref.sample(x, 0.6, k=2)[0] == 3
    assert ref.sample(x, 0.0, p=0.65)[2].tolist() == [False, True, False, True]
    assert ref.sample(x, 0.0, p=0.71)[2].tolist() == [False, True, True, True]
    assert ref.sample(x, 0.0, m=0.6)[2].tolist() == [False, True, False, True]
    assert ref.sample(x, 0.9, t=0.0)[0] == 1
    assert ref.sample(np.full(4, -np.inf), 0.5)[0] == -1
    assert ref.sample(np.array([1.0, 1.0, 1.0]), 0.0, k=2)[2].tolist() == [True, True, False]


def test_reference_attention_by_hand():
    from oracle import decode as ref
    q = np.array([[1.0, 0.0]])
    k = np.array([[[0.0, 5.0], [np.log(3.0), -2.0]]])
    v = np.array([[[4.0, 0.0], [0.0, 8.0]]])
    assert np.allclose(ref.attention(q, k, v, 1.0), [[1.0, 6.0]])      # weights 1/4 and 3/4
    assert np.allclose(ref.attention(q, k, v, 1.0, window=1), [[0.0, 8.0]])
    assert np.allclose(ref.attention(q, k, v, 1e9, softcap=np.log(3.0)), [[1.0, 6.0]])
    assert np.all(ref.attention(q, k[:, :0], v[:, :0], 1.0) == 0)


def test_reference_rotation_by_hand():
    from oracle import decode as ref
    x = np.array([[[1.0, 0.0, 0.0, 2.0]]])
    f = np.array([np.pi / 2, np.pi])
    half, _ = ref.rotate(x, np.abs(x), [1], f, "half")                  # pairs (0, 2), (1, 3)
    assert np.allclose(half, [[[0.0, 0.0, 1.0, -2.0]]])
    pairs, _ = ref.rotate(x, np.abs(x), [1], f, "pairs")                # pairs (0, 1), (2, 3)
    assert np.allclose(pairs, [[[0.0, 1.0, 0.0, -2.0]]])


# ------------------------------------------------------------------ the build
class Compiler:
    """Stands for nvcc: writes what a command names as its output; refuses a source."""

    def __init__(self, refuse=None):
        self.commands, self.refuse = [], refuse

    def __call__(self, cmd, **_):
        import types
        self.commands.append(cmd)
        if self.refuse and any(str(x).endswith(self.refuse) for x in cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    from quant_quantized_gemv_gb300 import build as b
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "SO", str(tmp_path / "libmq.so"))
    return b


def torch_at(path, version):
    import types
    path.mkdir(exist_ok=True)
    (path / "version.py").write_text(f"__version__ = '{version}'\n")
    return lambda name: types.SimpleNamespace(submodule_search_locations=[str(path)])


def test_the_library_builds_without_torch(elsewhere, monkeypatch, tmp_path):
    """The C ABI needs nvcc alone; the Python calls over torch's headers are left out."""
    cc = Compiler()
    monkeypatch.setattr(elsewhere, "find_spec", lambda name: None)
    monkeypatch.setattr(elsewhere.subprocess, "run", cc)
    assert elsewhere.build(force=True) == str(tmp_path / "libmq.so") and (tmp_path / "libmq.so").exists()
    assert not any("binding" in str(x) for c in cc.commands for x in c)
    assert not elsewhere._stale()


def test_the_library_is_linked_before_the_calls_over_torch(elsewhere, monkeypatch, tmp_path):
    cc = Compiler(refuse="binding.cpp")
    monkeypatch.setattr(elsewhere, "find_spec", torch_at(tmp_path / "torch", "1.0"))
    monkeypatch.setattr(elsewhere.subprocess, "run", cc)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        elsewhere.build(force=True)
    assert (tmp_path / "libmq.so").exists()
    cc.refuse = None
    monkeypatch.setattr(elsewhere, "find_spec", lambda name: None)
    assert not elsewhere._stale()


def test_another_torch_has_calls_of_its_own(elsewhere, monkeypatch, tmp_path):
    """What was compiled over one torch's headers is not taken for another's."""
    monkeypatch.setattr(elsewhere.subprocess, "run", Compiler())
    monkeypatch.setattr(elsewhere, "find_spec", torch_at(tmp_path / "torch", "1.0"))
    elsewhere.build()
    assert not elsewhere._stale()
    monkeypatch.setattr(elsewhere, "find_spec", torch_at(tmp_path / "torch", "1.1+x"))
    assert elsewhere._stale()
    elsewhere.build()
    assert not elsewhere._stale()
    monkeypatch.setattr(elsewhere.sysconfig, "get_config_var", lambda name: "cpython-399-there")
    assert elsewhere._stale()


def test_the_calls_are_those_of_the_torch_that_runs(mq):
    import torch
    from quant_quantized_gemv_gb300 import build as b
    assert torch.__version__ in b.binding() and mq._bind().__file__ == b.binding()


def test_a_folder_named_torch_is_no_torch(elsewhere, monkeypatch, tmp_path):
    import types
    monkeypatch.setattr(elsewhere.subprocess, "run", Compiler())
    for spec in (None, types.SimpleNamespace(submodule_search_locations=None),
                 types.SimpleNamespace(submodule_search_locations=[str(tmp_path / "torch")])):
        monkeypatch.setattr(elsewhere, "find_spec", lambda name: spec)
        assert elsewhere.binding() is None and elsewhere.build(force=True)
