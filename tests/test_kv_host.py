"""The paged cache's calls and the sampling without a GPU: every refusal of the C
calls answers before anything is launched, the binding's own checks, and the
oracle against hand-worked values.

The handle is a block of zeros: no refused call looks into it."""
import ctypes
import math

import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from oracle import kv_oracle as KO
from test_batch_host import OnDevice

A = 1 << 40  # an aligned address that no refused call reads
BAD, UNSUPPORTED, SMALL = bq.MOE_ERR_INVALID_ARG, bq.MOE_ERR_UNSUPPORTED, bq.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    bq.build_library()
    return bq.load_library()


@pytest.fixture(scope="module")
def handle():
    buf = (ctypes.c_uint8 * 4096)()
    return ctypes.cast(buf, ctypes.c_void_p), buf


def cache(**kw):
    a = dict(n_pages=10, kv_heads=2, page_rows=16, head_dim=64, k=A, v=A, k_scales=A, v_scales=A, table=A, n_seqs=3,
             table_stride=4)
    a.update(kw)
    return bq.KvCache(*[a[n] for n, _ in bq.KvCache._fields_])


CACHES = [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(table=None), BAD), (dict(k_scales=None), BAD),
    (dict(v_scales=None), BAD), (dict(n_pages=0), BAD), (dict(kv_heads=0), BAD), (dict(n_seqs=0), BAD),
    (dict(table_stride=0), BAD), (dict(k=A + 8), BAD), (dict(v=A + 2), BAD), (dict(k_scales=A + 4), BAD),
    (dict(v_scales=A + 8), BAD), (dict(table=A + 2), BAD), (dict(page_rows=8), UNSUPPORTED),
    (dict(page_rows=24), UNSUPPORTED), (dict(page_rows=512), UNSUPPORTED), (dict(page_rows=0), UNSUPPORTED),
    (dict(head_dim=8), UNSUPPORTED), (dict(head_dim=72), UNSUPPORTED), (dict(head_dim=272), UNSUPPORTED),
    (dict(kv_heads=129), UNSUPPORTED), (dict(n_seqs=4097), UNSUPPORTED),
    (dict(n_pages=1 << 30, page_rows=256), UNSUPPORTED), (dict(table_stride=1 << 27), UNSUPPORTED)]


def append(lib, h, c=None, **kw):
    a = dict(q=A, ldq=256, q_heads=4, k=A, ldk=128, v=A, ldv=128, rows=3, seq=A, pos=A, freq=A, rot=64, out=A, ldo=256)
    a.update(kw)
    return lib.moe_kv_append(h, a["q"], a["ldq"], a["q_heads"], a["k"], a["ldk"], a["v"], a["ldv"], a["rows"], a["seq"],
                             a["pos"], ctypes.byref(c or cache()), a["freq"], a["rot"], a["out"], a["ldo"], None)


def read(lib, h, c=None, **kw):
    a = dict(seq=A, pos=A, rows=3, k=A, ldk=128, v=A, ldv=128)
    a.update(kw)
    return lib.moe_kv_read(h, ctypes.byref(c or cache()), a["seq"], a["pos"], a["rows"], a["k"], a["ldk"], a["v"],
                           a["ldv"], None)


def attend(lib, h, c=None, **kw):
    a = dict(q=A, ldq=256, len=A, q_heads=4, scale=0.1, cap=0.0, window=0, out=A, ldo=256, lse=A, ws=A, bytes=1 << 34)
    a.update(kw)
    return lib.moe_kv_attend(h, a["q"], a["ldq"], ctypes.byref(c or cache()), a["len"], a["q_heads"], a["scale"],
                             a["cap"], a["window"], a["out"], a["ldo"], a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("change,status", CACHES)
def test_cache_refusals(lib, handle, change, status):
    h, c = handle[0], cache(**change)
    assert append(lib, h, c) == status and read(lib, h, c) == status and attend(lib, h, c) == status
    assert lib.moe_kv_attend_workspace_bytes(ctypes.byref(c), 4) == 0


@pytest.mark.parametrize("change,status", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(pos=None), BAD), (dict(q=None), BAD), (dict(out=None), BAD),
    (dict(rows=0), BAD), (dict(rows=-1), BAD), (dict(rows=(1 << 20) + 1), BAD), (dict(q_heads=0), BAD),
    (dict(q_heads=1025), UNSUPPORTED), (dict(ldq=248), BAD), (dict(ldq=260), BAD), (dict(ldk=120), BAD),
    (dict(ldv=132), BAD), (dict(ldo=8), BAD), (dict(ldo=264), BAD), (dict(q=A + 8, out=A), BAD), (dict(k=A + 2), BAD),
    (dict(v=A + 8), BAD), (dict(pos=A + 2), BAD), (dict(seq=A + 1), BAD), (dict(freq=A + 2), BAD), (dict(rot=-16), BAD),
    (dict(rot=0), BAD), (dict(freq=None), BAD), (dict(rot=24), UNSUPPORTED), (dict(rot=80), UNSUPPORTED)])
def test_append_refusals(lib, handle, change, status):
    assert append(lib, handle[0], **change) == status
    assert append(lib, None, **change) == BAD


@pytest.mark.parametrize("change,status", [
    (dict(pos=None), BAD), (dict(k=None, v=None), BAD), (dict(rows=0), BAD), (dict(rows=(1 << 20) + 1), BAD),
    (dict(ldk=120), BAD), (dict(ldv=129), BAD), (dict(k=A + 4), BAD), (dict(pos=A + 1), BAD), (dict(seq=A + 2), BAD)])
def test_read_refusals(lib, handle, change, status):
    assert read(lib, handle[0], **change) == status
    assert read(lib, None, **change) == BAD


@pytest.mark.parametrize("change,status", [
    (dict(q=None), BAD), (dict(len=None), BAD), (dict(out=None), BAD), (dict(ws=None), BAD), (dict(q_heads=0), BAD),
    (dict(q_heads=3), UNSUPPORTED), (dict(q_heads=130, ldq=8320, ldo=8320), UNSUPPORTED), (dict(ldq=248), BAD),
    (dict(ldo=257), BAD), (dict(q=A + 2), BAD), (dict(out=A + 8), BAD), (dict(len=A + 2), BAD), (dict(lse=A + 1), BAD),
    (dict(ws=A + 128), BAD), (dict(scale=math.nan), BAD), (dict(scale=math.inf), BAD), (dict(cap=-1.0), BAD),
    (dict(cap=math.nan), BAD), (dict(cap=math.inf), BAD), (dict(window=-1), BAD), (dict(bytes=0), SMALL)])
def test_attend_refusals(lib, handle, change, status):
    assert attend(lib, handle[0], **change) == status
    assert attend(lib, None, **change) == BAD


def test_attend_workspace(lib):
    for heads, dim in ((2, 64), (128, 64), (256, 64)):
        n = lib.moe_kv_attend_workspace_bytes(ctypes.byref(cache(kv_heads=2 if heads < 256 else 4, head_dim=dim)), heads)
        assert n > 0 and n % 256 == 0
    assert lib.moe_kv_attend_workspace_bytes(ctypes.byref(cache()), 3) == 0
    assert lib.moe_kv_attend_workspace_bytes(ctypes.byref(cache()), 0) == 0
    wide = dict(n_seqs=4096, table_stride=1 << 12, page_rows=256, kv_heads=8)  # 2^31 tiles of 16 positions
    assert lib.moe_kv_attend_workspace_bytes(ctypes.byref(cache(**wide)), 8) == 0
    wide["n_seqs"] = 4095
    assert lib.moe_kv_attend_workspace_bytes(ctypes.byref(cache(**wide)), 128) > 0
    assert lib.moe_kv_attend_workspace_bytes(ctypes.byref(cache(**wide)), 136) == 0


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), BAD), (dict(rules=None), BAD), (dict(uniform=None), BAD), (dict(tokens=None), BAD),
    (dict(rows=0), BAD), (dict(rows=4097), BAD), (dict(vocab=0), UNSUPPORTED), (dict(vocab=(1 << 28) + 1), UNSUPPORTED),
    (dict(ld=99), BAD), (dict(ld=(1 << 32) + 1), UNSUPPORTED), (dict(logits=A + 2), BAD), (dict(uniform=A + 1), BAD),
    (dict(top_k=A + 2), BAD), (dict(min_p=A + 2), BAD), (dict(tokens=A + 2), BAD), (dict(logprobs=A + 3), BAD)])
def test_sample_refusals(lib, handle, change, status):
    a = dict(logits=A, ld=100, rows=2, vocab=100, rules=1, uniform=A, temperature=A, top_k=A, top_p=A, min_p=A,
             tokens=A, logprobs=A)
    a.update(change)
    r = bq.SampleRules(a["uniform"], a["temperature"], a["top_k"], a["top_p"], a["min_p"])
    for h, want in ((handle[0], status), (None, BAD)):
        assert lib.moe_sample(h, a["logits"], a["ld"], a["rows"], a["vocab"], ctypes.byref(r) if a["rules"] else None,
                              a["tokens"], a["logprobs"], None) == want


# ------------------------------------------------------------------ the binding
torch = pytest.importorskip("torch")
B16, I8, F32, I32 = torch.bfloat16, torch.int8, torch.float32, torch.int32


def on(shape, dtype, device=0):
    return OnDevice(torch.zeros(shape, dtype=dtype), device)


@pytest.fixture
def moe(monkeypatch):
    monkeypatch.setattr(bq, "_current_device", lambda: 0)

    class Lib:
        def __getattr__(self, name):
            return lambda *a: bq.MOE_OK

    m = object.__new__(bq.Moe)
    m.lib, m.h = Lib(), None
    return m


def made(bits8=True, **kw):
    shape = (10, 2, 16, 64)
    a = dict(k=on(shape, I8 if bits8 else B16), v=on(shape, I8 if bits8 else B16), table=on((3, 4), I32),
             k_scales=on(shape[:3], F32) if bits8 else None, v_scales=on(shape[:3], F32) if bits8 else None)
    a.update(kw)
    return bq.make_kv_cache(**a)


def test_make_kv_cache():
    c = made()
    assert [getattr(c, n) for n in ("n_pages", "kv_heads", "page_rows", "head_dim", "n_seqs", "table_stride")] == \
        [10, 2, 16, 64, 3, 4]
    assert made(bits8=False).k_scales is None
    for bad in (dict(k=on((10, 2, 16, 64), B16)), dict(v=on((10, 2, 16, 32), I8)), dict(v_scales=None),
                dict(k_scales=on((10, 2, 8), F32)), dict(k_scales=on((10, 2, 16), B16)), dict(table=on((3, 4), F32)),
                dict(table=on(12, I32)), dict(v=on((10, 2, 16, 64), I8, 1)), dict(table=on((3, 4), I32, 1)),
                dict(k=on((10, 2, 1024), I8)), dict(table=OnDevice(torch.zeros((3, 8), dtype=I32)[:, :4], 0)),
                dict(k=OnDevice(torch.zeros((10, 2, 64, 16), dtype=I8).transpose(2, 3), 0))):
        with pytest.raises(ValueError):
            made(**bad)


@pytest.mark.parametrize("bad", [
    dict(k=on((3, 3, 64), B16)), dict(k=on((2, 2, 64), B16)), dict(v=on((3, 2, 64), F32)), dict(v=on((3, 96), B16)),
    dict(q=on((3, 4, 32), B16)), dict(q_out=on((3, 2, 64), B16)), dict(seqs=on(2, I32)), dict(positions=on(3, F32)),
    dict(inv_freq=on(32, B16)), dict(k=on((3, 2, 64), B16, 1)), dict(cache=1), dict(k=on((64, 2, 3), B16, 0)),
    dict(k=OnDevice(torch.zeros((3, 64, 2), dtype=B16).transpose(1, 2), 0))])
def test_append_shapes(moe, bad):
    a = dict(k=on((3, 2, 64), B16), v=on((3, 128), B16), positions=on(3, I32), seqs=on(3, I32), q=on((3, 4, 64), B16),
             q_out=on((3, 4, 64), B16), inv_freq=on(32, F32), cache=made())
    moe.kv_append(stream=1, **a)
    wide = OnDevice(torch.zeros((3, 512), dtype=B16)[:, 256:384], 0)  # part of a wider projection
    moe.kv_append(stream=1, **{**a, "k": wide})
    a.update(bad)
    if a["cache"] == 1:
        a["cache"] = made(**{n: on(s, d, 1) for n, s, d in (("k", (10, 2, 16, 64), I8), ("v", (10, 2, 16, 64), I8),
                          ("table", (3, 4), I32), ("k_scales", (10, 2, 16), F32), ("v_scales", (10, 2, 16), F32))})
    with pytest.raises(ValueError):
        moe.kv_append(stream=1, **a)


@pytest.mark.parametrize("bad", [
    dict(q=on((2, 4, 64), B16)), dict(q=on((3, 4, 64), F32)), dict(out=on((3, 2, 64), B16)), dict(lengths=on(2, I32)),
    dict(lengths=on(3, F32)), dict(lse=on((5, 3), F32)), dict(ws=on(8, F32)), dict(out=on((3, 4, 64), B16, 1))])
def test_attend_shapes(moe, bad):
    a = dict(q=on((3, 4, 64), B16), lengths=on(3, I32), cache=made(), out=on((3, 256), B16), ws=on(512, torch.uint8),
             scale=0.1, lse=on((3, 4), F32))
    moe.kv_attend(stream=1, **a)
    a.update(bad)
    with pytest.raises(ValueError):
        moe.kv_attend(stream=1, **a)


@pytest.mark.parametrize("bad", [
    dict(k_out=on((2, 2, 64), B16)), dict(v_out=on((3, 64, 2), B16)), dict(positions=on((3, 2), I32)),
    dict(seqs=on(3, F32))])
def test_read_shapes(moe, bad):
    a = dict(positions=on(3, I32), k_out=on((3, 2, 64), B16), v_out=on((3, 128), B16), seqs=on(3, I32))
    moe.kv_read(made(), stream=1, **a)
    a.update(bad)
    with pytest.raises(ValueError):
        moe.kv_read(made(), stream=1, **a)


@pytest.mark.parametrize("bad", [
    dict(logits=on((2, 100), F32)), dict(logits=on((3, 99), F32)), dict(logits=on((3, 100), B16)),
    dict(tokens=on(2, I32)), dict(logprobs=on(2, F32)), dict(top_k=on(3, F32)), dict(top_p=on(2, F32)),
    dict(uniform=on(2, F32)), dict(min_p=on(3, F32, 1))])
def test_sample_shapes(moe, bad):
    a = dict(logits=on((3, 100), F32), tokens=on(3, I32), logprobs=on(3, F32), uniform=on(3, F32),
             temperature=on(3, F32), top_k=on(3, I32), top_p=on(3, F32), min_p=on(3, F32))

    def call(a):
        r = bq.make_sample_rules(*[a[n] for n in ("uniform", "temperature", "top_k", "top_p", "min_p")])
        moe.sample(a["logits"], 3, 100, r, a["tokens"], logprobs=a["logprobs"], stream=1)
    call(a)
    with pytest.raises(ValueError):
        call({**a, **bad})


# ------------------------------------------------------------------ the oracle by hand
def test_oracle_rotation():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    got = KO.rotate(x, [1], [math.pi / 2, 0.0])[0, 0]
    # the pair (1, 3) turns by a quarter: (-3, 1); the pair (2, 4) and the rest stay
    assert np.allclose(got, [-3, 2, 1, 4, 5, 6], atol=1e-12)


def test_oracle_codes():
    q, s = KO.quantise(np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1, np.nan, 0, 0], [np.inf, 1, 1, 1]]))
    assert q.tolist() == [[127, -64, 0, 2], [0] * 4, [0] * 4, [0] * 4]  # ties to even
    assert s[0] == 1.0 and s[1] == 0.0 and np.isnan(s[2]) and np.isnan(s[3])


def test_oracle_attention():
    k, v = np.array([[1.0, 0.0], [0.0, 1.0]]), np.array([[3.0, 0.0], [0.0, 9.0]])
    out, lse, _, _ = KO.attend(np.array([math.log(2.0), 0.0]), k, v, 1.0)
    assert np.allclose(out, [2.0, 3.0]) and np.isclose(lse, math.log(3.0))  # weights 2/3 and 1/3
    out, _, _, _ = KO.attend(np.array([1e9, 0.0]), k, v, 1.0, softcap=math.log(2.0))  # capped at log 2
    assert np.allclose(out, [2.0, 3.0])
    out, lse, _, _ = KO.attend(np.ones(2), k[:0], v[:0], 1.0)
    assert not out.any() and lse == -np.inf


def test_oracle_sampling():
    l = np.log(np.array([1.0, 4.0, 2.0, 4.0, 0.5, 1.0]))  # weights 1 4 2 4 .5 1, of 12.5
    assert KO.sample(l, 0.0)[0] == 0 and KO.sample(l, 0.99)[0] == 5
    assert KO.sample(l, 0.5)[0] == 2 and KO.sample(l, 0.3)[0] == 1  # running sums 1 5 7 11 11.5 12.5
    assert KO.sample(l, 0.9, top_k=1) == (1, 0.0)  # the lower id of equals
    t, p = KO.sample(l, 0.99, top_k=3)
    assert t == 3 and np.isclose(p, math.log(0.4))
    assert [KO.sample(l, u, top_p=0.32)[0] for u in (0.0, 0.99)] == [1, 1]   # 4 / 12.5 is enough
    assert [KO.sample(l, u, top_p=0.33)[0] for u in (0.0, 0.99)] == [1, 3]
    assert [KO.sample(l, u, min_p=0.4)[0] for u in (0.0, 0.45, 0.99)] == [1, 2, 3]
    assert KO.sample(l, 0.99, temperature=0.0) == (1, 0.0)
    assert KO.sample(np.full(3, -np.inf), 0.5) == (-1, -np.inf)
    assert KO.sample(l, 1.0)[0] == 5 and KO.sample(l, -1.0)[0] == 0
