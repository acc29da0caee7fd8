"""The batched path (norm_quant, qdense, logits_process) without a GPU: every
refusal of its C calls answers before anything is launched, the binding's own
checks, and the oracle against hand-worked values.

The handle is a block of zeros: no refused call looks into it."""
import ctypes
import math

import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from oracle import batch_oracle as BO
from oracle.batch_oracle import to_bf16
from synth import gen

A = 1 << 40  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    bq.build_library()
    return bq.load_library()


@pytest.fixture(scope="module")
def handle():
    buf = (ctypes.c_uint8 * 4096)()
    return ctypes.cast(buf, ctypes.c_void_p), buf


def _norm(lib, h, **kw):
    a = dict(hidden=A, y=A, rows=4, width=64, norm=A, eps=1e-6, out=A, q=A, scales=A, x=A)
    a.update(kw)
    return lib.moe_norm_quant(h, a["hidden"], a["y"], a["rows"], a["width"], a["norm"], a["eps"], a["out"], a["q"],
                              a["scales"], a["x"], None)


@pytest.mark.parametrize("change,status", [
    (dict(hidden=None), bq.MOE_ERR_INVALID_ARG), (dict(q=None), bq.MOE_ERR_INVALID_ARG),
    (dict(scales=None), bq.MOE_ERR_INVALID_ARG), (dict(rows=0), bq.MOE_ERR_INVALID_ARG),
    (dict(rows=-1), bq.MOE_ERR_INVALID_ARG), (dict(rows=(1 << 20) + 1), bq.MOE_ERR_INVALID_ARG),
    (dict(width=0), bq.MOE_ERR_UNSUPPORTED), (dict(width=72), bq.MOE_ERR_UNSUPPORTED),
    (dict(width=16384 + 16), bq.MOE_ERR_UNSUPPORTED), (dict(hidden=A + 8), bq.MOE_ERR_INVALID_ARG),
    (dict(y=A + 2), bq.MOE_ERR_INVALID_ARG), (dict(norm=A + 4), bq.MOE_ERR_INVALID_ARG),
    (dict(out=A + 8), bq.MOE_ERR_INVALID_ARG), (dict(q=A + 8), bq.MOE_ERR_INVALID_ARG),
    (dict(x=A + 8), bq.MOE_ERR_INVALID_ARG), (dict(scales=A + 2), bq.MOE_ERR_INVALID_ARG),
    (dict(y=None), bq.MOE_ERR_INVALID_ARG),  # hidden_out without y
    (dict(eps=-1e-6), bq.MOE_ERR_INVALID_ARG), (dict(eps=math.nan), bq.MOE_ERR_INVALID_ARG),
    (dict(eps=2.0), bq.MOE_ERR_INVALID_ARG)])
def test_norm_quant_refuses(lib, handle, change, status):
    assert _norm(lib, handle[0], **change) == status
    assert _norm(lib, None, **change) in (status, bq.MOE_ERR_INVALID_ARG)


def _qdense(lib, h, **kw):
    a = dict(x=A, xs=A, rows=32, n=64, k=64, wq=A, wsc=A, cap=0.0, y=A, y32=A, ws=A, ws_bytes=1 << 30)
    a.update(kw)
    w = bq.QdenseWeights(a["n"], a["k"], a["wq"], a["wsc"])
    return lib.moe_qdense_forward(h, a["x"], a["xs"], a["rows"], ctypes.byref(w), a["cap"], a["y"], a["y32"], a["ws"],
                                  a["ws_bytes"], None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), bq.MOE_ERR_INVALID_ARG), (dict(xs=None), bq.MOE_ERR_INVALID_ARG),
    (dict(y=None, y32=None), bq.MOE_ERR_INVALID_ARG), (dict(rows=0), bq.MOE_ERR_INVALID_ARG),
    (dict(rows=65537), bq.MOE_ERR_INVALID_ARG), (dict(n=0), bq.MOE_ERR_UNSUPPORTED),
    (dict(n=(1 << 28) + 1), bq.MOE_ERR_UNSUPPORTED), (dict(k=8), bq.MOE_ERR_UNSUPPORTED),
    (dict(k=40), bq.MOE_ERR_UNSUPPORTED), (dict(k=16400), bq.MOE_ERR_UNSUPPORTED),
    (dict(wq=None), bq.MOE_ERR_INVALID_ARG), (dict(wsc=None), bq.MOE_ERR_INVALID_ARG),
    (dict(wq=A + 8), bq.MOE_ERR_INVALID_ARG), (dict(wsc=A + 2), bq.MOE_ERR_INVALID_ARG),
    (dict(x=A + 4), bq.MOE_ERR_INVALID_ARG), (dict(xs=A + 2), bq.MOE_ERR_INVALID_ARG),
    (dict(y=A + 1), bq.MOE_ERR_INVALID_ARG), (dict(y32=A + 2), bq.MOE_ERR_INVALID_ARG),
    (dict(cap=math.nan), bq.MOE_ERR_INVALID_ARG), (dict(cap=math.inf), bq.MOE_ERR_INVALID_ARG)])
def test_qdense_refuses(lib, handle, change, status):
    assert _qdense(lib, handle[0], **change) == status
    assert _qdense(lib, None, **change) in (status, bq.MOE_ERR_INVALID_ARG)


def test_qdense_workspace(lib, handle):
    def need(n, k, rows):
        w = bq.QdenseWeights(n, k, A, A)
        return lib.moe_qdense_workspace_bytes(ctypes.byref(w), rows)

    for rows in (1, 8):
        assert need(4096, 2816, rows) == 0
    for bad in ((0, 64, 32), (64, 40, 32), (64, 64, 0), (64, 64, 65537)):
        assert need(*bad) == 0
    n = need(64, 64, 32)
    if n:
        assert _qdense(lib, handle[0], ws=None) == bq.MOE_ERR_INVALID_ARG
        assert _qdense(lib, handle[0], ws=A + 16) == bq.MOE_ERR_INVALID_ARG
        assert _qdense(lib, handle[0], ws_bytes=n - 1) == bq.MOE_ERR_WORKSPACE


def _logits(lib, h, **kw):
    a = dict(logits=A, ld=100, rows=2, vocab=100, out=A + 4096, ld_out=100, tokens=A)
    r = dict(history=A, history_len=A, prompt_len=A, history_stride=8, repetition=A, presence=A, frequency=A,
             bias_ids=A, bias_values=A, bias_len=A, bias_stride=4, mask=A, mask_stride=4)
    for k, v in kw.items():
        (a if k in a else r)[k] = v
    rules = bq.LogitRules(**r)
    return lib.moe_logits_process(h, a["logits"], a["ld"], a["rows"], a["vocab"], ctypes.byref(rules), a["out"],
                                  a["ld_out"], a["tokens"], None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), bq.MOE_ERR_INVALID_ARG), (dict(out=None, tokens=None), bq.MOE_ERR_INVALID_ARG),
    (dict(rows=0), bq.MOE_ERR_INVALID_ARG), (dict(rows=4097), bq.MOE_ERR_INVALID_ARG),
    (dict(vocab=0), bq.MOE_ERR_UNSUPPORTED), (dict(vocab=(1 << 28) + 1), bq.MOE_ERR_UNSUPPORTED),
    (dict(ld=99), bq.MOE_ERR_INVALID_ARG), (dict(ld_out=99), bq.MOE_ERR_INVALID_ARG),
    (dict(ld=1 << 33), bq.MOE_ERR_UNSUPPORTED), (dict(out=A, ld_out=104), bq.MOE_ERR_INVALID_ARG),
    (dict(history_len=None), bq.MOE_ERR_INVALID_ARG), (dict(history_stride=0), bq.MOE_ERR_INVALID_ARG),
    (dict(history_stride=(1 << 24) + 1), bq.MOE_ERR_UNSUPPORTED), (dict(history=None), bq.MOE_ERR_INVALID_ARG),
    (dict(bias_values=None), bq.MOE_ERR_INVALID_ARG), (dict(bias_len=None), bq.MOE_ERR_INVALID_ARG),
    (dict(bias_stride=0), bq.MOE_ERR_INVALID_ARG), (dict(bias_ids=None), bq.MOE_ERR_INVALID_ARG),
    (dict(mask_stride=3), bq.MOE_ERR_INVALID_ARG), (dict(mask_stride=-1), bq.MOE_ERR_INVALID_ARG),
    (dict(mask=A + 2), bq.MOE_ERR_INVALID_ARG), (dict(history=A + 1), bq.MOE_ERR_INVALID_ARG),
    (dict(tokens=A + 2), bq.MOE_ERR_INVALID_ARG), (dict(bias_values=A + 2), bq.MOE_ERR_INVALID_ARG)])
def test_logits_process_refuses(lib, handle, change, status):
    assert _logits(lib, handle[0], **change) == status
    assert _logits(lib, None, **change) in (status, bq.MOE_ERR_INVALID_ARG)
    assert lib.moe_logits_process(handle[0], A, 8, 1, 8, None, A, 8, None, None) == bq.MOE_ERR_INVALID_ARG


def test_binding_checks():
    """The binding refuses host tensors before it hands out an address."""
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        bq.make_qdense_weights(4, 16, torch.zeros((4, 16), dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError):
        bq.make_logit_rules(history=torch.zeros((2, 4), dtype=torch.int32), history_len=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        bq.make_logit_rules(history=torch.zeros(4, dtype=torch.int32))
    assert bq.make_logit_rules().rows is None


class OnDevice:
    """What the binding asks of a tensor, on a device of its own."""

    def __init__(self, t, device):
        self.t, self.device = t, f"cuda:{device}"
        self.get_device, self.data_ptr = (lambda: device), (lambda: A)

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_other_devices(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(bq, "_current_device", lambda: 0)

    class Lib:
        def __getattr__(self, name):
            return lambda *a: bq.MOE_OK

    moe = object.__new__(bq.Moe)
    moe.lib, moe.h = Lib(), None

    def on(dev, shape, dtype):
        return OnDevice(torch.zeros(shape, dtype=dtype), dev)

    i8, f32, i32, b16 = torch.int8, torch.float32, torch.int32, torch.bfloat16
    # (T = 2, K = N = 16; a stream is given: there is no device here to ask for its own)
    calls = {
        "norm_quant": lambda d: moe.norm_quant(on(d[0], (2, 16), b16), 2, on(d[1], (2, 16), i8), on(d[2], 2, f32),
                                               stream=1),
        "qdense": lambda d: moe.qdense_forward(on(d[0], (2, 16), i8), on(d[1], 2, f32), 2, bq.make_qdense_weights(
            16, 16, on(d[2], (16, 16), i8), on(d[2], 16, f32)), y32=on(0, (2, 16), f32), stream=1),
        "logits": lambda d: moe.logits_process(on(d[0], (2, 16), f32), 2, 16, bq.make_logit_rules(mask=on(d[1], 1, i32)),
                                               tokens=on(d[2], 2, i32), stream=1),
    }
    for call in calls.values():
        call((0, 0, 0))
        for bad in ((1, 0, 0), (0, 1, 0), (0, 0, 1)):
            with pytest.raises(ValueError):
                call(bad)
    with pytest.raises(ValueError):  # one of the tensors elsewhere
        bq.make_qdense_weights(16, 16, on(0, (16, 16), i8), on(1, 16, f32))
    with pytest.raises(ValueError):
        bq.make_logit_rules(history=on(0, (2, 4), i32), history_len=on(1, 2, i32))


# ------------------------------------------------------------------ the oracle
def test_oracle_norm_quant_by_hand():
    # rms of (3, 4, 0, 0) is 2.5; weight 2 on the second: u = (3, 8, 0, 0)
    h = to_bf16(np.array([[1.0, 4.0, 0.0, 0.0], [0.0] * 4]))
    y = to_bf16(np.array([[2.0, 0.0, 0.0, 0.0], [0.0] * 4]))
    g = to_bf16(np.array([1.0, 2.0, 1.0, 1.0]))
    o = BO.norm_quant(h, y, g, eps=0.0 + 1e-12)
    assert np.array_equal(gen.bf16_bits_to_f64(o["s"][0]), [3.0, 4.0, 0.0, 0.0])
    assert o["q"][0].tolist() == [48, 127, 0, 0]  # 127 * 3 / 8 = 47.625
    assert abs(o["scales"][0] - 8 / 2.5 / 127) < 1e-12 and np.allclose(o["x"][0], [1.2, 3.2, 0, 0], atol=1e-9)
    assert o["q"][1].tolist() == [0] * 4 and o["scales"][1] == 0.0
    # a tie goes to the even code: 127 * 1 / 254 = 0.5, 127 * 3 / 254 = 1.5
    t = BO.norm_quant(to_bf16(np.array([[254.0, 1.0, 3.0, -1.0]])))
    assert t["q"][0].tolist() == [127, 0, 2, 0]
    bad = BO.norm_quant(to_bf16(np.array([[np.inf, 1.0], [np.nan, 1.0], [2.0, 1.0]])))
    assert np.isnan(bad["scales"][:2]).all() and np.isfinite(bad["scales"][2]) and not bad["q"][:2].any()


def test_oracle_qdense_by_hand():
    x, w = np.array([[1, -2, 127]], dtype=np.int8), np.array([[3, 4, -128], [0, 1, 0]], dtype=np.int8)
    assert BO.int_product(x, w).tolist() == [[3 - 8 - 127 * 128, -2]]
    z = BO.qdense(x, [0.5], w, [2.0, 4.0])
    assert z.tolist() == [[3 - 8 - 127 * 128, -4]]
    assert abs(BO.qdense(x, [0.5], w, [2.0, 4.0], 30.0)[0, 1] - 30 * math.tanh(-4 / 30)) < 1e-12


def test_oracle_logits_by_hand():
    lg = np.array([[2.0, -2.0, 1.0, 0.0, 5.0], [1.0, 1.0, 1.0, 1.0, 1.0]])
    rows = [dict(history=[0, 1, 1, 2, 1, 9], prompt=1, repetition=2.0, presence=0.25, frequency=0.5,
                 bias=[(3, 1.0), (3, 4.0), (-1, 9.0)]), {}]
    mask = np.array([[1, 1, 1, 1, 0], [0, 0, 1, 1, 0]], dtype=bool)
    v, _ = BO.logits(lg, rows, mask)
    # 0: in the prompt only; 1: three times after it; 2: once
    assert v[0].tolist() == [1.0, -4.0 - 1.5 - 0.25, 0.5 - 0.5 - 0.25, 4.0, -math.inf]
    assert BO.greedy(v).tolist() == [3, 2]
    assert BO.greedy(np.array([[-np.inf, np.nan], [np.inf, -3.0]])).tolist() == [-1, 1]
