"""The binding of the batched path checks shapes, not sizes alone: a matrix whose
rows have another width than the call's would be read, or written, in the wrong
places.  No GPU: the library is one that accepts every call."""
import pytest

import bit_affine_quantized_gb300 as bq
from test_batch_host import OnDevice

torch = pytest.importorskip("torch")
I8, F32, I32, B16 = torch.int8, torch.float32, torch.int32, torch.bfloat16
T, H, N = 4, 64, 48


@pytest.fixture
def moe(monkeypatch):
    monkeypatch.setattr(bq, "_current_device", lambda: 0)

    class Lib:
        def __getattr__(self, name):
            return lambda *a: bq.MOE_OK

    m = object.__new__(bq.Moe)
    m.lib, m.h = Lib(), None
    return m


def on(shape, dtype):
    return OnDevice(torch.zeros(shape, dtype=dtype), 0)


def norm(moe, T=T, **kw):
    a = dict(hidden=on((T, H), B16), q=on((T, H), I8), scales=on(T, F32), y=on((T, H), B16), norm=on(H, B16),
             hidden_out=on((T, H), B16), x_out=on((T, H), B16))
    a.update(kw)
    moe.norm_quant(a["hidden"], T, a["q"], a["scales"], y=a["y"], norm=a["norm"], hidden_out=a["hidden_out"],
                   x_out=a["x_out"], stream=1)


def qdense(moe, T=T, **kw):
    a = dict(x=on((T, H), I8), xs=on(T, F32), w=on((N, H), I8), ws=on(N, F32), y=on((T, N), B16), y32=on((T, N), F32))
    a.update(kw)
    moe.qdense_forward(a["x"], a["xs"], T, bq.make_qdense_weights(N, H, a["w"], a["ws"]), y=a["y"], y32=a["y32"],
                       stream=1)


def rules(**kw):
    a = dict(history=on((T, 8), I32), history_len=on(T, I32), prompt_len=on(T, I32), repetition=on(T, F32),
             presence=on(T, F32), frequency=on(T, F32), bias_ids=on((T, 3), I32), bias_values=on((T, 3), F32),
             bias_len=on(T, I32), mask=on((T, 2), I32))
    a.update(kw)
    return bq.make_logit_rules(**a)


@pytest.mark.parametrize("bad", [
    dict(hidden=on((T, 2 * H), B16)), dict(y=on((T, 2 * H), B16)), dict(hidden_out=on((T, H + 16), B16)),
    dict(x_out=on((3 * T, H // 2), B16)), dict(hidden=on((3 * T, H // 2), B16)), dict(q=on((T, H // 2), I8)),
    dict(norm=on((H, 2), B16)), dict(scales=on((T, 2), F32)), dict(hidden=on((2, T, H // 2 + 8), B16))])
def test_norm_quant_widths(moe, bad):
    norm(moe)
    with pytest.raises(ValueError):
        norm(moe, **bad)


@pytest.mark.parametrize("bad", [
    dict(x=on((T, 2 * H), I8)), dict(x=on((3 * T, H // 2), I8)), dict(xs=on((T, 2), F32)), dict(w=on((H, N), I8)),
    dict(w=on((N, 2 * H), I8)), dict(ws=on((N, 2), F32)), dict(y=on((T, N + 16), B16)), dict(y=on((T, 64), B16)),
    dict(y32=on((T, 2 * N), F32))])
def test_qdense_widths(moe, bad):
    qdense(moe)
    with pytest.raises(ValueError):
        qdense(moe, **bad)


@pytest.mark.parametrize("bad", [
    dict(bias_values=on((T, 5), F32)), dict(bias_values=on((2 * T, 2), F32)), dict(history_len=on((T, 2), I32)),
    dict(prompt_len=on((T, 2), I32)), dict(repetition=on((T, 2), F32)), dict(presence=on((2, T), F32)),
    dict(frequency=on((T, 8), F32)), dict(bias_len=on((T, 3), I32))])
def test_rules_widths(moe, bad):
    assert rules().rows == T
    with pytest.raises(ValueError):
        rules(**bad)


def test_tokens_of_the_logits(moe):
    lg = on((T, N), F32)
    moe.logits_process(lg, T, N, rules(), tokens=on(T, I32), stream=1)
    with pytest.raises(ValueError):
        moe.logits_process(lg, T, N, rules(), tokens=on((T, 2), I32), stream=1)


def test_shapes_that_say_the_same(moe):
    """Flat buffers, more rows than asked for, rows in several dimensions, vectors as a row or a column, the rows'
    exact size in another shape."""
    norm(moe, hidden=on(T * H, B16), y=on((2, 2, H), B16), hidden_out=on((T + 3, H), B16),
         x_out=on((T, 4, H // 4), B16))
    norm(moe, scales=on((T, 1), F32), norm=on((1, H), B16), q=on((2, 2, H), I8))
    norm(moe, T=1, q=on(H, I8), hidden=on(H, B16), scales=on((), F32))
    qdense(moe, y=on((T * 6, 8), B16))
    qdense(moe, x=on(T * H, I8), xs=on((1, T), F32), w=on(N * H, I8), y=on((T, 6, 8), B16), y32=on((9, N), F32))
    moe.qdense_forward(on((T, H), I8), on(T, F32), T, bq.make_qdense_weights(N, H, on((N, H), I8), on(N, F32)),
                       on((16, 64), torch.uint8), y32=on((T, N), F32), stream=1)
    rules(bias_values=on(T * 3, F32), history_len=on((T, 1), I32), repetition=on((1, T), F32), presence=on(T + 2, F32))
