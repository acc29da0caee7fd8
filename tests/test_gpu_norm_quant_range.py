"""norm_quant at the upper end of fp32 and bf16: a normalised value that either
cannot hold is told, not stored as an infinity."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from oracle import batch_oracle as BO
from oracle.batch_oracle import to_bf16
from synth import gen
from test_gpu_norm_quant import REL, moe, run  # noqa: F401  (moe: the fixture)

pytestmark = pytest.mark.gpu

TOP = float(np.float32(2.0 ** 127 * (2 - 2.0 ** -7)))  # bf16's largest value


@pytest.mark.parametrize("T", [3, 500])
@pytest.mark.parametrize("x_out", [True, False])
def test_scale_out_of_range(moe, T, x_out):  # noqa: F811
    """One value of 64, a weight of 1e38: r = 8 and m r = 8e38, though both are finite."""
    v = np.ones((T, 64))
    v[1] = 0
    v[1, 5] = 1.0
    g = np.ones(64)
    g[5] = 1e38
    h, gb = to_bf16(v), to_bf16(g)
    got = run(moe, h, g=gb, x_out=x_out, status=bq.MOE_ERR_NONFINITE)
    want = BO.norm_quant(h, g_bits=gb)
    assert np.isnan(got["scales"][1]) and not got["q"][1].any()
    rest = np.arange(T) != 1
    assert np.array_equal(got["q"][rest], want["q"][rest])
    assert np.all(np.abs(got["scales"] - want["scales"])[rest] <= REL * want["scales"][rest])
    if x_out:
        assert np.isnan(gen.bf16_bits_to_f64(got["x"][1])).all()
        assert np.isfinite(gen.bf16_bits_to_f64(got["x"][rest])).all()


@pytest.mark.parametrize("T", [1, 500])
def test_rows16_out_of_range(moe, T):  # noqa: F811
    """m r = 1.9999 * 2^127: fp32 holds it, bf16 rounds it to infinity."""
    v = np.full((T, 64), 1 - 2.0 ** -8)
    v[:, 0] = 1.0
    h, g = to_bf16(v), to_bf16(np.full(64, TOP))
    want = BO.norm_quant(h, g_bits=g, eps=0.0)
    assert np.all((127 * want["scales"] > 2.0 ** 127 * (2 - 2.0 ** -8)) & (127 * want["scales"] < 2.0 ** 128 * (1 - 2.0 ** -20)))
    got = run(moe, h, g=g, eps=0.0, x_out=False)
    assert np.array_equal(got["q"], want["q"]) and np.all(np.abs(got["scales"] - want["scales"]) <= REL * want["scales"])
    got = run(moe, h, g=g, eps=0.0, x_out=True, status=bq.MOE_ERR_NONFINITE)
    assert np.isnan(got["scales"]).all() and not got["q"].any() and np.isnan(gen.bf16_bits_to_f64(got["x"])).all()


@pytest.mark.parametrize("T", [1, 500])
def test_largest_rows16(moe, T):  # noqa: F811
    """Rows of ones with the largest weight: r = 1, and x is that weight."""
    h, g = to_bf16(np.ones((T, 64))), to_bf16(np.full(64, TOP))
    got = run(moe, h, g=g, eps=0.0)
    assert np.all(got["q"] == 127) and np.all(gen.bf16_bits_to_f64(got["x"]) == TOP)
    assert np.all(np.abs(got["scales"] - TOP / 127) <= REL * TOP / 127)
