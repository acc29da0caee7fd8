"""moe_sample at the vocabularies where a row's blocks change their form: those that
fill a block's shared memory, and the first that do not fit it."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from test_gpu_sample import check, draw, moe  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [360448, 360449, 524288, 786432 - 61, 786432, 786433])
@pytest.mark.parametrize("pad", [0, 3])
def test_vocabularies_about_a_blocks_memory(moe, V, pad):  # noqa: F811
    g = np.random.default_rng(V + pad)
    T = 6
    logits = g.standard_normal((T, V)) * 2.5 + 7 * (g.random((T, V)) < 400 / V)
    u, temp = g.random(T), g.uniform(0.6, 1.2, T)
    k, p, m = np.array([0, 50, 2000, 0, 0, 700]), np.array([1, 0.9, 1, 0.9, 1, 0.95]), np.array([0, 0, 0, 0, 0.02, 0.001])
    tokens, logp = draw(moe, logits, u, temp, k, p, m, stride=V + pad)
    assert moe.get_error() == bq.MOE_OK
    check(logits, tokens, logp, u, temp, k, p, m)
