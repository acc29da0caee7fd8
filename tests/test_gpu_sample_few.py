"""moe_sample where fewer tokens remain than top_k asks for: all of them stay, and
what the filters behind it leave is drawn from.  The bounds are test_gpu_sample's."""
import itertools

import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from test_gpu_sample import check, draw, moe  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = (5000, 40000, 262144, 1_000_003)  # one block; several; the most; rows that shared memory does not hold
MIN_P = float(np.float32(np.exp(-3.0)))


def rows(V):
    """(kept, more, logits, temperature, min_p, top_k): `kept` tokens within one of the largest, the others far below;
    the least logit that min-p allows lies between them, at no token, so the last 340 of 512 parts of the range that
    may remain are empty."""
    g = np.random.default_rng(V)
    for kept, more in itertools.product((300, 600, 1500, 3000), (1, 700)):
        l = np.zeros(V, np.float32)
        l[g.permutation(V)[:kept]] = g.uniform(5, 6, kept)
        yield kept, more, l, 1.0, MIN_P, kept + more


@pytest.mark.parametrize("top_p", [None, 0.9, 0.3])
@pytest.mark.parametrize("V", SIZES)
def test_min_p_leaves_fewer_than_top_k(moe, V, top_p):  # noqa: F811
    cases = list(rows(V))
    T = len(cases)
    logits = np.stack([c[2] for c in cases])
    m, k = np.array([c[4] for c in cases]), np.array([c[5] for c in cases])
    u = np.random.default_rng(1).random(T)
    p = None if top_p is None else np.full(T, top_p)
    tokens, logp = draw(moe, logits, u, None, k, p, m)
    assert moe.get_error() == bq.MOE_OK
    check(logits, tokens, logp, u, None, k, p, m)
    if top_p is None:
        for t, c in enumerate(cases):  # all that min-p leaves, in their order
            ids = np.flatnonzero(c[2] > 0)
            w = np.cumsum(np.exp(c[2][ids].astype(np.float64) - 6))
            near = [ids[min(np.searchsorted(w, x * w[-1], side="right"), len(ids) - 1)]
                    for x in np.float32(u[t]) + np.array([-1.0, 0.0, 1.0]) * 2.0 ** -20]
            assert tokens[t] in near


@pytest.mark.parametrize("top_p", [None, 0.9])
@pytest.mark.parametrize("V", (5000, 262144))
def test_few_logits_above_minus_infinity(moe, V, top_p):  # noqa: F811
    """Masked rows: 140 to 4000 tokens are left, and top_k is larger."""
    g = np.random.default_rng(V + 1)
    kept = np.array([140, 513, 700, 1500, 4000])
    T = len(kept)
    logits = np.full((T, V), -np.inf)
    for t, n in enumerate(kept):
        logits[t, g.permutation(V)[:n]] = g.standard_normal(n) * 2
    logits[2] = np.where(logits[2] > -np.inf, 1.5, -np.inf)  # all of one value
    u, k = g.random(T), kept + 300
    p = None if top_p is None else np.full(T, top_p)
    tokens, logp = draw(moe, logits, u, None, k, p)
    assert moe.get_error() == bq.MOE_OK
    check(logits, tokens, logp, u, None, k, p)
    if top_p is None:
        free, _ = draw(moe, logits, u)
        assert np.array_equal(tokens, free)  # top_k takes nothing away
