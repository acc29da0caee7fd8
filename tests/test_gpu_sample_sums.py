"""The sums of moe_sample: exact over the weights' fixed-point values, however many
tokens a row has and whatever else is in the call.

A weight is within 2^-21 of its value, so is every sum of them, and a share of the
whole within 2^-20 (NEAR).  The cuts below stand 2^-19 of the whole away from where
another token would come in, so they have one right answer."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from kv_cases import i32
from test_gpu_sample import NEAR, draw, f32, moe  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_a_long_tail_of_small_weights(moe):  # noqa: F811
    """A thousand large weights and 2^25 small ones, which together are a quarter of the whole: a chain of fp32
    additions over a thread's 4096 of them would be off by 2^-15 of their sum, and the cut by a token."""
    V, big = 1 << 25, 1000
    g = np.random.default_rng(1)
    at = g.permutation(V)[:big]
    logits = np.full((2, V), -1.5, np.float32)
    logits[:, at] = (10 + np.arange(big) * 1e-4).astype(np.float32)
    l = logits[0, at].astype(np.float64)
    w = np.exp(l - l[-1])
    whole = w.sum() + (V - big) * np.exp(-1.5 - l[-1])
    order = np.arange(big)[::-1]  # by weight
    upto = np.cumsum(w[order])
    n = int(np.searchsorted(upto, 0.6 * whole))
    p = np.float32([upto[n] / whole - 2.0 ** -19, upto[n] / whole + 2.0 ** -19])
    want = [n + 1, n + 2]  # the fewest that sum to the share
    for x, k in zip(p.astype(np.float64), want):  # (also after the rounding of p)
        assert upto[k - 2] < (x - NEAR) * whole and (x + NEAR) * whole < upto[k - 1]
    u = np.array([0.5, 0.5])
    tokens, logp = draw(moe, logits, u, None, None, p)
    assert moe.get_error() == bq.MOE_OK
    for t in range(2):
        kept = order[:want[t]]
        ids = kept[np.argsort(at[kept])]
        run = np.cumsum(w[ids])
        near = [ids[np.searchsorted(run, x * run[-1], side="right")] for x in (0.5 - NEAR, 0.5, 0.5 + NEAR)]
        assert tokens[t] in at[near]
        mine = w[np.flatnonzero(at == tokens[t])[0]]
        assert abs(logp[t] - np.log(mine / run[-1])) <= 2 * NEAR + 2.0 ** -22 * abs(logp[t])  # (a token more: 2^-10)


@pytest.mark.parametrize("V", [5000, 50257, 262144])
def test_a_row_alone_and_among_others(moe, V):  # noqa: F811
    """The number of rows decides how many blocks a row has, and nothing else: the same bits come out."""
    g = np.random.default_rng(V)
    T = 300
    logits = f32(g.standard_normal((T, V)) * g.uniform(0.5, 4, (T, 1)))
    u, p = f32(g.random(T)), f32(g.uniform(0.3, 0.9999, T))
    k = i32(np.where(np.arange(T) % 3 == 0, g.integers(1, 3000, T), 0))
    m = f32(np.where(np.arange(T) % 5 == 0, 0.01, 0.0))
    tokens, logp = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
    moe.sample(logits, T, V, bq.make_sample_rules(u, top_k=k, top_p=p, min_p=m), tokens, logprobs=logp)
    for a, n in ((0, 1), (7, 1), (20, 5), (40, 17), (100, 64), (299, 1)):
        s = slice(a, a + n)
        t2, l2 = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
        moe.sample(logits[s], n, V, bq.make_sample_rules(u[s], top_k=k[s], top_p=p[s], min_p=m[s]), t2, logprobs=l2)
        assert torch.equal(t2, tokens[s]) and torch.equal(l2, logp[s])
    assert moe.get_error() == bq.MOE_OK
