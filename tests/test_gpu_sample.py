"""moe_sample against the oracle.

A weight is within 2^-21 of its value (fp32 exponentials), so a share of the sum is
within 2^-20: a token is right if the oracle gives it for a random number and a
top_p within 2^-20 of the given ones, and its log-probability is within 2^-19 of
the oracle's (fp32's own rounding on top)."""
import itertools

import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from kv_cases import i32
from oracle import kv_oracle as KO

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

NEAR = 2.0 ** -20


@pytest.fixture(scope="module")
def moe():
    bq.build_library()
    m = bq.Moe()
    yield m
    m.close()


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()


def draw(moe, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, stride=None, probs=True):
    T, V = logits.shape
    ld = stride or V
    wide = torch.full((T, ld), np.nan, device="cuda")
    wide[:, :V] = f32(logits)
    r = bq.make_sample_rules(f32(u), *[None if x is None else f32(x) for x in (temperature,)],
                             None if top_k is None else i32(top_k), *[None if x is None else f32(x) for x in (top_p, min_p)])
    tokens = torch.full((T + 2,), 77, dtype=torch.int32, device="cuda")
    logp = torch.full((T + 2,), 77.0, device="cuda") if probs else None
    moe.sample(wide, T, V, r, tokens, logprobs=logp)
    torch.cuda.synchronize()
    assert tokens[T:].tolist() == [77, 77]
    return tokens[:T].cpu().numpy(), None if logp is None else logp[:T].cpu().numpy().astype(float)


def at(x, t, default):
    return default if x is None else float(np.float32(x[t]))


def check(logits, tokens, logp, u, temperature=None, top_k=None, top_p=None, min_p=None):
    l32 = np.asarray(logits, np.float32).astype(np.float64)
    for t in range(len(logits)):
        p, uu = at(top_p, t, 1.0), at(u, t, 0.0)
        k = 0 if top_k is None else int(top_k[t])
        found = []
        for du, dp in itertools.product((0, -NEAR, NEAR), (0, -NEAR, NEAR) if p < 1 else (0,)):
            found.append(KO.sample(l32[t], uu + du if uu < 1 else uu, at(temperature, t, 1.0), k,
                                   min(p + dp, 1 - 1e-12) if p < 1 else 1.0, at(min_p, t, 0.0)))
            token, lp = found[-1]
            if token == tokens[t] and (logp is None or lp == logp[t] or
                                       abs(lp - logp[t]) <= 2 * NEAR + 2.0 ** -22 * abs(lp)):
                break
        else:
            raise AssertionError((t, int(tokens[t]), None if logp is None else logp[t], found))


@pytest.mark.parametrize("V,pad", [(1, 0), (2, 0), (7, 3), (31, 0), (1000, 0), (4097, 1), (16384, 0), (16385, 0),
                                   (50257, 3), (100003, 13), (262144, 0), (300001, 0)])
def test_vocabularies(moe, V, pad):
    """Every combination of filters, a row each."""
    g = np.random.default_rng(V)
    rows = list(itertools.product((0, 1, 5, 64, 1000), (1.0, 0.95, 0.5, 0.01), (0.0, 0.05, 0.5)))
    T = len(rows)
    logits = g.standard_normal((T, V)) * np.exp(g.uniform(-1, 1.6, (T, 1))) + 8 * (g.random((T, V)) < 50 / V)
    k, p, m = [np.array(c) for c in zip(*rows)]
    u, temp = g.random(T), np.exp(g.uniform(-1, 1, T))
    tokens, logp = draw(moe, logits, u, temp, k, p, m, stride=V + pad)
    assert moe.get_error() == bq.MOE_OK
    check(logits, tokens, logp, u, temp, k, p, m)


@pytest.mark.parametrize("V", [33, 20000, 262144])
def test_without_filters(moe, V):
    g = np.random.default_rng(V)
    logits, u = g.standard_normal((9, V)) * 2, g.random(9)
    tokens, logp = draw(moe, logits, u)
    check(logits, tokens, logp, u)
    again, _ = draw(moe, logits, u, probs=False)
    assert np.array_equal(tokens, again)


@pytest.mark.parametrize("V", [64, 5000, 262144])
def test_equal_logits(moe, V):
    """All tokens equal: ties go by id, whatever the filter that cuts them."""
    T = 8
    logits = np.full((T, V), 3.25)
    k = np.array([0, 10, 10, 0, 0, V, 1, 40])
    p = np.array([1, 1, 1, 0.5, 0.5, 1, 1, 0.5])
    u = np.array([0, 0, 0.95, 0.0, 0.9, 0.5, 0.9, 0.99])
    tokens, logp = draw(moe, logits, u, np.full(T, 0.7), k, p, np.full(T, 0.1))
    # equal weights: kept n, the token floor(u n)
    n = np.array([V, 10, 10, V // 2, V // 2, V, 1, 20])
    assert tokens.tolist() == [int(np.floor(float(np.float32(a)) * b)) for a, b in zip(u, n)]
    assert np.allclose(logp, -np.log(n), rtol=1e-6, atol=1e-6)


def test_a_few_levels(moe):
    """Many ties at a few values; the cut falls among equals."""
    g = np.random.default_rng(5)
    T, V = 40, 30000
    logits = g.integers(-3, 3, (T, V)) * 1.5
    k = g.integers(1, V, T)
    u = g.random(T)
    tokens, logp = draw(moe, logits, u, None, k)
    check(logits, tokens, logp, u, None, k)
    p = g.random(T)
    tokens, logp = draw(moe, logits, u, None, None, p)
    check(logits, tokens, logp, u, None, None, p)
    tokens, logp = draw(moe, logits, u, None, k, p)
    check(logits, tokens, logp, u, None, k, p)


def test_random_numbers_at_the_ends(moe):
    V = 9000
    logits = np.random.default_rng(6).standard_normal((8, V))
    u = np.array([0.0, -1.0, np.nan, 1.0, 2.0, np.inf, 1 - 2.0 ** -24, 2.0 ** -149])
    tokens, _ = draw(moe, logits, u)
    assert tokens.tolist()[:6] == [0, 0, 0, V - 1, V - 1, V - 1] and tokens[6] >= V - 2 and tokens[7] == 0
    tokens, _ = draw(moe, logits, u, top_k=np.full(8, 3))
    ids = np.sort(np.argsort(-logits, axis=1)[:, :3], axis=1)
    assert tokens.tolist() == [ids[t, 2 if t in (3, 4, 5, 6) else 0] for t in range(8)]


def test_temperatures_and_filters_at_the_ends(moe):
    V, T = 5000, 14
    g = np.random.default_rng(7)
    logits = g.standard_normal((T, V)) * 3
    u = np.full(T, 0.999)
    temp = np.array([0, -1, np.nan, 1e-30, 2.0 ** -149, 1e-3, np.inf, 1e30] + [1.0] * 6)
    tokens, logp = draw(moe, logits, u, temp)
    top = logits.astype(np.float32).argmax(1)
    assert tokens[:5].tolist() == top[:5].tolist() and np.all(logp[:5] == 0)
    check(logits[5:6], tokens[5:6], logp[5:6], u[:1], temp[5:6])
    assert tokens[6] == int(0.999 * V) and tokens[7] == int(0.999 * V)
    assert np.allclose(logp[6:8], -np.log(V), rtol=1e-6)
    p = np.array([0, -1, np.nan, 1.0, 7.0, 1e-30, 1 - 2.0 ** -24] + [1.0] * 7)
    m = np.array([0] * 7 + [1.0, 2.0, np.nan, -1, 1e-30, 0.0, np.inf])
    k = np.array([0] * 12 + [-5, 1 << 30])
    tokens, logp = draw(moe, logits, u, None, k, p, m)
    plain, _ = draw(moe, logits, u)
    assert tokens[[0, 1, 5, 7, 8, 13]].tolist() == top[[0, 1, 5, 7, 8, 13]].tolist()
    assert tokens[[2, 3, 4, 9, 10, 12]].tolist() == plain[[2, 3, 4, 9, 10, 12]].tolist()
    check(logits[[6, 11]], tokens[[6, 11]], logp[[6, 11]], u[:2], None, None, p[[6, 11]], m[[6, 11]])


@pytest.mark.parametrize("V", [50, 40000])
def test_values_that_do_not_count(moe, V):
    """-inf is never drawn; NaN and +inf neither, and they are told; a row without a token."""
    g = np.random.default_rng(8)
    T = 6
    logits = g.standard_normal((T, V))
    logits[:, ::3] = -np.inf
    logits[1] = -np.inf
    logits[2] = -np.inf
    logits[2, 17] = -3e38
    logits[3, 7::9] = 3e38
    u = np.array([0.7, 0.5, 0.9, 0.3, 0.0, 0.999])
    tokens, logp = draw(moe, logits, u, top_k=np.array([0, 3, 3, 0, 5, 0]))
    assert moe.get_error() == bq.MOE_OK
    assert tokens[1] == -1 and logp[1] == -np.inf and tokens[2] == 17 and logp[2] == 0
    keep = [0, 3, 4, 5]
    check(logits[keep], tokens[keep], logp[keep], u[keep], None, [0, 0, 5, 0])
    logits[4, 5], logits[5, 1], logits[1, 4] = np.nan, np.inf, np.nan
    tokens, logp = draw(moe, logits, u)
    assert moe.get_error() == bq.MOE_ERR_NONFINITE
    assert tokens[1] == -1
    logits[4, 5] = logits[5, 1] = -np.inf
    check(logits[keep], tokens[keep], logp[keep], u[keep])


def test_values_close_together(moe):
    """Neighbouring floats: a cut goes by the logits, not by what an fp32 difference keeps of them."""
    V = 20000
    l = (np.float32(1000.0) + np.random.default_rng(9).integers(0, 50, (4, V)) * np.float32(2.0 ** -14)).astype(np.float32)
    l[:, 5] = -1000.0
    k, u = np.array([7, 100, 3000, 19999]), np.array([0.1, 0.5, 0.9, 0.99])
    tokens, logp = draw(moe, l, u, None, k)
    check(l, tokens, logp, u, None, k)


@pytest.mark.parametrize("V", [600, 40000])
def test_lists_of_every_length(moe, V):
    ks = [1, 2, 31, 32, 33, 63, 65, 127, 128, 129, 160, 255, 256, 257, 300, 479, 511, 512, 513]
    g = np.random.default_rng(V + 1)
    k, p, u = (np.array(c) for c in zip(*itertools.product(ks, (1.0, 0.9), (0.0, 0.37, 0.999))))
    logits = g.standard_normal((len(k), V)) * 2
    tokens, logp = draw(moe, logits, u, None, k, p)
    assert moe.get_error() == bq.MOE_OK
    check(logits, tokens, logp, u, None, k, p)


@pytest.mark.parametrize("V", [3000, 50000])
@pytest.mark.parametrize("few", [2, 7, 11])
def test_cuts_among_close_values(moe, V, few):
    """A few tokens far above, the others within 2^-few of each other: the cut lies in one bin of the first histogram."""
    g = np.random.default_rng(V + few)
    k, p, u = (np.array(c) for c in zip(*itertools.product((0, V // 9, V - 20), (1.0, 0.8, 0.3), (0.01, 0.5, 0.99))))
    logits = g.random((len(k), V)) * 2.0 ** -few
    logits[:, 5:V:V // 10] += 50
    temp = np.full(len(k), 10.0)  # (a far one counts as much as e^5 others)
    tokens, logp = draw(moe, logits, u, temp, k, p)
    assert moe.get_error() == bq.MOE_OK
    check(logits, tokens, logp, u, temp, k, p)


def test_shares_follow_the_weights(moe):
    """A thousand even random numbers pick each token as often as its weight says."""
    w = np.array([0.1, 0.0, 0.4, 0.25, 0.05, 0.2])
    T = 1000
    with np.errstate(divide="ignore"):
        logits = np.tile(np.log(w), (T, 1))
    tokens, _ = draw(moe, logits, (np.arange(T) + 0.5) / T)
    assert np.all(np.abs(np.bincount(tokens, minlength=6) - w * T) <= 1)


def test_most_rows(moe):
    T, V = 4096, 700
    g = np.random.default_rng(10)
    logits, u = g.standard_normal((T, V)) * 2, g.random(T)
    k, p = g.integers(0, 50, T), g.uniform(0.5, 1.2, T)
    tokens, logp = draw(moe, logits, u, None, k, p)
    check(logits, tokens, logp, u, None, k, p)


def test_a_vocabulary_of_millions(moe):
    V = 3_000_017
    g = np.random.default_rng(11)
    logits, u = g.standard_normal((3, V)) * 3, g.random(3)
    k, p = np.array([50, 0, 0]), np.array([0.9, 0.9, 1.0])
    tokens, logp = draw(moe, logits, u, None, k, p)
    check(logits, tokens, logp, u, None, k, p)


def test_a_graph_and_rows_in_any_place(moe):
    """Captured, replayed with new logits; rows off a 16-byte boundary."""
    T, V = 5, 3001
    wide = torch.zeros((T, V + 8), device="cuda")
    logits = wide[:, 3:3 + V]
    g = np.random.default_rng(12)
    u = f32(g.random(T))
    r = bq.make_sample_rules(u, top_p=f32(np.full(T, 0.9)))
    tokens, logp = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            moe.sample(logits, T, V, r, tokens, logprobs=logp)
    for _ in range(3):
        x = g.standard_normal((T, V)) * 3
        logits.copy_(f32(x))
        u.copy_(f32(g.random(T)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(x, tokens.cpu().numpy(), logp.cpu().numpy().astype(float), u.cpu().numpy(), None, None, np.full(T, 0.9))
