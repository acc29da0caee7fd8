"""moe_kv_attend's caps of any size: a capped score is as good, relative to itself, as
one that is not capped.

A score's error: 32 * 2^-22 of the sum of magnitudes behind it and 2^-22 of the
largest score (test_gpu_kv_attend's), and for the cap 2^-19 of the capped score: below
a quarter of the cap the series and its factors, 4 roundings; above it 1 - 2 / (E + 1)
with E within 2^-21.5 (the exponential 2^-22, its argument 2^-23), the sum, the division
and the difference within 2^-22: 2^-21 in all of a result of 0.245 or more.  A weight
changes by as much; the other terms are that file's."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from kv_cases import BF16, Cache, dev, f64, i32
from oracle import kv_oracle as KO
from test_gpu_kv_attend import moe, queries, run  # noqa: F401

pytestmark = pytest.mark.gpu


def check(cache, q, lengths, scale, softcap, out, lse):
    n, Hq, D = q.shape
    group = Hq // cache.heads
    got, got_lse = f64(out).reshape(n, Hq, D), f64(lse)
    weight = 2.0 ** -11 if cache.bits8 else BF16
    for s in range(n):
        k, v = cache.rows(np.full(lengths[s], s), np.arange(lengths[s]))
        for h in range(Hq):
            kh, vh = k[:, h // group], v[:, h // group]
            want, wl, mean, size = KO.attend(q[s, h], kh, vh, scale, softcap)
            top = np.abs(KO.scores(q[s, h], kh, scale, softcap)[0]).max()
            z = 32 * 2.0 ** -22 * size + 2.0 ** -22 * max(size, abs(wl)) + 2.0 ** -19 * top
            tol = mean * (weight + 2 * z + 2.0 ** -17) + BF16 * np.abs(want) * 1.01 + 1e-37
            if cache.bits8:
                tol = tol + lengths[s] * 2.0 ** -39 * np.abs(vh).max()
            assert np.all(np.abs(got[s, h] - want) <= tol), (s, h)
            assert abs(got_lse[s, h] - wl) <= z + 2.0 ** -17 + 2.0 ** -22 * abs(wl), (s, h, got_lse[s, h], wl)


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("softcap", [1e-3, 2.0, 8.0, 33.0, 1e3, 1e4, 1e6, 1e20, 1.2e38, 2e38, 3.4e38])
def test_caps_of_any_size(moe, bits8, softcap):  # noqa: F811
    lengths = [200, 33, 1]
    cache = Cache(36, lengths, 2, 64, 16, bits8)
    q = queries(37, 3, 4, 64)  # scores of some -12 .. 12: on both sides of a quarter of the smaller caps
    for scale in (0.25, -0.25):
        out, lse = run(moe, cache, dev(q), i32(lengths), scale, softcap)
        assert moe.get_error() == bq.MOE_OK
        check(cache, q, lengths, scale, softcap, out, lse)


@pytest.mark.parametrize("bits8", [False, True])
def test_large_scores_under_large_caps(moe, bits8):  # noqa: F811
    """Scores near a large cap: all but the largest have no weight, and the largest is the cap's."""
    lengths = [150, 20]
    cache = Cache(38, lengths, 1, 64, 16, bits8)
    q = queries(39, 2, 2, 64)
    for softcap, scale in ((1e6, 2e5), (1e20, 1e20), (2e38, 2e36)):
        out, lse = run(moe, cache, dev(q), i32(lengths), scale, softcap)
        assert moe.get_error() == bq.MOE_OK
        got, got_lse = f64(out), f64(lse)
        for s in range(2):
            k, v = cache.rows(np.full(lengths[s], s), np.arange(lengths[s]))
            for h in range(2):
                z = KO.scores(q[s, h], k[:, 0], scale, softcap)[0]
                first, second = np.sort(z)[::-1][:2]
                if first - second < 2.0 ** -12 * abs(first):
                    continue  # (within the scores' errors of each other)
                assert abs(got_lse[s, h] - first) <= 2.0 ** -12 * abs(first)
                # the output's rounding, and the weight's: of 1 none, of 1 times a row's scale half a step of fp16
                assert np.all(np.abs(got[s, h] - v[z.argmax(), 0]) <= (BF16 + 2.0 ** -11) * np.abs(v[z.argmax(), 0]) * 1.01 + 1e-6)


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("scale,softcap", [(3e38, 0.0), (-3e38, 0.0), (3e38, 1e-3), (1e30, 5.0), (3e38, 3e38)])
@pytest.mark.parametrize("size", [1.0, 40.0, 2.0 ** 100])
def test_scores_of_zero_of_large_queries(moe, bits8, scale, softcap, size):  # noqa: F811
    """Keys of zeros: every score is 0, whatever the query and the factors; the output is the mean of the values."""
    lengths = [77, 3]
    cache = Cache(40, lengths, 2, 64, 16, bits8)
    cache.k[:] = 0.0
    cache.upload()
    q = queries(41, 2, 4, 64) * size
    out, lse = run(moe, cache, dev(q), i32(lengths), scale, softcap)
    assert moe.get_error() == bq.MOE_OK
    check(cache, q, lengths, 0.0, 0.0, out, lse)
