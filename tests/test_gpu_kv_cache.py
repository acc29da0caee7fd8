"""moe_kv_append and moe_kv_read against the oracle: rotation, codes and scales,
rows through tables, what is left as it was, what is refused on the device.

A turned value is u c - w s in fp32: sine and cosine to 2^-22 (the angle to half a
unit of 2^-24 of a half turn, two units for the function), two products and a sum:
2^-21 (|u| + |w|) in all."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from kv_cases import BF16, F32, Cache, bf16, dev, f64, i32
from oracle import kv_oracle as KO

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TURN = 2.0 ** -21


@pytest.fixture(scope="module")
def moe():
    bq.build_library()
    m = bq.Moe()
    yield m
    m.close()


def error(moe):
    torch.cuda.synchronize()
    return moe.get_error()


def freqs(r):
    return (10000.0 ** (-np.arange(0, r, 2) / max(r, 1))).astype(np.float32)


def near(got, want, x, r):
    """Turned rows in bf16: half a step, and the rotation's own error."""
    size = np.zeros_like(x)
    h = r // 2
    size[..., :h] = size[..., h:r] = np.abs(x[..., :h]) + np.abs(x[..., h:r])
    return np.all(np.abs(got - want) <= BF16 * np.abs(want) * (1 + 2.0 ** -8) + 2 * TURN * size)


def check_rows(cache, seq, pos, k, v, want_k, x_k, r):
    """The rows that the GPU's cache holds now against turned keys and values."""
    got = {}
    for name, d, s in (("k", cache.dk, cache.dks), ("v", cache.dv, cache.dvs)):
        pages, page = f64(d), cache.table[seq, pos // cache.page]
        got[name] = pages[page, :, pos % cache.page]
        if s is not None:
            got[name + "s"] = f64(s)[page, :, pos % cache.page]
    if not cache.bits8:
        assert near(got["k"], want_k, x_k, r) and np.array_equal(got["v"], v)
        return
    q, m = KO.quantise(v)
    assert np.array_equal(got["v"], q) and np.all(np.abs(got["vs"] - m) <= 2 * F32 * m)
    _, m = KO.quantise(want_k)
    most = 2 * np.abs(x_k).max(-1)
    assert np.all(np.abs(got["ks"] - m) <= 2 * F32 * m + TURN * most / 127)
    off = np.abs(got["k"] * got["ks"][..., None] - want_k)
    # half a code, the scale's error at the largest code, the division's and the rotation's
    assert np.all(off <= (got["ks"] * 0.5 + 4 * F32 * 127 * got["ks"] + 2 * TURN * most)[..., None])


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,page,r", [
    (1, 16, 8, 256, 64, 256), (1, 1, 1, 16, 16, 16), (5, 4, 2, 64, 16, 64), (64, 32, 8, 128, 64, 128),
    (7, 9, 3, 80, 32, 64), (3, 6, 2, 96, 128, 0), (33, 5, 5, 192, 256, 192), (2, 128, 128, 48, 16, 16),
    (300, 3, 1, 112, 16, 112)])
def test_append_of_a_batch(moe, bits8, T, Hq, H, D, page, r):
    """One token per sequence, at the end of each; q, k and v as parts of one projection's rows."""
    g = np.random.default_rng(T + D)
    lengths = g.integers(0, 200, T)
    cache = Cache(1, lengths, H, D, page, bits8)
    qkv = bf16(g.standard_normal((T, (Hq + 2 * H) * D)))
    x = dev(qkv)
    q, k, v = [qkv[:, a * D:b * D].reshape(T, -1, D) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H))]
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    f = freqs(r)
    before = [t.clone() for t in (cache.dk, cache.dv)]
    moe.kv_append(x[:, Hq * D:(Hq + H) * D], x[:, (Hq + H) * D:], i32(lengths), cache.c, q=x[:, :Hq * D], q_out=out,
                  inv_freq=dev(f, torch.float32) if r else None)
    assert error(moe) == bq.MOE_OK
    assert near(f64(out), KO.rotate(q, lengths, f), q, r)
    seq = np.arange(T)
    check_rows(cache, seq, lengths, k, v, KO.rotate(k, lengths, f), k, r)
    # nothing else was written
    for a, b in zip(before, (cache.dk, cache.dv)):
        page_ids = torch.from_numpy(cache.table[seq, lengths // page].astype(np.int64)).cuda()
        at = torch.from_numpy(lengths % page).cuda()
        a[page_ids, :, at] = b[page_ids, :, at]
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("T,H,D,page", [(1, 2, 64, 16), (15, 1, 128, 16), (17, 3, 80, 16), (500, 4, 128, 64),
                                        (1000, 8, 256, 256)])
def test_append_of_a_prompt_and_read_back(moe, bits8, T, H, D, page):
    """Rows of one prompt, given out of order, without queries; then the rows read back twice over."""
    g = np.random.default_rng(T)
    cache = Cache(2, [0, T + 40], H, D, page, bits8, room=3)
    k, v = bf16(g.standard_normal((2, T, H, D)))
    pos = g.permutation(T) + 5
    f = freqs(D)
    moe.kv_append(dev(k), dev(v), i32(pos), cache.c, seqs=i32(np.ones(T)), inv_freq=dev(f, torch.float32))
    assert error(moe) == bq.MOE_OK
    check_rows(cache, np.ones(T, int), pos, k, v, KO.rotate(k, pos, f), k, D)
    # the cache as it stands now, read in another order, positions named again, rows of a wider matrix
    cache.k, cache.v = f64(cache.dk), f64(cache.dv)
    if bits8:
        cache.ks, cache.vs = f64(cache.dks), f64(cache.dvs)
    n = 2 * T + 3
    seq, pos = np.ones(n, int), g.integers(0, T + 40, n)
    ko = torch.full((n, H * D + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.kv_read(cache.c, i32(pos), ko[:, 8:8 + H * D], vo, seqs=i32(seq))
    assert error(moe) == bq.MOE_OK
    wk, wv = cache.rows(seq, pos)
    for got, want in ((f64(ko)[:, 8:8 + H * D].reshape(n, H, D), wk), (f64(vo), wv)):
        # the fp32 product's rounding may move a value across a rounding border of bf16
        assert np.all(np.abs(got - want) <= BF16 * np.abs(want) * (1 + 2.0 ** -8))
        if not bits8:
            assert np.array_equal(got, want)
    assert np.all(f64(ko)[:, :8] == 7) and np.all(f64(ko)[:, 8 + H * D:] == 7)
    one = torch.empty_like(vo)
    moe.kv_read(cache.c, i32(pos), v_out=one, seqs=i32(seq))
    assert torch.equal(one, vo)


def test_far_positions(moe):
    """Angles of far positions: the rotation is as good as at the first."""
    pos = np.array([0, 1, 4097, 1 << 20, (1 << 30) - 1])
    T, D = len(pos), 64
    g = np.random.default_rng(3)
    q = bf16(g.standard_normal((T, 2, D)))
    kv = dev(np.zeros((T, 1, D)))
    pages = torch.zeros((1, 1, 16, D), dtype=torch.bfloat16, device="cuda")
    c = bq.make_kv_cache(pages, torch.zeros_like(pages), i32(np.full((1, 1), 0)))
    f = freqs(D)
    out = dev(q)
    # (sequence 7 is not there: only the queries are turned, in place)
    moe.kv_append(kv, kv, i32(pos), c, seqs=i32(np.full(T, 7)), q=out, q_out=out, inv_freq=dev(f, torch.float32))
    assert error(moe) == bq.MOE_ERR_BAD_EXPERT_ID
    assert near(f64(out), KO.rotate(q, pos, f), q, D)
    assert not pages.any()


@pytest.mark.parametrize("bits8", [False, True])
def test_rows_left_out_and_rows_that_are_not_there(moe, bits8):
    T, H, D, page = 6, 2, 64, 16
    cache = Cache(4, [20, 20], H, D, page, bits8)
    before = [t.clone() for t in (cache.dk, cache.dv)]
    g = np.random.default_rng(4)
    k = dev(g.standard_normal((T, H, D)))
    out = torch.full((T, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    q = dev(g.standard_normal((T, 1, D)))
    seq, pos = np.array([0, 0, 2, -1, 1, 1]), np.array([-1, -(1 << 31), 3, 3, 1 << 20, 32])  # (32: behind the table)
    moe.kv_append(k, k, i32(pos), cache.c, seqs=i32(seq), q=q, q_out=out)
    assert error(moe) == bq.MOE_ERR_BAD_EXPERT_ID
    assert torch.equal(out[2:], q[2:]) and bool((out[:2] == 7).all())
    for a, b in zip(before, (cache.dk, cache.dv)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    moe.kv_append(k[:2], k[:2], i32(pos[:2]), cache.c, seqs=i32(seq[:2]))
    assert error(moe) == bq.MOE_OK
    ko, vo = [torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    moe.kv_read(cache.c, i32(pos), ko, vo, seqs=i32(seq))
    assert error(moe) == bq.MOE_ERR_BAD_EXPERT_ID
    for t in (ko, vo):
        assert bool((t[:2] == 7).all()) and not t[2:].any()


def test_rows_that_are_not_finite(moe):
    """8-bit rows with a NaN or an infinity: codes 0 and the scale NaN; other heads as always.  Zeros: scale 0."""
    T, H, D = 4, 3, 32
    cache = Cache(5, [0] * T, H, D, 16, True)
    g = np.random.default_rng(5)
    k, v = bf16(g.standard_normal((2, T, H, D)))
    k[0, 1, 5], v[1, 2, 31], k[2, 0, 0], v[3, 0] = np.nan, np.inf, -np.inf, 0.0
    moe.kv_append(dev(k), dev(v), i32(np.zeros(T)), cache.c)
    assert error(moe) == bq.MOE_ERR_NONFINITE
    for x, d, s in ((k, cache.dk, cache.dks), (v, cache.dv, cache.dvs)):
        q, m = KO.quantise(x)
        page = cache.table[:, 0]
        assert np.array_equal(f64(d)[page, :, 0], q)
        assert np.allclose(f64(s)[page, :, 0], m, rtol=2 * F32, atol=0, equal_nan=True)
    out = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    moe.kv_read(cache.c, i32(np.zeros(T)), out)
    assert np.array_equal(np.isnan(f64(out)).all(-1), np.isin(np.arange(T * H), [1, 6]).reshape(T, H))


@pytest.mark.parametrize("size", [1e-38, 3e38, 1e-30, 1e30, 2.0 ** -126])
def test_values_at_the_ends_of_the_range(moe, size):
    T, H, D = 3, 1, 16
    cache = Cache(6, [0] * T, H, D, 16, True)
    v = bf16(np.random.default_rng(6).uniform(-1, 1, (T, H, D)) * size)
    moe.kv_append(dev(v), dev(v), i32(np.zeros(T)), cache.c)
    assert error(moe) == bq.MOE_OK
    q, m = KO.quantise(v)
    page = cache.table[:, 0]
    assert np.array_equal(f64(cache.dv)[page, :, 0], q) and np.array_equal(f64(cache.dk)[page, :, 0], q)
    assert np.all(np.abs(f64(cache.dvs)[page, :, 0] - m) <= 2 * F32 * m + 2.0 ** -149)


def test_pages_past_32_bits_of_bytes(moe):
    """A pool of more than 4 GiB: the last page is written and read where it lies."""
    H, D, page, n = 8, 256, 256, 4200
    kv = torch.zeros((n, H, page, D), dtype=torch.int8, device="cuda")
    s = torch.zeros((n, H, page), device="cuda")
    c = bq.make_kv_cache(kv, torch.zeros_like(kv), i32([[0, n - 1]]), s, torch.zeros_like(s))
    x = bf16(np.random.default_rng(7).standard_normal((2, H, D)))
    pos = i32([255, 511])
    out = torch.empty((2, H, D), dtype=torch.bfloat16, device="cuda")
    moe.kv_append(dev(x), dev(x), pos, c, seqs=i32([0, 0]))
    moe.kv_read(c, pos, out, seqs=i32([0, 0]))
    assert error(moe) == bq.MOE_OK
    q, m = KO.quantise(x)
    assert np.array_equal(f64(kv[0, :, 255]), q[0]) and np.array_equal(f64(kv[n - 1, :, 255]), q[1])
    assert int(kv.count_nonzero()) == int(np.count_nonzero(q))
    want = q * m[..., None]
    assert np.all(np.abs(f64(out) - want) <= BF16 * np.abs(want) * (1 + 2.0 ** -8))


def test_another_stream_and_a_graph(moe):
    T, H, D = 9, 2, 128
    cache = Cache(8, [30] * T, H, D, 16, True)
    g = np.random.default_rng(8)
    k, pos = dev(g.standard_normal((T, H, D))), i32(np.full(T, 30))
    out = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            moe.kv_append(k, k, pos, cache.c)
            moe.kv_read(cache.c, pos, out)
    for _ in range(2):
        x = bf16(g.standard_normal((T, H, D)))
        k.copy_(dev(x))
        torch.cuda.synchronize()
        graph.replay()
        assert error(moe) == bq.MOE_OK
        q, m = KO.quantise(x)
        want = q * m[..., None]
        assert np.all(np.abs(f64(out) - want) <= BF16 * np.abs(want) * (1 + 2.0 ** -8))
