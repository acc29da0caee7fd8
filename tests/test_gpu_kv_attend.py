"""moe_kv_attend against the oracle, a query head at a time.

What an output may be off by, with p the weights, A the weighted mean of the
values' magnitudes and S the sum of magnitudes behind a score:
  a weight's rounding            half a step of bf16 (bf16 cache) or fp16 (8 bits), of A
  a score's error                32 * 2^-22 S + 2^-22 |z|: fp32 sums in at most 16 steps of 16 products and
                                 the factors; capped scores 2^-20 of the cap more; a weight changes by as much
  sums over positions, joins     2^-17 of A
  a small weight (8 bits)        a weight times its row's scale is held as fp16 in units of U 2^-14, U the power of two
                                 at or below the largest scale s: below fp16's normal numbers (2^-14) it is off by up
                                 to half of 2^-24, times 2^-14 U <= 2^-14 s: 2^-39 s.  Times a code of up to 127, over
                                 the positions, divided by a sum of weights of 1 or more: positions 2^-39 127 s, and
                                 127 s is the largest magnitude of a value, as every row has a code of 127
  the output's rounding          half a step of bf16"""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from kv_cases import BF16, Cache, bf16, dev, f64, i32
from oracle import kv_oracle as KO

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    bq.build_library()
    m = bq.Moe()
    yield m
    m.close()


def run(moe, cache, q, lengths, scale, softcap=0.0, window=0, out=None, **kw):
    n, Hq, D = q.shape
    out = torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((n, Hq), 7.0, device="cuda")
    ws = torch.full((moe.kv_attend_workspace_bytes(cache.c, Hq),), 255, dtype=torch.uint8, device="cuda")
    moe.kv_attend(q, lengths, cache.c, out, ws, scale=scale, softcap=softcap, window=window, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def check(cache, q, lengths, scale, softcap, window, out, lse, heads=None):
    n, Hq, D = q.shape
    group = Hq // cache.heads
    got, got_lse = f64(out).reshape(n, Hq, D), f64(lse)
    weight = 2.0 ** -11 if cache.bits8 else BF16
    for s in range(n):
        first = max(0, int(lengths[s]) - window) if window else 0
        pos = np.arange(first, max(first, int(lengths[s])))
        k, v = cache.rows(np.full(len(pos), s), pos)
        for h in range(Hq) if heads is None else heads:
            want, wl, mean, size = KO.attend(q[s, h], k[:, h // group], v[:, h // group], scale, softcap)
            if len(pos) == 0:
                assert not got[s, h].any() and got_lse[s, h] == -np.inf
                continue
            z = 32 * 2.0 ** -22 * size + 2.0 ** -22 * max(size, abs(wl)) + 2.0 ** -20 * softcap
            tol = mean * (weight + 2 * z + 2.0 ** -17) + BF16 * np.abs(want) * 1.01 + 1e-37
            if cache.bits8:
                tol = tol + len(pos) * 2.0 ** -39 * np.abs(v[:, h // group]).max()
            off = np.abs(got[s, h] - want)
            assert np.all(off <= tol), (s, h, float((off / tol).max()))
            assert abs(got_lse[s, h] - wl) <= z + 2.0 ** -17 + 2.0 ** -22 * abs(wl), (s, h, got_lse[s, h], wl)


def queries(seed, n, Hq, D):
    return bf16(np.random.default_rng(seed).standard_normal((n, Hq, D)) * 2)


SHAPES = [  # kv heads, queries to a head, head size, page
    (8, 2, 256, 64), (1, 1, 16, 16), (2, 4, 64, 16), (4, 8, 128, 64), (3, 3, 80, 32), (2, 5, 96, 16), (1, 16, 192, 256),
    (2, 16, 256, 128), (1, 33, 64, 32), (1, 64, 128, 16), (5, 1, 112, 64), (2, 7, 48, 256), (1, 9, 240, 16)]
LENGTHS = [[1], [0], [16, 17, 15], [300, 0, 1, 2, 31, 32, 33, 64], [5, 0, 0, 0, 900], [1500, 63, 65, 127, 129, 255, 257]]


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("H,group,D,page", SHAPES)
def test_shapes(moe, bits8, H, group, D, page):
    for i, lengths in enumerate(LENGTHS):
        cache = Cache(10 + i, lengths, H, D, page, bits8)
        q = queries(20 + i, len(lengths), H * group, D)
        out, lse = run(moe, cache, dev(q), i32(lengths), D ** -0.5)
        assert moe.get_error() == bq.MOE_OK
        check(cache, q, lengths, D ** -0.5, 0.0, 0, out, lse)


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("softcap,window,scale", [(50.0, 0, 0.125), (0.0, 1, 0.125), (0.0, 64, 0.125), (3.0, 100, -0.3),
                                                  (0.0, 1 << 30, 0.0), (0.5, 33, 2.0)])
def test_caps_and_windows(moe, bits8, softcap, window, scale):
    lengths = [0, 1, 50, 64, 99, 100, 101, 517, 1030]
    for H, group, D, page in ((2, 3, 64, 16), (1, 12, 128, 64)):
        cache = Cache(30, lengths, H, D, page, bits8)
        q = queries(31, len(lengths), H * group, D)
        out, lse = run(moe, cache, dev(q), i32(lengths), scale, softcap, window)
        assert moe.get_error() == bq.MOE_OK
        check(cache, q, lengths, scale, softcap, window, out, lse)


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("scale,softcap", [(1e10, 1e-30), (3e38, 0.0), (3e38, 1e-3), (-3e38, 2.0)])
def test_scores_of_zero_at_any_scale(moe, bits8, scale, softcap):
    """Queries of zeros: every score is 0 however large the factors are, the output the mean of the values."""
    cache = Cache(35, [77, 3], 2, 64, 16, bits8)
    q = np.zeros((2, 4, 64))
    out, lse = run(moe, cache, dev(q), i32([77, 3]), scale, softcap)
    assert moe.get_error() == bq.MOE_OK
    check(cache, q, [77, 3], 0.0, 0.0, 0, out, lse)


@pytest.mark.parametrize("bits8", [False, True])
def test_a_long_sequence(moe, bits8):
    """One head's positions go to many blocks, next to sequences of a few."""
    lengths = [70001, 3, 0, 20000]
    cache = Cache(40, lengths, 1, 64, 32, bits8)
    q = queries(41, 4, 4, 64)
    out, lse = run(moe, cache, dev(q), i32(lengths), 0.2)
    assert moe.get_error() == bq.MOE_OK
    check(cache, q, lengths, 0.2, 0.0, 0, out, lse)
    again, _ = run(moe, cache, dev(q), i32(lengths), 0.2)
    assert torch.equal(out, again)  # bit by bit


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("n,H,most,few", [(40, 2, 500, ()), (100, 2, 900, ()), (150, 1, 1500, (0,)), (700, 3, 190, ()),
                                          (700, 3, 120, (6000,)), (60, 4, 60, (1400, 1900)), (300, 1, 40, (1500, 0, 1400)),
                                          (31, 5, 64, (700,)), (152, 1, 1, ()), (153, 1, 33, ())])
def test_how_sequences_share_the_blocks(moe, bits8, n, H, most, few):
    """Items that a block or a warp has whole, beside longer ones that are cut."""
    g = np.random.default_rng(n + most)
    lengths = g.integers(0, most + 1, n)
    for i, L in enumerate(few):
        lengths[(i + 1) * n // (len(few) + 1)] = L
    cache = Cache(45, lengths, H, 64, 16, bits8)
    q = queries(46, n, 2 * H, 64)
    out, lse = run(moe, cache, dev(q), i32(lengths), 0.15)
    assert moe.get_error() == bq.MOE_OK
    check(cache, q, lengths, 0.15, 0.0, 0, out, lse, heads=(0, 2 * H - 1))
    again, _ = run(moe, cache, dev(q), i32(lengths), 0.15)
    assert torch.equal(out, again)


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("n", [1000, 4096])
def test_many_sequences(moe, bits8, n):
    g = np.random.default_rng(n)
    lengths = g.integers(0, 40, n)
    lengths[::7] = 0
    lengths[-1] = 3
    cache = Cache(50, lengths, 2, 16, 16, bits8)
    q = queries(51, n, 2, 16)
    out, lse = run(moe, cache, dev(q), i32(lengths), 0.25)
    assert moe.get_error() == bq.MOE_OK
    check(cache, q, lengths, 0.25, 0.0, 0, out, lse)


@pytest.mark.parametrize("bits8", [False, True])
def test_scores_far_apart(moe, bits8):
    """One position takes everything, first, in the middle or last; equal scores; the running maximum grows."""
    L, D = 400, 64
    for at in (0, 200, 399, None):
        cache = Cache(60, [L], 1, D, 16, bits8)
        q = np.ones((1, 1, D))
        page, row = cache.table[0, np.arange(L) // 16], np.arange(L) % 16
        k = np.ones((L, D)) * (np.linspace(-1, 1, L)[:, None] if at is None else 0.0)
        if at is not None:
            k[at] = 2.0
        if bits8:
            codes, m = KO.quantise(k)
            cache.k[page, 0, row], cache.ks[page, 0, row] = codes, m.astype(np.float32)
        else:
            cache.k[page, 0, row] = bf16(k)
        cache.upload()
        out, lse = run(moe, cache, dev(q), i32([L]), 4.0)
        check(cache, q, [L], 4.0, 0.0, 0, out, lse)


@pytest.mark.parametrize("size", [1e-25, 1e-6, 1e4, 1e12])
def test_scales_of_any_size(moe, size):
    """8-bit values whose rows' scales differ widely; queries far from one."""
    lengths = [333, 20]
    cache = Cache(70, lengths, 2, 64, 16, True)
    g = np.random.default_rng(70)
    cache.vs = (cache.vs * size * np.exp(g.standard_normal(cache.vs.shape) * 3)).astype(np.float32).astype(float)
    cache.ks = (cache.ks / np.float32(size)).astype(np.float32).astype(float)
    cache.upload()
    q = bf16(queries(71, 2, 4, 64) * size)
    out, lse = run(moe, cache, dev(q), i32(lengths), 0.125)
    assert moe.get_error() == bq.MOE_OK
    check(cache, q, lengths, 0.125, 0.0, 0, out, lse)


@pytest.mark.parametrize("bits8", [False, True])
def test_pages_that_are_not_there(moe, bits8):
    """Positions of a page outside the pool are left out and told; a sequence of such pages alone is empty."""
    lengths = [100, 40, 64]
    cache = Cache(80, lengths, 2, 64, 16, bits8)
    cache.table[0, 2], cache.table[0, 6], cache.table[2, :4] = -1, 1 << 20, cache.k.shape[0]
    cache.upload()
    q = queries(81, 3, 4, 64)
    out, lse = run(moe, cache, dev(q), i32(lengths), 0.125)
    assert moe.get_error() == bq.MOE_ERR_BAD_EXPERT_ID
    keep = [np.array([p for p in range(L) if 0 <= cache.table[s, p // 16] < cache.k.shape[0]], int)
            for s, L in enumerate(lengths)]
    got = f64(out)
    for s, pos in enumerate(keep):
        k, v = cache.rows(np.full(len(pos), s), pos)
        for h in range(4):
            want, wl, mean, size = KO.attend(q[s, h], k[:, h // 2], v[:, h // 2], 0.125)
            assert np.all(np.abs(got[s, h] - want) <= mean * (BF16 + 2.0 ** -12) + BF16 * np.abs(want) * 1.01)
    assert not got[2].any() and bool((lse[2] == -np.inf).all())
    # outside a window they do not matter
    out, lse = run(moe, cache, dev(q), i32([92, 40, 0]), 0.125, window=20)
    assert moe.get_error() == bq.MOE_OK


@pytest.mark.parametrize("bits8", [False, True])
def test_lengths_outside_the_table(moe, bits8):
    cache = Cache(90, [64, 64], 1, 32, 16, bits8, room=0)
    q = queries(91, 2, 2, 32)
    out, lse = run(moe, cache, dev(q), i32([1 << 30, -5]), 0.2)
    assert moe.get_error() == bq.MOE_OK
    check(cache, q, [64, 0], 0.2, 0.0, 0, out, lse)


def test_a_nan_that_is_looked_at(moe):
    """It comes out for the heads that look at it, and for no others."""
    for bits8 in (False, True):
        cache = Cache(100, [40, 40], 2, 64, 16, bits8)
        p, r = cache.table[0, 1], 3
        if bits8:
            cache.vs[p, 1, r] = np.nan
        else:
            cache.v[p, 1, r] = np.nan
        cache.upload()
        q = queries(101, 2, 4, 64)
        out, _ = run(moe, cache, dev(q), i32([40, 40]), 0.1)
        got = np.isnan(f64(out))
        assert got[0, 2:].all() and not got[0, :2].any() and not got[1].any()


@pytest.mark.parametrize("bits8", [False, True])
def test_rows_that_lie_apart(moe, bits8):
    """Queries out of a wider projection, outputs into a wider matrix, shared and repeated pages."""
    lengths, H, D = [70, 70, 33], 2, 64
    cache = Cache(110, lengths, H, D, 16, bits8)
    cache.table[1] = cache.table[0]  # the same prefix
    cache.table[2, 1] = cache.table[2, 0]  # one page twice (a ring)
    cache.upload()
    q = queries(111, 3, 6, D)
    wide = torch.full((3, 6 * D + 40), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + 6 * D] = dev(q).reshape(3, -1)
    out = torch.full((3, 6 * D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 6), device="cuda")
    ws = torch.empty(moe.kv_attend_workspace_bytes(cache.c, 6), dtype=torch.uint8, device="cuda")
    moe.kv_attend(wide[:, 16:16 + 6 * D], i32(lengths), cache.c, out[:, :6 * D], ws, scale=0.125, lse=lse)
    assert moe.get_error() == bq.MOE_OK
    check(cache, q, lengths, 0.125, 0.0, 0, out[:, :6 * D], lse)
    assert bool((out[:, 6 * D:] == 7).all())


@pytest.mark.parametrize("bits8", [False, True])
def test_graphs_that_share_a_workspace(moe, bits8):
    """Two captured calls of one handle and workspace, replayed in turn; lengths and pages change in between."""
    shapes = [([600, 50, 0], 1, 8, 128), ([40, 3000], 2, 2, 64)]
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    jobs = []
    for i, (lengths, H, group, D) in enumerate(shapes):
        cache = Cache(120 + i, lengths, H, D, 32, bits8)
        q = queries(121 + i, len(lengths), H * group, D)
        job = dict(cache=cache, q=q, dq=dev(q), n=i32(lengths), lengths=lengths, out=torch.empty_like(dev(q)),
                   lse=torch.empty(q.shape[:2], device="cuda"), g=torch.cuda.CUDAGraph())
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st), torch.cuda.graph(job["g"], stream=st):
            moe.kv_attend(job["dq"], job["n"], cache.c, job["out"], ws, scale=0.1, lse=job["lse"])
        jobs.append(job)
    for turn in range(3):
        for job in jobs:
            lengths = [max(0, n - 17 * turn) for n in job["lengths"]]
            job["n"].copy_(i32(lengths))
            torch.cuda.synchronize()
            job["g"].replay()
            torch.cuda.synchronize()
            assert moe.get_error() == bq.MOE_OK
            check(job["cache"], job["q"], lengths, 0.1, 0.0, 0, job["out"], job["lse"])


@pytest.mark.parametrize("bits8", [False, True])
def test_a_graph_whose_lengths_change(moe, bits8):
    """Replays in which the blocks share the items in another way each time: all empty, short, one long, all long."""
    H, n, most = 2, 90, 1900
    cache = Cache(47, np.full(n, most), H, 64, 16, bits8)
    q = queries(48, n, 2 * H, 64)
    out, lse = torch.empty((n, 2 * H, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((n, 2 * H), device="cuda")
    ws = torch.empty(moe.kv_attend_workspace_bytes(cache.c, 2 * H), dtype=torch.uint8, device="cuda")
    dq, held = dev(q), torch.zeros(n, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            moe.kv_attend(dq, held, cache.c, out, ws, scale=0.15, lse=lse)
    r = np.random.default_rng(49)
    long = r.integers(0, 50, n)
    long[37] = most
    few = np.zeros(n, int)
    few[[3, 80]] = 1700, 40
    for lengths in (np.zeros(n, int), r.integers(0, 65, n), long, few, np.full(n, most), r.integers(0, 400, n), np.zeros(n, int), long):
        out.fill_(7.0)
        lse.fill_(7.0)
        held.copy_(i32(lengths))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        assert moe.get_error() == bq.MOE_OK
        check(cache, q, lengths, 0.15, 0.0, 0, out, lse, heads=(1, 2))


def test_two_handles_on_two_streams():
    """A handle and a workspace each: calls that may run at the same time."""
    bq.build_library()
    jobs = []
    for i in range(2):
        lengths = [900 + 50 * i, 20, 4000]
        cache = Cache(130 + i, lengths, 2, 128, 64, i == 1)
        q = queries(131 + i, 3, 8, 128)
        m = bq.Moe()
        jobs.append((m, cache, q, lengths, dev(q), i32(lengths), torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda"),
                     torch.empty((3, 8), device="cuda"),
                     torch.empty(m.kv_attend_workspace_bytes(cache.c, 8), dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for m, cache, q, lengths, dq, n, out, lse, ws, st in jobs:
            m.kv_attend(dq, n, cache.c, out, ws, scale=0.1, lse=lse, stream=st)
    torch.cuda.synchronize()
    for m, cache, q, lengths, dq, n, out, lse, ws, st in jobs:
        assert m.get_error() == bq.MOE_OK
        check(cache, q, lengths, 0.1, 0.0, 0, out, lse)
        m.close()


def test_pages_past_32_bits_of_bytes(moe):
    H, D, page, n = 8, 256, 256, 4200
    kv = torch.zeros((n, H, page, D), dtype=torch.int8, device="cuda")
    s = torch.zeros((n, H, page), device="cuda")
    g = np.random.default_rng(140)
    k, v = g.standard_normal((2, 256, H, D))
    c = bq.make_kv_cache(kv, kv.clone(), i32([[n - 1]]), s, s.clone())
    moe.kv_append(dev(k), dev(v), i32(np.arange(256)), c, seqs=i32(np.zeros(256)))
    cache = Cache(141, [1], H, D, page, True)
    small = bq.make_kv_cache(*[t[n - 1:] for t in c.keep[:2]], i32([[0]]), *[t[n - 1:] for t in c.keep[2:4]])
    q = queries(142, 1, 2 * H, D)
    outs = []
    for cc in (c, small):  # the same page by another table: the same bits
        cache.c = cc
        outs.append(run(moe, cache, dev(q), i32([250]), 0.06)[0])
    assert moe.get_error() == bq.MOE_OK
    assert torch.equal(*outs) and bool(outs[0].any())
