"""The dense 8-bit projection on a GB300 (moe_qdense_forward) against the exact
integer product.

Where sum |x||w| stays below 2^24 every partial sum is an integer that fp32
holds, so whatever the order the product is exact and what is left are three
roundings (the sum to fp32, times x_scale, times w_scale): 3 * 2^-24 of the
value.  Beyond that the tensor cores' fp32 accumulators may lose up to 2^-23
of the largest partial sum for each of the K / 16 additions.  Up to 8 rows the
sums are integers throughout.  A bf16 output adds 2^-8, a softcap a relative
4 * 2^-24 of its two divisions and products and tanhf's own error (2 ulp)."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from oracle import batch_oracle as BO
from synth import gen

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

F32 = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    bq.build_library()
    m = bq.Moe()
    yield m
    m.close()


def codes(seed, T, K, kind="bell"):
    rng = np.random.default_rng(seed)
    if kind == "bell":
        return np.clip(np.rint(rng.standard_normal((T, K)) * 30), -127, 127).astype(np.int8)
    if kind == "full":
        return rng.integers(-128, 128, (T, K)).astype(np.int8)
    return np.full((T, K), {"max": 127, "min": -128}[kind], dtype=np.int8)


def bound(x, w, xs, ws):
    """Absolute error allowed for the fp32 output without a softcap."""
    T, K = x.shape
    scale = np.abs(np.asarray(xs, np.float64))[:, None] * np.abs(np.asarray(ws, np.float64))[None, :]
    exact = BO.int_product(x, w)
    most = BO.int_product(np.abs(x.astype(np.int16)), np.abs(w.astype(np.int16)))
    lost = np.where((most < 2 ** 24) | (T <= 8), 0.0, (K / 16) * 2.0 ** -23 * most)
    return (lost + 3 * F32 * np.abs(exact)) * scale * (1 + 2.0 ** -20)


def run(moe, x, xs, w, ws, softcap=0.0, y=True, y32=True):
    T, N = x.shape[0], w.shape[0]
    wd = bq.make_qdense_weights(N, w.shape[1], torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    n = moe.qdense_workspace_bytes(wd, T)
    work = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    # one row more than asked for: it has to stay as it is
    a = torch.full((T + 1, N), 1234, dtype=torch.int16, device="cuda") if y else None
    b = torch.full((T + 1, N), 77.0, device="cuda") if y32 else None
    moe.qdense_forward(torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), T, wd, work, y=a, y32=b, softcap=softcap)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    assert a is None or torch.all(a[T] == 1234)
    assert b is None or torch.all(b[T] == 77.0)
    return (None if a is None else a[:T].cpu().numpy().view(np.uint16), None if b is None else b[:T].cpu().numpy())


def scales(seed, T, N):
    rng = np.random.default_rng(seed)
    return (rng.uniform(0.005, 0.02, T).astype(np.float32), rng.uniform(0.0005, 0.002, N).astype(np.float32))


SHAPES = [(1, 1, 16), (1, 2816, 2816), (1, 4097, 208), (2, 33, 64), (3, 130, 1072), (5, 700, 16384), (8, 515, 704),
          (9, 1, 16), (9, 128, 64), (16, 129, 80), (17, 2816, 704), (24, 1411, 2816), (64, 300, 4096), (100, 127, 1072),
          (128, 2816, 4096), (129, 257, 128), (255, 64, 2816), (257, 512, 704), (333, 1411, 1072), (1000, 384, 256),
          (2049, 130, 48), (40, 40000, 64),
          # more tiles than SMs: the last round in halves of tiles (one of them past the last row)
          (512, 10240, 144), (520, 7000, 64), (4112, 1280, 64), (4097, 1290, 80),
          # one tile or part per block, with more stages of K than a block holds at once
          # pairs of blocks on tiles of up to 128 rows, the second block's channels not there in the last
          (48, 20000, 1600), (70, 19600, 1168), (128, 9900, 704), (333, 3900, 784), (1000, 1300, 1040),
          (20, 300, 16), (128, 1, 48), (16, 8200, 4096), (24, 12800, 2832), (9, 5000, 80), (96, 1300, 1936), (64, 19400, 2176),
          # tiles shared by clusters of every size; K that ends inside a stage and inside its first half
          (40, 128, 2816), (150, 128, 1040), (100, 1408, 2832), (64, 2816, 1120), (200, 704, 4112), (33, 5632, 528)]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_matches_exact_product(moe, T, N, K):
    x, w = codes(T, T, K), codes(N + 1, N, K)
    xs, ws = scales(K, T, N)
    y16, y32 = run(moe, x, xs, w, ws)
    want = BO.qdense(x, xs, w, ws)
    err = np.abs(y32.astype(np.float64) - want)
    assert np.all(err <= bound(x, w, xs, ws)), f"worst {np.max(err - bound(x, w, xs, ws))}"
    assert np.array_equal(y16, gen.to_bf16_bits(y32.astype(np.float64)))


@pytest.mark.parametrize("T", [1, 8, 9, 70, 300])
@pytest.mark.parametrize("xk,wk", [("full", "full"), ("max", "min"), ("min", "min"), ("min", "max")])
def test_largest_codes(moe, T, xk, wk):
    """Every code at its limit, sums far beyond 2^24."""
    N, K = 140, 4096
    x, w = codes(1, T, K, xk), codes(2, N, K, wk)
    xs, ws = scales(3, T, N)
    _, y32 = run(moe, x, xs, w, ws, y=False)
    assert np.all(np.abs(y32 - BO.qdense(x, xs, w, ws)) <= bound(x, w, xs, ws))


@pytest.mark.parametrize("T,N,K", [(1, 1000, 704), (6, 77, 2816), (24, 4096, 704), (200, 300, 704)])
def test_softcap(moe, T, N, K):
    x, w = codes(5, T, K), codes(6, N, K)
    xs, ws = scales(7, T, N)
    xs = xs * np.float32(40.0)
    y16, y32 = run(moe, x, xs, w, ws, softcap=30.0)
    want = BO.qdense(x, xs, w, ws, 30.0)
    assert np.abs(want).max() > 20
    assert np.all(np.abs(y32 - want) <= bound(x, w, xs, ws) + 12 * F32 * np.abs(want))
    assert np.array_equal(y16, gen.to_bf16_bits(y32.astype(np.float64)))


@pytest.mark.parametrize("T", [4, 60])
def test_each_output_alone(moe, T):
    x, w = codes(8, T, 704), codes(9, 200, 704)
    xs, ws = scales(10, T, 200)
    y16, y32 = run(moe, x, xs, w, ws)
    assert np.array_equal(run(moe, x, xs, w, ws, y=False)[1], y32)
    assert np.array_equal(run(moe, x, xs, w, ws, y32=False)[0], y16)


@pytest.mark.parametrize("T", [4, 60])
def test_nan_and_zero_scales(moe, T):
    """A NaN row scale (a row that norm_quant gave up) makes its row NaN and no other."""
    x, w = codes(8, T, 64), codes(9, 50, 64)
    x[1] = 0
    xs, ws = scales(10, T, 50)
    xs[1], xs[2] = np.nan, 0.0
    _, y32 = run(moe, x, xs, w, ws, y=False)
    assert np.isnan(y32[1]).all() and not y32[2].any() and np.isfinite(np.delete(y32, 1, 0)).all()


@pytest.mark.parametrize("T,N,K", [(1, 4096, 2816), (24, 5000, 704), (300, 1411, 1072)])
def test_repeated_calls_are_bit_identical(moe, T, N, K):
    x, w = codes(11, T, K, "full"), codes(12, N, K, "full")
    xs, ws = scales(13, T, N)
    first = run(moe, x, xs, w, ws, y=False)[1]
    for _ in range(4):
        assert np.array_equal(run(moe, x, xs, w, ws, y=False)[1], first)


@pytest.mark.parametrize("T", [3, 40])
def test_captured_and_replayed(moe, T):
    N, K = 900, 704
    w = codes(14, N, K)
    xs, ws = scales(15, T, N)
    wd = bq.make_qdense_weights(N, K, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    work = torch.empty(moe.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
    xd, xsd = torch.zeros((T, K), dtype=torch.int8, device="cuda"), torch.from_numpy(xs).cuda()
    outs = [torch.empty((T, N), device="cuda") for _ in range(2)]
    moe.qdense_forward(xd, xsd, T, wd, work, y32=outs[0])  # attributes are set before the capture
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graphs = []
        for o in outs:  # two graphs that share one workspace, replayed in turn
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                moe.qdense_forward(xd, xsd, T, wd, work, y32=o, stream=st)
            graphs.append(g)
        got = []
        for seed in (16, 17):
            x = codes(seed, T, K)
            xd.copy_(torch.from_numpy(x))
            for g in graphs:
                g.replay()
            got.append((x, [o.clone() for o in outs]))
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    for x, both in got:
        for o in both:
            assert np.all(np.abs(o.cpu().numpy() - BO.qdense(x, xs, w, ws)) <= bound(x, w, xs, ws))


@pytest.mark.parametrize("T", [1, 5, 16, 40, 128, 150, 300, 700])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_outputs_off_a_boundary(moe, T, off):
    """Outputs and scales that start off a 16-byte boundary, the values around them left alone."""
    N, K = 1412, 1040
    x, w = codes(60, T, K), codes(61, N, K)
    xs, ws = scales(62, T, N)
    shift = lambda v: torch.cat([torch.zeros(off, device="cuda"), torch.from_numpy(v).cuda()])[off:]
    wd = bq.make_qdense_weights(N, K, torch.from_numpy(w).cuda(), shift(ws))
    work = torch.empty(moe.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
    a = torch.full((T * N + 8,), 1234, dtype=torch.int16, device="cuda")
    b = torch.full((T * N + 8,), 1234.0, device="cuda")
    moe.qdense_forward(torch.from_numpy(x).cuda(), shift(xs), T, wd, work, y=a[off:off + T * N], y32=b[off:off + T * N])
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    z, lim = BO.qdense(x, xs, w, ws), bound(x, w, xs, ws)
    got = b.cpu().numpy()
    assert np.all(np.abs(got[off:off + T * N].reshape(T, N) - z) <= lim)
    bits = a.cpu().numpy().view(np.uint16)
    y16 = (bits[off:off + T * N].astype(np.uint32) << 16).view(np.float32).reshape(T, N)
    assert np.all(np.abs(y16 - z) <= lim + 2.0 ** -8 * (np.abs(z) + lim))
    for v in (got, a.cpu().numpy()):
        assert np.all(v[:off] == 1234) and np.all(v[off + T * N:] == 1234)


@pytest.mark.parametrize("T,N,K", [(2, 3000, 2816), (7, 3000, 2816), (16, 8200, 4096), (24, 12800, 2832),
                                   (90, 2816, 2816), (333, 700, 2816), (30, 20000, 704), (300, 5000, 704)])
def test_the_same_on_every_call(moe, T, N, K):
    """Sums are added in a fixed order: every call gives the same bits."""
    x, w = codes(50, T, K), codes(51, N, K)
    xs, ws = scales(52, T, N)
    wd = bq.make_qdense_weights(N, K, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    work = torch.empty(moe.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
    xd, xsd = torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda()
    y = torch.empty((T, N), device="cuda")
    moe.qdense_forward(xd, xsd, T, wd, work, y32=y)
    first, same = y.clone(), torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(100):
        y.zero_()
        for _ in range(3):
            moe.qdense_forward(xd, xsd, T, wd, work, y32=y)
        same &= (y == first).all()
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK and bool(same)
    some = np.unique(np.linspace(0, N - 1, 400).astype(int))
    assert np.all(np.abs(first.cpu().numpy()[:, some] - BO.qdense(x, xs, w[some], ws[some]))
                  <= bound(x, w[some], xs, ws[some]))


@pytest.mark.parametrize("T", [1, 5, 12])
def test_weights_beyond_32_bits(moe, T):
    """A matrix whose last rows start more than 2^31 bytes into it."""
    N, K = 140000, 16384
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    w = torch.randint(-40, 41, (N, K), generator=g, device="cuda", dtype=torch.int8)
    x = codes(30, T, K)
    xs, _ = scales(31, T, 1)
    ws = torch.full((N,), 0.001, device="cuda")
    wd = bq.make_qdense_weights(N, K, w, ws)
    work = torch.empty(moe.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
    y = torch.empty((T, N), device="cuda")
    moe.qdense_forward(torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), T, wd, work, y32=y)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    for a in (0, 70000, N - 300):
        part = w[a:a + 300].cpu().numpy()
        s = np.full(300, np.float32(0.001))
        assert np.all(np.abs(y[:, a:a + 300].cpu().numpy() - BO.qdense(x, xs, part, s)) <= bound(x, part, xs, s))


def test_outputs_beyond_32_bits(moe):
    """An output with more than 2^31 values."""
    T, N, K = 2100, 1050000, 16
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    x, w = codes(32, T, K), codes(33, N, K)
    xs, ws = scales(34, T, N)
    wd = bq.make_qdense_weights(N, K, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    work = torch.empty(moe.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
    y = torch.empty((T, N), device="cuda")
    moe.qdense_forward(torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), T, wd, work, y32=y)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    for t in (0, 1024, T - 1):
        got = y[t].cpu().numpy()[None]
        assert np.all(np.abs(got - BO.qdense(x[t:t + 1], xs[t:t + 1], w, ws)) <= bound(x[t:t + 1], w, xs[t:t + 1], ws))


def test_two_handles_at_once(moe):
    """Calls of two handles on two streams, each with its own workspace."""
    N, K = 3000, 704
    w = codes(40, N, K)
    other = bq.Moe()
    jobs = []
    for i, (m, T) in enumerate(((moe, 40), (other, 300))):
        x = codes(41 + i, T, K)
        xs, ws = scales(43 + i, T, N)
        wd = bq.make_qdense_weights(N, K, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
        work = torch.empty(m.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
        jobs.append((m, torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), T, wd, work,
                     torch.empty((T, N), device="cuda"), torch.cuda.Stream(), x, xs, ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for m, xd, xsd, T, wd, work, y, st, *_ in jobs:
            m.qdense_forward(xd, xsd, T, wd, work, y32=y, stream=st)
    torch.cuda.synchronize()
    for m, _, _, T, _, _, y, _, x, xs, ws in jobs:
        assert m.get_error() == bq.MOE_OK
        assert np.all(np.abs(y.cpu().numpy() - BO.qdense(x, xs, w, ws)) <= bound(x, w, xs, ws))
    other.close()


def test_binding_refuses(moe):
    x, w = torch.zeros((20, 64), dtype=torch.int8, device="cuda"), torch.zeros((8, 64), dtype=torch.int8, device="cuda")
    s = torch.ones(20, device="cuda")
    wd = bq.make_qdense_weights(8, 64, w, s[:8])
    ws = torch.empty(moe.qdense_workspace_bytes(wd, 20), dtype=torch.uint8, device="cuda")
    y = torch.empty((20, 8), device="cuda")
    for bad in (dict(x=x[:19]), dict(x=x.float()), dict(s=s[:3]), dict(y=y[:19]), dict(y=y.half())):
        a = dict(x=x, s=s, y=y)
        a.update(bad)
        with pytest.raises(ValueError):
            moe.qdense_forward(a["x"], a["s"], 20, wd, ws, y32=a["y"])
    with pytest.raises(ValueError):
        bq.make_qdense_weights(9, 64, w, s)
    if ws.numel():
        with pytest.raises(bq.MoeError):
            moe.qdense_forward(x, s, 20, wd, None, y32=y)
        with pytest.raises(bq.MoeError):
            moe.qdense_forward(x, s, 20, wd, ws[:256], y32=y)
