"""Residual addition, root-mean-square norm and 8-bit rows on a GB300
(moe_norm_quant) against the float64 oracle.

The stored sum and the codes must be equal: both are the roundings of exact
values (csrc/norm_quant.cu gives the argument for the codes).  The scale
m r / 127 takes, in units of 2^-24 relative to its value: the sum of squares
at most 16 products of a thread and 10 shuffle steps (26 roundings, halved by
the square root: 13), the mean, + eps, square root, reciprocal, times m, over
127 (6 more): 19, so 20 * 2^-24.  The bf16 rows add half a bf16 step, 2^-8."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from oracle import batch_oracle as BO
from oracle.batch_oracle import to_bf16
from synth import gen

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

F32 = 2.0 ** -24
REL = 20 * F32


@pytest.fixture(scope="module")
def moe():
    bq.build_library()
    m = bq.Moe()
    yield m
    m.close()


def dev16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()


def host16(t):
    return t.cpu().numpy().view(np.uint16)


def rows(seed, T, H, scale=1.0):
    rng = np.random.default_rng(seed)
    return to_bf16(rng.standard_normal((T, H)) * np.exp(rng.standard_normal((T, 1))) * scale)


def run(moe, h, y=None, g=None, eps=1e-6, x_out=True, in_place=False, status=bq.MOE_OK, stream=None):
    T, H = h.shape
    hd, yd, gd = dev16(h), None if y is None else dev16(y), None if g is None else dev16(g)
    out = hd if in_place else (torch.empty_like(hd) if y is not None else None)
    q = torch.full((T, H), 99, dtype=torch.int8, device="cuda")
    s = torch.full((T,), -7.0, device="cuda")
    x = torch.empty_like(hd) if x_out else None
    moe.norm_quant(hd, T, q, s, y=yd, norm=gd, eps=eps, hidden_out=out, x_out=x, stream=stream)
    torch.cuda.synchronize()
    assert moe.get_error() == status
    return {"s": None if out is None else host16(out), "q": q.cpu().numpy(), "scales": s.cpu().numpy().astype(np.float64),
            "x": host16(x) if x_out else None, "h": host16(hd)}


def check(got, want):
    if got["s"] is not None:
        assert np.array_equal(got["s"], want["s"])
    assert np.array_equal(got["q"], want["q"])
    assert np.array_equal(np.isnan(got["scales"]), np.isnan(want["scales"]))
    fine = ~np.isnan(want["scales"])
    assert np.all(np.abs(got["scales"] - want["scales"])[fine] <= REL * want["scales"][fine])
    if got["x"] is not None:
        x, w = gen.bf16_bits_to_f64(got["x"])[fine], want["x"][fine]
        assert np.all(np.abs(x - w) <= (2.0 ** -8 + REL) * np.abs(w) + 2.0 ** -133)


@pytest.mark.parametrize("T,H", [(600, 16384), (460, 8208), (500, 48), (1, 16), (3, 48), (1, 2816), (130, 2816), (5, 1360), (2, 8192), (3, 8208), (2, 16384),
                                 (700, 64)])
@pytest.mark.parametrize("add,weight", [(True, True), (True, False), (False, True), (False, False)])
def test_matches_oracle(moe, T, H, add, weight):
    h = rows(T * H, T, H)
    y = rows(T * H + 1, T, H) if add else None
    g = to_bf16(np.random.default_rng(5).uniform(0.5, 1.5, H)) if weight else None
    check(run(moe, h, y, g), BO.norm_quant(h, y, g))


def test_codes_without_rows16_and_in_place(moe):
    h, y = rows(1, 9, 704), rows(2, 9, 704)
    want = BO.norm_quant(h, y)
    got = run(moe, h, y, x_out=False, in_place=True)
    check(got, want)
    assert np.array_equal(got["h"], want["s"])
    # the sum is not wanted: the input stays as it was
    hd, yd = dev16(h), dev16(y)
    q, s = torch.empty((9, 704), dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda")
    moe.norm_quant(hd, 9, q, s, y=yd)
    torch.cuda.synchronize()
    assert np.array_equal(host16(hd), h) and np.array_equal(q.cpu().numpy(), want["q"])


def test_ties_go_to_even(moe):
    """Rows whose quotients 127 u / m are half integers, m = 254: u odd."""
    u = np.zeros((1, 256))
    u[0, :255] = np.arange(-127, 128)
    u[0, 255] = 254
    h = to_bf16(u)
    check(run(moe, h), BO.norm_quant(h))


@pytest.mark.parametrize("scale", [2.0 ** -70, 2.0 ** -50, 2.0 ** 50, 2.0 ** 55])
def test_far_ranges(moe, scale):
    """Rows far from 1: the codes do not depend on a power of two; with eps = 0
    the normalised rows do not either."""
    h = rows(3, 4, 512, 1.0)
    small = to_bf16(gen.bf16_bits_to_f64(h) * scale)
    a = BO.norm_quant(small, eps=0.0)
    got = run(moe, small, eps=1e-6, x_out=False)
    assert np.array_equal(got["q"], a["q"])
    check(got, BO.norm_quant(small, eps=float(np.float32(1e-6))))


@pytest.mark.parametrize("top", [-100, -120, -125, -130])
def test_smallest_rows(moe, top):
    """Largest values of 2^top, down to bf16's subnormal numbers (steps of 2^-133)."""
    rng = np.random.default_rng(-top)
    step = max(2.0 ** (top - 7), 2.0 ** -133)
    v = rng.integers(-round(2.0 ** top / step), round(2.0 ** top / step) + 1, (3, 320)) * step
    v[:, 0] = 2.0 ** top
    bits = to_bf16(v)
    got, want = run(moe, bits, x_out=False), BO.norm_quant(bits, eps=float(np.float32(1e-6)))
    assert np.array_equal(got["q"], want["q"])
    # m r / 127 in fp32, a step of 2^-149 where it is subnormal
    assert np.all(np.abs(got["scales"] - want["scales"]) <= REL * want["scales"] + 2.0 ** -149)


def test_eps_zero(moe):
    """Rows of zeros stay zeros; rows whose squares leave fp32's range are told."""
    h = rows(8, 3, 320)
    h[1] = 0
    got, want = run(moe, h, eps=0.0, x_out=True), BO.norm_quant(h[[0, 2]], eps=0.0)
    assert got["scales"][1] == 0.0 and not got["q"][1].any() and not got["x"][1].any()
    check({k: (v[[0, 2]] if v is not None else None) for k, v in got.items()}, want)
    small = to_bf16(np.full((1, 64), 2.0 ** -90))
    got = run(moe, small, eps=0.0, x_out=False, status=bq.MOE_ERR_NONFINITE)
    assert np.isnan(got["scales"]).all() and not got["q"].any()


def test_zero_rows(moe):
    h = rows(4, 5, 320)
    h[2] = 0
    got = run(moe, h)
    check(got, BO.norm_quant(h))
    assert got["scales"][2] == 0.0 and not got["q"][2].any() and not got["x"][2].any()


def test_weight_of_zeros(moe):
    h = rows(4, 2, 320)
    check(run(moe, h, g=np.zeros(320, np.uint16)), BO.norm_quant(h, g_bits=np.zeros(320, np.uint16)))


@pytest.mark.parametrize("where", [0, 17, 319])
@pytest.mark.parametrize("value", [0x7F80, 0xFF80, 0x7FC0])
def test_non_finite_rows(moe, where, value):
    h, y = rows(6, 4, 320), rows(7, 4, 320)
    h[1, where] = value
    want = BO.norm_quant(h, y)
    got = run(moe, h, y, status=bq.MOE_ERR_NONFINITE)
    fine = [0, 2, 3]
    assert np.array_equal(got["s"][fine], want["s"][fine]) and np.array_equal(got["q"], want["q"])
    assert np.isnan(got["scales"][1]) and np.isnan(gen.bf16_bits_to_f64(got["x"][1])).all()
    assert np.isfinite(got["scales"][fine]).all()


def test_sum_of_squares_out_of_range(moe):
    h = to_bf16(np.full((2, 64), 2.0 ** 66))
    h[1] = to_bf16(np.ones(64))
    got = run(moe, h, status=bq.MOE_ERR_NONFINITE)
    assert np.isnan(got["scales"][0]) and not got["q"][0].any() and got["q"][1].tolist() == [127] * 64


def test_rows_behind_the_last_stay(moe):
    h = rows(8, 4, 160)
    q = torch.full((4, 160), 55, dtype=torch.int8, device="cuda")
    s = torch.full((4,), 3.5, device="cuda")
    moe.norm_quant(dev16(h), 2, q, s)
    torch.cuda.synchronize()
    assert torch.all(q[2:] == 55) and torch.all(s[2:] == 3.5)
    assert np.array_equal(q[:2].cpu().numpy(), BO.norm_quant(h[:2])["q"])


def test_captured_and_on_another_stream(moe):
    h, y = rows(9, 6, 2816), rows(10, 6, 2816)
    want = BO.norm_quant(h, y)
    hd, yd = dev16(np.zeros_like(h)), dev16(np.zeros_like(h))
    out, q, s = torch.empty_like(hd), torch.empty((6, 2816), dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            moe.norm_quant(hd, 6, q, s, y=yd, hidden_out=out, stream=st)
        hd.copy_(dev16(h))
        yd.copy_(dev16(y))
        g.replay()
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    assert np.array_equal(q.cpu().numpy(), want["q"]) and np.array_equal(host16(out), want["s"])


def test_rows_beyond_32_bits(moe):
    """A matrix with more than 2^31 values."""
    T, H = 270000, 8192
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    h = torch.zeros((T, H), dtype=torch.int16, device="cuda")
    some = rows(50, 3, H)
    at = [0, 140000, T - 1]
    for i, t in enumerate(at):
        h[t] = torch.from_numpy(some[i].view(np.int16)).cuda()
    q, s = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.norm_quant(h, T, q, s)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    want = BO.norm_quant(some)
    assert np.array_equal(q[at].cpu().numpy(), want["q"])
    assert np.all(np.abs(s[at].cpu().numpy() - want["scales"]) <= REL * want["scales"])
    assert int((s != 0).sum()) == 3 and int(q.count_nonzero()) == int(np.count_nonzero(want["q"]))


def test_binding_refuses(moe):
    h = dev16(rows(1, 4, 64))
    q, s = torch.empty((4, 64), dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    for bad in (dict(hidden=h[:2]), dict(hidden=h.float()), dict(hidden=h.t()), dict(q=q.float()), dict(scales=s[:3]),
                dict(y=h[:1]), dict(norm=h[0, :32]), dict(hidden=h.cpu())):
        a = dict(hidden=h, q=q, scales=s, y=None, norm=None)
        a.update(bad)
        with pytest.raises(ValueError):
            moe.norm_quant(a["hidden"], 4, a["q"], a["scales"], y=a["y"], norm=a["norm"])
    with pytest.raises(bq.MoeError):
        moe.norm_quant(h, 4, q, s, hidden_out=h)  # no y
