"""Penalties, biases, grammar masks and the greedy token on a GB300
(moe_logits_process) against the float64 oracle.

Every operation rounds once to fp32, so a processed logit is off by at most
2^-24 times the sum of the magnitudes of its operations' results (the oracle
returns that sum); one without a rule is unchanged.  The token must be the
first index of the largest of the GPU's own results."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from oracle import batch_oracle as BO

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    bq.build_library()
    m = bq.Moe()
    yield m
    m.close()


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def pack(mask):
    T, V = mask.shape
    bits = np.zeros((T, (V + 31) // 32 * 32), dtype=np.uint64)
    bits[:, :V] = mask
    words = (bits.reshape(T, -1, 32) << np.arange(32, dtype=np.uint64)).sum(axis=2)
    return words.astype(np.uint32).view(np.int32)


def make(seed, T, V, L=0, B=0, mask=None, penalties=("repetition", "presence", "frequency"), prompt=True, spread=50):
    """Rules as arrays and as the oracle's rows."""
    rng = np.random.default_rng(seed)
    a, rows = {}, [dict() for _ in range(T)]
    if L:
        few = rng.integers(0, V, (T, spread))
        a["history"] = np.where(rng.random((T, L)) < 0.7, np.take_along_axis(few, rng.integers(0, spread, (T, L)), 1),
                                rng.integers(0, V, (T, L))).astype(np.int32)
        a["history_len"] = rng.integers(0, L + 1, T).astype(np.int32)
        a["history_len"][0] = L
        if prompt:
            a["prompt_len"] = (a["history_len"] * rng.random(T)).astype(np.int32)
        for name, lo, hi in (("repetition", 1.0, 1.5), ("presence", -0.5, 1.0), ("frequency", 0.0, 0.5)):
            if name in penalties:
                a[name] = rng.uniform(lo, hi, T).astype(np.float32)
        for t in range(T):
            rows[t]["history"] = a["history"][t, :a["history_len"][t]].tolist()
            rows[t]["prompt"] = int(a["prompt_len"][t]) if prompt else 0
            for name in penalties:
                rows[t][name] = float(a[name][t])
    if B:
        a["bias_ids"] = rng.integers(0, V, (T, B)).astype(np.int32)
        a["bias_values"] = (5 * rng.standard_normal((T, B))).astype(np.float32)
        a["bias_len"] = rng.integers(0, B + 1, T).astype(np.int32)
        a["bias_len"][-1] = B
        for t in range(T):
            k = a["bias_len"][t]
            rows[t]["bias"] = list(zip(a["bias_ids"][t, :k].tolist(), a["bias_values"][t, :k].astype(float).tolist()))
    m = None
    if mask is not None:
        m = rng.random((T, V)) < mask
        a["mask"] = pack(m)
    return a, rows, m


def run(moe, lg, a, tokens=True, out="own", status=bq.MOE_OK):
    """out: "own" a buffer of its own, "in" in place, "pad" rows further apart, None tokens only."""
    T, V = lg.shape
    d = cuda(lg)
    rules = bq.make_logit_rules(**{k: cuda(v) for k, v in a.items()})
    if out == "in":
        o = d
    elif out == "pad":
        wide = torch.full((T + 1, V + 7), 5.5, device="cuda")
        o = wide[:T, :V]
    else:
        o = None if out is None else torch.full((T, V), 5.5, device="cuda")
    tk = torch.full((T + 1,), -5, dtype=torch.int32, device="cuda") if tokens else None
    moe.logits_process(d, T, V, rules, out=o, tokens=tk)
    torch.cuda.synchronize()
    assert moe.get_error() == status
    if out == "pad":
        assert torch.all(wide[:, V:] == 5.5) and torch.all(wide[T] == 5.5)
    if out != "in":
        assert torch.equal(d.view(torch.int32), cuda(lg).view(torch.int32))
    if tokens:
        assert tk[T] == -5
    return None if o is None else o.cpu().numpy(), tk[:T].cpu().numpy() if tokens else None


def check(lg, got, tk, rows, mask):
    want, mag = BO.logits(lg, rows, mask)
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fine = np.isfinite(want)
    assert np.all(np.abs(got[fine] - want[fine]) <= 2.0 ** -24 * 1.001 * mag[fine])
    untouched = (mag == 0) & fine
    assert np.array_equal(got[untouched], lg[untouched])
    if tk is not None:
        assert np.array_equal(tk, BO.greedy(got))


def logits_of(seed, T, V):
    return (4 * np.random.default_rng(seed).standard_normal((T, V))).astype(np.float32)


@pytest.mark.parametrize("out", ["own", "in", "pad"])
@pytest.mark.parametrize("T,V,L,B,mask", [
    (1, 1, 3, 2, 0.5), (1, 31, 5, 0, None), (3, 33, 40, 7, 0.5), (2, 4096, 300, 0, None), (5, 4097, 0, 9, None),
    (4, 5003, 0, 0, 0.3), (7, 1000, 2000, 1, 0.9), (1, 70001, 500, 300, None), (17, 8192, 100, 40, 0.1),
    (2, 262144, 3000, 300, 0.25), (3, 20000, 0, 0, None), (300, 129, 20, 5, 0.5),
    # blocks that take parts of several rows; lists longer than what stays in registers, at odd strides
    (40, 20000, 60, 12, 0.5), (200, 9001, 33, 0, None), (3, 30000, 5001, 2500, 0.5), (2, 40960, 9000, 1100, None)])
def test_matches_oracle(moe, T, V, L, B, mask, out):
    lg = logits_of(T * V, T, V)
    a, rows, m = make(V + L, T, V, L, B, mask)
    got, tk = run(moe, lg, a, out=out)
    check(lg, got, tk, rows, m)


@pytest.mark.parametrize("penalties", [("repetition",), ("presence",), ("frequency",), ()])
@pytest.mark.parametrize("prompt", [True, False])
def test_single_penalties(moe, penalties, prompt):
    lg = logits_of(3, 4, 3000)
    a, rows, m = make(9, 4, 3000, L=200, penalties=penalties, prompt=prompt)
    got, tk = run(moe, lg, a)
    check(lg, got, tk, rows, m)


def test_tokens_only_and_logits_only(moe):
    lg = logits_of(4, 6, 9000)
    a, rows, m = make(10, 6, 9000, 100, 20, 0.5)
    got, tk = run(moe, lg, a)
    assert np.array_equal(run(moe, lg, a, out=None)[1], tk)
    assert np.array_equal(run(moe, lg, a, tokens=False)[0], got)


def test_counts_are_exact_over_a_long_history(moe):
    """One token over and over, and prompt lengths at and past both ends."""
    V, L = 500, 70000
    a = dict(history=np.full((4, L), 7, np.int32), history_len=np.array([L, L, L, L + 50], np.int32),
             prompt_len=np.array([0, L, L + 5, -3], np.int32), frequency=np.full(4, 0.001, np.float32),
             presence=np.full(4, 0.25, np.float32), repetition=np.full(4, 1.25, np.float32))
    lg = np.ones((4, V), np.float32)
    got, _ = run(moe, lg, a)
    f = np.float32
    pen = f(f(f(1.0) / f(1.25)) - f(f(0.001) * f(L))) - f(0.25)
    assert got[0, 7] == pen and got[3, 7] == pen and got[1, 7] == f(0.8) and got[2, 7] == f(0.8)
    assert np.all(np.delete(got, 7, 1) == 1.0)


@pytest.mark.parametrize("L", [4096, 4097, 4099, 4127, 5000, 8195, 12289, 20003])
@pytest.mark.parametrize("stride", [0, 1])
def test_every_token_of_a_long_history_counts(moe, L, stride):
    """Histories at and past what stays in registers; a vocabulary of one
    segment, so that every token is the segment's, and rows off a boundary."""
    V, T = 777, 3
    rng = np.random.default_rng(L)
    h = rng.integers(0, V, (T, L + stride)).astype(np.int32)
    n = np.array([L, L - 1, max(L - 40, 0)], dtype=np.int32)
    p = np.array([0, 4100, L // 2], dtype=np.int32)
    r = bq.make_logit_rules(history=cuda(h), history_len=cuda(n), prompt_len=cuda(p),
                            frequency=torch.full((T,), 1.0, device="cuda"))
    lg = torch.zeros((T, V), device="cuda")
    out = torch.empty_like(lg)
    moe.logits_process(lg, T, V, r, out=out)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    want = np.stack([-np.bincount(h[t, p[t]:n[t]], minlength=V) for t in range(T)])
    assert np.array_equal(out.cpu().numpy(), want.astype(np.float32))


def test_rows_with_nothing_left(moe):
    lg = logits_of(5, 4, 6000)
    lg[3] = -np.inf
    mask = np.ones((4, 6000), bool)
    mask[1] = False
    a, rows, _ = make(11, 4, 6000, 50)
    a["mask"] = pack(mask)
    got, tk = run(moe, lg, a)
    check(lg, got, tk, rows, mask)
    assert tk[1] == -1 and tk[3] == -1 and np.isneginf(got[1]).all() and tk[0] >= 0


def test_non_finite_logits(moe):
    """Under the mask they are gone; elsewhere they are passed on, skipped and recorded."""
    lg = logits_of(6, 3, 5000)
    lg[:, 10], lg[:, 11], lg[:, 12] = np.nan, np.inf, -np.inf
    mask = np.ones((3, 5000), bool)
    mask[:, 10:12] = False
    got, tk = run(moe, lg, dict(mask=pack(mask)))
    assert np.isneginf(got[:, 10:13]).all() and np.array_equal(tk, BO.greedy(got))
    got, tk = run(moe, lg, {}, status=bq.MOE_ERR_NONFINITE)
    assert np.isnan(got[:, 10]).all() and np.isposinf(got[:, 11]).all() and np.array_equal(tk, BO.greedy(got))
    low = np.full((1, 300), np.finfo(np.float32).min, np.float32)  # the type's lowest value is a value
    assert run(moe, low, {})[1][0] == 0


def test_ties_and_zeros(moe):
    lg = np.full((2, 9000), -1.0, np.float32)
    lg[0, [8999, 4500, 77]] = 2.0
    lg[1, 100:] = 0.0
    lg[1, 100:8000] = -0.0
    assert run(moe, lg, {})[1].tolist() == [77, 100]


def test_ids_outside_the_vocabulary(moe):
    lg = logits_of(7, 2, 700)
    a, rows, _ = make(12, 2, 700, 40, 6)
    a["history"][:, 3], a["history"][:, 5], a["bias_ids"][1, 2] = -1, 700, 1 << 30
    rows[0]["history"], rows[1]["history"] = (a["history"][t, :a["history_len"][t]].tolist() for t in range(2))
    for t in range(2):
        k = a["bias_len"][t]
        rows[t]["bias"] = list(zip(a["bias_ids"][t, :k].tolist(), a["bias_values"][t, :k].astype(float).tolist()))
    got, tk = run(moe, lg, a, status=bq.MOE_ERR_BAD_EXPERT_ID)
    check(lg, got, tk, rows, None)


def test_one_bias_entry_of_a_token_counts(moe):
    V = 5000
    ids = np.zeros((1, 600), np.int32) + 4200
    ids[0, ::3] = 17
    vals = np.arange(600, dtype=np.float32)[None]
    got, tk = run(moe, np.zeros((1, V), np.float32), dict(bias_ids=ids, bias_values=vals, bias_len=np.array([599], np.int32)))
    assert got[0, 4200] == 598.0 and got[0, 17] == 597.0 and got[0].sum() == 1195.0 and tk[0] == 4200


def test_one_mask_for_every_row(moe):
    lg = logits_of(8, 5, 4100)
    m = np.random.default_rng(1).random((1, 4100)) < 0.2
    got, tk = run(moe, lg, dict(mask=pack(m)[0]))
    check(lg, got, tk, [{}] * 5, np.repeat(m, 5, 0))


def test_views_that_start_off_a_boundary(moe):
    """Rows whose starts lie at every offset from a 16-byte boundary."""
    V = 4103
    big = cuda(logits_of(9, 4, V + 3))
    want, tk = run(moe, big[:, 1:V + 1].cpu().numpy(), {})
    src = big[:, 1:V + 1]
    for off in range(4):
        wide = torch.full((4, V + 9), 3.25, device="cuda")
        dst = wide[:, off:V + off]
        t = torch.empty(4, dtype=torch.int32, device="cuda")
        moe.logits_process(src, 4, V, bq.make_logit_rules(), out=dst, tokens=t)
        torch.cuda.synchronize()
        assert moe.get_error() == bq.MOE_OK
        assert np.array_equal(dst.cpu().numpy(), want) and np.array_equal(t.cpu().numpy(), tk)
        assert torch.all(wide[:, :off] == 3.25) and torch.all(wide[:, V + off:] == 3.25)


def test_captured_histories_that_grow(moe):
    """A captured call reads the history that stands in its buffers when it is replayed."""
    T, V, L = 3, 6000, 64
    a, _, _ = make(13, T, V, L, 8, 0.5)
    d = {k: cuda(v) for k, v in a.items()}
    lg = logits_of(14, T, V)
    x, out, tk = cuda(lg), torch.empty((T, V), device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
    rules = bq.make_logit_rules(**d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            moe.logits_process(x, T, V, rules, out=out, tokens=tk, stream=st)
        for n in (1, 40, L):
            d["history_len"].fill_(n)
            d["prompt_len"].fill_(n // 3)
            g.replay()
            a["history_len"][:], a["prompt_len"][:] = n, n // 3
            st.synchronize()
            want, wtk = run(moe, lg, a)
            assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(tk.cpu().numpy(), wtk)


def test_many_rows(moe):
    T, V = 4096, 300
    lg = logits_of(15, T, V)
    a, rows, m = make(16, T, V, 12, 3, 0.4, spread=5)
    got, tk = run(moe, lg, a)
    check(lg, got, tk, rows, m)


def test_offsets_beyond_32_bits(moe):
    """A row of logits that starts more than 2^32 bytes into its matrix."""
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    V, ld = 2000, (1 << 30) + 5
    buf = torch.empty(2 * ld, device="cuda")  # 8 GB, the second row past 4 GB
    lg = logits_of(17, 2, V)
    view = buf.as_strided((2, V), (ld, 1))
    view.copy_(torch.from_numpy(lg))
    tk = torch.empty(2, dtype=torch.int32, device="cuda")
    moe.logits_process(view, 2, V, bq.make_logit_rules(), out=view, tokens=tk)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    assert np.array_equal(view.cpu().numpy(), lg) and np.array_equal(tk.cpu().numpy(), BO.greedy(lg))


def test_binding_refuses(moe):
    lg = torch.zeros((2, 100), device="cuda")
    for bad in (dict(rows=3), dict(vocab=101), dict(lg=lg.t()), dict(lg=lg.half()), dict(out=lg[:, :50])):
        a = dict(lg=lg, rows=2, vocab=100, out=lg)
        a.update(bad)
        with pytest.raises(ValueError):
            moe.logits_process(a["lg"], a["rows"], a["vocab"], bq.make_logit_rules(), out=a["out"])
    short = bq.make_logit_rules(mask=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        moe.logits_process(lg, 2, 100, short, out=lg)
    one = bq.make_logit_rules(history=torch.zeros((1, 4), dtype=torch.int32, device="cuda"),
                              history_len=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        moe.logits_process(lg, 2, 100, one, out=lg)
