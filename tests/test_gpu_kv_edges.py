"""Calls of the cache and the sampling that their documentation allows at the ends
of their ranges: the most rows and heads, one handle on two streams, the launch
trace, rows behind the last."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from kv_cases import Cache, bf16, dev, f64, i32
from oracle import kv_oracle as KO
from test_gpu_batch_trace import in_order, stamps
from test_gpu_kv_attend import check as check_attend
from test_gpu_kv_cache import error, freqs, near
from test_gpu_sample import check as check_sample

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    bq.build_library()
    m = bq.Moe()
    yield m
    m.close()


def test_most_rows(moe):
    """2^20 rows of one sequence, appended and read back."""
    T, D, page = 1 << 20, 16, 256
    g = np.random.default_rng(1)
    v = torch.from_numpy(g.integers(-127, 128, (T, 1, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    v[:, 0, 0] = 127.0  # (a row's largest magnitude: the codes are the values)
    kv = torch.zeros((T // page, 1, page, D), dtype=torch.int8, device="cuda")
    s = torch.zeros((T // page, 1, page), device="cuda")
    c = bq.make_kv_cache(kv, kv.clone(), i32(np.arange(T // page)[None]), s, s.clone())
    pos, seq = torch.arange(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    moe.kv_append(v, v, pos, c, seqs=seq)
    out = torch.empty_like(v)
    moe.kv_read(c, pos, v_out=out, seqs=seq)
    assert error(moe) == bq.MOE_OK
    assert torch.equal(out, v) and torch.equal(kv.flatten(0, 2), v[:, 0].to(torch.int8))
    assert bool((s == 1.0).all())


@pytest.mark.parametrize("bits8", [False, True])
def test_most_heads(moe, bits8):
    """128 key heads of 256, eight queries to each."""
    lengths, H, D = [33, 5], 128, 256
    cache = Cache(2, lengths, H, D, 32, bits8)
    g = np.random.default_rng(2)
    x = bf16(g.standard_normal((2, (1024 + 2 * H) * D)))
    d = dev(x)
    q_out = torch.empty((2, 1024, D), dtype=torch.bfloat16, device="cuda")
    f = freqs(D)
    moe.kv_append(d[:, 1024 * D:(1024 + H) * D], d[:, (1024 + H) * D:], i32(lengths), cache.c, q=d[:, :1024 * D],
                  q_out=q_out, inv_freq=dev(f, torch.float32))
    assert error(moe) == bq.MOE_OK
    q = x[:, :1024 * D].reshape(2, 1024, D)
    assert near(f64(q_out), KO.rotate(q, lengths, f), q, D)
    cache.k, cache.v = f64(cache.dk), f64(cache.dv)
    if bits8:
        cache.ks, cache.vs = f64(cache.dks), f64(cache.dvs)
    out, lse = torch.empty_like(q_out), torch.empty((2, 1024), device="cuda")
    ws = torch.empty(moe.kv_attend_workspace_bytes(cache.c, 1024), dtype=torch.uint8, device="cuda")
    after = np.array(lengths) + 1
    moe.kv_attend(q_out, i32(after), cache.c, out, ws, scale=1 / 16, lse=lse)
    assert error(moe) == bq.MOE_OK
    check_attend(cache, f64(q_out), after, 1 / 16, 0.0, 0, out, lse, heads=range(0, 1024, 37))


def test_rows_between_padding_of_a_batch(moe):
    """A padded batch: rows that are left out between others, many rows to a block."""
    T, H, D = 3000, 1, 16
    g = np.random.default_rng(3)
    pos = np.where(np.arange(T) % 3 == 1, -1, np.arange(T))
    cache = Cache(3, [T], H, D, 16, False)
    before = f64(cache.dk)
    k = bf16(g.standard_normal((T, H, D)))
    out = torch.full((T, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    q = bf16(g.standard_normal((T, 2, D)))
    moe.kv_append(dev(k), dev(k), i32(pos), cache.c, seqs=i32(np.zeros(T)), q=dev(q), q_out=out)
    assert error(moe) == bq.MOE_OK
    on, at = pos >= 0, np.arange(T)
    want = before.copy()
    want[cache.table[0, at[on] // 16], :, at[on] % 16] = k[on]
    assert np.array_equal(f64(cache.dk), want, equal_nan=True)
    assert np.array_equal(f64(out)[on], q[on]) and np.all(f64(out)[~on] == 7)
    ko = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.kv_read(cache.c, i32(pos), ko, seqs=i32(np.zeros(T)))
    assert error(moe) == bq.MOE_OK
    assert np.array_equal(f64(ko)[on], k[on]) and np.all(f64(ko)[~on] == 7)


def test_one_handle_on_two_streams(moe):
    """Appends, reads and samples of one handle may run at the same time: they keep nothing in it but errors."""
    g = np.random.default_rng(4)
    T, V, H, D = 20, 70000, 4, 128
    jobs = []
    for i in range(2):
        cache = Cache(4 + i, [50] * T, H, D, 16, True)
        k = bf16(g.standard_normal((T, H, D)))
        x = g.standard_normal((T, V)) * 3
        u, p = g.random(T), g.uniform(0.6, 0.99, T)
        lg = torch.from_numpy(x.astype(np.float32)).cuda()
        rules = bq.make_sample_rules(*[torch.from_numpy(a.astype(np.float32)).cuda() for a in (u,)],
                                     top_p=torch.from_numpy(p.astype(np.float32)).cuda())
        jobs.append(dict(cache=cache, k=k, dk=dev(k), pos=i32(np.full(T, 50)), out=dev(np.zeros((T, H, D))), x=x, u=u, p=p,
                         lg=lg, rules=rules, tokens=torch.empty(T, dtype=torch.int32, device="cuda"),
                         logp=torch.empty(T, device="cuda"), st=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for j in jobs:
            moe.kv_append(j["dk"], j["dk"], j["pos"], j["cache"].c, stream=j["st"])
            moe.kv_read(j["cache"].c, j["pos"], j["out"], stream=j["st"])
            moe.sample(j["lg"], T, V, j["rules"], j["tokens"], logprobs=j["logp"], stream=j["st"])
    assert error(moe) == bq.MOE_OK
    for j in jobs:
        q, m = KO.quantise(j["k"])
        want = q * m[..., None]
        assert np.all(np.abs(f64(j["out"]) - want) <= 2.0 ** -8 * np.abs(want) * 1.01)
        check_sample(j["x"], j["tokens"].cpu().numpy(), j["logp"].cpu().numpy().astype(float), j["u"], None, None, j["p"])


def test_every_launch_is_stamped(moe):
    """Each of the calls takes one group of the launch trace."""
    cache = Cache(6, [40, 700], 2, 64, 16, True)
    k = dev(np.ones((2, 2, 64)))
    q = dev(np.ones((2, 4, 64)))
    ws = torch.empty(moe.kv_attend_workspace_bytes(cache.c, 4), dtype=torch.uint8, device="cuda")
    lg = torch.randn((3, 50000), device="cuda")
    rules = bq.make_sample_rules(torch.rand(3, device="cuda"), top_k=i32([0, 5, 700]))
    tokens = torch.empty(3, dtype=torch.int32, device="cuda")
    calls = [lambda: moe.kv_append(k, k, i32([40, 700]), cache.c), lambda: moe.kv_read(cache.c, i32([3, 4]), k),
             lambda: moe.kv_attend(q, i32([40, 700]), cache.c, torch.empty_like(q), ws, scale=0.1),
             lambda: moe.sample(lg, 3, 50000, rules, tokens)]
    for call in calls:
        got = stamps(moe, call)
        assert [any(g) for g in got] == [True] + [False] * 5, got
        assert in_order(got[0]), got[0]


def test_attention_of_one_sequence_many_times(moe):
    """The counters are clean after every call, whatever the shape of the one before."""
    g = np.random.default_rng(7)
    shapes = [([4000], 1, 8, 128, True), ([7] * 300, 2, 2, 16, False), ([100, 9000, 1], 3, 1, 80, False), ([2], 8, 2, 256, True)]
    cases = []
    for i, (lengths, H, group, D, bits8) in enumerate(shapes):
        cache = Cache(70 + i, lengths, H, D, 64, bits8)
        q = bf16(g.standard_normal((len(lengths), H * group, D)))
        ws = torch.empty(moe.kv_attend_workspace_bytes(cache.c, H * group), dtype=torch.uint8, device="cuda")
        cases.append([cache, q, dev(q), i32(lengths), lengths, ws, None])
    for turn in range(30):
        for c in cases:
            out, lse = torch.empty_like(c[2]), torch.empty(c[1].shape[:2], device="cuda")
            moe.kv_attend(c[2], c[3], c[0].c, out, c[5], scale=0.1, lse=lse)
            if c[6] is None:
                torch.cuda.synchronize()
                check_attend(c[0], c[1], c[4], 0.1, 0.0, 0, out, lse)
                c[6] = out
            assert torch.equal(out, c[6])  # bit by bit
    assert error(moe) == bq.MOE_OK


@pytest.mark.parametrize("bits8", [False, True])
def test_rows_behind_the_last_sequence(moe, bits8):
    """Outputs of more rows than there are sequences: those behind the last stay as they were."""
    lengths = [30, 0, 5]
    cache = Cache(90, lengths, 2, 64, 16, bits8)
    q = bf16(np.random.default_rng(9).standard_normal((5, 4, 64)))
    out, lse = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((5, 4), 7.0, device="cuda")
    ws = torch.empty(moe.kv_attend_workspace_bytes(cache.c, 4), dtype=torch.uint8, device="cuda")
    moe.kv_attend(dev(q), i32(lengths + [9, 9]), cache.c, out, ws, scale=0.1, lse=lse)
    assert error(moe) == bq.MOE_OK
    check_attend(cache, q[:3], lengths, 0.1, 0.0, 0, out[:3], lse)
    assert bool((out[3:] == 7).all()) and bool((lse[3:] == 7).all())


def test_workspace_behind_its_size_is_left_alone(moe):
    """The call writes no byte past the size that it asks for, on shapes that use all kinds of parts."""
    for lengths, H, group, D, bits8 in (([60000, 9], 1, 16, 256, False), ([3000] * 40, 2, 8, 128, True), ([700] * 90, 3, 1, 64, True)):
        cache = Cache(91, lengths, H, D, 64, bits8)
        n = moe.kv_attend_workspace_bytes(cache.c, H * group)
        ws = torch.full((n + 4096,), 85, dtype=torch.uint8, device="cuda")
        q = dev(np.ones((len(lengths), H * group, D)))
        moe.kv_attend(q, i32(lengths), cache.c, torch.empty_like(q), ws[:n], scale=0.1)
        assert error(moe) == bq.MOE_OK and bool((ws[n:] == 85).all())
        with pytest.raises(bq.MoeError) as e:
            moe.kv_attend(q, i32(lengths), cache.c, torch.empty_like(q), ws[:n - 1], scale=0.1)
        assert e.value.status == bq.MOE_ERR_WORKSPACE
