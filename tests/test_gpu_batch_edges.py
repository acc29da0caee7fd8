"""Calls of the batched path that its documentation allows at the ends of their
ranges: the most rows, one handle on two streams, inputs that are one tensor."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from oracle import batch_oracle as BO
from test_gpu_norm_quant import REL, dev16, host16, moe, rows  # noqa: F401  (moe: the fixture)
from test_gpu_qdense import bound, codes, scales

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T", [65535, 65536])
@pytest.mark.parametrize("N,K", [(200, 64), (33, 144)])
def test_most_rows_of_a_projection(moe, T, N, K):  # noqa: F811
    x, w = codes(1, T, K), codes(2, N, K)
    xs, ws = scales(3, T, N)
    wd = bq.make_qdense_weights(N, K, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    work = torch.empty(moe.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
    y = torch.full((T, N), np.nan, device="cuda")
    moe.qdense_forward(torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), T, wd, work, y32=y)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    assert np.all(np.abs(y.cpu().numpy() - BO.qdense(x, xs, w, ws)) <= bound(x, w, xs, ws))


def test_most_rows_of_a_norm(moe):  # noqa: F811
    T, H = 1 << 20, 16
    h = rows(4, T, H)
    q, s = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.norm_quant(dev16(h), T, q, s)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    want = BO.norm_quant(h)
    assert np.array_equal(q.cpu().numpy(), want["q"])
    assert np.all(np.abs(s.cpu().numpy() - want["scales"]) <= REL * want["scales"])


def test_hidden_added_to_itself(moe):  # noqa: F811
    """hidden and y are one tensor, and the sum goes back into it."""
    h = rows(5, 7, 704)
    want = BO.norm_quant(h, h)
    hd = dev16(h)
    q, s = torch.empty((7, 704), dtype=torch.int8, device="cuda"), torch.empty(7, device="cuda")
    moe.norm_quant(hd, 7, q, s, y=hd)
    torch.cuda.synchronize()
    assert np.array_equal(host16(hd), h) and np.array_equal(q.cpu().numpy(), want["q"])


@pytest.mark.parametrize("T", [5, 16, 300])
def test_one_handle_on_two_streams(moe, T):  # noqa: F811
    """Projections of one handle that may run at the same time, a workspace each."""
    N, K = 3000, 704
    w = codes(6, N, K)
    jobs = []
    for i in range(2):
        x = codes(7 + i, T, K)
        xs, ws = scales(9 + i, T, N)
        wd = bq.make_qdense_weights(N, K, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
        work = torch.empty(moe.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
        jobs.append((torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), wd, work, torch.empty((T, N), device="cuda"),
                     torch.cuda.Stream(), x, xs, ws))
    torch.cuda.synchronize()
    for _ in range(30):
        for xd, xsd, wd, work, y, st, *_ in jobs:
            moe.qdense_forward(xd, xsd, T, wd, work, y32=y, stream=st)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    for *_, y, _, x, xs, ws in jobs:
        assert np.all(np.abs(y.cpu().numpy() - BO.qdense(x, xs, w, ws)) <= bound(x, w, xs, ws))


@pytest.mark.parametrize("T", [16, 300])
def test_graph_and_eager_calls_in_turn(moe, T):  # noqa: F811
    """A captured projection replayed between eager ones that use its workspace, in one stream."""
    N, K = 900, 704
    w = codes(20, N, K)
    xs, ws = scales(21, T, N)
    wd = bq.make_qdense_weights(N, K, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    work = torch.empty(moe.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
    a, b = codes(22, T, K), codes(23, T, K)
    ad, bd, xsd = torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda(), torch.from_numpy(xs).cuda()
    ya, yb = torch.empty((T, N), device="cuda"), torch.empty((T, N), device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            moe.qdense_forward(ad, xsd, T, wd, work, y32=ya)
        for _ in range(20):
            g.replay()
            moe.qdense_forward(bd, xsd, T, wd, work, y32=yb)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    for x, y in ((a, ya), (b, yb)):
        assert np.all(np.abs(y.cpu().numpy() - BO.qdense(x, xs, w, ws)) <= bound(x, w, xs, ws))
