"""Launch tracing (moe_set_trace) of the batched path's calls: every launch
takes one group of four slots and stamps its entry, the time past its dependency
wait and its exit."""
import pytest

import bit_affine_quantized_gb300 as bq

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

GROUPS = 6


@pytest.fixture(scope="module")
def moe():
    bq.build_library()
    m = bq.Moe()
    yield m
    m.close()


def stamps(moe, call):
    trace = torch.zeros((GROUPS, 4), dtype=torch.int64, device="cuda")
    moe.set_trace(trace, GROUPS)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        moe.set_trace(None, 0)
    assert moe.get_error() == bq.MOE_OK
    return [[v & (2 ** 64 - 1) for v in row] for row in trace.tolist()]


def in_order(group):
    entry, waited, _, end = group
    return 0 < 2 ** 64 - 1 - entry <= 2 ** 64 - 1 - waited <= end


def projection(T, N, K):
    w = torch.ones((N, K), dtype=torch.int8, device="cuda")
    wd = bq.make_qdense_weights(N, K, w, torch.ones(N, device="cuda"))
    x, xs = torch.ones((T, K), dtype=torch.int8, device="cuda"), torch.ones(T, device="cuda")
    y = torch.empty((T, N), device="cuda")

    def call(moe):
        ws = torch.empty(moe.qdense_workspace_bytes(wd, T), dtype=torch.uint8, device="cuda")
        return lambda: moe.qdense_forward(x, xs, T, wd, ws, y32=y)
    return call


# one row, few rows; one tile or part of one per block, whole tiles, pairs of blocks
SHAPES = [(1, 300, 704), (5, 300, 704), (16, 704, 2816), (24, 40000, 704), (300, 5000, 704)]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_every_launch_is_stamped(moe, T, N, K):
    """Entry, dependency wait and exit of each launch of a projection."""
    got = stamps(moe, projection(T, N, K)(moe))
    used = [g for g in got if any(g)]
    assert 1 <= len(used) <= 2 and all(in_order(g) for g in used), got


def test_exit_is_the_last_blocks(moe):
    """A launch of many short blocks: its exit is the last one's, not the first's."""
    T, H = 300000, 1024
    if torch.cuda.mem_get_info()[0] < 4 << 30:
        pytest.skip("needs 4 GB")
    h = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.norm_quant(h, T, q, s)
    torch.cuda.synchronize()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))

    def call():
        begin.record()
        moe.norm_quant(h, T, q, s)
        end.record()

    group = stamps(moe, call)[0]
    assert in_order(group)
    assert group[3] - (2 ** 64 - 1 - group[0]) > 0.5e6 * begin.elapsed_time(end)  # ns against ms


@pytest.mark.parametrize("T,N,K", [(1, 300000, 704), (5, 300000, 704), (24, 300000, 704), (4000, 5000, 704)])
def test_exit_of_a_projection(moe, T, N, K):
    """Its last launch leaves no later than a launch behind it passes its dependency wait."""
    call = projection(T, N, K)(moe)
    h = torch.ones((1, 64), dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty((1, 64), dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    call()
    moe.norm_quant(h, 1, q, s)
    trace = torch.zeros((GROUPS, 4), dtype=torch.int64, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    moe.set_trace(trace, GROUPS)
    with torch.cuda.graph(graph, stream=stream):  # the launches follow each other whatever the host does
        call()
        moe.norm_quant(h, 1, q, s)
    moe.set_trace(None, 0)
    graph.replay()
    trace.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    used = [g for g in ([v & (2 ** 64 - 1) for v in row] for row in trace.tolist()) if any(g)]
    assert all(in_order(g) for g in used)
    first, last, behind = used[0], used[-2], used[-1]
    lived, waited = last[3] - (2 ** 64 - 1 - first[0]), 2 ** 64 - 1 - behind[1]
    # (the blocks end together: what is left are the last stores and the next launch's start)
    assert last[3] <= waited and waited - last[3] < max(4000, lived // 4)


@pytest.mark.parametrize("T,N,K,launches", [(1, 300, 704, 1), (8, 300, 704, 1), (16, 704, 2816, 1), (24, 40000, 704, 2),
                                            (300, 5000, 704, 2)])
def test_groups_in_a_row(moe, T, N, K, launches):
    """Launches take groups one after another: a projection between two norms
    leaves none between them, whether it widens its rows in a launch before or in
    the same one."""
    call = projection(T, N, K)(moe)
    h = torch.ones((1, 64), dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty((1, 64), dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")

    def chain():
        moe.norm_quant(h, 1, q, s)
        call()
        moe.norm_quant(h, 1, q, s)

    got = stamps(moe, chain)
    assert [any(g) for g in got] == [i < launches + 2 for i in range(GROUPS)], got
    assert all(in_order(g) for g in got[:launches + 2])
    for a, b in zip(got, got[1:launches + 2]):
        assert a[3] <= b[3]  # in the stream's order


def test_one_group_is_enough_for_one_launch(moe):
    """A call that makes one launch is stamped in a buffer of one group."""
    call = projection(16, 704, 2816)(moe)
    trace = torch.zeros((1, 4), dtype=torch.int64, device="cuda")
    moe.set_trace(trace, 1)
    call()
    torch.cuda.synchronize()
    moe.set_trace(None, 0)
    assert moe.get_error() == bq.MOE_OK and bool((trace[0, :2] != 0).all())
