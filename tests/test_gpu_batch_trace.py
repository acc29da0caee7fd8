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
