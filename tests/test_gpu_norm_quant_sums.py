"""The sum of squares of norm_quant's rows where every rounding goes one way.

test_gpu_norm_quant.py allows a scale 20 * 2^-24: 16 squares a thread, 10 steps
of the block's sum, 6 more operations.  The rows here lose half a unit of the
running sum at nearly every addition: a thread's squares are 1 and then 31 times
2^-24, each a tie that goes to the even neighbour, 1; the last ones of some lanes
leave whole units, so that the sums of pairs of lanes are ties as well."""
import numpy as np
import pytest

from oracle import batch_oracle as BO
from oracle.batch_oracle import to_bf16
from test_gpu_norm_quant import check, moe, run  # noqa: F401  (moe: the fixture)

pytestmark = pytest.mark.gpu

# units of 2^-23 that each lane's sum ends with
UNITS = [0, 0, 0, 0, 0, 0, 0, 2, 0, 0, 0, 0, 0, 0, 3, 6, 1, 1, 1, 1, 1, 1, 1, 7, 2, 2, 2, 2, 5, 5, 7, 7]


def losing_row():
    """1024 values: lane l's 32, in the order in which a chain of fused
    multiply-adds over its four vectors of eight takes them (odd ones first)."""
    v = np.full((32, 32), 2.0 ** -12)
    v[:, 0] = 1.0
    for lane, k in enumerate(UNITS):
        if k:  # the largest bf16 value whose square is below k + 1/2 units
            bits = np.float32(np.sqrt((k + 0.5) * 2.0 ** -23 * (1 - 2.0 ** -40))).view(np.uint32) & 0xFFFF0000
            v[lane, 31] = np.uint32(bits).view(np.float32)
    row = np.empty(1024)
    for lane in range(32):
        for k in range(32):
            row[(lane + 32 * (k // 8)) * 8 + (k % 8) // 2 * 2 + (k % 2 == 0)] = v[lane, k]
    return row


@pytest.mark.parametrize("eps,top", [(5.4797154e-05, 1.515625), (3.2322467e-05, 1.5), (5.6824247e-06, 1.4375),
                                     (2.6592394e-05, 1.484375), (5.682283e-06, 1.4375)])
@pytest.mark.parametrize("T", [600, 100])
def test_scale_of_rows_that_lose_at_every_addition(moe, T, eps, top):  # noqa: F811
    h = to_bf16(np.tile(losing_row(), (T, 1)))
    g = to_bf16(np.full(1024, top))
    eps = float(np.float32(eps))
    check(run(moe, h, g=g, eps=eps), BO.norm_quant(h, g_bits=g, eps=eps))
