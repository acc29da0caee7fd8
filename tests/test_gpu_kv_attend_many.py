"""moe_kv_attend with more sequences than a block has threads, so that a thread counts
several: items that all fit a block, which then stay whole, and one that does not.
The bounds are test_gpu_kv_attend's."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from kv_cases import Cache, dev, i32
from test_gpu_kv_attend import check, moe, queries, run  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("n,H,D,most,long", [(600, 1, 64, 1500, 0), (1100, 2, 16, 500, 0), (1100, 1, 16, 500, 9000),
                                             (520, 1, 256, 600, 0), (513, 3, 16, 1537, 1600), (4096, 1, 16, 150, 2100)])
def test_more_sequences_than_threads(moe, bits8, n, H, D, most, long):  # noqa: F811
    g = np.random.default_rng(n + most)
    lengths = g.integers(0, most + 1, n)
    if long:
        lengths[n // 3] = long
    cache = Cache(150, lengths, H, D, 64, bits8)
    q = queries(151, n, 2 * H, D)
    out, lse = run(moe, cache, dev(q), i32(lengths), 0.15)
    assert moe.get_error() == bq.MOE_OK
    check(cache, q, lengths, 0.15, 0.0, 0, out, lse, heads=(2 * H - 1,))
    again, _ = run(moe, cache, dev(q), i32(lengths), 0.15)
    assert torch.equal(out, again)
