"""The dense 8-bit projection where its tiles end: channels that end inside a
warp's 32, in every form of the tensor-core kernel; bounds as in
test_gpu_qdense.py."""
import numpy as np
import pytest

import bit_affine_quantized_gb300 as bq
from oracle import batch_oracle as BO
from synth import gen
from test_gpu_qdense import F32, bound, codes, moe, run, scales  # noqa: F401  (moe: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T,N,K", [
    (70, 19585, 1168), (128, 9889, 704), (100, 39009, 80),       # whole tiles of up to 128 rows, several per warp
    (300, 5007, 704), (512, 10223, 144), (1000, 1281, 1040), (250, 31, 80),  # pairs of blocks, halves of tiles
    (128, 2785, 4096), (333, 1411, 1072), (16, 705, 2816), (24, 33, 80)])    # parts of tiles
def test_channels_that_end_inside_a_warp(moe, T, N, K):  # noqa: F811
    """With a softcap and both outputs; every call gives the same bits."""
    x, w = codes(T, T, K), codes(N, N, K)
    xs, ws = scales(K, T, N)
    xs = xs * np.float32(20.0)
    want = BO.qdense(x, xs, w, ws, 30.0)
    y16, y32 = run(moe, x, xs, w, ws, softcap=30.0)
    assert np.all(np.abs(y32 - want) <= bound(x, w, xs, ws) + 12 * F32 * np.abs(want))
    assert np.array_equal(y16, gen.to_bf16_bits(y32.astype(np.float64)))
    for _ in range(3):
        assert np.array_equal(run(moe, x, xs, w, ws, softcap=30.0, y=False)[1], y32)


@pytest.mark.parametrize("T,N,K", [(3, 700, 12272), (3, 700, 12288), (4, 131, 12288), (3, 33, 16384), (4, 1027, 16384),
                                   (5, 131, 12288), (8, 515, 16384), (8, 515, 12272), (2, 515, 16384)])
@pytest.mark.parametrize("kind", ["bell", "full"])
def test_few_wide_rows(moe, T, N, K, kind):  # noqa: F811
    """3 to 8 rows on both sides of the width up to which their widened codes fit
    a block's shared memory; the sums are integers on both."""
    x, w = codes(T, T, K, kind), codes(N, N, K, kind)
    xs, ws = scales(K, T, N)
    y16, y32 = run(moe, x, xs, w, ws)
    assert np.all(np.abs(y32 - BO.qdense(x, xs, w, ws)) <= bound(x, w, xs, ws))
    assert np.array_equal(y16, gen.to_bf16_bits(y32.astype(np.float64)))


@pytest.mark.parametrize("T,N,K", [(16, 704, 2816), (128, 2816, 4096), (300, 5000, 704)])
def test_workspace_edges(moe, T, N, K):  # noqa: F811
    """A workspace of exactly the size asked for, what lies around it left alone;
    a smaller one and none are refused, whether the call uses it or not."""
    x, w = codes(70, T, K), codes(71, N, K)
    xs, ws = scales(72, T, N)
    wd = bq.make_qdense_weights(N, K, torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda())
    n = moe.qdense_workspace_bytes(wd, T)
    assert n == (T * K * 2 + 255) // 256 * 256
    room = torch.full((n + 512,), 77, dtype=torch.uint8, device="cuda")
    y = torch.empty((T, N), device="cuda")
    xd, xsd = torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda()
    moe.qdense_forward(xd, xsd, T, wd, room[256:256 + n], y32=y)
    torch.cuda.synchronize()
    assert moe.get_error() == bq.MOE_OK
    assert bool((room[:256] == 77).all()) and bool((room[256 + n:] == 77).all())
    assert np.all(np.abs(y.cpu().numpy() - BO.qdense(x, xs, w, ws)) <= bound(x, w, xs, ws))
    for bad in (None, room[256:256 + n - 256], room[16:16 + n]):
        with pytest.raises(bq.MoeError):
            moe.qdense_forward(xd, xsd, T, wd, bad, y32=y)
