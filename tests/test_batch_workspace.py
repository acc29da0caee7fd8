"""The workspace of qdense_forward: its size and its refusals, whatever the size
function says (no refused call looks into the handle, a block of zeros)."""
import ctypes

import pytest

import bit_affine_quantized_gb300 as bq
from test_batch_host import A, _qdense, handle, lib  # noqa: F401  (handle, lib: the fixtures)


@pytest.mark.parametrize("rows", [1, 2, 8, 9, 16, 128, 333, 4096, 65536])
@pytest.mark.parametrize("n,k", [(64, 64), (4096, 2816), (1411, 1072), (1, 16), (1 << 28, 16384)])
def test_size(lib, rows, n, k):  # noqa: F811
    """Nothing up to 8 rows; then the rows widened to 2 bytes, in whole 256 bytes, the same on every device."""
    w = bq.QdenseWeights(n, k, A, A)
    want = 0 if rows <= 8 else (rows * k * 2 + 255) // 256 * 256
    assert lib.moe_qdense_workspace_bytes(ctypes.byref(w), rows) == want


@pytest.mark.parametrize("rows", [9, 32, 4096])
def test_refusals(lib, handle, rows):  # noqa: F811
    need = (rows * 64 * 2 + 255) // 256 * 256
    assert _qdense(lib, handle[0], rows=rows, ws=None) == bq.MOE_ERR_INVALID_ARG
    assert _qdense(lib, handle[0], rows=rows, ws=A + 16) == bq.MOE_ERR_INVALID_ARG
    assert _qdense(lib, handle[0], rows=rows, ws_bytes=need - 1) == bq.MOE_ERR_WORKSPACE
    assert _qdense(lib, handle[0], rows=rows, ws_bytes=0) == bq.MOE_ERR_WORKSPACE
