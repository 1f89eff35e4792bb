"""The cache append at its smallest head counts and on values that are not numbers."""
import pytest
import torch

from helpers import cuda_ok
from test_gpu_attention import BF16, F16, F32, I8, check_append

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def bq():
    import bit_quantized_decode_gb300 as pkg
    pkg._lib.load()
    pkg._lib.clear_device_error()
    yield pkg
    assert pkg._lib.device_error() == 0


@pytest.mark.parametrize("x_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("dtype", [BF16, I8])
@pytest.mark.parametrize("rot,layout", [(64, "half"), (16, "interleaved"), (0, "half")])
def test_fewer_heads_than_a_warp_takes(bq, rot, layout, dtype, x_dtype):
    """One query, one key and one value head of 64: three of the four heads that a warp has lanes for.  Rows behind each other
    and apart."""
    check_append(bq, 3, [5, 1], [10, 0], 16, 1, 1, 64, dtype, x_dtype, rot, layout, True)
    check_append(bq, 4, [3], [17], 16, 1, 1, 64, dtype, x_dtype, rot, layout, False, wide=8)
