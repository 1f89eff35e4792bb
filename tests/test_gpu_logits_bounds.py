"""What the order of the steps of the logit rules decides, on the GPU."""
import pytest
import torch

from helpers import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("values,want", [([1e8, -1e8], 1.0), ([1e8, -1e8, 2.0], 3.0), ([3.0, 1e8, -1e8], 1.0), ([-1e8, 0.25, 1e8, 0.5], 1.5)])
def test_biases_are_summed_before_they_meet_the_logit(values, want):
    """A logit of 1: biases added to it one by one would swallow it.  In fp32, 1e8 has steps of 8."""
    import bit_quantized_decode_gb300 as bq
    ids, vals = torch.full((1, 64), -1, dtype=torch.int32), torch.zeros((1, 64))
    for j, v in enumerate(values):
        ids[0, 5 * j], vals[0, 5 * j] = 700, v
    x = torch.ones((1, 1000), device="cuda")
    y = bq.LogitRules(1000, bias_ids=ids.cuda(), bias_values=vals.cuda())(x).cpu()
    assert float(y[0, 700]) == want and float(y.sum()) == 999.0 + want
