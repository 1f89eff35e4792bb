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


@pytest.mark.parametrize("D,rot", [(64, 0), (64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("x_dtype", [F32, BF16])
def test_a_nan_stays_in_its_head_of_an_int8_cache(bq, x_dtype, D, rot):
    """A NaN among a head's values, in its rotated part and behind it, and a head of nothing else: the scale says so.  The
    other heads of the row and other rows are as without."""
    Hq, Hkv, T = 3, 3, 4
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()                      # noqa: E731
    batch = bq.KVBatch(i32([[0, 1]]), i32([0]), i32([0, T]), T)
    x = torch.randn((T, (Hq + 2 * Hkv) * D), generator=torch.Generator().manual_seed(1)).to(x_dtype)
    bad = x.clone().view(T, Hq + 2 * Hkv, D)
    bad[0, Hq, 5] = bad[1, Hq + 2, D - 1] = bad[2, Hq + Hkv + 1, 0] = float("nan")
    bad[3, Hq + 1], bad[3, Hq + Hkv] = float("nan"), float("nan")
    hit = {"k": [(0, 0), (1, 2), (3, 1)], "v": [(2, 1), (3, 0)]}
    caches = []
    for t in (x, bad.view(T, -1)):
        cache = bq.KVCache.empty(2, 16, Hkv, D, I8)
        rope = bq.RopeTable.build(8, rot) if rot else None
        bq.CachedAttention(cache, Hq, rope=rope).append(t.cuda(), batch)
        caches.append(cache)
    for codes, scale, which in (("k", "k_scale", "k"), ("v", "v_scale", "v")):
        a, b = (getattr(c, codes)[0, :, :T].cpu().transpose(0, 1).clone() for c in caches)
        sa, sb = (getattr(c, scale)[0, :, :T].cpu().t().clone() for c in caches)
        for t, h in hit[which]:
            assert bool(torch.isnan(sb[t, h])) and bool((b[t, h] == 0).all()), (which, t, h)
            a[t, h], sa[t, h], sb[t, h] = 0, 0.0, 0.0
        assert torch.equal(a, b) and torch.equal(sa, sb)
