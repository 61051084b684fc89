"""What cache_append stores of values that are not finite: the same for both input types."""
import pytest
import torch

import fp4_microscaling_tensor_b200 as mx
import oracle
from cache_helpers import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", (mx.E4M3, mx.UE5M3))
@pytest.mark.parametrize("block", (16, 64))
def test_nans_do_not_count_for_their_blocks_scale(cuda_device, fmt, block):
    """A block's scale and its other values are as if its NaNs were zeros, also where every other value
    of it is a NaN, or all are (the scale is zero then); a NaN reads as 6 times the scale; an infinity
    has the largest scale."""
    table, zero = i32([[1, 0]], cuda_device), i32([0], cuda_device)
    x = torch.randn(1, 7, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    x[0, 0, 0, 3], x[0, 1, 0, :16], x[0, 2, 0, 15] = torch.nan, torch.nan, -torch.nan
    x[0, 3, 0, 0], x[0, 3, 0, 5], x[0, 4, 0, 9] = torch.inf, torch.nan, -torch.inf
    x[0, 5, 0, ::2], x[0, 6] = torch.nan, torch.nan
    bad = x.isnan()
    stored = []
    for dtype in (torch.bfloat16, torch.float32):
        cache = mx.KVCache(2, 1, 64, page_size=16, block=block, fmt=fmt, device=cuda_device)
        k, v = (t.to(dtype).to(cuda_device) for t in (x, x.nan_to_num(0.0, torch.inf, -torch.inf)))
        mx.cache_append(cache, k, v, table, zero)
        ko, vo = (t.cpu() for t in mx.cache_read(cache, table, zero, None, 7, out_dtype=torch.float32))
        assert torch.isfinite(ko).all() and torch.equal(cache.k_scales, cache.v_scales)
        assert torch.equal(ko[~bad], vo[~bad])
        scale = mx.dequantize(torch.full((7, 32), 0x22, dtype=torch.uint8, device=cuda_device),
                              cache.k_scales[1, 0, :7].contiguous(), block, fmt,
                              out_dtype=torch.float32).cpu().view(x.shape)
        assert torch.equal(ko[bad], 6 * scale[bad]) and not ko[0, 6].any()
        assert ko[0, 3, 0, 0] == 6 * oracle.scale_max(fmt) == -ko[0, 4, 0, 9] == ko[0, 3, 0, 5]
        stored.append([t.cpu() for t in (cache.k_codes, cache.k_scales, cache.v_codes)])
    for a, b in zip(*stored):
        assert torch.equal(a, b)
