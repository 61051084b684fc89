"""The paged FP4 cache: append against the oracle's quantizer, bit for bit, read against its
dequantizer, and everything around the written positions left as it was."""
import numpy as np
import pytest
import torch

import fp4_microscaling_tensor_b200 as mx
import oracle
from cache_helpers import G_ONE, i32, pages_for, place, poisoned
from gpu_helpers import assert_same, bits, special_values_bf16, u8

pytestmark = pytest.mark.gpu


def buffers(cache):
    return [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


def to_oracle(x):
    x = x.detach().contiguous().cpu()
    return bits(x) if x.dtype == torch.bfloat16 else x.numpy().reshape(-1)


def check_append(cache, table, k, v, start, count, device):
    """Appends and compares the whole pool with a host copy that only the oracle has written to."""
    want = buffers(cache)
    host = mx.KVCache.from_buffers(*want, fmt=cache.fmt, k_g=cache.k_g, v_g=cache.v_g)
    tokens = k.shape[1]
    for b in range(k.shape[0]):
        n = tokens if count is None else min(max(count[b], 0), tokens)
        pos = start[b] + np.arange(n)
        inside = (pos >= 0) & (pos < table.shape[1] * cache.page_size)
        ids = np.where(inside, table[b, np.where(inside, pos // cache.page_size, 0)], -1)
        keep = np.nonzero((ids >= 0) & (ids < cache.pages))[0]
        if not len(keep):
            continue
        for x, which, g in ((k, "k", cache.k_g), (v, "v", cache.v_g)):
            rows = x[b][torch.from_numpy(keep).to(device)]
            p, s = oracle.quantize(to_oracle(rows), len(keep) * cache.kv_heads, cache.head_dim,
                                   cache.block, cache.fmt, g)
            place(host, table, b, pos[keep], which, p.reshape(len(keep), cache.kv_heads, -1),
                  s.reshape(len(keep), cache.kv_heads, -1))
    mx.cache_append(cache, k, v, i32(table, device), i32(start, device),
                    count=None if count is None else i32(count, device))
    torch.cuda.synchronize()
    for got, ref, what in zip(buffers(cache), want, ("k_codes", "k_scales", "v_codes", "v_scales")):
        assert_same(u8(got), u8(ref), what)


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("fmt", (mx.E4M3, mx.UE5M3))
@pytest.mark.parametrize("head_dim,block,page", ((64, 16, 16), (64, 64, 256), (128, 32, 64),
                                                 (128, 128, 32), (256, 16, 128), (256, 64, 16)))
def test_append_matches_the_quantizer(cuda_device, head_dim, block, page, fmt, dtype):
    rng = np.random.default_rng(head_dim + block + fmt)
    kvh, tokens = 3, 37
    g = (0x0155, 0x2E66) if fmt == mx.UE5M3 else (G_ONE, 0x2E66)
    start, count = [0, page - 1, 5, 1000], [37, 20, 0, 37]
    table, pages = pages_for([1100] * 4, page, 2, rng)
    cache = poisoned(pages, kvh, head_dim, page, block, fmt, *g, rng, cuda_device)
    shape = (4, tokens, kvh, head_dim)
    k, v = (special_values_bf16(fmt, gb, int(np.prod(shape)), seed=s).view(shape).to(cuda_device)
            .to(dtype) for gb, s in zip(g, (1, 2)))
    if dtype == torch.float32:  # bits below bf16's
        k, v = (x * (1 + torch.rand(shape, generator=torch.Generator().manual_seed(9)).to(x.device)
                     * 2.0 ** -9) for x in (k, v))
        k, v = (x.clamp(-3e38, 3e38) for x in (k, v))
    check_append(cache, table, k, v, start, count, cuda_device)


def test_append_strided_and_one_token(cuda_device):
    """Slices of a fused projection, one token a sequence, no counts; a transposed layout."""
    rng = np.random.default_rng(4)
    table, pages = pages_for([300] * 5, 64, 1, rng)
    cache = poisoned(pages, 4, 128, 64, 32, mx.E4M3, G_ONE, G_ONE, rng, cuda_device)
    qkv = torch.randn(5, 1, 16 + 8, 128, device=cuda_device).bfloat16()
    check_append(cache, table, qkv[:, :, 16:20], qkv[:, :, 20:], [0, 63, 64, 255, 299], None,
                 cuda_device)
    heads_first = torch.randn(5, 4, 19, 128, device=cuda_device)
    check_append(cache, table, heads_first.transpose(1, 2), heads_first.flip(0).transpose(1, 2),
                 [0, 40, 64, 255, 281], [19, 19, 1, 7, 18], cuda_device)
    shared = torch.randn(1, 1, 4, 128, device=cuda_device).bfloat16().expand(5, 3, 4, 128)
    check_append(cache, table, shared, shared, [7] * 5, None, cuda_device)


def test_positions_without_a_page_are_left_alone(cuda_device):
    """Table entries that name no page, positions beyond the table and negative ones: nothing is
    written for them, they read as zeros, the other positions are not disturbed."""
    rng = np.random.default_rng(5)
    table, pages = pages_for([64] * 4, 16, 1, rng)
    table[0, 1], table[1, 2] = -1, pages
    table[2, 0] = np.iinfo(np.int32).max
    cache = poisoned(pages, 2, 64, 16, 32, mx.UE5M3, G_ONE, G_ONE, rng, cuda_device)
    k, v = (torch.randn(4, 70, 2, 64, device=cuda_device).bfloat16() for _ in range(2))
    start = [0, 0, 0, -3]
    check_append(cache, table, k, v, start, None, cuda_device)
    ko, vo = mx.cache_read(cache, i32(table, cuda_device), i32(start, cuda_device), None, 70)
    codes, scales = mx.quantize(k, 32, "ue5m3")
    y = mx.dequantize(codes, scales, 32, "ue5m3")
    for b in range(4):
        pos = start[b] + np.arange(70)
        ids = [table[b, p // 16] if 0 <= p < 64 else -1 for p in pos]
        ok = torch.tensor([0 <= i < pages for i in ids], device=cuda_device)
        assert torch.equal(ko[b][ok], y[b][ok]) and not ko[b][~ok].any() and not vo[b][~ok].any()


@pytest.mark.parametrize("fmt", (mx.E4M3, mx.UE5M3))
@pytest.mark.parametrize("head_dim,block,page", ((64, 32, 16), (128, 16, 64), (256, 128, 32)))
def test_read_matches_the_dequantizer(cuda_device, head_dim, block, page, fmt):
    """Every code byte and every scale code the quantizer can write, both output types; rows behind
    the counts keep their mark."""
    rng = np.random.default_rng(head_dim)
    kvh, lengths = 3, [1, 100, 0, 333]
    table, pages = pages_for(lengths, page, 2, rng)
    g = (0x0155, 0x2E66)
    cache = poisoned(pages, kvh, head_dim, page, block, fmt, *g, rng, cuda_device)
    top = 0x7F if fmt == mx.E4M3 else 0x100
    for t in (cache.k_scales, cache.v_scales):
        t.copy_(torch.from_numpy(rng.integers(0, top, tuple(t.shape), dtype=np.uint8)))
    start, count, tokens = [0, 7, 0, 11], [1, 93, 0, 322], 322
    for dtype in (torch.bfloat16, torch.float32):
        out = [torch.full((4, tokens, kvh, head_dim), 5.0, dtype=dtype, device=cuda_device)
               for _ in range(2)]
        r = mx.cache_read(cache, i32(table, cuda_device), i32(start, cuda_device),
                          i32(count, cuda_device), tokens, k_out=out[0], v_out=out[1])
        assert r[0] is out[0] and r[1] is out[1]
        for y, c, s, gb in ((out[0], cache.k_codes, cache.k_scales, g[0]),
                            (out[1], cache.v_codes, cache.v_scales, g[1])):
            for b, n in enumerate(count):
                pos = start[b] + np.arange(n)
                ids, slot = torch.from_numpy(table[b, pos // page].astype(np.int64)), pos % page
                ref = oracle.dequantize(u8(c.cpu()[ids, :, slot]), u8(s.cpu()[ids, :, slot]),
                                        n * kvh, head_dim, block, fmt, gb,
                                        out_bf16=dtype == torch.bfloat16) if n else np.zeros(0, np.uint32)
                ref = ref if dtype == torch.bfloat16 else ref.view(np.uint32)
                assert_same(bits(y[b, :n]), ref, f"sequence {b} {dtype}")
                assert (y[b, n:] == 5.0).all()
    # new outputs: zeros behind the counts; strided outputs
    ko, vo = mx.cache_read(cache, i32(table, cuda_device), i32(start, cuda_device),
                           i32(count, cuda_device), tokens)
    wide = torch.zeros(4, tokens, 2, kvh, head_dim, dtype=torch.bfloat16, device=cuda_device)
    mx.cache_read(cache, i32(table, cuda_device), i32(start, cuda_device), i32(count, cuda_device),
                  tokens, k_out=wide[:, :, 0], v_out=wide[:, :, 1])
    assert torch.equal(wide[:, :, 0].view(torch.int16), ko.view(torch.int16))
    assert torch.equal(wide[:, :, 1].view(torch.int16), vo.view(torch.int16))
    assert not ko[2].any()


def test_infinities_and_nans_store_no_nan_scale(cuda_device):
    """What is not finite is stored as something finite, and only in its own block."""
    for fmt in (mx.E4M3, mx.UE5M3):
        for dtype in (torch.bfloat16, torch.float32):
            cache = mx.KVCache(2, 1, 64, page_size=16, block=32, fmt=fmt, device=cuda_device)
            k = torch.ones(1, 4, 1, 64, dtype=dtype, device=cuda_device)
            k[0, 0, 0, 3] = torch.inf
            k[0, 1, 0, 3] = -torch.inf
            k[0, 2, 0, 3] = torch.nan
            k[0, 3, 0, :32] = torch.nan
            table, zero = i32([[1, 0]], cuda_device), i32([0], cuda_device)
            mx.cache_append(cache, k, k, table, zero)
            ko, vo = mx.cache_read(cache, table, zero, None, 4, out_dtype=torch.float32)
            assert torch.isfinite(ko).all() and torch.isfinite(vo).all()
            # a block of ones: 1 / 6 = 1.333 * 2^-3 rounds to the scale 1.375 * 2^-3 in both formats
            # (neighbours 1.25 and 1.375), and each element 1 / 0.171875 = 5.8 to 6: 1.03125
            assert (ko[..., 32:] == 1.03125).all() and torch.equal(ko, vo)
            assert ko[0, 0, 0, 3] == 6 * oracle.scale_max(fmt) == -ko[0, 1, 0, 3]


def test_long_cache_offsets(cuda_device):
    """Pages whose bytes lie beyond 2^32 of the codes (a pool of more than 4 GiB)."""
    page, kvh, dim = 256, 8, 256
    per = kvh * page * dim // 2
    pages = (1 << 32) // per + 4
    cache = mx.KVCache(pages, kvh, dim, page_size=page, block=128, fmt="e4m3", device=cuda_device)
    k, v = (torch.randn(2, 300, kvh, dim, device=cuda_device).bfloat16() for _ in range(2))
    table = i32([[pages - 1, 0], [pages - 3, 2]], cuda_device)
    zero = i32([0, 0], cuda_device)
    mx.cache_append(cache, k, v, table, zero)
    ko, vo = mx.cache_read(cache, table, zero, None, 300)
    for x, y in ((k, ko), (v, vo)):
        c, s = mx.quantize(x, 128, "e4m3")
        assert torch.equal(mx.dequantize(c, s, 128, "e4m3"), y)
