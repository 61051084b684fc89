"""cache_attention with many query rows per key/value head (the tensor-core tiles), and what the cache's
kernels do at the edges of how they cut their work (bounds: cache_helpers.attend)."""
import numpy as np
import pytest
import torch

import fp4_microscaling_tensor_b200 as mx
import oracle
from cache_helpers import (G_ONE, assert_close, attend, chain_mask, check_attention, fill, i32,
                           normal_bf16, pages_for, poisoned, random_tree)
from test_gpu_cache import check_append

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def nobody_gave_up():
    """No bounded wait of a tensor-core kernel runs out."""
    yield
    assert mx.matmul_gave_up() == 0


def setup(lengths, kvh, head_dim, page, block, fmt, rng, device, sigma=1.0):
    g = (0x0155, 0x2E66) if fmt == mx.UE5M3 else (G_ONE, 0x2E66)
    table, pages = pages_for(lengths, page, 2, rng)
    cache = poisoned(pages, kvh, head_dim, page, block, fmt, *g, rng, device)
    return cache, table, fill(cache, table, lengths, rng, sigma)


def scale_for(cache):
    return cache.head_dim ** -0.5 / oracle.fp16_value(cache.k_g)


@pytest.mark.parametrize("fmt", (mx.E4M3, mx.UE5M3))
@pytest.mark.parametrize("head_dim,block,page", ((64, 32, 16), (128, 16, 32), (256, 64, 64)))
def test_rows_around_a_tile(cuda_device, head_dim, block, page, fmt):
    """33 to 300 rows per key/value head, lengths that end inside a chunk, short counts."""
    rng = np.random.default_rng(head_dim)
    lengths, counts = [300, 301, 384, 127, 520, 33], [300, 257, 129, 127, 128, 33]
    cache, table, kv = setup(lengths, 2, head_dim, page, block, fmt, rng, cuda_device)
    q = normal_bf16((6, 300, 2, head_dim), 1, cuda_device)
    check_attention(cache, table, lengths, counts, kv, q, scale=scale_for(cache))


@pytest.mark.parametrize("head_dim", (64, 128, 256))
def test_positions_without_a_page(cuda_device, head_dim):
    rng = np.random.default_rng(2)
    lengths, tokens = [310, 200, 64], 40
    cache, table, kv = setup(lengths, 1, head_dim, 16, 32, mx.UE5M3, rng, cuda_device)
    table[0, 2], table[0, 19], table[1, 0], table[2, 1] = -1, cache.pages, -7, 1 << 30
    q = normal_bf16((3, tokens, 8, head_dim), 3, cuda_device)
    out, lse = mx.cache_attention(cache, q, i32(table, cuda_device), i32(lengths, cuda_device),
                                  lse=True, scale=scale_for(cache))
    for b, n in enumerate(lengths):
        ids = table[b, np.arange(n) // 16]
        mask = ((ids >= 0) & (ids < cache.pages))[None] & chain_mask(n, tokens)
        ref = attend(q[b].float().cpu().numpy().astype(np.float64), *kv[b], mask, scale_for(cache))
        assert_close(out[b].float().cpu().numpy(), ref[0], ref[2], f"sequence {b}")
        assert_close(lse[b].cpu().numpy(), ref[1], ref[3], f"sequence {b} lse")
    table[:] = -1  # nothing is there: every row is empty
    out, lse = mx.cache_attention(cache, q, i32(table, cuda_device), i32(lengths, cuda_device), lse=True)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("head_dim", (64, 128, 256))
def test_every_scale_code(cuda_device, head_dim):
    """Random codes with every finite scale code: small q keeps the scores in range."""
    rng = np.random.default_rng(4)
    for fmt, top in ((mx.E4M3, 0x7F), (mx.UE5M3, 0x100)):
        lengths = [190, 70]
        table, pages = pages_for(lengths, 32, 0, rng)
        cache = poisoned(pages, 1, head_dim, 32, 16, fmt, G_ONE, G_ONE, rng, cuda_device)
        for t in (cache.k_scales, cache.v_scales):
            t.copy_(torch.from_numpy(rng.integers(0, top, tuple(t.shape), dtype=np.uint8)))
        kv = []
        for b, n in enumerate(lengths):
            ids, slot = table[b, np.arange(n) // 32].astype(np.int64), np.arange(n) % 32
            kv.append([np.asarray(oracle.dequantize(
                c.cpu().numpy()[ids, :, slot].reshape(-1), s.cpu().numpy()[ids, :, slot].reshape(-1),
                n, head_dim, 16, fmt, G_ONE, out_bf16=False), np.float64).reshape(n, 1, head_dim)
                for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))])
        size = 448.0 if fmt == mx.E4M3 else 122880.0
        q = normal_bf16((2, 70, 4, head_dim), 5, cuda_device, sigma=3.0 / size)
        check_attention(cache, table, lengths, [70, 33], kv, q, scale=0.05)


@pytest.mark.parametrize("sigma,scale", ((1e-30, 1e30), (1e30, 1e-30), (40.0, None), (0.0, None)))
def test_query_ranges(cuda_device, sigma, scale):
    """Tiny and huge queries, scores in the hundreds, all-zero rows; a row whose values span 2^24; a
    negative scale, and none."""
    rng = np.random.default_rng(6)
    lengths = [150, 90]
    table, pages = pages_for(lengths, 16, 0, rng)
    cache = poisoned(pages, 2, 128, 16, 32, mx.E4M3, G_ONE, G_ONE, rng, cuda_device)
    kv = fill(cache, table, lengths, rng)
    q = normal_bf16((2, 40, 4, 128), 7, cuda_device, sigma=sigma)
    q[0, 0, 0] *= torch.exp2(torch.arange(128, device=cuda_device) % 25 - 24.0)
    q[0, 1, 3] = 0
    s = 128 ** -0.5 if scale is None else scale * 128 ** -0.5
    check_attention(cache, table, lengths, None, kv, q, scale=s)
    check_attention(cache, table, lengths, [40, 37], kv, q, scale=-s)
    check_attention(cache, table, lengths, None, kv, q, scale=0.0)


@pytest.mark.parametrize("head_dim", (64, 256))
def test_one_bad_query_row_stays_alone(cuda_device, head_dim):
    rng = np.random.default_rng(8)
    cache, table, kv = setup([200], 1, head_dim, 16, 32, mx.E4M3, rng, cuda_device)
    q = normal_bf16((1, 150, 2, head_dim), 9, cuda_device)
    args = (i32(table, cuda_device), i32([200], cuda_device))
    ref = mx.cache_attention(cache, q, *args)
    bad = q.clone()
    bad[0, 3, 1, 5], bad[0, 149, 0, 0] = torch.nan, torch.inf
    out = mx.cache_attention(cache, bad, *args)
    keep = torch.ones(1, 150, 2, dtype=torch.bool)
    keep[0, 3, 1] = keep[0, 149, 0] = False
    assert torch.equal(out[keep], ref[keep]) and out[0, 3, 1].isnan().all()


@pytest.mark.parametrize("tokens", (1, 40))
@pytest.mark.parametrize("batch", (1, 5, 33, 130, 600))
def test_many_sequences(cuda_device, batch, tokens):
    """Every way in which a block's threads add the sequences up; empty ones among them."""
    rng = np.random.default_rng(batch)
    lengths = [0 if i % 7 == 3 else int(n) for i, n in enumerate(rng.integers(1, 90, batch))]
    counts = [min(n, tokens) if i % 5 else min(n, 1) for i, n in enumerate(lengths)]
    cache, table, kv = setup(lengths, 1, 64, 16, 32, mx.E4M3, rng, cuda_device)
    q = normal_bf16((batch, tokens, 2, 64), batch, cuda_device)
    check_attention(cache, table, lengths, counts, kv, q, scale=scale_for(cache))


@pytest.mark.parametrize("head_dim,heads", ((128, 16), (256, 7)))
def test_many_tiles(cuda_device, head_dim, heads):
    """More row tiles than a warp looks at at once."""
    rng = np.random.default_rng(head_dim)
    lengths, counts = [900, 710], [690, 700]
    cache, table, kv = setup(lengths, 1, head_dim, 64, 32, mx.UE5M3, rng, cuda_device)
    q = normal_bf16((2, 700, heads, head_dim), 2, cuda_device)
    check_attention(cache, table, lengths, counts, kv, q, scale=scale_for(cache))


@pytest.mark.parametrize("tokens", (1, 20, 40, 260))
def test_one_segment_in_many_pieces(cuda_device, tokens):
    """One head over a long sequence: every thread block has a piece of the same rows."""
    rng = np.random.default_rng(tokens)
    lengths = [33333]
    cache, table, kv = setup(lengths, 1, 64, 128, 64, mx.E4M3, rng, cuda_device)
    q = normal_bf16((1, tokens, 1, 64), tokens, cuda_device)
    check_attention(cache, table, lengths, None, kv, q, scale=scale_for(cache))


def test_trees_over_short_sequences(cuda_device):
    """64 drafted tokens, sequences that begin with them or end in a chunk of them."""
    rng = np.random.default_rng(10)
    lengths, counts = [64, 65, 130, 200, 191], [64, 64, 63, 64, 1]
    cache, table, kv = setup(lengths, 2, 128, 16, 16, mx.E4M3, rng, cuda_device)
    tree = np.stack([random_tree(rng, 64) for _ in lengths])
    tree[1, 5] = 0  # a token that sees the old positions only
    q = normal_bf16((5, 64, 8, 128), 11, cuda_device)
    check_attention(cache, table, lengths, counts, kv, q, tree=tree, scale=scale_for(cache))


@pytest.mark.parametrize("tokens", (1, 40))
def test_out_in_place_of_q(cuda_device, tokens):
    rng = np.random.default_rng(12)
    lengths = [3000, 77, 500]
    cache, table, kv = setup(lengths, 2, 128, 32, 32, mx.E4M3, rng, cuda_device)
    q = normal_bf16((3, tokens, 16, 128), 13, cuda_device)
    args = (i32(table, cuda_device), i32(lengths, cuda_device))
    ref = mx.cache_attention(cache, q, *args)
    assert mx.cache_attention(cache, q, *args, out=q) is q and torch.equal(q, ref)


def test_captured_tiles(cuda_device):
    """Two calls in one graph; lengths, counts and queries change between replays, while another
    stream uses the same cache."""
    rng = np.random.default_rng(14)
    cache, table, kv = setup([1500, 1500], 2, 128, 64, 32, mx.E4M3, rng, cuda_device)
    tb, ln, ct = i32(table, cuda_device), i32([60, 60], cuda_device), i32([50, 50], cuda_device)
    q = normal_bf16((2, 50, 16, 128), 15, cuda_device)
    out, out2 = torch.zeros_like(q), torch.zeros_like(q)

    def once():
        mx.cache_attention(cache, q, tb, ln, count=ct, out=out)
        mx.cache_attention(cache, out, tb, ln, count=ct, out=out2)
    once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    side = torch.cuda.Stream()
    side_q = normal_bf16((2, 50, 16, 128), 16, cuda_device)
    torch.cuda.synchronize()
    for n, c in (([60, 50], [50, 50]), ([1500, 0], [50, 0]), ([700, 1499], [1, 33])):
        ln.copy_(i32(n, cuda_device)), ct.copy_(i32(c, cuda_device))
        q.normal_()
        out.zero_(), out2.zero_()
        torch.cuda.synchronize()
        mx.cache_attention(cache, side_q, tb, ln, count=ct, stream=side)
        graph.replay()
        torch.cuda.synchronize()
        got, got2 = out.clone(), out2.clone()
        out.zero_(), out2.zero_()
        once()
        assert torch.equal(got, out) and torch.equal(got2, out2) and got.any()


def test_attention_beyond_4_gib(cuda_device):
    """Pages whose bytes lie beyond 2^32 of the codes give the bits of a small pool."""
    page, kvh, dim, n = 256, 8, 256, 300
    pages = (1 << 32) // (kvh * page * dim // 2) + 4
    k, v = (normal_bf16((1, n, kvh, dim), s, cuda_device) for s in (1, 2))
    zero, ln = i32([0], cuda_device), i32([n], cuda_device)
    got = []
    for pool, ids in ((4, [[1, 0]]), (pages, [[pages - 1, pages - 3]])):
        cache = mx.KVCache(pool, kvh, dim, page_size=page, block=64, fmt="e4m3", device=cuda_device)
        table = i32(ids, cuda_device)
        mx.cache_append(cache, k, v, table, zero)
        for tokens in (1, 40):
            q = normal_bf16((1, tokens, 16, dim), tokens, cuda_device)
            got.append(mx.cache_attention(cache, q, table, ln))
        del cache
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3]) and got[0].any()


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("batch,tokens,kvh,dim", ((1, 1, 1, 64), (1, 100, 4, 256), (7, 333, 5, 64),
                                                 (64, 1, 8, 128), (2, 3000, 3, 64)))
def test_append_and_read_sizes(cuda_device, batch, tokens, kvh, dim, dtype):
    """From one item per block to full tiles."""
    rng = np.random.default_rng(tokens)
    table, pages = pages_for([tokens + 3] * batch, 32, 1, rng)
    cache = poisoned(pages, kvh, dim, 32, 32, mx.E4M3, G_ONE, G_ONE, rng, cuda_device)
    k, v = (normal_bf16((batch, tokens, kvh, dim), s, cuda_device).to(dtype) for s in (1, 2))
    if dtype == torch.float32:
        k, v = k * 1.0009765625, v / 3
    start = [b % 4 for b in range(batch)]
    check_append(cache, table, k, v, start, None, cuda_device)
    ko, vo = mx.cache_read(cache, i32(table, cuda_device), i32(start, cuda_device), None, tokens,
                           out_dtype=dtype)
    for x, y in ((k, ko), (v, vo)):
        c, s = mx.quantize(x, 32, "e4m3")
        assert torch.equal(mx.dequantize(c, s, 32, "e4m3", out_dtype=dtype), y)
