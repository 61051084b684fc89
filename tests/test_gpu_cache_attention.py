"""cache_attention against float64 attention over the oracle's values (bounds: cache_helpers.attend).
The caches' other slots hold NaN or the largest scales, so anything read from outside a sequence
shows."""
import numpy as np
import pytest
import torch

import fp4_microscaling_tensor_b200 as mx
from cache_helpers import (G_ONE, check_attention, fill, i32, normal_bf16, pages_for, poisoned,
                           random_tree)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def nobody_gave_up():
    """No bounded wait of a tensor-core kernel runs out."""
    yield
    assert mx.matmul_gave_up() == 0


def setup(lengths, kvh, head_dim, page, block, fmt, rng, device, g=None, sigma=1.0):
    g = g or ((0x0155, 0x2E66) if fmt == mx.UE5M3 else (G_ONE, 0x2E66))
    table, pages = pages_for(lengths, page, 2, rng)
    cache = poisoned(pages, kvh, head_dim, page, block, fmt, *g, rng, device)
    return cache, table, fill(cache, table, lengths, rng, sigma)


def scale_for(cache):
    """1 / sqrt(d) for keys of unit size before the factor g."""
    import oracle
    return cache.head_dim ** -0.5 / oracle.fp16_value(cache.k_g)


EDGES = [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 1025]


@pytest.mark.parametrize("fmt", (mx.E4M3, mx.UE5M3))
@pytest.mark.parametrize("head_dim,block,page", ((64, 16, 16), (64, 64, 64), (128, 16, 32),
                                                 (128, 32, 64), (128, 128, 256), (256, 16, 16),
                                                 (256, 32, 128), (256, 128, 64)))
def test_single_tokens(cuda_device, head_dim, block, page, fmt):
    rng = np.random.default_rng(head_dim + block)
    cache, table, kv = setup(EDGES, 2, head_dim, page, block, fmt, rng, cuda_device)
    q = normal_bf16((len(EDGES), 1, 16, head_dim), 1, cuda_device)
    check_attention(cache, table, EDGES, None, kv, q, scale=scale_for(cache))


@pytest.mark.parametrize("group", (1, 2, 3, 4, 5, 7, 8, 12, 16, 17, 33, 64))
def test_head_groups(cuda_device, group):
    rng = np.random.default_rng(group)
    lengths = [77, 300, 5]
    cache, table, kv = setup(lengths, 3, 64, 32, 32, mx.E4M3, rng, cuda_device)
    q = normal_bf16((3, 2, 3 * group, 64), group, cuda_device)
    check_attention(cache, table, lengths, [2, 2, 1], kv, q, scale=scale_for(cache))


@pytest.mark.parametrize("head_dim", (64, 128, 256))
@pytest.mark.parametrize("tokens", (2, 3, 4, 9, 16, 33, 70, 130, 300))
def test_chains(cuda_device, tokens, head_dim):
    """Chains from two tokens to chunks of a prompt; counts from none to all, sequences that hold
    nothing but the chain."""
    rng = np.random.default_rng(tokens)
    counts = [tokens, tokens - 1, 0, 1, tokens]
    lengths = [tokens, tokens + 64, 30, 1, 500 + tokens]
    cache, table, kv = setup(lengths, 2, head_dim, 64, 32, mx.UE5M3, rng, cuda_device)
    q = normal_bf16((5, tokens, 8, head_dim), 2, cuda_device)
    check_attention(cache, table, lengths, counts, kv, q, scale=scale_for(cache))


@pytest.mark.parametrize("head_dim", (64, 128, 256))
@pytest.mark.parametrize("tokens", (1, 2, 7, 31, 48, 63, 64))
def test_trees(cuda_device, tokens, head_dim):
    """Random ancestor words, several roots, bit 63; tokens that see nothing of the tree (and, in a
    sequence that holds nothing else, nothing at all)."""
    rng = np.random.default_rng(tokens)
    counts = [tokens, max(1, tokens - 3), tokens, tokens]
    lengths = [700, 129, tokens, 64 + tokens]
    tree = np.stack([random_tree(rng, tokens, r) for r in (1, 3, 1, 1)])
    tree[2, tokens // 2] = 0     # sees nothing
    tree[3, :] = 0               # sees what came before only
    tree[0, -1] |= np.uint64(1 << 63)  # a token that is not there, unless tokens is 64
    cache, table, kv = setup(lengths, 2, head_dim, 32, 16 if head_dim == 64 else 32, mx.E4M3, rng,
                             cuda_device)
    q = normal_bf16((4, tokens, 16, head_dim), 3, cuda_device)
    out, lse = check_attention(cache, table, lengths, counts, kv, q, tree=tree, scale=scale_for(cache))
    assert not out[2, tokens // 2].any() and (lse[2, tokens // 2] == -torch.inf).all()


def test_empty_sequences_and_counts(cuda_device):
    """Lengths of zero; counts above the length (the missing positions are nobody's) and outside
    [0, tokens]."""
    rng = np.random.default_rng(0)
    cache, table, kv = setup([0, 40, 3], 1, 128, 16, 32, mx.E4M3, rng, cuda_device)
    q = normal_bf16((3, 5, 4, 128), 5, cuda_device)
    out, lse = mx.cache_attention(cache, q, i32(table, cuda_device), i32([0, 40, 3], cuda_device),
                                  count=i32([5, 99, 5], cuda_device), lse=True,
                                  scale=scale_for(cache))
    assert not out[0].any() and (lse[0] == -torch.inf).all()
    assert not out[2, :2].any() and (lse[2, :2] == -torch.inf).all()  # positions -2 and -1
    check_attention(cache, table, [0, 40, 3], [0, 5, 3], kv,
                    torch.cat((q[:2], q[2:].roll(-2, 1))), scale=scale_for(cache))
    ref = mx.cache_attention(cache, q[2:, 2:], i32(table[2:], cuda_device), i32([3], cuda_device),
                             scale=scale_for(cache))
    assert torch.equal(out[2:, 2:], ref)
    none = mx.cache_attention(cache, q, i32(table, cuda_device), i32([-4, 40, 3], cuda_device),
                              count=i32([1, -7, 0], cuda_device), scale=scale_for(cache))
    assert not none.any()


def test_positions_without_a_page_are_not_attended(cuda_device):
    rng = np.random.default_rng(1)
    lengths = [100, 260, 64]
    cache, table, kv = setup(lengths, 2, 128, 16, 32, mx.UE5M3, rng, cuda_device)
    table[0, 2], table[1, 0], table[2, 3] = -1, cache.pages, np.iinfo(np.int32).min
    q = normal_bf16((3, 1, 8, 128), 8, cuda_device)
    out, lse = mx.cache_attention(cache, q, i32(table, cuda_device), i32(lengths, cuda_device),
                                  lse=True, scale=scale_for(cache))
    from cache_helpers import assert_close, attend
    for b, n in enumerate(lengths):
        ids = table[b, np.arange(n) // 16]
        mask = ((ids >= 0) & (ids < cache.pages))[None]
        ref = attend(q[b].float().cpu().numpy().astype(np.float64), *kv[b], mask, scale_for(cache))
        assert_close(out[b].float().cpu().numpy(), ref[0], ref[2], f"sequence {b}")
        assert_close(lse[b].cpu().numpy(), ref[1], ref[3], f"sequence {b} lse")
    # a length beyond what the table reaches is cut to it
    long = mx.cache_attention(cache, q, i32(table, cuda_device), i32([10 ** 9] * 3, cuda_device),
                              scale=scale_for(cache))
    cut = mx.cache_attention(cache, q, i32(table, cuda_device),
                             i32([table.shape[1] * 16] * 3, cuda_device), scale=scale_for(cache))
    assert torch.equal(long[1], cut[1])


def test_every_scale_code_and_code_byte(cuda_device):
    """Random codes with every finite scale code: small q keeps the scores in range."""
    import oracle
    rng = np.random.default_rng(2)
    for fmt, top in ((mx.E4M3, 0x7F), (mx.UE5M3, 0x100)):
        lengths = [190, 33]
        table, pages = pages_for(lengths, 32, 0, rng)
        cache = poisoned(pages, 2, 128, 32, 16, fmt, G_ONE, G_ONE, rng, cuda_device)
        for t in (cache.k_scales, cache.v_scales):
            t.copy_(torch.from_numpy(rng.integers(0, top, tuple(t.shape), dtype=np.uint8)))
        kv = []
        for b, n in enumerate(lengths):
            ids, slot = table[b, np.arange(n) // 32].astype(np.int64), np.arange(n) % 32
            kv.append([np.asarray(oracle.dequantize(
                c.cpu().numpy()[ids, :, slot].reshape(-1), s.cpu().numpy()[ids, :, slot].reshape(-1),
                n * 2, 128, 16, fmt, G_ONE, out_bf16=False), np.float64).reshape(n, 2, 128)
                for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))])
        size = 448.0 if fmt == mx.E4M3 else 122880.0
        q = normal_bf16((2, 3, 8, 128), 6, cuda_device, sigma=3.0 / size)
        check_attention(cache, table, lengths, [3, 2], kv, q, scale=0.05)


@pytest.mark.parametrize("sigma,scale", ((1e-30, 1e30), (1e30, 1e-30), (40.0, None), (0.0, None)))
def test_query_ranges(cuda_device, sigma, scale):
    """Tiny and huge queries, scores in the hundreds, all-zero rows; values of one row that span 2^24;
    a negative scale."""
    rng = np.random.default_rng(3)
    lengths = [150, 40]
    cache, table, kv = setup(lengths, 2, 128, 16, 32, mx.E4M3, rng, cuda_device, g=(G_ONE, G_ONE))
    q = normal_bf16((2, 2, 8, 128), 7, cuda_device, sigma=sigma)
    q[0, 0, 0] *= torch.exp2(torch.arange(128, device=cuda_device) % 25 - 24.0)
    q[0, 1, 3] = 0
    s = 128 ** -0.5 if scale is None else scale * 128 ** -0.5
    check_attention(cache, table, lengths, None, kv, q, scale=s)
    check_attention(cache, table, lengths, [1, 2], kv, q, scale=-s)


def test_one_bad_query_row_stays_alone(cuda_device):
    """A NaN or infinity in one head's query reaches that row only."""
    rng = np.random.default_rng(8)
    cache, table, kv = setup([90], 2, 64, 16, 32, mx.E4M3, rng, cuda_device)
    q = normal_bf16((1, 2, 8, 64), 9, cuda_device)
    args = (i32(table, cuda_device), i32([90], cuda_device))
    ref = mx.cache_attention(cache, q, *args)
    bad = q.clone()
    bad[0, 0, 1, 5], bad[0, 1, 6, 0] = torch.nan, torch.inf
    out = mx.cache_attention(cache, bad, *args)
    keep = torch.ones(1, 2, 8, dtype=torch.bool)
    keep[0, 0, 1] = keep[0, 1, 6] = False
    assert torch.equal(out[keep], ref[keep]) and out[0, 0, 1].isnan().all()


def test_strides_and_padding(cuda_device):
    """q a slice of a fused projection, out a slice of a wider tensor, heads before tokens."""
    rng = np.random.default_rng(10)
    lengths = [300, 70]
    cache, table, kv = setup(lengths, 4, 128, 64, 16, mx.UE5M3, rng, cuda_device)
    for tokens in (1, 40):
        qkv = normal_bf16((2, tokens, 24, 128), tokens, cuda_device)
        q = qkv[:, :, :16]
        ref, _ = check_attention(cache, table, lengths, None, kv, q, scale=scale_for(cache))
        wide = torch.full((2, 20, tokens, 128), 3.0, dtype=torch.bfloat16, device=cuda_device)
        out = mx.cache_attention(cache, q.transpose(1, 2).contiguous().transpose(1, 2),
                                 i32(table, cuda_device), i32(lengths, cuda_device),
                                 out=wide[:, 2:18].transpose(1, 2), scale=scale_for(cache))
        assert torch.equal(out, ref)
        assert (wide[:, :2] == 3).all() and (wide[:, 18:] == 3).all()


@pytest.mark.parametrize("tokens", (1, 24))
def test_long_sequences_and_repeats(cuda_device, tokens):
    """A long and a short sequence in one call (the long one is split over many thread blocks);
    repeated calls give the same bits, whatever else runs."""
    rng = np.random.default_rng(11)
    lengths = [20000, 31, 9001]
    cache, table, kv = setup(lengths, 1, 64, 64, 32, mx.E4M3, rng, cuda_device)
    q = normal_bf16((3, tokens, 4, 64), 12, cuda_device)
    first = check_attention(cache, table, lengths, None, kv, q, scale=scale_for(cache))
    side = torch.cuda.Stream()
    args = dict(lse=True, scale=scale_for(cache))
    ids = (i32(table, cuda_device), i32(lengths, cuda_device))
    torch.cuda.synchronize()
    for _ in range(5):
        other = mx.cache_attention(cache, q, *ids, stream=side, **args)
        here = mx.cache_attention(cache, q, *ids, **args)
        torch.cuda.synchronize()
        for x in (here, other):
            assert torch.equal(x[0], first[0]) and torch.equal(x[1], first[1])


def test_decoding_together(cuda_device):
    """The operators as a decoder uses them: a padded prompt enters the cache and attends to it,
    single tokens follow, a tree of drafts is verified and its accepted path appended behind each
    other; at each step attention equals the float64 one over everything appended so far."""
    rng = np.random.default_rng(12)
    kvh, heads, d, page, block = 2, 8, 64, 16, 32
    prompts, room = [45, 17, 33], 100
    table, pages = pages_for([room] * 3, page, 2, rng)
    cache = poisoned(pages, kvh, d, page, block, mx.E4M3, G_ONE, G_ONE, rng, cuda_device)
    tb = i32(table, cuda_device)
    held = [[np.zeros((0, kvh, d)), np.zeros((0, kvh, d))] for _ in range(3)]

    def values(x):
        c, s = mx.quantize(x.contiguous(), block, "e4m3")
        return mx.dequantize(c, s, block, "e4m3").float().cpu().numpy().astype(np.float64)

    def step(tokens, counts, tree=None, seed=0):
        qkv = normal_bf16((3, tokens, heads + 2 * kvh, d), 100 + seed, cuda_device)
        k, v = qkv[:, :, heads:heads + kvh], qkv[:, :, heads + kvh:]
        start = [h[0].shape[0] for h in held]
        mx.cache_append(cache, k, v, tb, i32(start, cuda_device), count=i32(counts, cuda_device))
        now = [[np.concatenate((h[i], values(x)[b, :counts[b]])) for i, x in enumerate((k, v))]
               for b, h in enumerate(held)]
        lengths = [s + c for s, c in zip(start, counts)]
        check_attention(cache, table, lengths, counts, now, qkv[:, :, :heads], tree=tree)
        return k, v, start, now

    held = step(max(prompts), prompts, seed=0)[3]
    for i in range(3):
        held = step(1, [1, 1, 1], seed=1 + i)[3]
    tree = np.stack([random_tree(rng, 12) for _ in range(3)])
    k, v, start, _ = step(12, [12, 12, 12], tree=tree, seed=9)
    paths = []
    for b in range(3):
        leaf = 11 - b
        paths.append([j for j in range(12) if (int(tree[b, leaf]) >> j) & 1])
    most = max(len(p) for p in paths)
    pick = torch.tensor([p + [0] * (most - len(p)) for p in paths], device=cuda_device)
    at = pick[:, :, None, None].expand(-1, -1, kvh, d)
    mx.cache_append(cache, k.gather(1, at), v.gather(1, at), tb, i32(start, cuda_device),
                    count=i32([len(p) for p in paths], cuda_device))
    held = [[np.concatenate((h[i], values(x)[b, paths[b]])) for i, x in enumerate((k, v))]
            for b, h in enumerate(held)]
    step(1, [1, 0, 1], seed=20)


def test_captured_and_replayed(cuda_device):
    """Append and attention in one graph; lengths, table and inputs change between replays."""
    rng = np.random.default_rng(13)
    lengths = [130, 64]
    cache, table, kv = setup([400, 400], 2, 128, 64, 32, mx.E4M3, rng, cuda_device, g=(G_ONE, G_ONE))
    tb, ln = i32(table, cuda_device), i32(lengths, cuda_device)
    st = torch.zeros_like(ln)
    x = torch.empty(2, 1, 12, 128, dtype=torch.bfloat16, device=cuda_device)
    x.normal_()

    def once():
        torch.sub(ln, 1, out=st)
        mx.cache_append(cache, x[:, :, 8:10], x[:, :, 10:], tb, st)
        return mx.cache_attention(cache, x[:, :, :8], tb, ln)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = once()
    for n in ([131, 65], [399, 66], [1, 400]):
        ln.copy_(i32(n, cuda_device))
        x.normal_()
        graph.replay()
        got = out.clone()
        assert torch.equal(got, once()) and got.any()
