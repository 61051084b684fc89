"""cache_attention at the borders of what its kernels skip or round: trees whose tokens do not see the
first drafted one, at every place of that one in a masked run; scores of any size float32 holds; many
small weights beside a few large ones (bounds: cache_helpers.attend)."""
import numpy as np
import pytest
import torch

import fp4_microscaling_tensor_b200 as mx
from cache_helpers import (G_ONE, assert_close, chain_mask, check_attention, fill, i32,
                           normal_bf16, pages_for, place, poisoned, random_tree)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def nobody_gave_up():
    """No bounded wait of a tensor-core kernel runs out."""
    yield
    assert mx.matmul_gave_up() == 0


def setup(lengths, kvh, head_dim, page, rng, device):
    table, pages = pages_for(lengths, page, 2, rng)
    cache = poisoned(pages, kvh, head_dim, page, 32, mx.E4M3, G_ONE, G_ONE, rng, device)
    return cache, table, fill(cache, table, lengths, rng)


def forest(rng, tokens):
    """Words of several trees: the first token sees itself only, the last but one nothing, the last
    itself only; the others hang below one of `tokens` / 3 roots."""
    words = random_tree(rng, tokens, max(1, tokens // 3))
    words[-2:] = 0, 1 << (tokens - 1)
    return words


@pytest.mark.parametrize("head_dim,tokens,heads", ((64, 4, 1), (64, 4, 8), (128, 4, 4), (256, 4, 2),
                                                   (64, 36, 1), (128, 36, 1), (256, 36, 1),
                                                   (128, 48, 6)))
def test_forests_behind_any_length(cuda_device, head_dim, tokens, heads):
    """Words without bit 0, the drafted tokens behind 0 to 160 and about 256 old positions: rows that
    reach both kernels, one tile and more."""
    rng = np.random.default_rng(head_dim + tokens + heads)
    lengths = [base + tokens for base in [*range(161), 254, 255, 256, 383, 384]]
    cache, table, kv = setup(lengths, 1, head_dim, 16, rng, cuda_device)
    tree = np.stack([forest(rng, tokens) for _ in lengths])
    tree[::3] = np.uint64(1) << np.arange(tokens, dtype=np.uint64)  # every token sees itself only
    q = normal_bf16((len(lengths), tokens, heads, head_dim), 1, cuda_device)
    check_attention(cache, table, lengths, None, kv, q, tree=tree)


def test_forests_of_equal_sequences(cuda_device):
    """More segments than thread blocks: 64 sequences of 131 positions, 8 key/value heads."""
    rng = np.random.default_rng(5)
    lengths = [131] * 64
    cache, table, kv = setup(lengths, 8, 64, 16, rng, cuda_device)
    tree = np.tile(np.uint64(1) << np.arange(4, dtype=np.uint64), (64, 1))
    q = normal_bf16((64, 4, 8, 64), 2, cuda_device)
    check_attention(cache, table, lengths, None, kv, q, tree=tree)


EXPONENTS = (10, 17, 20, 23, 26, 29, 40, 90, 115)  # of the queries' size


@pytest.mark.parametrize("tokens", (2, 40))
@pytest.mark.parametrize("head_dim", (64, 128, 256))
def test_one_score_far_above_the_rest(cuda_device, head_dim, tokens):
    """Huge queries: the largest score leads by more than its own float32 error, so a row is that
    position's values, and lse its score."""
    rng = np.random.default_rng(head_dim)
    lengths = [300, 2900]
    cache, table, kv = setup(lengths, 1, head_dim, 64, rng, cuda_device)
    ids, ln = i32(table, cuda_device), i32(lengths, cuda_device)
    checked = 0
    for e in EXPONENTS:
        q = normal_bf16((2, tokens, 4, head_dim), e, cuda_device) * 2.0 ** e
        out, lse = mx.cache_attention(cache, q, ids, ln, lse=True)
        qn, on, ln_ = (x.float().cpu().numpy().astype(np.float64) for x in (q, out, lse))
        assert np.isfinite(on).all() and np.isfinite(ln_).all(), e
        for b, n in enumerate(lengths):
            k, v = (x[:, 0] for x in kv[b])
            for h in range(4):
                s = qn[b, :, h] @ k.T * head_dim ** -0.5
                off = (head_dim * 2.0 ** -23 * head_dim ** -0.5 * (np.abs(qn[b, :, h]) @ np.abs(k).T)
                       + np.abs(s) * 2.0 ** -22).max(-1)
                s = np.where(chain_mask(n, tokens), s, -np.inf)
                top = s.argmax(-1)
                order = np.sort(s, -1)
                # 30: what the others add is below n 2^-40
                clear = order[:, -1] - order[:, -2] > 2 * off + 30
                checked += clear.sum()
                want = v[top[clear]]
                # the one weight in 11 bits, and bf16
                assert_close(on[b, clear, h], want, (2.0 ** -8 + 2.0 ** -10) * np.abs(want) + 1e-9,
                             f"2^{e}, sequence {b}")
                assert_close(ln_[b, clear, h], order[clear, -1],
                             off[clear] + np.abs(order[clear, -1]) * 2.0 ** -22, f"2^{e} lse")
    assert checked > 0.9 * 8 * tokens * (len(EXPONENTS) - 1)  # (at 2^10 some rows are closer)


@pytest.mark.parametrize("tokens", (1, 40))
@pytest.mark.parametrize("fmt", (mx.E4M3, mx.UE5M3))
@pytest.mark.parametrize("head_dim", (64, 128, 256))
def test_equal_scores_of_any_size(cuda_device, head_dim, fmt, tokens):
    """Every position has the same key, so every row is a mean of values whatever the score's size and
    sign: what rounds the score must not reach the weights."""
    rng = np.random.default_rng(head_dim)
    lengths = [40, 2000]
    table, pages = pages_for(lengths, 32, 1, rng)
    cache = poisoned(pages, 1, head_dim, 32, 32, fmt, G_ONE, G_ONE, rng, cuda_device)
    kv = fill(cache, table, lengths, rng)
    one = 0x38 if fmt == mx.E4M3 else 0x78  # the scale 1
    code = rng.integers(0, 256, head_dim // 2, dtype=np.uint8) & 0x77  # magnitudes only
    mags = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    key = np.stack((mags[code & 7], mags[code >> 4]), -1).reshape(-1)
    for b, n in enumerate(lengths):
        place(cache, table, b, np.arange(n), "k", np.tile(code, (n, 1, 1)),
              np.full((n, 1, head_dim // 32), one, np.uint8))
    ids, ln = i32(table, cuda_device), i32(lengths, cuda_device)
    for e in EXPONENTS:
        for sign in (1, -1):
            q = torch.full((2, tokens, 3, head_dim), sign * 1.0078125 * 2.0 ** e,
                           dtype=torch.bfloat16, device=cuda_device)
            q[:, :, 1] *= 1.0234375
            out, lse = mx.cache_attention(cache, q, ids, ln, lse=True, scale=0.1234567)
            on, ln_ = (x.double().cpu().numpy() for x in (out, lse))
            for b, n in enumerate(lengths):
                seen = n - tokens + 1 + np.arange(tokens)
                v = kv[b][1][:, 0]
                mean, mag = (np.cumsum(x, 0)[seen - 1] / seen[:, None] for x in (v, np.abs(v)))
                tol = (2.0 ** -11 + 2 * n * 2.0 ** -23) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(mean)
                for h in range(3):
                    assert_close(on[b, :, h], mean, tol, f"{sign} 2^{e}, sequence {b}")
                    s = float(q[b, 0, h, 0]) * key.sum() * float(np.float32(0.1234567))
                    ref = s + np.log(seen)
                    assert_close(ln_[b, :, h], ref, 2.0 ** -21 + n * 2.0 ** -23 + np.abs(ref) *
                                 (2.0 ** -22 + head_dim * 2.0 ** -23), f"{sign} 2^{e} lse")


@pytest.mark.parametrize("tokens", (1, 40))
def test_scores_too_small_to_tell_apart(cuda_device, tokens):
    """A scale so small that all weights are equal, behind positions that have no page: the first
    positions that a warp sees may give it no score at all."""
    rng = np.random.default_rng(3)
    lengths = [700, 90]
    cache, table, kv = setup(lengths, 1, 64, 16, rng, cuda_device)
    table[:, :5] = -1
    q = normal_bf16((2, tokens, 4, 64), 4, cuda_device)
    out, lse = mx.cache_attention(cache, q, i32(table, cuda_device), i32(lengths, cuda_device),
                                  lse=True, scale=1e-38)
    for b, n in enumerate(lengths):
        for t in range(tokens):
            v = kv[b][1][80:n - tokens + t + 1, 0]
            if not len(v):
                assert not out[b, t].any() and torch.isneginf(lse[b, t]).all()
                continue
            mean, mag = v.mean(0), np.abs(v).mean(0)
            tol = (2.0 ** -11 + 2 * n * 2.0 ** -23) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(mean)
            for h in range(4):
                assert_close(out[b, t, h].double().cpu().numpy(), mean, tol, f"sequence {b}, {t}")
            assert (lse[b, t] - np.log(len(v))).abs().max() < 2.0 ** -20 + n * 2.0 ** -23


@pytest.mark.parametrize("batch,tokens", ((444, 1), (100, 1), (148, 40), (30, 300)))
@pytest.mark.parametrize("head_dim,fmt", ((64, mx.E4M3), (128, mx.UE5M3), (256, mx.E4M3)))
def test_many_small_weights_beside_a_few_large_ones(cuda_device, head_dim, fmt, batch, tokens):
    """A position in 8192 has a score x above the rest (in log2) and a value of 0, the rest have 1:
    what the rest add up to must not be lost.  (All sequences share their pages; x reaches to where a
    weight is 2^-29 of the largest.)

    Bound: a weight, relative to the largest, is rounded by 2^-11 of itself and 2^-32; the rest as in
    cache_helpers.attend, with scores that are exact but for their scaling (2^-22 x) and the
    exponential (2^-21)."""
    n, page = 131072 if batch == 444 else 65536, 256
    one = 0x38 if fmt == mx.E4M3 else 0x78  # the scale 1
    shape = (n // page, 1, page, head_dim // 2)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device=cuda_device) for _ in range(2))
    sink = torch.arange(n, device=cuda_device) % 8192 == 5
    k.view(n, -1)[sink] = 0x22    # 1, 1
    v.view(n, -1)[~sink] = 0x22
    scales = torch.full((n // page, 1, page, head_dim // 32), one, dtype=torch.uint8,
                        device=cuda_device)
    cache = mx.KVCache.from_buffers(k, scales, v, scales, fmt=fmt)
    table = torch.arange(n // page, dtype=torch.int32, device=cuda_device).expand(batch, -1)
    q = torch.ones(batch, tokens, 1, head_dim, dtype=torch.bfloat16, device=cuda_device)
    seen = n - tokens + 1 + np.arange(tokens)
    sinks = (seen - 6) // 8192 + 1
    for x in (20.0, 24.9, 25.1, 27.0, 29.0):
        scale = float(np.float32(x * np.log(2) / head_dim))
        out, lse = mx.cache_attention(cache, q, table, i32([n] * batch, cuda_device), lse=True,
                                      scale=scale)
        w = np.exp(-scale * head_dim)
        total = sinks + (seen - sinks) * w
        want = (seen - sinks) * w / total
        e = 2.0 ** -22 * x + 2.0 ** -21
        tol = (2 * e + 2.0 ** -11 + 2 * n * 2.0 ** -23) * want + n * 2.0 ** -32 / total
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want
        on, ln = (t.double().cpu().numpy()[:, :, 0] for t in (out, lse))
        for b in range(batch):
            assert_close(on[b], np.tile(want[:, None], head_dim), tol[:, None], f"2^-{x}, {b}")
            assert_close(ln[b], scale * head_dim + np.log(total), e + n * 2.0 ** -23 + 2.0 ** -17,
                         f"2^-{x}, {b} lse")


def test_the_count_of_ended_waits_is_read_behind_every_stream(cuda_device):
    """matmul_gave_up synchronizes the device: work on a stream that the default one does not wait for
    is over when it returns, so nothing that the work would add is missed."""
    a = torch.randn(8192, 8192, device=cuda_device).bfloat16()
    side, over = torch.cuda.Stream(), torch.cuda.Event()
    assert mx.matmul_gave_up() == 0  # (a first call loads the kernels, which waits by itself)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(60):  # about 40 ms
            b = a @ a
        over.record()
    assert mx.matmul_gave_up() == 0
    assert over.query()
    del b


@pytest.mark.parametrize("tokens", (1, 40))
def test_streams_by_handle(cuda_device, tokens):
    """A stream's handle, the default stream's (0) too, does what the stream object does."""
    rng = np.random.default_rng(tokens)
    lengths = [300, 90]
    cache, table, kv = setup(lengths, 1, 64, 16, rng, cuda_device)
    q = normal_bf16((2, tokens, 4, 64), 4, cuda_device)
    args = (i32(table, cuda_device), i32(lengths, cuda_device))
    ref = mx.cache_attention(cache, q, *args, lse=True)
    read = mx.cache_read(cache, args[0], i32([0, 0], cuda_device), args[1], 300)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        got = mx.cache_attention(cache, q, *args, lse=True, stream=stream)
        back = mx.cache_read(cache, args[0], i32([0, 0], cuda_device), args[1], 300, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip((*ref, *read), (*got, *back)):
            assert torch.equal(a, b)
