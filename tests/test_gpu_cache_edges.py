"""cache_attention at the borders of what its kernels skip or round: trees whose tokens do not see the
first drafted one, at every place of that one in a masked run (bounds: cache_helpers.attend)."""
import numpy as np
import pytest
import torch

import fp4_microscaling_tensor_b200 as mx
from cache_helpers import (G_ONE, check_attention, fill, normal_bf16, pages_for, poisoned,
                           random_tree)

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
