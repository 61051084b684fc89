"""A paged FP4 cache on the host for the cache tests: values by the oracle, attention in float64."""
import numpy as np
import torch

import fp4_microscaling_tensor_b200 as mx
import oracle
from fp4_microscaling_tensor_b200 import inputs

G_ONE = 0x3C00


def pages_for(lengths, page, extra, rng):
    """A table of shuffled page numbers for sequences of these lengths (unused entries -1) and the
    number of pages: `extra` of them belong to nobody."""
    need = [-(-n // page) for n in lengths]
    ids = rng.permutation(sum(need) + extra)
    table = np.full((len(lengths), max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, len(ids)


def poisoned(pages, kv_heads, head_dim, page, block, fmt, kg, vg, rng, device):
    """A cache whose every slot holds random codes and the worst scales: NaN (E4M3) or the largest
    (UE5M3)."""
    bufs = []
    for _ in range(2):
        bufs.append(rng.integers(0, 256, (pages, kv_heads, page, head_dim // 2), dtype=np.uint8))
        bufs.append(np.full((pages, kv_heads, page, head_dim // block),
                            0x7F if fmt == mx.E4M3 else 0xFF, np.uint8))
    return mx.KVCache.from_buffers(*(torch.from_numpy(b).to(device) for b in bufs), fmt=fmt, k_g=kg,
                                   v_g=vg)


def place(cache, table, b, pos, which, codes, scales):
    """Writes codes / scales [n, kv_heads, ...] (numpy) of positions pos of sequence b."""
    ids = torch.from_numpy(table[b, pos // cache.page_size].astype(np.int64)).to(cache.device)
    slot = torch.from_numpy(pos % cache.page_size).to(cache.device)
    c, s = (cache.k_codes, cache.k_scales) if which == "k" else (cache.v_codes, cache.v_scales)
    c[ids, :, slot] = torch.from_numpy(codes).to(cache.device)
    s[ids, :, slot] = torch.from_numpy(scales).to(cache.device)


def fill(cache, table, lengths, rng, sigma=1.0):
    """Fills the sequences' positions with quantized normals (by the oracle).  Returns their values
    in float64: per sequence (k, v) [length, kv_heads, head_dim]."""
    out = []
    for b, n in enumerate(lengths):
        kv = []
        for which, g in (("k", cache.k_g), ("v", cache.v_g)):
            x = (rng.standard_normal((n * cache.kv_heads, cache.head_dim)) * sigma
                 * oracle.fp16_value(g)).astype(np.float32)
            p, s = oracle.quantize(x, n * cache.kv_heads, cache.head_dim, cache.block, cache.fmt, g)
            y = oracle.dequantize(p, s, n * cache.kv_heads, cache.head_dim, cache.block, cache.fmt,
                                  g, out_bf16=False)
            kv.append(np.asarray(y, np.float64).reshape(n, cache.kv_heads, cache.head_dim))
            place(cache, table, b, np.arange(n), which,
                  p.reshape(n, cache.kv_heads, cache.head_dim // 2),
                  s.reshape(n, cache.kv_heads, cache.head_dim // cache.block))
        out.append(kv)
    return out


def chain_mask(length, count):
    base = length - count
    return np.arange(length)[None, :] <= base + np.arange(count)[:, None]


def tree_mask(length, count, words):
    m = np.zeros((count, length), bool)
    base = length - count
    for t in range(count):
        for p in range(length):
            j = p - base
            m[t, p] = j < 0 or bool((int(words[t]) >> j) & 1)
    return m


def attend(q, k, v, mask, scale):
    """float64 attention of q [count, heads, d] over k, v [length, kv_heads, d].  Returns out, lse
    and their bounds.

    Bounds, for n positions.  The kernel's products of a query and a key are exact and summed in
    float32 in an unspecified order: each score is off by at most d 2^-23 scale sum |q k| (twice the
    round-to-nearest bound, allowing truncating adders), plus 2^-22 of itself for its scaling, plus
    2^-21 for the exponential; call the largest of these e.  A weight is then off by a factor
    exp(+-e), and so is the sum of weights: 2 e of A = sum p |v| together.  Rounding the weights to
    binary16 gives 2^-11 A, and 2^-25 max |v| for each weight below the normal range; summing n
    products in float32 n 2^-23 A, the weights' sum as much again; and bf16 outputs 2^-8 |out|.  lse
    is off by e, n 2^-23 and 2^-22 of itself."""
    heads, d = q.shape[1], q.shape[2]
    group = heads // k.shape[1]
    n = k.shape[0]
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    tol, tol_lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for h in range(heads):
        kk, vv = k[:, h // group], v[:, h // group]
        s = q[:, h] @ kk.T * scale
        off = d * 2.0 ** -23 * abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T) + np.abs(s) * 2.0 ** -22
        s = np.where(mask, s, -np.inf)
        e = np.where(mask, off, 0).max(-1, initial=0.0) + 2.0 ** -21
        m = s.max(-1, initial=-np.inf, keepdims=True)
        w = np.where(mask, np.exp(s - np.where(np.isinf(m), 0, m)), 0)
        total = w.sum(-1)
        live = total > 0
        p = w / np.where(live, total, 1)[:, None]
        out[:, h] = p @ vv
        mag = p @ np.abs(vv)
        top = np.abs(vv).max(initial=0.0)
        lse[live, h] = np.log(total[live]) + m[live, 0]
        tol[:, h] = ((2 * e + 2.0 ** -11 + 2 * n * 2.0 ** -23)[:, None] * mag
                     + n * 2.0 ** -25 * top) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(out[:, h])
        tol_lse[:, h] = e + n * 2.0 ** -23 + np.where(live, np.abs(np.where(live, lse[:, h], 0)), 0) * 2.0 ** -22
    return out, lse, tol, tol_lse


def assert_close(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = got == ref  # infinities
    err = np.where(same, 0.0, np.abs(np.where(same, 0.0, got) - np.where(same, 0.0, ref)))
    bad = ~(err <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err - tol)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; worst at {i}: got {got[i]}, "
                             f"oracle {ref[i]}, bound {tol[i]}")


def i32(x, device):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)


def check_attention(cache, table, lengths, counts, kv, q, tree=None, scale=None, device="cuda",
                    **call):
    """Runs cache_attention (out and lse prefilled with a mark) and checks every row against the
    oracle, and that rows behind a sequence's count keep the mark."""
    batch, tokens, heads, d = q.shape
    out = torch.full(tuple(q.shape), 77.0, dtype=torch.bfloat16, device=device)
    lse = torch.full((batch, tokens, heads), 77.0, dtype=torch.float32, device=device)
    td = None if tree is None else torch.from_numpy(tree.view(np.int64)).to(device)
    r = mx.cache_attention(cache, q, i32(table, device), i32(lengths, device),
                           count=None if counts is None else i32(counts, device), tree=td,
                           scale=scale, out=out, lse=lse, **call)
    assert r[0] is out and r[1] is lse
    torch.cuda.synchronize()
    qn, on, ln = (x.float().cpu().numpy().astype(np.float64) for x in (q, out, lse))
    for b in range(batch):
        c = tokens if counts is None else counts[b]
        mask = (chain_mask(lengths[b], c) if tree is None
                else tree_mask(lengths[b], c, tree[b]))
        ref = attend(qn[b, :c], kv[b][0], kv[b][1], mask, d ** -0.5 if scale is None else scale)
        what = f"sequence {b} (length {lengths[b]}, {c} tokens)"
        assert_close(on[b, :c], ref[0], ref[2], what)
        assert_close(ln[b, :c], ref[1], ref[3], what + " lse")
        assert (on[b, c:] == 77.0).all() and (ln[b, c:] == 77.0).all(), what + ": padding written"
    return out, lse


def random_tree(rng, count, roots=1):
    """Ancestor words of a random tree: token i >= roots hangs below one drawn before it."""
    words = []
    for i in range(count):
        words.append((1 << i) | (words[rng.integers(0, i)] if i >= roots else 0))
    return np.array(words, np.uint64)


def normal_bf16(shape, seed, device, sigma=1.0):
    return inputs.normal(shape, sigma, seed=seed, device=device)
