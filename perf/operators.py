"""Measured cases of the operators on a paged FP4 key/value cache: writing keys and values into it as
they are quantized, reading them back, and attention over it (single tokens, chains and trees of
drafted tokens, chunks of a prompt).

``run`` computes a case either with elementary torch operations (``own`` false) or with the
library's own calls (``own`` true); ``exact`` gives the same outputs from the definition in 64 bits.

Layout of a cache (one layer): codes [pages, kv_heads, page_size, head_dim / 2] (two E2M1 codes per
byte, the even element in the low nibble), scales [pages, kv_heads, page_size, head_dim / block]
(E4M3 or UE5M3), for keys and for values, each with an FP16 factor g; value = E2M1 * scale * g.
Position p of sequence b is slot p % page_size of page table[b, p / page_size].
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- the cases -----------------------------------------------------------------------------------

def _attention(name, batch, tokens, length, heads, kv_heads, head_dim, page, block, fmt, tree=False,
               spread=0.0, drop=0):
    """length: the longest sequence (its new tokens included); spread: how much shorter the others
    may be, as a share; drop: how many of its `tokens` new tokens a sequence may lack."""
    return dict(name=name, op="attention", batch=batch, tokens=tokens, length=length, heads=heads,
                kv_heads=kv_heads, head_dim=head_dim, page=page, block=block, fmt=fmt, tree=tree,
                spread=spread, drop=drop, type=BF16)


def _cache(name, op, batch, tokens, length, kv_heads, head_dim, page, block, fmt, spread, type):
    """op append: `tokens` new tokens a sequence (less by up to `spread`) behind a sequence that
    ends up at most `length` long; op read: the first positions."""
    return dict(name=name, op=op, batch=batch, tokens=tokens, length=length, kv_heads=kv_heads,
                head_dim=head_dim, page=page, block=block, fmt=fmt, spread=spread, type=type)


def listed():
    return [
        # one user's next token in a short conversation, 64 query heads on 8 key/value heads (the
        # head layout of the 70B-shaped layers): latency
        _attention("decode_one_777", 1, 1, 777, 64, 8, 128, 16, 32, "ue5m3"),
        # a serving batch, every sequence at its own length: the usual step
        _attention("decode_64x8191", 64, 1, 8191, 64, 8, 128, 64, 16, "e4m3", spread=0.9),
        # two long documents: the cache streams, few rows
        _attention("decode_2x131071", 2, 1, 131071, 64, 8, 128, 64, 32, "ue5m3", spread=0.3),
        # chains of three drafted tokens, a key/value head for each query head, small heads
        _attention("chain_16x4000_mha", 16, 3, 4000, 32, 32, 64, 32, 16, "e4m3", spread=0.6,
                   drop=2),
        # trees of 48 drafted tokens to verify at once
        _attention("tree_8x6001", 8, 48, 6001, 64, 8, 128, 64, 32, "ue5m3", tree=True, spread=0.5,
                   drop=7),
        # a chunk of a long prompt over what is in the cache already: the tensor cores' work
        _attention("prompt_2048_of_16384", 1, 2048, 16384, 64, 8, 128, 64, 32, "e4m3"),
        # one token for each of 64 sequences enters the cache (and is read back): latency
        _cache("append_64x1", "append", 64, 1, 5000, 8, 128, 64, 16, "e4m3", 0.0, BF16),
        # four padded prompts enter the cache
        _cache("append_4x8192", "append", 4, 8192, 9000, 8, 128, 64, 32, "ue5m3", 0.6, BF16),
        # fp32 keys and values, odd counts, small pages
        _cache("append_f32_7x333", "append", 7, 333, 1000, 5, 64, 16, 64, "e4m3", 0.5, F32),
        # one short sequence is read back, wide heads, to fp32
        _cache("read_1x100_f32", "read", 1, 100, 100, 4, 256, 32, 128, "ue5m3", 0.0, F32),
        # eight long prefixes are read back for a kernel that wants bf16
        _cache("read_8x16000", "read", 8, 16000, 16000, 8, 128, 64, 32, "ue5m3", 0.4, BF16),
    ]


#: what bounds a drawn case: values of the keys read or written, and score entries
_MOST_VALUES, _MOST_SCORES = 2.0e8, 2.0e9


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    head_dim = rng.choice((64, 128, 128, 128, 256))
    block = rng.choice([n for n in (16, 32, 64, 128) if n <= head_dim])
    kv_heads = rng.choice((1, 2, 4, 5, 8, 8, 16))
    page = rng.choice((16, 32, 64, 128))
    fmt = rng.choice(("e4m3", "ue5m3"))
    op = rng.choice(("attention", "attention", "attention", "append", "read"))
    if op != "attention":
        batch = _log(rng, 1, 64)
        most = max(1, int(_MOST_VALUES / (2 * batch * kv_heads * head_dim)))
        tokens = 1 if op == "append" and rng.random() < 0.3 else _log(rng, 1, min(most, 20000))
        length = tokens + (_log(rng, 1, 4000) if op == "append" else 0)
        return dict(op=op, batch=batch, tokens=tokens, length=length, kv_heads=kv_heads,
                    head_dim=head_dim, page=page, block=block, fmt=fmt,
                    spread=rng.choice((0.0, 0.5, 0.9)), type=rng.choice((BF16, BF16, F32)))
    kind = rng.choice(("one", "one", "chain", "tree", "prompt"))
    group = rng.choice((1, 2, 4, 5, 7, 8, 8, 12, 16))
    tokens = dict(one=1, chain=rng.randint(2, 9), tree=rng.randint(5, 64),
                  prompt=_log(rng, 65, 2048))[kind]
    batch = _log(rng, 1, 4 if kind == "prompt" else 16 if kind == "tree" else 96)
    per = min(_MOST_VALUES / (batch * kv_heads * head_dim),
              _MOST_SCORES / (batch * kv_heads * group * tokens * (head_dim / 128)), 131072)
    tokens = int(max(1, min(tokens, per)))
    length = max(tokens, _log(rng, min(per, 8), per))
    return dict(op=op, batch=batch, tokens=tokens, length=length, heads=kv_heads * group,
                kv_heads=kv_heads, head_dim=head_dim, page=page, block=block, fmt=fmt,
                tree=kind == "tree", spread=rng.choice((0.0, 0.5, 0.95)),
                drop=rng.randint(0, tokens - 1) if kind in ("chain", "tree") else 0,
                type=BF16)


def _spread(n, most, share, phase):
    """n whole numbers in [most * (1 - share), most], the first one `most`; always the same ones."""
    return [max(1, int(most * (1 - share * ((b * 0.6180339887 + phase * (b > 0)) % 1.0))))
            for b in range(n)]


def _sizes(case):
    """(start, count) of each sequence: its tokens before this call, and its new tokens (append,
    attention) or the tokens to read (from position 0)."""
    n = case["batch"]
    if case["op"] == "read":
        return [0] * n, _spread(n, case["tokens"], case["spread"], 0.3)
    if case["op"] == "append":
        count = _spread(n, case["tokens"], case["spread"], 0.3)
        before = case["length"] - case["tokens"]
        return [int(before * ((b * 0.7548776662) % 1.0)) for b in range(n)], count
    count = [case["tokens"] - (b * 5) % (case["drop"] + 1) for b in range(n)]
    length = _spread(n, case["length"], case["spread"], 0.0)
    length = [max(a, c) for a, c in zip(length, count)]
    return [a - c for a, c in zip(length, count)], count


def work(case):
    start, count = _sizes(case)
    hd, n = case["kv_heads"] * case["head_dim"], sum(count)
    stored = 2 * hd * (0.5 + 1.0 / case["block"])  # bytes of a token's keys and values
    wide = 2 * hd * (2 if case["type"] == BF16 else 4)
    if case["op"] == "read":
        return {"bytes": n * (stored + wide), "flops": 0}
    if case["op"] == "append":  # read k and v, write the cache; read that, write the values
        return {"bytes": n * (2 * stored + 2 * wide), "flops": 0}
    q = n * case["heads"] * case["head_dim"]
    pairs = sum(c * s + (c * (c + 1)) // 2 for s, c in zip(start, count))  # a tree: at most these
    return {"bytes": sum(s + c for s, c in zip(start, count)) * stored
            + q * (2 + 2) + 4 * n * case["heads"],
            "flops": 4.0 * pairs * case["heads"] * case["head_dim"]}


# ---- quantization in plain torch -----------------------------------------------------------------

def _g(bits):
    """Value of a binary16 bit pattern."""
    e, m = bits >> 10, bits & 1023
    return m * 2.0 ** -24 if e == 0 else (1 + m / 1024.0) * 2.0 ** (e - 15)


def _g_bits(fmt):
    """The caches' FP16 factors (keys, values): 1 with E4M3; with UE5M3 what puts the largest keys
    and values near the top of its range."""
    return (0x3C00, 0x3C00) if fmt == "e4m3" else (0x038E, 0x0060)


def _quantize(x, block, fmt, g):
    """(codes, scale codes) of x [..., d]: blocks of `block` along the last dimension, scale =
    RNE(absmax / (6 g)) saturating, element = RNE(x / (scale g)) saturating, in 64 bits."""
    v = x.double().unflatten(-1, (-1, block))
    u = v.abs().amax(-1) / (6 * g)
    bias, top = (7, 0x7E) if fmt == "e4m3" else (15, 0xFF)
    e = (torch.frexp(u)[1] - 1).clamp(min=1 - bias)           # u = m 2^e, subnormals share the last
    m = torch.round(torch.ldexp(u, 3 - e))                    # 8..16, below 8 for subnormals
    sc = ((e + bias - 1) * 8 + m.long()).clamp(max=top)       # a carry moves into the exponent
    s = _scale_values(fmt, x.device)[sc].unsqueeze(-1) * g
    a = torch.where(s > 0, v.abs() / s, 0.0).clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = torch.round(a / step) * step
    mag = torch.where(r < 2, r * 2, torch.where(r < 4, r + 2, r / 2 + 4)).to(torch.uint8)
    code = (mag | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sc.to(torch.uint8)


def _scale_values(fmt, device):
    c = torch.arange(256, device=device)
    bias = 7 if fmt == "e4m3" else 15
    sign = 1.0
    if fmt == "e4m3":
        sign, c = torch.where(c < 128, 1.0, -1.0), c & 127
    e, m = c >> 3, (c & 7).double()
    return sign * torch.where(e == 0, m * 2.0 ** (-bias - 2), (8 + m) * torch.exp2((e - bias - 3).double()))


def _values(codes, scales, fmt, g):
    """The 32-bit values (exact) of codes [..., d / 2] with scales [..., d / block]."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    q = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    s = (_scale_values(fmt, codes.device) * g).float()[scales.long()]
    return (q.unflatten(-1, (s.shape[-1], -1)) * s.unsqueeze(-1)).flatten(-2)


# ---- inputs --------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * seed + 17)
    b, d, kvh, page, block, fmt = (case[k] for k in ("batch", "head_dim", "kv_heads", "page", "block",
                                                     "fmt"))
    start, count = _sizes(case)
    need = [-(-(s + c) // page) for s, c in zip(start, count)]
    width, pages = max(need), sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev).int()
    table = torch.full((b, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    gk, gv = _g_bits(fmt)
    gain = torch.where(torch.rand(kvh, 1, d, generator=gen, device=dev) < 0.04, 5.0, 0.8)  # some
    # channels of the keys are much larger than the others
    pool = [torch.zeros(pages, kvh, page, n, dtype=torch.uint8, device=dev)
            for n in (d // 2, d // block, d // 2, d // block)]
    st = dict(case=case, pool=pool, table=table, gk=gk, gv=gv,
              start=torch.tensor(start, dtype=torch.int32, device=dev),
              count=torch.tensor(count, dtype=torch.int32, device=dev))
    kind = _DT[case["type"]]
    if case["op"] == "append":
        t = case["tokens"]
        # keys and values are slices of one projection's output, as a layer hands them over
        kv = normal(b, t, 2, kvh, d).to(kind)
        kv[:, :, 0] *= gain[:, 0]
        st.update(k=kv[:, :, 0], v=kv[:, :, 1])
    else:
        step = max(1, 32_000_000 // (kvh * page * d))
        for i in range(0, pages, step):
            n = min(step, pages - i)
            k = (normal(n, kvh, page, d) * gain).bfloat16()
            pool[0][i:i + n], pool[1][i:i + n] = _quantize(k, block, fmt, _g(gk))
            v = (normal(n, kvh, page, d) * 0.7).bfloat16()
            pool[2][i:i + n], pool[3][i:i + n] = _quantize(v, block, fmt, _g(gv))
    if case["op"] != "attention":
        shape = (b, case["tokens"], kvh, d)
        st.update(k_out=torch.zeros(shape, dtype=kind, device=dev),
                  v_out=torch.zeros(shape, dtype=kind, device=dev))
        return st
    t, h = case["tokens"], case["heads"]
    # queries are a slice of the projection's output too
    st["q"] = normal(b, t, h + 2 * kvh, d).bfloat16()[:, :, :h]
    st["length"] = st["start"] + st["count"]
    st["out"] = torch.zeros(b, t, h, d, dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.zeros(b, t, h, device=dev)
    st["tree"] = None
    if case["tree"]:
        # token i > 0 hangs below a token drawn among those before it; a token sees its ancestors
        # and itself (bit j of word i: token i sees token j)
        parent = (torch.rand(b, t, generator=gen, device=dev)
                  * torch.arange(t, device=dev)).long().cpu().tolist()
        words = []
        for row in parent:
            seen = []
            for i, p in enumerate(row):
                seen.append((1 << i) | (seen[p] if i else 0))
            words.append([w - (1 << 64) if w >> 63 else w for w in seen])
        st["tree"] = torch.tensor(words, dtype=torch.int64, device=dev)
    return st


# ---- one pass ------------------------------------------------------------------------------------

def _slots(st, tokens):
    """(page, slot, valid) of positions start + 0 .. tokens - 1 of every sequence."""
    page, t = st["case"]["page"], torch.arange(tokens, device=st["table"].device)
    pos = st["start"].long()[:, None] + t
    valid = t < st["count"][:, None]
    ids = st["table"].long().gather(1, (pos // page).clamp(max=st["table"].shape[1] - 1))
    return ids.clamp(min=0), pos % page, valid


def _plain_append(st):
    c = st["case"]
    ids, slot, valid = _slots(st, c["tokens"])
    ids, slot = ids[valid], slot[valid]
    for x, at, g in ((st["k"], 0, st["gk"]), (st["v"], 2, st["gv"])):
        codes, scales = _quantize(x[valid], c["block"], c["fmt"], _g(g))
        st["pool"][at][ids, :, slot] = codes
        st["pool"][at + 1][ids, :, slot] = scales


def _plain_read(st):
    c = st["case"]
    ids, slot, valid = _slots(st, c["tokens"])
    ids, slot = ids[valid], slot[valid]
    for out, at, g in ((st["k_out"], 0, st["gk"]), (st["v_out"], 2, st["gv"])):
        p = st["pool"]
        out[valid] = _values(p[at][ids, :, slot], p[at + 1][ids, :, slot], c["fmt"], _g(g)).to(out.dtype)
    return st["k_out"], st["v_out"]


def _whole(st):
    """Keys and values [batch, kv_heads, positions, head_dim] of every sequence, in 32 bits."""
    c = st["case"]
    page, n = c["page"], st["table"].shape[1] * c["page"]
    ids = st["table"].long().clamp(min=0)
    p = st["pool"]
    k = _values(p[0][ids], p[1][ids], c["fmt"], _g(st["gk"])).transpose(1, 2).flatten(2, 3)
    v = _values(p[2][ids], p[3][ids], c["fmt"], _g(st["gv"])).transpose(1, 2).flatten(2, 3)
    return k[:, :, :c["length"]], v[:, :, :c["length"]], min(n, c["length"])


def _seen(st, n):
    """[batch, tokens, n]: whether a new token sees a position."""
    c, dev = st["case"], st["table"].device
    pos, t = torch.arange(n, device=dev), torch.arange(c["tokens"], device=dev)
    j = pos - st["start"][:, None]  # the position's place among the new tokens
    if st["tree"] is None:
        return j[:, None, :] <= t[:, None]
    bit = (st["tree"][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    return (j < 0)[:, None, :] | ((bit == 1) & (j < c["tokens"])[:, None, :])


def _plain_attention(st):
    c = st["case"]
    b, t, h, kvh, d = (c[k] for k in ("batch", "tokens", "heads", "kv_heads", "head_dim"))
    k, v, n = _whole(st)
    q = st["q"].float().reshape(b, t, kvh, h // kvh, d).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5).unflatten(2, (t, h // kvh))
    # a new token that a sequence lacks is behind its end: nobody sees it
    s.masked_fill_(~_seen(st, n)[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (t, h // kvh))
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + total.log()).squeeze(-1)
    valid = torch.arange(t, device=q.device) < st["count"][:, None]
    order = lambda x: x.transpose(1, 2).flatten(2, 3)  # noqa: E731  heads behind the tokens
    st["out"].copy_(torch.where(valid[..., None, None], order(o), st["out"].float()))
    st["lse"].copy_(torch.where(valid[..., None], order(lse), st["lse"]))
    return st["out"], st["lse"]


def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "attention":
            return _plain_attention(st)
        if c["op"] == "append":
            _plain_append(st)
        return _plain_read(st)
    import fp4_microscaling_tensor_b200 as mx
    cache = st.get("cache")
    if cache is None:  # the handle that a program keeps beside the cache's memory
        cache = st["cache"] = mx.KVCache.from_buffers(*st["pool"], fmt=c["fmt"], k_g=st["gk"],
                                                      v_g=st["gv"])
    if c["op"] == "attention":
        return mx.cache_attention(cache, st["q"], st["table"], st["length"], count=st["count"],
                                  tree=st["tree"], out=st["out"], lse=st["lse"])
    if c["op"] == "append":
        mx.cache_append(cache, st["k"], st["v"], st["table"], st["start"], count=st["count"])
    return mx.cache_read(cache, st["table"], st["start"], st["count"], c["tokens"],
                         k_out=st["k_out"], v_out=st["v_out"])


# ---- the definition in 64 bits -------------------------------------------------------------------

def _exact_scales(fmt, device):
    """Values of the scale codes, from their bits."""
    mant, bias = 3, (7 if fmt == "e4m3" else 15)
    out = []
    for c in range(127 if fmt == "e4m3" else 256):
        e, m = divmod(c, 1 << mant)
        out.append(math.ldexp(m, 1 - bias - mant) if e == 0 else math.ldexp((1 << mant) + m, e - bias - mant))
    return torch.tensor(out, dtype=torch.float64, device=device)


def _nearest(x, grid):
    """Index of the nearest grid value, ties to the even index, the last one for what lies above."""
    hi = torch.bucketize(x, grid).clamp(1, len(grid) - 1)
    below, above = x - grid[hi - 1], grid[hi] - x
    up = (below > above) | ((below == above) & (hi % 2 == 0))
    return torch.where(up, hi, hi - 1)


def _exact_round_trip(x, block, fmt, g):
    grid, fp4 = _exact_scales(fmt, x.device), torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    v = x.double().reshape(*x.shape[:-1], x.shape[-1] // block, block)
    s = grid[_nearest(v.abs().max(-1).values / 6 / g, grid)][..., None] * g
    q = fp4[_nearest((v.abs() / torch.where(s == 0, torch.inf, s)), fp4)] * s
    return torch.copysign(q, v).reshape(x.shape)


def _exact_values(codes, scales, fmt, g):
    fp4 = torch.tensor(_E2M1, dtype=torch.float64, device=codes.device)
    nib = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.long, device=codes.device)
    nib[..., ::2], nib[..., 1::2] = codes % 16, codes // 16
    x = torch.where(nib >= 8, -fp4[nib % 8], fp4[nib % 8])
    s = _exact_scales(fmt, codes.device)[scales.long()] * g
    return x * s.repeat_interleave(x.shape[-1] // s.shape[-1], dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    start, count = _sizes(case)
    page, b, table = case["page"], case["batch"], st["table"].long()
    gk, gv = _g(st["gk"]), _g(st["gv"])

    def stored(i, first, n):
        """Keys and values [n, kv_heads, head_dim] of positions first .. first + n - 1."""
        pos = torch.arange(first, first + n, device=table.device)
        ids, slot = table[i, pos // page], pos % page
        kc, ks, vc, vs = (p[ids, :, slot] for p in st["pool"])
        return _exact_values(kc, ks, case["fmt"], gk), _exact_values(vc, vs, case["fmt"], gv)

    if case["op"] != "attention":
        k, v = (torch.zeros(x.shape, dtype=torch.float64, device=x.device)
                for x in (st["k_out"], st["v_out"]))
        for i in range(b):
            n = count[i]
            if case["op"] == "read":
                k[i, :n], v[i, :n] = stored(i, 0, n)
            else:
                k[i, :n] = _exact_round_trip(st["k"][i, :n], case["block"], case["fmt"], gk)
                v[i, :n] = _exact_round_trip(st["v"][i, :n], case["block"], case["fmt"], gv)
        return k, v
    t, h, d = case["tokens"], case["heads"], case["head_dim"]
    if 4.0 * b * t * h * d * case["length"] > 4e13:
        return None
    out = torch.zeros(b, t, h, d, dtype=torch.float64, device=table.device)
    lse = torch.zeros(b, t, h, dtype=torch.float64, device=table.device)
    group = h // case["kv_heads"]
    for i in range(b):
        n, c = start[i] + count[i], count[i]
        k, v = stored(i, 0, n)
        seen = torch.ones(c, n, dtype=torch.bool, device=table.device)
        if st["tree"] is None:
            seen[:, start[i]:] = torch.ones(c, c, device=table.device).tril() > 0
        else:
            words = st["tree"][i].tolist()
            seen[:, start[i]:] = torch.tensor([[bool((words[x] >> y) & 1) for y in range(c)]
                                               for x in range(c)], device=table.device)
        for head in range(h):
            s = st["q"][i, :c, head].double() @ k[:, head // group].T / math.sqrt(d)
            s = s.masked_fill(~seen, -math.inf)
            lse[i, :c, head] = torch.logsumexp(s, -1)
            out[i, :c, head] = torch.softmax(s, -1) @ v[:, head // group]
    return out, lse
