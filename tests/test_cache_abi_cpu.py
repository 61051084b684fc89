"""The cache calls reject bad arguments on the host before anything is enqueued (fake addresses;
every accepted call is stopped by an armed failure)."""
import ctypes
import math

import pytest

from fp4_microscaling_tensor_b200 import _lib

L = _lib.lib
OK, INV, UNS, MIS, WS, CUDA = range(6)
A = 0x10000  # a fake address; never dereferenced
BF16, F32 = _lib.MX_BF16, _lib.MX_F32
INT64_MAX = (1 << 63) - 1


def cache(**over):
    f = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, pages=4, kv_heads=2, page_size=64,
             head_dim=128, block=32, fmt=0, k_global_scale_fp16=0x3C00, v_global_scale_fp16=0x3C00)
    f.update(over)
    return _lib.Cache(**f)


S = _lib.Strides(1024, 256, 128, 1)


def append(c=None, k=A, v=A, xt=BF16, ks=S, vs=S, b=2, t=3, table=A, ts=8, w=8, start=A, count=None):
    return L.mx_cache_append(c or cache(), k, v, xt, ks, vs, b, t, table, ts, w, start, count, None)


def read(c=None, table=A, ts=8, w=8, start=A, count=None, b=2, t=3, k=A, v=A, yt=BF16, ks=S, vs=S):
    return L.mx_cache_read(c or cache(), table, ts, w, start, count, b, t, k, v, yt, ks, vs, None)


def attend(c=None, q=A, qs=S, b=2, t=3, heads=8, table=A, ts=8, w=8, length=A, count=None, tree=None,
           scale=0.1, out=A, os=S, lse=None, ws=A, n=None):
    n = L.mx_cache_attention_workspace_size(2, 3, 8, 2, 128) if n is None else n
    return L.mx_cache_attention(c or cache(), q, qs, b, t, heads, table, ts, w, length, count, tree,
                                scale, out, os, lse, ws, n, None)


def stopped(status):
    """The call passed its checks (the armed failure ended it before anything was enqueued)."""
    return status == CUDA and L.mx_test_fail_next_calls(0) == 0


def arm():
    L.mx_test_fail_next_calls(1)


@pytest.mark.parametrize("call", (append, read, attend))
def test_cache_descriptors(call):
    for field, bad in (("pages", 0), ("pages", -1), ("pages", 1 << 31), ("kv_heads", 0),
                       ("kv_heads", -2), ("kv_heads", 1025), ("fmt", 2), ("fmt", -1),
                       ("k_global_scale_fp16", 0), ("k_global_scale_fp16", 0x7C00),
                       ("v_global_scale_fp16", 0x8001), ("v_global_scale_fp16", 0x7E00),
                       ("k_codes", None), ("k_scales", None), ("v_codes", None), ("v_scales", None)):
        assert call(cache(**{field: bad})) == INV, (field, bad)
    for field, bad in (("head_dim", 96), ("head_dim", 0), ("head_dim", 512), ("head_dim", -64),
                       ("block", 8), ("block", 4), ("block", 256), ("block", 48), ("block", 0),
                       ("page_size", 8), ("page_size", 48), ("page_size", 512), ("page_size", 0),
                       ("page_size", -16)):
        assert call(cache(**{field: bad})) == UNS, (field, bad)
    assert call(cache(head_dim=64, block=128)) == UNS
    for field in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert call(cache(**{field: A + 8})) == MIS
    for d in (64, 128, 256):
        for n in (16, 32, 64):
            for p in (16, 32, 64, 128, 256):
                for f in (0, 1):
                    arm()
                    more = dict(n=1 << 40) if call is attend else {}
                    assert stopped(call(cache(head_dim=d, block=n, page_size=p, fmt=f), **more))


@pytest.mark.parametrize("call", (append, read, attend))
def test_batches_and_tables(call):
    first = "length" if call is attend else "start"
    for bad in (dict(b=-1), dict(t=-1), dict(b=1 << 31), dict(t=1 << 31), dict(w=-1), dict(w=1 << 31),
                dict(ts=-1), dict(table=None), {first: None}):
        assert call(**bad) == INV, bad
    for bad in (dict(table=A + 2), {first: A + 1}, dict(count=A + 2)):
        assert call(**bad) == MIS, bad
    assert call(b=0) == OK and call(t=0) == OK
    arm()
    assert stopped(call(table=A + 4, count=A + 4, **{first: A + 12}))
    arm()
    assert stopped(call(w=0, table=None))  # no pages at all: every position is nobody's


def test_outside_tensors():
    odd, neg = _lib.Strides(1024, 260, 128, 1), _lib.Strides(1024, -256, 128, 1)
    for call, names in ((append, ("k", "v")), (read, ("k", "v")), (attend, ("q", "out"))):
        for name in names:
            st = {"k": "ks", "v": "vs", "q": "qs", "out": "os"}[name]
            assert call(**{name: None}) == INV
            assert call(**{name: A + 8}) == MIS
            assert call(**{st: None}) == INV
            assert call(**{st: neg}) == INV
            assert call(**{st: odd}) == MIS      # 260 bf16 = 520 bytes: not whole 16-byte pieces
    assert append(xt=3) == INV and read(yt=-1) == INV
    arm()
    assert stopped(append(xt=F32, ks=odd, vs=odd))  # 260 fp32 are
    arm()
    assert stopped(append(t=1, ks=odd, vs=neg))     # a dimension with one entry
    for call in (append, read):
        arm()
        assert stopped(call(ks=_lib.Strides(0, 0, 0, 1)) if call is append else call())


def test_attention_arguments():
    assert attend(heads=7) == INV and attend(heads=0) == INV and attend(heads=-8) == INV
    assert attend(heads=2 * 65) == UNS
    assert attend(t=65, tree=A, n=1 << 40) == UNS
    assert attend(t=1 << 30, heads=4, n=1 << 40) == UNS       # 2^31 query rows of a kv head
    assert attend(w=(1 << 24) + 1, n=1 << 40) == UNS          # tables that reach beyond 2^30
    arm()
    assert stopped(attend(w=1 << 24))
    assert attend(scale=math.inf) == INV and attend(scale=math.nan) == INV
    assert attend(tree=A + 4) == MIS
    assert attend(lse=A + 2) == MIS
    assert attend(ws=None) == WS and attend(n=0) == WS
    assert attend(ws=A + 4) == MIS
    size = L.mx_cache_attention_workspace_size(2, 3, 8, 2, 128)
    assert attend(n=size - 1) == WS
    arm()
    assert stopped(attend(n=size, tree=A + 8, lse=A + 4, count=A))
    arm()
    assert stopped(attend(t=64, tree=A, n=1 << 40))
    arm()
    assert stopped(attend(t=5000, n=1 << 40, scale=-1.0))


def test_workspace_sizes():
    size = L.mx_cache_attention_workspace_size
    assert size(1, 1, 8, 8, 128) > 0
    for bad in ((-1, 1, 8, 8, 128), (1, -1, 8, 8, 128), (1, 1, 9, 8, 128), (1, 1, 0, 8, 128),
                (1, 1, 8, 0, 128), (1, 1, 8, 8, 96), (1, 1, 65, 1, 128), (1, 1, 8, 2000, 128),
                (1 << 31, 1, 8, 8, 128)):
        assert size(*bad) == 0, bad
    # bounded however long and wide the call is
    assert size((1 << 31) - 1, (1 << 31) - 1, 1024 * 64, 1024, 256) < 1 << 31


def test_python_checks_without_a_device():
    import torch
    import fp4_microscaling_tensor_b200 as mx
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError):  # not on a device
        mx.KVCache.from_buffers(z(2, 2, 16, 64), z(2, 2, 16, 4), z(2, 2, 16, 64), z(2, 2, 16, 4))
    for bad in (dict(head_dim=96), dict(block=8), dict(block=256), dict(head_dim=64, block=128),
                dict(pages=0), dict(kv_heads=0), dict(page_size=0)):
        with pytest.raises(ValueError):
            mx.KVCache(**{**dict(pages=1, kv_heads=1, head_dim=128, device="cpu"), **bad})
    assert ctypes.sizeof(_lib.Cache) == 64
