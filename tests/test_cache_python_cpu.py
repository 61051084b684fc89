"""What the Python cache calls refuse before anything reaches the library (CPU tensors stand in for a
device's; no call gets through)."""
import types

import pytest
import torch

import fp4_microscaling_tensor_b200 as mx
from fp4_microscaling_tensor_b200 import api

CPU = torch.device("cpu")
BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


@pytest.fixture
def calls(monkeypatch):
    """The calls that would have reached the library."""
    made = []
    monkeypatch.setattr(api, "_call", lambda fn, where, *args: made.append(where))
    return made


def cache():
    return types.SimpleNamespace(device=CPU, head_dim=64, kv_heads=2, _desc=None, _workspaces={})


def zeros(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def numbers(n=3, dtype=I32):
    return torch.zeros(n, dtype=dtype)


META = dict(device="meta", dtype=I32)  # another device
BATCH = [dict(table=zeros(3, 4, dtype=I64)), dict(table=zeros(2, 4, dtype=I32)),
         dict(table=zeros(12, dtype=I32)), dict(table=zeros(3, 8, dtype=I32)[:, ::2]),
         dict(table=torch.zeros(3, 4, **META)), dict(first=numbers(2)), dict(first=numbers(dtype=I64)),
         dict(first=numbers(6)[::2]), dict(first=torch.zeros(3, **META)), dict(count=numbers(4)),
         dict(count=numbers(dtype=F32)), dict(count=numbers(6)[::2])]


def append(c, k=zeros(3, 5, 2, 64), v=zeros(3, 5, 2, 64), table=zeros(3, 4, dtype=I32),
           first=numbers(), count=None):
    mx.cache_append(c, k, v, table, first, count=count)


def read(c, table=zeros(3, 4, dtype=I32), first=numbers(), count=None, tokens=5, **out):
    mx.cache_read(c, table, first, count, tokens, **out)


def attend(c, q=zeros(3, 5, 8, 64), table=zeros(3, 4, dtype=I32), first=numbers(), **rest):
    mx.cache_attention(c, q, table, first, **{"workspace": zeros(16, dtype=torch.uint8), **rest})


@pytest.mark.parametrize("bad", BATCH + [
    dict(k=zeros(3, 5, 2, 128)), dict(v=zeros(3, 4, 2, 64)), dict(v=zeros(3, 5, 2, 64, dtype=F32)),
    dict(k=zeros(15, 2, 64)), dict(k=zeros(3, 5, 2, 64, dtype=torch.float16)),
    dict(k=zeros(3, 5, 4, 64), v=zeros(3, 5, 4, 64)), dict(v=zeros(3, 5, 2, 128)[..., ::2]),
    dict(k=torch.zeros(3, 5, 2, 64, dtype=BF16, device="meta"))])
def test_append_refuses(calls, bad):
    append(cache())
    assert calls.pop() == "mx_cache_append"
    with pytest.raises(ValueError):
        append(cache(), **bad)
    assert not calls


@pytest.mark.parametrize("bad", BATCH + [
    dict(k_out=zeros(3, 5, 2, 128)), dict(k_out=zeros(3, 4, 2, 64)),
    dict(v_out=zeros(3, 5, 2, 64, dtype=torch.float16)),
    dict(k_out=zeros(3, 5, 2, 64), v_out=zeros(3, 5, 2, 64, dtype=F32)),
    dict(k_out=zeros(3, 1, 2, 64).expand(3, 5, 2, 64)), dict(v_out=zeros(3, 5, 2, 128)[..., ::2])])
def test_read_refuses(calls, bad):
    read(cache())
    assert calls.pop() == "mx_cache_read"
    with pytest.raises(ValueError):
        read(cache(), **bad)
    assert not calls


@pytest.mark.parametrize("bad", BATCH + [
    dict(q=zeros(3, 5, 7, 64)), dict(q=zeros(3, 5, 0, 64)), dict(q=zeros(3, 5, 8, 128)),
    dict(q=zeros(3, 5, 8, 64, dtype=F32)), dict(q=zeros(3, 5, 8, 128)[..., ::2]),
    dict(tree=zeros(3, 4, dtype=I64)), dict(tree=zeros(3, 5, dtype=I32)),
    dict(tree=zeros(3, 10, dtype=I64)[:, ::2]), dict(out=zeros(3, 5, 4, 64)),
    dict(out=zeros(3, 5, 8, 64, dtype=F32)), dict(out=zeros(3, 1, 8, 64).expand(3, 5, 8, 64)),
    dict(lse=zeros(3, 5, 8)), dict(lse=zeros(3, 8, 5, dtype=F32)),
    dict(lse=zeros(3, 5, 16, dtype=F32)[..., ::2]), dict(workspace=zeros(16, dtype=F32)),
    dict(workspace=zeros(32, dtype=torch.uint8)[::2]),
    dict(workspace=torch.zeros(16, dtype=torch.uint8, device="meta"))])
def test_attention_refuses(calls, bad):
    attend(cache())
    assert calls.pop() == "mx_cache_attention"
    with pytest.raises(ValueError):
        attend(cache(), **bad)
    assert not calls
