"""The stream's bookkeeping on the CPU: the norm and the cached attention are
stood in for by plain code that refuses what the library's call refuses, so
what is tested is which rows are written, which lengths each call gets, and
that a step which is refused leaves the stream as it was."""
import math
import types

import pytest
import torch

from dynamic_block_sparse_pool_b200 import DSAError, _lib, ops, window_layer

H, HK, D = 4, 2, 8


class Plan:
    table = torch.zeros(1)

    def at(self, pos):
        return self


def norm(xq, xk, wq, wk, plan, eps):
    return xq.transpose(1, 2).contiguous(), xk.transpose(1, 2).contiguous()


def decode(q, k, v, lens, left, sink, scale=None):
    if not q.is_contiguous() or not 1 <= q.shape[2] <= 128:
        raise DSAError(_lib.DSA_ERR_INVALID_ARG, "dsa_window_attn_decode", "Nq must be 1..128")
    if q.dtype != k.dtype or q.shape[0] != k.shape[0] or q.shape[1] % k.shape[1]:
        raise ValueError("caches must match q")
    out = torch.empty_like(q)
    for b, n in enumerate(lens.tolist()):
        t = (n - q.shape[2] + torch.arange(q.shape[2]))[:, None]
        u = torch.arange(k.shape[2])[None]
        ok = u <= t
        if left >= 0:
            ok &= (u < sink) | (u >= t - left)
        kk, vv = (x[b].repeat_interleave(q.shape[1] // k.shape[1], 0) for x in (k, v))
        s = (q[b] @ kk.transpose(1, 2) / math.sqrt(D)).masked_fill(~ok, -math.inf)
        out[b] = torch.softmax(s, -1) @ vv
    return out


@pytest.fixture
def stream(monkeypatch):
    monkeypatch.setattr(window_layer, "ops", types.SimpleNamespace(
        **{**vars(ops), "qk_norm_rope": norm, "window_attn_decode": decode}))

    def make(capacity=400, mask=window_layer.Mask(70, 0, 3)):
        s = window_layer.Stream(2, H, HK, capacity, D, Plan(), mask, dtype=torch.float64)
        s.k.zero_()  # rows that no query sees are multiplied by 0 here
        s.v.zero_()
        return s
    return make


def rows(n, seed=0, b=2, heads=H + 2 * HK, dtype=torch.float64):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(b, n, heads, D, generator=g, dtype=torch.float64).to(dtype)


def whole(qkv, mask):
    q, k, v = (x.transpose(1, 2) for x in (qkv[:, :, :H], qkv[:, :, H:H + HK], qkv[:, :, H + HK:]))
    n = qkv.shape[1]
    t, u = torch.arange(n)[:, None], torch.arange(n)[None]
    ok = (u <= t) & ((u < mask.sink) | (u >= t - mask.left))
    k, v = (x.repeat_interleave(H // HK, 1) for x in (k, v))
    return torch.softmax((q @ k.transpose(2, 3) / math.sqrt(D)).masked_fill(~ok, -math.inf), -1) @ v


@pytest.mark.parametrize("steps", [(129,), (300, 1), (1, 128, 2), (5, 257, 1, 37), (400,)])
def test_a_step_takes_any_number_of_tokens(stream, steps):
    s = stream()
    qkv = rows(sum(steps))
    got, at = [], 0
    for n in steps:
        got.append(s.step(qkv[:, at:at + n], torch.zeros(n, 1)))
        at += n
        assert s.length == at and s.lens.tolist() == [at, at]
    assert torch.allclose(torch.cat(got, 2), whole(qkv, s.mask), rtol=0, atol=1e-12)


def test_no_tokens(stream):
    s = stream()
    out = s.step(rows(0), torch.zeros(0, 1))
    assert out.shape == (2, H, 0, D) and s.length == 0


def state(s):
    return s.length, s.lens.tolist(), s.k[:, :, :s.length].clone(), s.v[:, :, :s.length].clone()


def same(a, b):
    return a[:2] == b[:2] and all(torch.equal(x, y) for x, y in zip(a[2:], b[2:]))


@pytest.mark.parametrize("bad", [
    dict(n=371),                                  # past the capacity
    dict(n=5, b=1),                               # would be broadcast over the streams
    dict(n=5, heads=H + 2),                       # one key head: would be broadcast over the cache's
    dict(n=5, dtype=torch.float32),               # would be converted into the cache
])
def test_what_a_step_refuses_leaves_the_stream_unchanged(stream, bad):
    s = stream()
    qkv = rows(60)
    s.step(qkv[:, :30], torch.zeros(30, 1))
    before = state(s)
    with pytest.raises(ValueError):
        s.step(rows(**bad), torch.zeros(bad["n"], 1))
    assert same(before, state(s))
    out = s.step(qkv[:, 30:], torch.zeros(30, 1))
    assert torch.allclose(out, whole(qkv, s.mask)[:, :, 30:], rtol=0, atol=1e-12)


@pytest.mark.parametrize("n,fails", [(1, 0), (300, 0), (300, 2)])
def test_a_failed_attention_leaves_the_stream_unchanged(stream, monkeypatch, n, fails):
    s = stream()
    qkv = rows(30 + n)
    s.step(qkv[:, :30], torch.zeros(30, 1))
    before, calls = state(s), []

    def failing(*a, **kw):
        calls.append(1)
        if len(calls) > fails:
            raise torch.OutOfMemoryError("no room for the workspace")
        return decode(*a, **kw)

    monkeypatch.setattr(window_layer.ops, "window_attn_decode", failing)
    with pytest.raises(torch.OutOfMemoryError):
        s.step(qkv[:, 30:], torch.zeros(n, 1))
    assert same(before, state(s))
    monkeypatch.setattr(window_layer.ops, "window_attn_decode", decode)
    out = s.step(qkv[:, 30:], torch.zeros(n, 1))
    assert torch.allclose(out, whole(qkv, s.mask)[:, :, 30:], rtol=0, atol=1e-12)
