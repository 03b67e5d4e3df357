"""The window attention as a layer uses it: from the fused projection's output
to the attention's, back to the projection's gradient, and token by token.

    qkv [B, N, H + 2 Hk, D] -> qk_norm_rope -> window_attn_fwd -> out [B, H, N, D]

`forward` and `backward` are one training step; with keep8 what lies between
them is held in 8 bits (the rows of q and k before their norm, and v), and the
backward first repeats the forward from them: its gradients are those of the
step on the values that the rows stand for.  (The output and lse of the first
forward do not belong to those values.  With them the rows of P would not sum to
1 nor those of dS to 0, and dQ, a small difference of large sums where the keys
share a common part, would be off several times as far: by 12 % in place of 3 %
for keys with a common part of three times their spread and one outlying
column.)  `Stream` is the cached form.  This module only strings the calls
together and moves v between the projection's token-major layout and the
attention's head-major one.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import ops
from .ops import Act8


_MOST_NEW = 128  # tokens that window_attn_decode takes of each stream


class Mask(NamedTuple):
    """Key u is visible at position t iff u <= t + right and (u < sink or
    u >= t - left); a negative bound is no bound."""

    left: int = -1
    right: int = 0
    sink: int = 0


class Saved(NamedTuple):
    """What the backward needs of a forward."""

    xq: Union[torch.Tensor, Act8]      # rows before the norm, [B, N, H, D]
    xk: Union[torch.Tensor, Act8]
    q: Optional[torch.Tensor]          # None with keep8: recomputed
    k: Optional[torch.Tensor]
    v: Union[torch.Tensor, Act8]       # [B, Hk, N, D]
    out: Union[torch.Tensor, Tuple[()]]  # () and None with keep8: recomputed
    lse: Optional[torch.Tensor]
    wq: Optional[torch.Tensor]
    wk: Optional[torch.Tensor]
    plan: ops.RopePlan
    eps: float
    mask: Mask
    scale: Optional[float]


def _split(qkv: torch.Tensor, heads: int):
    Hk = (qkv.shape[2] - heads) // 2
    if Hk < 1 or heads + 2 * Hk != qkv.shape[2] or heads % Hk:
        raise ValueError(f"{qkv.shape[2]} rows per token are not {heads} query heads and twice the key heads")
    return qkv[:, :, :heads], qkv[:, :, heads:heads + Hk], qkv[:, :, heads + Hk:]


def forward(qkv: torch.Tensor, heads: int, wq: Optional[torch.Tensor], wk: Optional[torch.Tensor],
            plan: ops.RopePlan, mask: Mask, eps: float = 1e-6, scale: Optional[float] = None,
            keep8: bool = False):
    """(out [B, H, N, D], Saved) of qkv [B, N, H + 2 Hk, D] (queries, keys,
    values of each token)."""
    xq, xk, xv = _split(qkv, heads)
    v = xv.transpose(1, 2).contiguous()
    if keep8:
        q, k, q8, k8 = ops.qk_norm_rope(xq, xk, wq, wk, plan, eps, save8=True)
    else:
        q, k = ops.qk_norm_rope(xq, xk, wq, wk, plan, eps)
    out, lse = ops.window_attn_fwd(q, k, v, mask.left, mask.right, mask.sink, scale=scale, want_lse=not keep8)
    if keep8:
        saved = Saved(q8, k8, None, None, ops.pack8(v), (), None, wq, wk, plan, eps, mask, scale)
    else:
        saved = Saved(xq, xk, q, k, v, out, lse, wq, wk, plan, eps, mask, scale)
    return out, saved


def backward(dout: torch.Tensor, s: Saved):
    """(dqkv [B, N, H + 2 Hk, D], dwq, dwk) for dout [B, H, N, D]."""
    q, k, v, out, lse = s.q, s.k, s.v, s.out, s.lse
    if q is None:
        q, k = ops.qk_norm_rope(s.xq, s.xk, s.wq, s.wk, s.plan, s.eps, dtype=dout.dtype)
        v = ops.unpack8(s.v, dout.dtype)
        out, lse = ops.window_attn_fwd(q, k, v, s.mask.left, s.mask.right, s.mask.sink, scale=s.scale)
    B, H, N, D = q.shape
    Hk = k.shape[1]
    dq, dk, dv = ops.window_attn_bwd(q, k, v, out, dout, lse, s.mask.left, s.mask.right, s.mask.sink,
                                     scale=s.scale)
    dqkv = torch.empty(B, N, H + 2 * Hk, D, device=dout.device, dtype=dout.dtype)
    dxq, dxk, dxv = _split(dqkv, H)
    _, _, dwq, dwk = ops.qk_norm_rope_bwd(dq, dk, s.xq, s.xk, s.wq, s.wk, s.plan, s.eps, dxq, dxk)
    dxv.copy_(dv.transpose(1, 2))
    return dqkv, dwq, dwk


class Stream:
    """Cached causal window attention of a batch of streams.

    step() takes the newest tokens' qkv [B, n, H + 2 Hk, D] and their
    positions, appends their keys and values and returns their outputs
    [B, H, n, D].  n is any number, a whole prompt's too: the cached attention
    takes 128 new tokens a call, so more are attended to in pieces.  A step
    that is refused leaves the stream as it was.  Every stream grows by the
    same n per step; `lens` (device) is what the kernel reads, `length` the
    same number on the host, so a step cannot be captured and replayed."""

    def __init__(self, B: int, heads: int, key_heads: int, capacity: int, head_dim: int,
                 plan: ops.RopePlan, mask: Mask, wq: Optional[torch.Tensor] = None,
                 wk: Optional[torch.Tensor] = None, eps: float = 1e-6, scale: Optional[float] = None,
                 dtype: torch.dtype = torch.bfloat16):
        if mask.right != 0:
            raise ValueError("a stream is causal: right must be 0")
        dev = plan.table.device
        self.heads, self.plan, self.mask = heads, plan, mask
        self.wq, self.wk, self.eps, self.scale = wq, wk, eps, scale
        self.k = torch.empty(B, key_heads, capacity, head_dim, device=dev, dtype=dtype)
        self.v = torch.empty_like(self.k)
        self.lens = torch.zeros(B, device=dev, dtype=torch.int32)
        self.length = 0

    def step(self, qkv: torch.Tensor, pos: torch.Tensor) -> torch.Tensor:
        cache, n = self.k, qkv.shape[1] if qkv.dim() == 4 else -1
        if n < 0 or qkv.shape != (cache.shape[0], n, self.heads + 2 * cache.shape[1], cache.shape[3]) \
                or qkv.dtype != cache.dtype or qkv.device != cache.device:
            raise ValueError(f"a step of this stream takes [{cache.shape[0]}, n, {self.heads + 2 * cache.shape[1]}, "
                             f"{cache.shape[3]}] of {cache.dtype} on {cache.device}")
        if self.length + n > cache.shape[2]:
            raise ValueError(f"{self.length} + {n} tokens exceed the capacity of {cache.shape[2]}")
        xq, xk, xv = _split(qkv, self.heads)
        q, k = ops.qk_norm_rope(xq, xk, self.wq, self.wk, self.plan.at(pos), self.eps)
        if n == 0:
            return q
        # rows past `lens` are not read: they count once every piece is on its way
        cache[:, :, self.length:self.length + n] = k
        self.v[:, :, self.length:self.length + n] = xv.transpose(1, 2)
        outs, at = [], 0
        try:
            for piece in (q,) if n <= _MOST_NEW else (x.contiguous() for x in q.split(_MOST_NEW, 2)):
                self.lens += piece.shape[2]
                at += piece.shape[2]
                outs.append(ops.window_attn_decode(piece, cache, self.v, self.lens, self.mask.left, self.mask.sink,
                                                   self.scale))
            out = outs[0] if len(outs) == 1 else torch.cat(outs, 2)
        except BaseException:
            self.lens -= at
            raise
        self.length += n
        return out
