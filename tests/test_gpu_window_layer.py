"""The norm with rotation, the window attention and the 8-bit rows together, as
a layer's training step and as a stream, against the same chain in 64 bits.

The chain in 64 bits rounds to bf16 where the layer stores bf16 (q, k, out,
dq, dk), so what is left between the two are the operators' own roundings: at
most three per output -- the weights before the second product, the output,
and a stored value that falls on the other side of a rounding border -- of half
a step, 2^-8 of a value at most and 2^-8 / sqrt(3) in the mean: the 2-norm of
the difference is held to 2^-7 of the result's.  fp32: sums of up to N terms of
fp32 roundings in a chain of four operators, 2^-24 * 4 * N with N <= 400:
2^-13.  A stream's tokens against the whole forward: two computations of the
same values, each within that."""
import math

import pytest
import torch

from dynamic_block_sparse_pool_b200 import ops, window_layer
from test_gpu_qk_norm_rope import angles, turn
from test_gpu_window_attn import visible

pytestmark = pytest.mark.gpu

LIMIT = {torch.bfloat16: 2.0 ** -7, torch.float32: 2.0 ** -13}


class _Round(torch.autograd.Function):
    """Rounds the value to the stored type, and the gradient that comes back."""

    @staticmethod
    def forward(ctx, x, dtype):
        ctx.dtype = dtype
        return x.to(dtype).double()

    @staticmethod
    def backward(ctx, g):
        return g.to(ctx.dtype).double(), None


def chain(qkv, H, wq, wk, c, s, mask, dtype):
    Hk = (qkv.shape[2] - H) // 2
    x = [qkv[:, :, :H], qkv[:, :, H:H + Hk], qkv[:, :, H + Hk:]]
    q, k = (_Round.apply(turn(t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w, c, s, False)
                         .transpose(1, 2), dtype) for t, w in ((x[0], wq), (x[1], wk)))
    v = x[2].transpose(1, 2)
    rep = lambda t: t.repeat_interleave(H // Hk, 1)  # noqa: E731
    ok = visible(q.shape[2], q.shape[2], 0, *mask)
    p = torch.softmax((q @ rep(k).transpose(2, 3) / math.sqrt(q.shape[3])).masked_fill(~ok, -math.inf), -1)
    return p @ rep(v)


def near(got, ref, limit, what):
    r = float((got.double().cpu() - ref).norm() / ref.norm())
    assert r <= limit, (what, r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,D,grid,prefix,mask", [
    (1, 4, 4, 64, (3, 7, 9), 20, (63, 63, 20)),
    (2, 6, 2, 128, (5, 6, 8), 0, (100, 0, 7)),
])
def test_training_step(B, H, Hk, D, grid, prefix, mask, dtype):
    N = prefix + grid[0] * grid[1] * grid[2]
    g = torch.Generator().manual_seed(N)
    qkv = torch.randn(B, N, H + 2 * Hk, D, generator=g).to(dtype).cuda()
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    dout = torch.randn(B, H, N, D, generator=g).to(dtype).cuda()
    plan = ops.RopePlan.grid(*grid, D, n_prefix=prefix)
    m = window_layer.Mask(*mask)
    out, saved = window_layer.forward(qkv, H, wq, wk, plan, m)
    dqkv, dwq, dwk = window_layer.backward(dout, saved)
    ops.device_status()
    c, s = angles(plan.pos.cpu(), plan.pairs, 10000.0, D)
    leaves = [t.double().cpu().requires_grad_() for t in (qkv, wq, wk)]
    ref = chain(leaves[0], H, leaves[1], leaves[2], c, s, mask, dtype)
    ref.backward(dout.double().cpu())
    lim = LIMIT[dtype]
    near(out, ref.detach(), lim, "out")
    for got, leaf, what in ((dqkv, leaves[0], "dqkv"), (dwq, leaves[1], "dwq"), (dwk, leaves[2], "dwk")):
        near(got, leaf.grad, lim, what)

    # the same step with what is kept in 8 bits: the outputs are the same, the
    # gradients those of the values the rows stand for.  A row's codes are off
    # by at most amax / 254, here at most 4.5 sigma / 254 = 1.8 % of sigma, 1 %
    # in the mean.  Two such rows meet in a score (their norms are near
    # sqrt(D), so a score moves by about 1.4 % of its own spread), and v and out
    # by 1 % each: 3 % in all, held to 5 %.
    out8, saved8 = window_layer.forward(qkv, H, wq, wk, plan, m, keep8=True)
    assert torch.equal(out8, out)
    assert sum(t.element_size() * t.numel() for a in (saved8.xq, saved8.xk, saved8.v, saved8.out) for t in a) \
        < 1.07 * (2 * H + 2 * Hk) * B * N * D  # a byte per value and a scale per row
    got8 = window_layer.backward(dout, saved8)
    ops.device_status()
    for a, leaf, what in zip(got8, leaves, ("dqkv8", "dwq8", "dwk8")):
        near(a, leaf.grad, 0.05, what)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_stream_is_the_forward_of_its_tokens(dtype):
    B, H, Hk, D, N = 2, 4, 2, 64, 150
    g = torch.Generator().manual_seed(11)
    qkv = torch.randn(B, N, H + 2 * Hk, D, generator=g).to(dtype).cuda()
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    pos = torch.stack([torch.arange(N), 500 + torch.arange(N)])[..., None]  # two streams at different places
    plan = ops.RopePlan(pos, (D // 2,), theta=500000.0)
    m = window_layer.Mask(40, 0, 4)
    want, _ = window_layer.forward(qkv, H, wq, wk, plan, m)
    st = window_layer.Stream(B, H, Hk, N, D, plan, m, wq, wk, dtype=dtype)
    got, at = [], 0
    for n in (64, 1, 1, 2, 1, 30, 1, 50):
        got.append(st.step(qkv[:, at:at + n].contiguous(), pos[:, at:at + n]))
        at += n
    ops.device_status()
    assert at == N
    near(torch.cat(got, 2), want.double().cpu(), 2 * LIMIT[dtype], "stream")
    with pytest.raises(ValueError, match="capacity"):
        st.step(qkv[:, :1].contiguous(), pos[:, :1])
