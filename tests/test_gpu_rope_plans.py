"""Rotation tables and plans: bases that fp32 cannot represent, one base for each
axis, given table lengths, a first frame and a token order.

A table entry is a cosine or sine of an angle that is exact to about 2^-51 of
itself (a 64-bit power and product), so below 3e6 turned by 2e-9 at most, and
rounded once: half a step of a value up to 1 is 2^-25.  The outputs of the norm
with rotation are held to the bound of its own tests."""
import pytest
import torch

from dynamic_block_sparse_pool_b200 import ops
from test_gpu_qk_norm_rope import angles, close, forward64, inputs

pytestmark = pytest.mark.gpu

BASES = [10000.0, 10000.0 * 8 ** (128 / 126), 500000.0 * 4 ** (64 / 62), 1.0e6 / 3, 1.1]


@pytest.mark.parametrize("theta", BASES)
@pytest.mark.parametrize("positions,pairs", [(7, 1), (131072, 64), (100000, 21)])
def test_table(positions, pairs, theta):
    got = ops.rope_table(positions, pairs, theta).double().cpu()
    f = torch.tensor([theta ** (-i / pairs) for i in range(pairs)], dtype=torch.float64)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    err = (got - torch.stack([a.cos(), a.sin()], -1)).abs().max()
    assert float(err) <= 2.0 ** -25 + 2e-9


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("theta", BASES[1:3])
def test_scaled_bases_far_out(theta, halves):
    B, N, H, D = 1, 40, 3, 128
    xq, xk, wq, wk, _, _ = inputs(B, N, H, H, D, torch.float32, seed=2)
    pos = 100000 + 13 * torch.arange(N)[None, :, None]
    plan = ops.RopePlan(pos, (D // 2,), theta=theta, halves=halves)
    q, k = ops.qk_norm_rope(xq, xk, wq, wk, plan)
    ops.device_status()
    c, s = angles(pos, (D // 2,), theta, D)
    close(q, *forward64(xq, wq, 1e-6, c, s, halves), torch.float32, 16)
    close(k, *forward64(xk, wk, 1e-6, c, s, halves), torch.float32, 16)


def test_a_base_for_each_axis_and_given_lengths():
    N, H, D = 50, 2, 64
    xq, xk, wq, wk, _, _ = inputs(1, N, H, H, D, torch.float32, seed=3)
    g = torch.Generator().manual_seed(0)
    pos = torch.stack([torch.randint(-1, n, (N,), generator=g) for n in (30, 7, 11)], 1)
    pairs, thetas, lengths = (10, 9, 5), (10000.0, 256.0, 33.3), (40, 7, 12)
    plan = ops.RopePlan(pos, pairs, theta=thetas, lengths=lengths)
    assert plan.lengths == lengths and plan.table.shape == (40 * 10 + 7 * 9 + 12 * 5, 2)
    a = torch.zeros(1, N, D // 2, dtype=torch.float64)
    m = 0
    for x, (n, t) in enumerate(zip(pairs, thetas)):
        for i in range(n):
            a[0, :, m] = pos[:, x].double().clamp(min=0) * t ** (-i / n)
            m += 1
    c, s = a.cos()[:, :, None], a.sin()[:, :, None]
    q, k = ops.qk_norm_rope(xq, xk, wq, wk, plan)
    # room that `lengths` left: other positions of the same tables
    far = pos.clone()
    far[:, 0] = 39
    ops.qk_norm_rope(xq, xk, wq, wk, plan.at(far))
    ops.device_status()
    close(q, *forward64(xq, wq, 1e-6, c, s, False), torch.float32, 16)
    close(k, *forward64(xk, wk, 1e-6, c, s, False), torch.float32, 16)


@pytest.mark.parametrize("prefix", [0, 5])
def test_grid_in_another_order_from_a_later_frame(prefix):
    T, Y, X, H, D = 3, 5, 6, 2, 128
    N = prefix + T * Y * X
    order = ops.HilbertOrder(T, Y, X, n_prefix=prefix)
    perm = order.perm.cpu().long()
    row = ops.RopePlan.grid(T, Y, X, D, n_prefix=prefix, t0=4)
    along = ops.RopePlan.grid(T, Y, X, D, n_prefix=prefix, t0=4, order=order.perm)
    assert row.lengths == (T + 4, Y, X) and int(row.pos[0, prefix, 0]) == 4
    assert torch.equal(along.pos[0].cpu(), row.pos[0].cpu()[perm])
    assert bool((row.pos[0, :prefix] == -1).all())
    xq, xk, wq, wk, _, _ = inputs(1, N, H, H, D, torch.bfloat16, seed=4)
    want = ops.qk_norm_rope(xq, xk, wq, wk, row)
    # rows taken in that order with the plan of that order: the outputs in that order
    got = ops.qk_norm_rope(xq[:, perm].contiguous(), xk[:, perm].contiguous(), wq, wk, along)
    ops.device_status()
    assert all(torch.equal(a, order.gather(b)) for a, b in zip(got, want))
