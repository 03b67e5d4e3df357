"""The layer's step with what lies between its passes held in 8 bits: its
gradients are those of the step on the values that the rows stand for.  The
chain in 64 bits therefore starts from those values; the bounds are the ones of
the step that keeps everything (test_gpu_window_layer.py), since the operators
and their roundings are the same.  Weights of 2 make the softmax peaked: a row
of weights that does not belong to the scores would show."""
import pytest
import torch

from dynamic_block_sparse_pool_b200 import ops, window_layer
from test_gpu_qk_norm_rope import angles
from test_gpu_window_layer import LIMIT, chain, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("weight", [1.0, 2.0])
@pytest.mark.parametrize("B,H,Hk,D,grid,prefix,mask", [
    (1, 4, 4, 64, (3, 7, 9), 20, (63, 63, 20)),
    (2, 6, 2, 128, (5, 6, 8), 0, (100, 0, 7)),
])
def test_gradients_of_the_values_held(B, H, Hk, D, grid, prefix, mask, weight, dtype):
    N = prefix + grid[0] * grid[1] * grid[2]
    g = torch.Generator().manual_seed(N)
    qkv = torch.randn(B, N, H + 2 * Hk, D, generator=g).to(dtype).cuda()
    wq, wk = ((weight * (1 + 0.2 * torch.randn(D, generator=g))).cuda() for _ in range(2))
    dout = torch.randn(B, H, N, D, generator=g).to(dtype).cuda()
    plan = ops.RopePlan.grid(*grid, D, n_prefix=prefix)
    _, saved = window_layer.forward(qkv, H, wq, wk, plan, window_layer.Mask(*mask), keep8=True)
    got = window_layer.backward(dout, saved)
    ops.device_status()
    held = lambda a: a.codes.double().cpu() * a.scales.double().cpu()[..., None]  # noqa: E731
    v = held(saved.v).to(dtype).double().transpose(1, 2)  # v is a stored value of the type, the rows are not
    rows = torch.cat([held(saved.xq), held(saved.xk), v], 2)
    c, s = angles(plan.pos.cpu(), plan.pairs, 10000.0, D)
    leaves = [rows.requires_grad_()] + [t.double().cpu().requires_grad_() for t in (wq, wk)]
    chain(leaves[0], H, leaves[1], leaves[2], c, s, mask, dtype).backward(dout.double().cpu())
    for a, leaf, what in zip(got, leaves, ("dqkv", "dwq", "dwk")):
        near(a, leaf.grad, LIMIT[dtype], what)
